// Expert products in BF16 over ragged row segments: expert e owns rows [offs[e], offs[e+1]) of any
// count, with no padding between experts.
//
//   OP 0   y[r, n] = sum_k x[r, k] w[e, n, k]
//   OP 1   dx[r, k] = sum_n dy[r, n] w[e, n, k]
//   OP 2   dw[e, n, k] = sum_{r of e} dy[r, n] x[r, k]        (x BF16, or MXFP8 codes and scales)
//
// BF16 operands, FP32 accumulation in the matrix cores, one rounding at the store. A code of the
// MXFP8 checkpoint has four significant bits, so its product with the scale is a BF16 number and
// enters the same matrix instruction unrounded.
#include "kernels.h"
#include "mx_device.h"

namespace mxf {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// The contract of offs (offs[0] = 0, non-decreasing, offs[E] <= M) and, for a row tile index t, the
// expert and rows that it covers; whole wavefronts, the same answer in every lane. Lane i looks at
// expert 64 j + i; tiles are counted in expert order.
struct RowTile {
  bool ok;        // offsets hold
  int64_t tiles;  // row tiles of all experts
  int e;          // -1: t is past the last tile
  int64_t m0, m1; // rows of the tile
};
__device__ __forceinline__ RowTile find_row_tile(const int32_t* offs, int E, int64_t M, int bm, int64_t t) {
  const int lane = threadIdx.x & 63;
  RowTile r = {true, 0, -1, 0, 0};
  bool bad = false;
  for (int base = 0; base < E; base += 64) {
    const int i = base + lane;
    const int32_t lo = i < E ? offs[i] : 0, hi = i < E ? offs[i + 1] : 0;
    if (i < E && (lo > hi || lo < 0 || hi > M || (i == 0 && lo != 0))) bad = true;
    const int32_t n = i < E && hi > lo ? (hi - lo + bm - 1) / bm : 0;
    int32_t pre = n;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int32_t v = __shfl_up(pre, o);
      if (lane >= o) pre += v;
    }
    const int64_t first = r.tiles + pre - n;
    const uint64_t hit = __ballot(n > 0 && t >= first && t < first + n);
    if (hit) {
      const int l = __ffsll((unsigned long long)hit) - 1;
      const int32_t k = (int32_t)(t - __shfl(first, l));
      const int32_t elo = __shfl(lo, l), ehi = __shfl(hi, l);
      r.e = base + l;
      r.m0 = (int64_t)elo + (int64_t)k * bm;
      r.m1 = r.m0 + bm < ehi ? r.m0 + bm : ehi;
    }
    r.tiles += __shfl(pre, 63);
  }
  r.ok = !__any(bad);
  return r;
}

// The same contract without a tile.
__device__ __forceinline__ bool ragged_ok(const int32_t* offs, int E, int64_t M) {
  bool bad = false;
  for (int i = threadIdx.x & 63; i < E; i += 64) {
    const int32_t lo = offs[i], hi = offs[i + 1];
    if (lo > hi || lo < 0 || hi > M || (i == 0 && lo != 0)) bad = true;
  }
  return !__any(bad);
}

__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Any size and alignment: 128 x 128 tiles of four wavefronts, 32 contraction steps at a time, elements
// loaded one by one and laid contraction-contiguous in LDS.
constexpr int AT = 128, AK = 32, AP = AK + 8;

template <int OP, bool X8>
__global__ __launch_bounds__(256) void grouped_any_kernel(GroupedParams p, int64_t col_tiles) {
  __shared__ uint16_t sa[AT * AP], sb[AT * AP];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int64_t om = OP == 2 ? p.N : p.M, on = OP == 0 ? p.N : p.K;
  int e;
  int64_t m0, m1, n0, c0, c1;  // output rows [m0, m1), columns from n0, contraction [c0, c1)
  if constexpr (OP == 2) {
    const int64_t row_tiles = (om + AT - 1) / AT;
    const bool ok = ragged_ok(p.offs, p.E, p.M);
    if (blockIdx.x == 0 && tid == 0 && p.status) *p.status = ok ? 0 : 1;
    if (!ok) return;
    const int64_t t = blockIdx.x;
    n0 = t % col_tiles * AT;
    m0 = t / col_tiles % row_tiles * AT;
    m1 = m0 + AT < om ? m0 + AT : om;
    e = (int)(t / col_tiles / row_tiles);
    c0 = p.offs[e];
    c1 = p.offs[e + 1];
  } else {
    const RowTile r = find_row_tile(p.offs, p.E, p.M, AT, blockIdx.x / col_tiles);
    if (blockIdx.x == 0 && tid == 0 && p.status) *p.status = r.ok ? 0 : 1;
    if (!r.ok || r.e < 0) return;
    e = r.e;
    m0 = r.m0;
    m1 = r.m1;
    n0 = blockIdx.x % col_tiles * AT;
    c0 = 0;
    c1 = OP == 0 ? p.K : p.N;
  }
  const uint16_t* b = OP == 2 ? p.b : p.b + (int64_t)e * p.N * p.K;
  f32x16 acc[2][2] = {};
  const int wr = (wid >> 1) * 64, wc = (wid & 1) * 64;
  for (int64_t k0 = c0; k0 < c1; k0 += AK) {
    for (int i = tid; i < AT * AK; i += 256) {
      // consecutive threads walk the operand's contiguous axis
      const int kk = OP == 2 ? i / AT : i % AK, rr = OP == 2 ? i % AT : i / AK;
      const int64_t row = m0 + rr, k = k0 + kk;
      const bool in = row < m1 && k < c1;
      sa[rr * AP + kk] = in ? (OP == 2 ? p.a[k * p.lda + row] : p.a[row * p.lda + k]) : (uint16_t)0;
    }
    for (int i = tid; i < AT * AK; i += 256) {
      const int kk = OP == 0 ? i % AK : i / AT, rr = OP == 0 ? i / AK : i % AT;
      const int64_t col = n0 + rr, k = k0 + kk;
      uint16_t v = 0;
      if (col < on && k < c1) {
        if constexpr (OP == 0) {
          v = b[col * p.K + k];
        } else if constexpr (X8) {
          const float f = __builtin_amdgcn_cvt_f32_fp8((int)p.bq[k * p.K + col], 0);
          v = (uint16_t)bf16_bits(f * e8m0_value(p.bs[k * ((p.K + 31) / 32) + (col >> 5)]));
        } else {
          v = OP == 1 ? b[k * p.K + col] : b[k * p.ldb + col];
        }
      }
      sb[rr * AP + kk] = v;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < AK / 16; ++s) {
      bf16x8 fa[2], fb[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int o = s * 16 + 8 * (lane >> 5);
        fa[i] = *reinterpret_cast<const bf16x8*>(&sa[(wr + i * 32 + (lane & 31)) * AP + o]);
        fb[i] = *reinterpret_cast<const bf16x8*>(&sb[(wc + i * 32 + (lane & 31)) * AP + o]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
    }
    __syncthreads();
  }
  // accumulator: lane l holds column l % 32 and rows 8 (q / 4) + 4 (l / 32) + q % 4 of a 32 x 32 block
  const int64_t base = OP == 2 ? (int64_t)e * p.N * p.K : 0;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) {
        const int64_t row = m0 + wr + i * 32 + 8 * (q >> 2) + 4 * (lane >> 5) + (q & 3);
        const int64_t col = n0 + wc + j * 32 + (lane & 31);
        if (row < m1 && col < on) {
          const int64_t o = base + row * p.ldc + col;
          if (p.out_f32) {
            float* c = reinterpret_cast<float*>(p.c) + o;
            *c = p.accum ? *c + acc[i][j][q] : acc[i][j][q];
          } else {
            reinterpret_cast<uint16_t*>(p.c)[o] = (uint16_t)bf16_bits(acc[i][j][q]);
          }
        }
      }
}

}  // namespace mxf

hipError_t mxf_launch_grouped(int op, const mxf::GroupedParams& p, int ncu, hipStream_t st) {
  using namespace mxf;
  (void)ncu;
  const int64_t on = op == 0 ? p.N : p.K;
  const int64_t ct = (on + AT - 1) / AT;
  const int64_t rt = op == 2 ? p.E * ((p.N + AT - 1) / AT) : p.M / AT + (p.E < p.M ? p.E : p.M);
  const int64_t blocks = rt * ct;
  if (blocks == 0) return hipSuccess;
  if (blocks > 0xFFFFFF) return hipErrorInvalidValue;  // fewer than 2^32 threads
  const dim3 g((unsigned)blocks), b(256);
  if (op == 0)
    hipLaunchKernelGGL((grouped_any_kernel<0, false>), g, b, 0, st, p, ct);
  else if (op == 1)
    hipLaunchKernelGGL((grouped_any_kernel<1, false>), g, b, 0, st, p, ct);
  else if (p.bq)
    hipLaunchKernelGGL((grouped_any_kernel<2, true>), g, b, 0, st, p, ct);
  else
    hipLaunchKernelGGL((grouped_any_kernel<2, false>), g, b, 0, st, p, ct);
  return hipGetLastError();
}
