// MXFP4 operands for gfx950: quantisation of a matrix along its rows and columns, and reading back.
//
// Rule (OCP MX v1.0): a group of 32 shares the scale 2^e, e = clamp(floor(log2 amax) - 2, -127, 127), and an element is the
// E2M1 number (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) nearest to v / 2^e, ties to the even code, saturated to 6. With
// E4M3 elements (products take an 8-bit left operand) the 2 is an 8 and the largest 448, as in quantize.hip. A
// group with amax 0 has scale byte 0; one that holds a NaN or an infinity has byte 255 and codes of the largest
// magnitude (E4M3: NaN). The amax is taken on the FP32 bits without the sign, whose order is that of the magnitudes, NaN
// last; its exponent field less 2 (8), not below 0, is the byte. v_cvt_scalef32_pk_fp4_f32 divides by the scale, rounds
// to nearest even and saturates.
//
// Layout: per 128 of the contraction a panel of codes [rows][64 bytes] (E4M3: two panels, 64 of the contraction each) and a
// plane of scale words [rows][4], so what the products load is contiguous whatever the rows they start at. The
// contraction is padded to 128 with zero codes and scale bytes.
//
// A block takes a tile of 128 x 128: a quarter of a wavefront reads 8 rows of it, 8 columns a lane, so a row group is
// four lanes, a column group the same column of four quarters, and all four outputs of the tile are contiguous runs (8 KB
// of codes, 512 bytes of scales), put together in LDS. A tile's amax takes four exchanges of packed pairs for the columns and two for
// the rows. BF16 values go through in pairs (v_cvt_scalef32_pk_fp4_bf16, 16-bit magnitudes), FP32 ones one by one.
//
// FP32 is bound by HBM: 16 weights of 2816 x 2048, rows 76 us (418 MB, 5.5 TB/s), and as BF16 read back 35 (235 MB, 6.6 TB/s). BF16
// is not: 24576 x 2048 rows 24.8 (127 MB, 5.1 TB/s), in both directions 28.7. Gathered rows (a plan's, topk 6) would be read topk times
// from memory where a token's experts' rows land on different XCDs; each XCD takes few column tiles of all rows, whose piece of x its
// L2 then holds: 25.4 us for 24576 x 2048 in both directions, 18 MB read, 58 written; the vector instructions are issued 64% of the
// time (the codes and two amax exchanges), LDS is busy 11%, a quarter of it with conflicts.
#include "chunk.h"
#include "kernels.h"
#include "ragged.h"

namespace mxf {

constexpr int kTile = 128;

template <bool E4M3>
struct GroupScale {
  float xf;       // 2^e
  float lim;      // E4M3: 448 * 2^e, the hardware's conversion does not saturate
  uint32_t nan;   // all ones in the magnitude bits of codes of a group that is not finite
  uint32_t byte;
};
template <bool E4M3>
__device__ __forceinline__ GroupScale<E4M3> group_scale(uint32_t amax) {
  constexpr uint32_t EMAX = E4M3 ? 8u : 2u;
  const uint32_t ef = amax >> 23;
  GroupScale<E4M3> g;
  const bool bad = ef == 255u;
  g.byte = bad ? 255u : ef > EMAX ? ef - EMAX : 0u;
  g.xf = bad ? 1.0f : __uint_as_float(g.byte ? g.byte << 23 : 0x00400000u);
  g.lim = 448.0f * g.xf;
  g.nan = bad ? (E4M3 ? 0x7F7F7F7Fu : 0x77777777u) : 0u;
  return g;
}
// Eight values as codes: one word of E2M1 (element 0 in the lowest bits) or two of E4M3.
__device__ __forceinline__ uint32_t codes4(const float (&v)[8], const GroupScale<false>& g) {
  uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, v[0], v[1], g.xf, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], g.xf, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], g.xf, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], g.xf, 3);
  return r | g.nan;
}
__device__ __forceinline__ uint2 codes8(const float (&v)[8], const GroupScale<true>& g) {
  s16x2 r[2] = {};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = __builtin_amdgcn_fmed3f(v[4 * i + j], -g.lim, g.lim);
    r[i] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r[i], c[0], c[1], g.xf, false);
    r[i] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r[i], c[2], c[3], g.xf, true);
  }
  return make_uint2(__builtin_bit_cast(uint32_t, r[0]) | g.nan, __builtin_bit_cast(uint32_t, r[1]) | g.nan);
}

// The same of packed BF16 pairs, which need no unpacking.
__device__ __forceinline__ uint32_t codes4(const uint32_t (&v)[4], const GroupScale<false>& g) {
  uint32_t r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, __builtin_bit_cast(bf16x2, v[0]), g.xf, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, v[1]), g.xf, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, v[2]), g.xf, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, v[3]), g.xf, 3);
  return r | g.nan;
}
__device__ __forceinline__ uint2 codes8(const uint32_t (&v)[4], const GroupScale<true>& g) {
  Scale s;
  const uint32_t lim = g.byte == 255u ? 0u : (g.byte + 8u) << 7 | 0x60u;  // 448 * 2^e
  s.lim2 = lim | lim << 16;
  s.xf = g.xf;
  s.nanmask = g.nan;
  s.byte = g.byte;
  return make_uint2(cvt4(v[0], v[1], s), cvt4(v[2], v[3], s));
}

// Staging of a tile's codes in LDS: 64-byte rows; 8 rows further another PAD bytes, so that the lanes of a write fall on
// different banks.
template <int PAD>
__device__ __forceinline__ int staged(int row) {
  return row * 64 + (row >> 3) * PAD;
}

template <class T, bool E4M3, bool ROW, bool COL, Ends E>
__global__ __launch_bounds__(256) void mxfp4_quantize_kernel(Mx4Params p, unsigned col_tiles, unsigned row_tiles) {
  constexpr int NP = E4M3 ? 2 : 1;  // code panels per 128 of the contraction
  constexpr int PADR = 64, PADC = E4M3 ? 32 : 16;
  constexpr int SIZER = kTile * 64 + 16 * PADR, SIZEC = kTile * 64 + 16 * PADC;
  __shared__ __attribute__((aligned(16))) uint8_t rc[ROW ? NP * SIZER : 16], cc[COL ? NP * SIZEC : 16];
  __shared__ __attribute__((aligned(16))) uint8_t rs[kTile * 4], cs[kTile * 4];
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, cg = lane & 15, rl = lane >> 4;
  unsigned ct = blockIdx.x % col_tiles, band = blockIdx.x / col_tiles;
  if (p.row_assign) {  // a token's rows are far apart: each XCD takes few columns of all rows, which its L2 then holds
    const unsigned pos = xcd_run(blockIdx.x, gridDim.x);
    ct = pos / row_tiles;
    band = pos % row_tiles;
  }
  const int64_t b = band / row_tiles, rt = band % row_tiles;
  const int64_t r0 = rt * kTile, c0 = (int64_t)ct * kTile;
  const T* x = reinterpret_cast<const T*>(p.x) + b * p.xs;
  const int64_t n_assign = p.tokens * p.topk, first = r0 + w * 32 + rl * 8;
  const int left = (int)min<int64_t>(p.cols - c0, 1 << 20) - cg * 8;  // columns from the lane's first

  int64_t end = p.rows, from[8];
  bool in[8];
  if (p.row_assign) {
    int32_t a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = p.row_assign[min<int64_t>(first + i, p.rows - 1)];
    end = min<int64_t>(p.offs[p.E], p.rows);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      in[i] = first + i < end && a[i] >= 0 && a[i] < n_assign;
      from[i] = in[i] ? (int64_t)(((uint64_t)(uint32_t)a[i] * p.topk_mul) >> p.topk_shift) : 0;  // a / topk
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      in[i] = first + i < end;
      from[i] = in[i] ? first + i : 0;
    }
  }
  if (r0 >= end) return;
  constexpr int VEC = Elem<T>::VEC, NV = 8 / VEC;
  u32x4_t raw[8][NV] = {};
  if (!p.row_assign || p.tokens > 0) {  // (else pad rows alone)
    const int c = (int)c0 + cg * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < NV; ++j) raw[i][j] = load_chunk<T, E>(x + from[i] * p.ldx, c + j * VEC, (int)p.cols);
    bool all = left >= 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) all = all && in[i];
    if (!__all(all)) {  // a ragged edge, or pad rows
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          raw[i][j] = chunk_of<T, E>(raw[i][j], left - j * VEC);
#pragma unroll
          for (int k = 0; k < 4; ++k) raw[i][j][k] = in[i] && left > j * VEC ? raw[i][j][k] : 0u;
        }
    }
  }

  // a group's eight of the lane's values with its scale: codes into LDS, the scale byte by one of its lanes
  const auto put_row = [&](int i, uint32_t amax, const auto& v) {
    amax = max(amax, dpp_xor1(amax));
    amax = max(amax, dpp_xor2(amax));
    const GroupScale<E4M3> g = group_scale<E4M3>(amax);
    const int row = w * 32 + rl * 8 + i;
    if constexpr (E4M3)
      *reinterpret_cast<uint2*>(rc + (cg >> 3) * SIZER + staged<PADR>(row) + (cg & 7) * 8) = codes8(v, g);
    else
      *reinterpret_cast<uint32_t*>(rc + staged<PADR>(row) + cg * 4) = codes4(v, g);
    if ((cg & 3) == 0) rs[row * 4 + (cg >> 2)] = (uint8_t)g.byte;
  };
  const auto put_col = [&](int j, uint32_t amax, const auto& v) {
    const GroupScale<E4M3> g = group_scale<E4M3>(amax);
    const int col = cg * 8 + j;
    if constexpr (E4M3)
      *reinterpret_cast<uint2*>(cc + (w >> 1) * SIZEC + staged<PADC>(col) + (w & 1) * 32 + rl * 8) = codes8(v, g);
    else
      *reinterpret_cast<uint32_t*>(cc + staged<PADC>(col) + w * 16 + rl * 4) = codes4(v, g);
    if (rl == 0) cs[col * 4 + w] = (uint8_t)g.byte;
  };
  if constexpr (sizeof(T) == 2) {
    // magnitudes of BF16 pairs as packed 16-bit integers
    if constexpr (ROW) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t v[4], m = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[k] = raw[i][0][k];
          m = pk_max_u16(m, mag2(v[k]));
        }
        put_row(i, max(m & 0xFFFFu, m >> 16) << 16, v);
      }
    }
    if constexpr (COL) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {  // columns 2 k and 2 k + 1
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = pk_max_u16(m, mag2(raw[i][0][k]));
        m = pk_max_u16(m, (uint32_t)__shfl_xor((int)m, 16));
        m = pk_max_u16(m, (uint32_t)__shfl_xor((int)m, 32));
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = pack_lo(raw[2 * i][0][k], raw[2 * i + 1][0][k]);
          hi[i] = pack_hi(raw[2 * i][0][k], raw[2 * i + 1][0][k]);
        }
        put_col(2 * k, m << 16, lo);
        put_col(2 * k + 1, m & 0xFFFF0000u, hi);
      }
    }
  } else {
    if constexpr (ROW) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v[8];
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          m = max(m, raw[i][k / VEC][k % VEC] & 0x7FFFFFFFu);
          v[k] = __uint_as_float(raw[i][k / VEC][k % VEC]);
        }
        put_row(i, m, v);
      }
    }
    if constexpr (COL) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float v[8];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          m = max(m, raw[i][k / VEC][k % VEC] & 0x7FFFFFFFu);
          v[i] = __uint_as_float(raw[i][k / VEC][k % VEC]);
        }
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        put_col(k, m, v);
      }
    }
  }
  __syncthreads();
  if constexpr (ROW) {
    const int64_t at = (b * col_tiles + ct) * p.rows + r0;
    const int n = (int)min<int64_t>(end - r0, kTile);
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      uint8_t* o = p.q + (NP * (b * col_tiles + ct) * p.rows + u * p.rows + r0) * 64;
#pragma unroll
      for (int t = tid; t < kTile * 4; t += 256)
        if (t < n * 4)
          *reinterpret_cast<uint4*>(o + t * 16) =
              *reinterpret_cast<const uint4*>(rc + u * SIZER + staged<PADR>(t >> 2) + (t & 3) * 16);
    }
    if (tid < n) reinterpret_cast<uint32_t*>(p.s)[at + tid] = reinterpret_cast<const uint32_t*>(rs)[tid];
  }
  if constexpr (COL) {
    const int64_t at = (b * row_tiles + rt) * p.cols + c0;
    const int n = (int)min<int64_t>(p.cols - c0, kTile);
#pragma unroll
    for (int u = 0; u < NP; ++u) {
      uint8_t* o = p.qt + (NP * (b * row_tiles + rt) * p.cols + u * p.cols + c0) * 64;
#pragma unroll
      for (int t = tid; t < kTile * 4; t += 256)
        if (t < n * 4)
          *reinterpret_cast<uint4*>(o + t * 16) =
              *reinterpret_cast<const uint4*>(cc + u * SIZEC + staged<PADC>(t >> 2) + (t & 3) * 16);
    }
    if (tid < n) reinterpret_cast<uint32_t*>(p.st)[at + tid] = reinterpret_cast<const uint32_t*>(cs)[tid];
  }
}

// Reading back: a block takes 128 rows of one 128-wide piece, a lane 16 bytes of output.
template <class T, bool E4M3>
__global__ __launch_bounds__(256) void mxfp4_dequantize_kernel(Mx4Params p, unsigned col_tiles, unsigned row_tiles) {
  constexpr int NP = E4M3 ? 2 : 1, VEC = Elem<T>::VEC, LPR = 128 / VEC, RPI = 64 / LPR, N = 32 / RPI;  // lanes per row, rows at a time
  constexpr int BITS = VEC * (E4M3 ? 8 : 4);                                                           // of a lane's codes
  const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6, l = lane % LPR, rl = lane / LPR;
  const unsigned ct = blockIdx.x % col_tiles, band = blockIdx.x / col_tiles;
  const int64_t b = band / row_tiles, r0 = (int64_t)(band % row_tiles) * kTile + w * 32 + rl;
  const int64_t plane = (b * col_tiles + ct) * p.rows, c0 = (int64_t)ct * kTile + l * VEC;
  const int64_t panel = NP * plane + (E4M3 ? (l * VEC >> 6) * p.rows : 0);
  const int n = (int)min<int64_t>(p.cols - c0, VEC), at = l * BITS / 8 % 64;
  uint32_t k[N][2];
  uint32_t sc[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t r = min<int64_t>(r0 + RPI * i, p.rows - 1);
    const uint8_t* q = p.q + (panel + r) * 64 + at;
    k[i][1] = 0;
    if constexpr (BITS == 16)
      k[i][0] = *reinterpret_cast<const uint16_t*>(q);
    else
      k[i][0] = *reinterpret_cast<const uint32_t*>(q);
    if constexpr (BITS == 64) k[i][1] = *reinterpret_cast<const uint32_t*>(q + 4);
    sc[i] = p.s[(plane + r) * 4 + (l * VEC >> 5)];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t r = r0 + RPI * i;
    const float scale = ckpt_scale(sc[i]);
    float f[VEC];
    if constexpr (E4M3) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) f[j] = ckpt_value(k[i], j, scale);
    } else {
#pragma unroll
      for (int j = 0; j < VEC / 2; ++j) {
        const f32x2 u = j == 0   ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(k[i][0], 1.0f, 0)
                        : j == 1 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(k[i][0], 1.0f, 1)
                        : j == 2 ? __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(k[i][0], 1.0f, 2)
                                 : __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(k[i][0], 1.0f, 3);
        f[2 * j] = u[0] * scale;
        f[2 * j + 1] = u[1] * scale;
      }
    }
    T* o = reinterpret_cast<T*>(p.out) + (b * p.rows + r) * p.cols + c0;
    if (r < p.rows) store_chunk<T, INSIDE>(o, f, n);
  }
}

}  // namespace mxf

namespace {

using namespace mxf;

template <class T, bool E4M3, bool ROW, bool COL>
hipError_t launch_as(const Mx4Params& p, hipStream_t st) {
  const int64_t ct = (p.cols + kTile - 1) / kTile, rt = (p.rows + kTile - 1) / kTile;
  const dim3 grid((unsigned)(p.batch * ct * rt)), block(256);
  constexpr int VEC = Elem<T>::VEC;
  auto* fn = p.cols % VEC == 0 ? mxfp4_quantize_kernel<T, E4M3, ROW, COL, EXACT>
             : p.cols > VEC    ? mxfp4_quantize_kernel<T, E4M3, ROW, COL, INSIDE>
                               : mxfp4_quantize_kernel<T, E4M3, ROW, COL, TINY>;
  hipLaunchKernelGGL(fn, grid, block, 0, st, p, (unsigned)ct, (unsigned)rt);
  return hipGetLastError();
}
template <class T, bool E4M3>
hipError_t launch_quantize(const Mx4Params& p, hipStream_t st) {
  if (p.q && p.qt) return launch_as<T, E4M3, true, true>(p, st);
  return p.q ? launch_as<T, E4M3, true, false>(p, st) : launch_as<T, E4M3, false, true>(p, st);
}
template <class T, bool E4M3>
hipError_t launch_dequantize(const Mx4Params& p, hipStream_t st) {
  const int64_t ct = (p.cols + kTile - 1) / kTile, rt = (p.rows + kTile - 1) / kTile;
  hipLaunchKernelGGL((mxfp4_dequantize_kernel<T, E4M3>), dim3((unsigned)(p.batch * ct * rt)), dim3(256), 0, st, p,
                     (unsigned)ct, (unsigned)rt);
  return hipGetLastError();
}

}  // namespace

hipError_t mxf_launch_mxfp4_quantize(const Mx4Params& p, bool f32, bool e4m3, hipStream_t st) {
  if (f32) return e4m3 ? launch_quantize<float, true>(p, st) : launch_quantize<float, false>(p, st);
  return e4m3 ? launch_quantize<uint16_t, true>(p, st) : launch_quantize<uint16_t, false>(p, st);
}

hipError_t mxf_launch_mxfp4_dequantize(const Mx4Params& p, bool f32, bool e4m3, hipStream_t st) {
  if (f32) return e4m3 ? launch_dequantize<float, true>(p, st) : launch_dequantize<float, false>(p, st);
  return e4m3 ? launch_dequantize<uint16_t, true>(p, st) : launch_dequantize<uint16_t, false>(p, st);
}
