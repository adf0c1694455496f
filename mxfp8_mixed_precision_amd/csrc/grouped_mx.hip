// Expert products on MXFP4 operands (mxfp4.hip has the layout), for gfx950.
//
//   forward          y[r, n] = sum_k x[r, k] w[e, n, k]          rows [offs[e], offs[e+1]) of x, any count
//   weight gradient  dw[e, n, k] = sum_{r of e} dy[r, n] x[r, k]  from the column operands of dy and x, offsets multiples of 128
//
// The input gradient is a forward product of dy with the column operand of w. The right operand is E2M1, the left E2M1 or
// E4M3. v_mfma_scale_f32_32x32x64_f8f6f4 multiplies the codes, applies both scales and adds to FP32. Within eight
// neighbouring products it keeps 13 places below the largest's exponent, which holds all of E2M1 x E2M1 (2.8e-7 over 16384
// random terms) but not of E4M3 x E2M1 (4e-5).
#include "chunk.h"
#include "kernels.h"
#include "mx_device.h"
#include "ragged.h"

namespace mxf {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Operand layout in registers: for 64 of the contraction lane l = r + 32 g (r < 32, g < 2) holds row r's E2M1 codes
// [32 g, 32 g + 32), 16 bytes, and the scale of that group; of E4M3 codes [16 g, 16 g + 16) and [32 + 16 g, 48 + 16 g), and
// the scale of group g all the same.
//
// Block tile BM x BN, four wavefronts in a 2 x 2 grid. The contraction advances 128 at a time (one panel); a stage
// in LDS is the rows' panel pieces as they lie (64-byte rows, 16-byte chunk c of row r at c ^ ((r / 4) % 4), so that 16
// consecutive rows at one chunk index hit 16 different bank groups) and their scale words. Direct loads fill a ring of S stages.
// Rows that do not exist load as zeros (bounded loads), the contraction is padded by the layout.
template <int BM, int BN, bool A8, int S_>
struct MxTile {
  static constexpr int S = S_;
  static constexpr int FM = BM / 64, FN = BN / 64;
  static constexpr int NPA = A8 ? 2 : 1;
  static constexpr int NLA = NPA * BM / 64, NLB = BN / 64;  // 1 KB loads per wavefront and stage
  static constexpr int NSC = (BM + BN) / 64;                 // 256-byte loads of scale words per stage
  static constexpr int NS = (NSC + 3) / 4;                   // per wavefront (the last ones may load nothing)
  static constexpr int L = NLA + NLB + NS;
  static constexpr int B_OFF = NPA * BM * 64, S_OFF = B_OFF + BN * 64;
  static constexpr int STAGE = S_OFF + NS * 1024;
  static constexpr int PITCH16 = BN + 8, PITCH32 = BN + 4;  // epilogue staging rows (elements)
  static constexpr int EPI16 = BM * PITCH16 * 2, EPI32 = BM / 2 * PITCH32 * 4;
  static constexpr int max3(int a, int b, int c) { return a > b ? (a > c ? a : c) : (b > c ? b : c); }
  static constexpr int LDS = max3(S * STAGE, EPI16, EPI32);
};

// One operand's place for a tile: its first panel's row and its first plane's, bytes from one panel (plane) to the next.
struct MxOperand {
  const uint8_t* q;
  const uint8_t* s;
  int64_t panel, plane;
};

template <int BM, int BN, bool A8, bool F32, int S>
__device__ __forceinline__ void mx_tile(uint8_t* smem, const MxOperand& a, const MxOperand& b, int mr, int nc, int KT,
                                        void* out, int64_t ldc, bool accum) {
  using T = MxTile<BM, BN, A8, S>;
  constexpr int FM = T::FM, FN = T::FN;
  const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid >> 1, wn = wid & 1, r32 = lane & 31, g = lane >> 5;
  const uint32_t lds0 = lds_addr(smem);

  // E4M3: wavefronts 0 and 1 load the stage's first panel, 2 and 3 its second
  i32x4 ra = descriptor(a.q + (A8 ? (wid >> 1) * a.panel : 0)), rb = descriptor(b.q);
  const uint64_t step_a = (uint64_t)(T::NPA * a.panel), step_b = (uint64_t)b.panel;
  const uint32_t chunk = ((lane & 3) ^ ((lane >> 4) & 3)) * 16;
  const int row_a = (A8 ? (wid & 1) : wid) * T::NLA * 16 + (lane >> 2), row_b = wid * T::NLB * 16 + (lane >> 2);
  uint32_t va[T::NLA], vb[T::NLB], vs[T::NS];
#pragma unroll
  for (int i = 0; i < T::NLA; ++i) va[i] = row_a + 16 * i < mr ? (row_a + 16 * i) * 64 + chunk : kNoElement;
#pragma unroll
  for (int i = 0; i < T::NLB; ++i) vb[i] = row_b + 16 * i < nc ? (row_b + 16 * i) * 64 + chunk : kNoElement;
  i32x4 rs[T::NS];
  uint64_t step_s[T::NS];
#pragma unroll
  for (int i = 0; i < T::NS; ++i) {
    const int j = wid + 4 * i;  // rows 64 j of A, then of B
    const bool of_a = j < BM / 64;
    const int row = (of_a ? j : j - BM / 64) * 64 + lane;
    rs[i] = descriptor(of_a ? a.s : b.s);
    step_s[i] = (uint64_t)(of_a ? a.plane : b.plane);
    vs[i] = j < T::NSC && row < (of_a ? mr : nc) ? row * 4 : kNoElement;
  }
  int issued = 0;
  auto issue = [&](uint32_t st) {  // the next stage into the slot at st
    const bool in = issued < KT;
#pragma unroll
    for (int i = 0; i < T::NLA; ++i) buffer_to_lds(ra, in ? va[i] : kNoElement, st + (wid * T::NLA + i) * 1024);
#pragma unroll
    for (int i = 0; i < T::NLB; ++i) buffer_to_lds(rb, in ? vb[i] : kNoElement, st + T::B_OFF + (wid * T::NLB + i) * 1024);
#pragma unroll
    for (int i = 0; i < T::NS; ++i) buffer_to_lds4(rs[i], in ? vs[i] : kNoElement, st + T::S_OFF + (wid + 4 * i) * 256);
    move_on(ra, step_a);
    move_on(rb, step_b);
#pragma unroll
    for (int i = 0; i < T::NS; ++i) move_on(rs[i], step_s[i]);
    ++issued;
  };
  const int ma = wm * (BM / 2) + r32, nb = wn * (BN / 2) + r32;
  auto swz = [](int row, int c) { return row * 64 + ((c ^ ((row >> 2) & 3)) << 4); };

  f32x16 acc[FM][FN];
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(lds0 + s * T::STAGE);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;

  uint32_t slot = 0, next = (S - 1) * T::STAGE;
#pragma unroll 1
  for (int kt = 0; kt < KT; ++kt) {
    wait_vmcnt<(S - 2) * T::L>();  // stage kt has landed
    __syncthreads();               // for every wavefront, and all have read the stage before it, whose slot is next
    issue(lds0 + next);
    const uint32_t st = lds0 + slot;
    uint32_t sa[FM], sb[FN];
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = *(const __attribute__((address_space(3))) uint32_t*)(uintptr_t)(st + T::S_OFF + (ma + 32 * i) * 4) >> (8 * g);
#pragma unroll
    for (int j = 0; j < FN; ++j)
      sb[j] = *(const __attribute__((address_space(3))) uint32_t*)(uintptr_t)(st + T::S_OFF + BM * 4 + (nb + 32 * j) * 4) >> (8 * g);
#pragma unroll
    for (int ks = 0; ks < 2; ++ks) {
      i32x8 fa[FM], fb[FN];
#pragma unroll
      for (int i = 0; i < FM; ++i) {
        if constexpr (A8) {
          const u32x4_t lo = lds16_at(st + ks * BM * 64 + swz(ma, g))[i * 128];
          const u32x4_t hi = lds16_at(st + ks * BM * 64 + swz(ma, 2 + g))[i * 128];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            fa[i][q] = (int)lo[q];
            fa[i][4 + q] = (int)hi[q];
          }
        } else {
          const u32x4_t v = lds16_at(st + swz(ma, 2 * ks + g))[i * 128];
          fa[i] = (i32x8){(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
        }
      }
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const u32x4_t v = lds16_at(st + T::B_OFF + swz(nb, 2 * ks + g))[j * 128];
        fb[j] = (i32x8){(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
      }
      // the operands swap places: a lane holds one output row and, in runs of four accumulators, four neighbouring columns
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          if (ks == 0)
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[j], fa[i], acc[i][j], 4, A8 ? 0 : 4, 0, (int)sb[j], 0,
                                                                        (int)sa[i]);
          else
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[j], fa[i], acc[i][j], 4, A8 ? 0 : 4, 2, (int)sb[j], 2,
                                                                        (int)sa[i]);
        }
    }
    next = slot;
    slot = slot == (S - 1) * T::STAGE ? 0 : slot + T::STAGE;
  }
  wait_vmcnt<0>();  // no load may still target LDS
  __syncthreads();  // the slots become the epilogue's staging

  // Epilogue: the tile goes through LDS so that stores are 16-byte runs along output rows.
  if constexpr (!F32) {
    uint16_t* cs = reinterpret_cast<uint16_t*>(smem);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint2*>(cs + (ma + i * 32) * T::PITCH16 + wn * (BN / 2) + j * 32 + 8 * c + 4 * g) =
              make_uint2(bf16x2_bits(acc[i][j][4 * c], acc[i][j][4 * c + 1]), bf16x2_bits(acc[i][j][4 * c + 2], acc[i][j][4 * c + 3]));
    __syncthreads();
    constexpr int CPR = BN / 8;
#pragma unroll 2
    for (int t = tid; t < BM * CPR; t += 256) {
      const int r = t / CPR, c = t % CPR * 8;
      if (r < mr && c < nc) {
        uint16_t* o = reinterpret_cast<uint16_t*>(out) + (int64_t)r * ldc + c;
        if (c + 8 <= nc)
          __builtin_nontemporal_store(*reinterpret_cast<const u32x4_t*>(cs + r * T::PITCH16 + c), reinterpret_cast<u32x4_any*>(o));
        else
          for (int e = 0; c + e < nc; ++e) o[e] = cs[r * T::PITCH16 + c + e];
      }
    }
    return;
  }
  float* cs = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int half = 0; half < 2; ++half) {  // half the rows at a time
    if (half) __syncthreads();
    if (wm == half) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<float4*>(cs + (i * 32 + r32) * T::PITCH32 + wn * (BN / 2) + j * 32 + 8 * c + 4 * g) =
                make_float4(acc[i][j][4 * c], acc[i][j][4 * c + 1], acc[i][j][4 * c + 2], acc[i][j][4 * c + 3]);
    }
    __syncthreads();
    constexpr int CPR = BN / 4;
#pragma unroll 2
    for (int t = tid; t < BM / 2 * CPR; t += 256) {
      const int r = t / CPR, c = t % CPR * 4, row = half * (BM / 2) + r;
      if (row < mr && c < nc) {
        u32x4_t v = *reinterpret_cast<const u32x4_t*>(cs + r * T::PITCH32 + c);
        float* o = reinterpret_cast<float*>(out) + (int64_t)row * ldc + c;
        if (c + 4 <= nc) {
          if (accum) {
            u32x4_t u;
            __builtin_memcpy(&u, o, 16);
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = __float_as_uint(__uint_as_float(v[q]) + __uint_as_float(u[q]));
          }
          __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(o));
        } else {
          const float* s = cs + r * T::PITCH32 + c;
          for (int e = 0; c + e < nc; ++e) o[e] = accum ? o[e] + s[e] : s[e];
        }
      }
    }
  }
}

template <bool F32>
__device__ __forceinline__ void* out_at(void* c, int64_t i) {
  return F32 ? (void*)(reinterpret_cast<float*>(c) + i) : (void*)(reinterpret_cast<uint16_t*>(c) + i);
}

// Forward: row tiles in groups of GM, all column tiles of a group before the next, so that the tiles in flight on an XCD
// share rows of x and columns of w in its L2.
template <int BM, int BN, bool A8, bool F32, int S>
__global__ __launch_bounds__(256, 2) void grouped_mx_rows_kernel(GroupedMxParams p, int col_tiles) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[MxTile<BM, BN, A8, S>::LDS];
  const RowTiles rt = count_row_tiles(p.offs, p.E, p.M, BM);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) *p.status = rt.ok ? 0 : 1;
  if (!rt.ok) return;
  const uint32_t total = (uint32_t)rt.tiles * (uint32_t)col_tiles;
  if (blockIdx.x >= total) return;
  const uint32_t pos = xcd_run(blockIdx.x, total);
  constexpr uint32_t GM = 4;
  const uint32_t per = GM * (uint32_t)col_tiles, grp = pos / per, in = pos - grp * per;
  const uint32_t rows = min(GM, (uint32_t)rt.tiles - grp * GM);
  const RowTile r = find_row_tile(rt, p.offs, p.E, BM, (int)(grp * GM + in % rows));
  const int64_t n0 = (int64_t)(in / rows) * BN, P = (p.K + 127) >> 7;
  const MxOperand a = {p.a + (int64_t)r.m0 * 64, p.as + (int64_t)r.m0 * 4, p.M * 64, p.M * 4};
  const MxOperand b = {p.b + (r.e * P * p.N + n0) * 64, p.bs + (r.e * P * p.N + n0) * 4, p.N * 64, p.N * 4};
  mx_tile<BM, BN, A8, F32, S>(smem, a, b, r.m1 - r.m0, (int)min(p.N - n0, (int64_t)BN), (int)P,
                              out_at<F32>(p.c, r.m0 * p.ldc + n0), p.ldc, false);
}

// The contract of the weight gradient's offsets: as ragged_ok, and multiples of 128.
__device__ __forceinline__ bool panels_ok(const int32_t* offs, int E, int64_t M) {
  bool bad = false;
  for (int i = threadIdx.x & 63; i < E; i += 64) bad = bad || (offs[i + 1] & 127) != 0;
  return ragged_ok(offs, E, M) && !__any(bad);
}

// Weight gradient: one grid of output tiles per expert, experts with the most rows first.
template <int BM, int BN, bool A8, bool F32, int S>
__global__ __launch_bounds__(256, 2) void grouped_mx_dw_kernel(GroupedMxParams p, int row_tiles, int col_tiles) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[MxTile<BM, BN, A8, S>::LDS];
  const bool ok = panels_ok(p.offs, p.E, p.M);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) *p.status = ok ? 0 : 1;
  if (!ok) return;
  const uint32_t per = (uint32_t)row_tiles * (uint32_t)col_tiles;
  const Segment sg = by_length(p.offs, p.E, (int)(blockIdx.x / per));
  if (p.accum && sg.hi == sg.lo) return;  // nothing to add
  const uint32_t pos = xcd_run(blockIdx.x % per, per);
  constexpr uint32_t GM = 4;
  const uint32_t grp = pos / (GM * (uint32_t)col_tiles), in = pos - grp * (GM * (uint32_t)col_tiles);
  const uint32_t rows = min(GM, (uint32_t)row_tiles - grp * GM);
  const int64_t m0 = (int64_t)(grp * GM + in % rows) * BM, n0 = (int64_t)(in / rows) * BN;
  const int64_t p0 = sg.lo >> 7;
  const MxOperand a = {p.a + ((A8 ? 2 : 1) * p0 * p.N + m0) * 64, p.as + (p0 * p.N + m0) * 4, p.N * 64, p.N * 4};
  const MxOperand b = {p.b + (p0 * p.K + n0) * 64, p.bs + (p0 * p.K + n0) * 4, p.K * 64, p.K * 4};
  mx_tile<BM, BN, A8, F32, S>(smem, a, b, (int)min(p.N - m0, (int64_t)BM), (int)min(p.K - n0, (int64_t)BN),
                              (sg.hi - sg.lo) >> 7, out_at<F32>(p.c, (int64_t)sg.e * p.N * p.K + m0 * p.K + n0), p.K, p.accum);
}

}  // namespace mxf

namespace {

using namespace mxf;

template <int B, bool A8, bool F32, int S>
hipError_t launch_rows(const GroupedMxParams& p, hipStream_t st) {
  const int64_t ct = (p.N + B - 1) / B;
  int64_t rt = p.M / B + (p.E < p.M ? p.E : p.M);  // every expert may end inside a tile
  if (rt == 0) rt = 1;                             // (one block looks at the offsets)
  hipLaunchKernelGGL((grouped_mx_rows_kernel<B, B, A8, F32, S>), dim3((unsigned)(rt * ct)), dim3(256), 0, st, p, (int)ct);
  return hipGetLastError();
}
template <int B, bool A8, bool F32, int S>
hipError_t launch_dw(const GroupedMxParams& p, hipStream_t st) {
  const int64_t rt = (p.N + B - 1) / B, ct = (p.K + B - 1) / B;
  hipLaunchKernelGGL((grouped_mx_dw_kernel<B, B, A8, F32, S>), dim3((unsigned)(p.E * rt * ct)), dim3(256), 0, st, p, (int)rt,
                     (int)ct);
  return hipGetLastError();
}
template <bool A8, bool F32>
hipError_t launch(bool wgrad, const GroupedMxParams& p, int ncu, hipStream_t st) {
  (void)ncu;
  constexpr int S = A8 ? 3 : 4;
  return wgrad ? launch_dw<128, A8, F32, S>(p, st) : launch_rows<128, A8, F32, S>(p, st);
}

}  // namespace

hipError_t mxf_launch_grouped_mx(bool wgrad, const GroupedMxParams& p, bool a8, int ncu, hipStream_t st) {
  if (a8) return p.out_f32 ? launch<true, true>(wgrad, p, ncu, st) : launch<true, false>(wgrad, p, ncu, st);
  return p.out_f32 ? launch<false, true>(wgrad, p, ncu, st) : launch<false, false>(wgrad, p, ncu, st);
}
