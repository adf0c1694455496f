// Expert products on MXFP4 operands (mxfp4.hip has the layout), for gfx950.
//
//   forward          y[r, n] = sum_k x[r, k] w[e, n, k]          rows [offs[e], offs[e+1]) of x, any count
//   weight gradient  dw[e, n, k] = sum_{r of e} dy[r, n] x[r, k]  from the column operands of dy and x, offsets multiples of 128
//
// The input gradient is a forward product of dy with the column operand of w. The right operand is E2M1, the left E2M1 or
// E4M3. v_mfma_scale_f32_32x32x64_f8f6f4 multiplies the codes, applies both scales and adds to FP32. Within eight
// neighbouring products it keeps 13 places below the largest's exponent, which holds all of E2M1 x E2M1 (2.8e-7 over 16384
// random terms) but not of E4M3 x E2M1. So E4M3 codes go in two parts, magnitudes from 2 on and those below, zeros in the place of
// the others: products of the first are multiples of 2^-3 (codes of 2^-2, E2M1 of 2^-1) with exponents up to 10, of the second
// multiples of 2^-10 with exponents up to 2, and both fit. That doubles the instructions, which E4M3 halves the rate of already.
#include <type_traits>

#include "chunk.h"
#include "kernels.h"
#include "mx_device.h"
#include "ragged.h"

namespace mxf {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// The E4M3 codes of magnitudes from 2 on (bit 6 of a byte), zeros in the place of the others.
__device__ __forceinline__ int large_codes(int v) {
  // (selectors 8 to 11 fill a byte with bit 15 or 31 of the second or first word)
  return v & (int)__builtin_amdgcn_perm((uint32_t)v << 1, (uint32_t)v << 9, 0x0B090A08u);
}

// Operand layout in registers: for 64 of the contraction lane l = r + 32 g (r < 32, g < 2) holds row r's E2M1 codes
// [32 g, 32 g + 32), 16 bytes, and the scale of that group; of E4M3 codes [16 g, 16 g + 16) and [32 + 16 g, 48 + 16 g), and
// the scale of group g all the same.
//
// Block tile BM x BN, four wavefronts in a 2 x 2 grid. The contraction advances 128 at a time (one panel); a stage
// in LDS is the rows' panel pieces as they lie (64-byte rows, 16-byte chunk c of row r at c ^ ((r / 4) % 4), so that 16
// consecutive rows at one chunk index hit 16 different bank groups) and their scale words. Direct loads fill a ring of S stages.
// Rows that do not exist load as zeros (bounded loads), the contraction is padded by the layout.
//
// Measured (us; instructions alone at 7.2 PFLOP/s, E4M3 x E2M1 4.6): weight gradient of 24576 x 2816 x 2048, 16 experts, into FP32 114
// (compute 40, the 369 MB of stores 61, one after the other in a tile; into BF16 94, added to FP32 251); forward of 24576 x 2816 x
// 2048 with E4M3 rows 192-205 (instructions 123, matrix cores busy 72%), 8192^3 632-686 (478, 86%).
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

// Kilobyte I of a wavefront's run of an operand (an instruction's offset moves both sides, up to 4 KB).
template <int I>
__device__ __forceinline__ void load_run(i32x4 rsrc, uint32_t voff, uint32_t lds) {
  buffer_to_lds_off<(I % 4) * 1024>(rsrc, voff + I / 4 * 4096, lds + I / 4 * 4096);
}
// fn(0), fn(1), ... fn(N - 1) with constants.
template <int N, int I = 0, class Fn>
__device__ __forceinline__ void each(Fn&& fn) {
  if constexpr (I < N) {
    fn(std::integral_constant<int, I>());
    each<N, I + 1>(fn);
  }
}

template <int BM, int BN, bool A8, bool F32, int S>
__device__ __forceinline__ void mx_tile(uint8_t* smem, const MxOperand& a, const MxOperand& b, int mr, int nc, int KT,
                                        void* out, int64_t ldc, bool accum) {
  using T = MxTile<BM, BN, A8, S>;
  constexpr int FM = T::FM, FN = T::FN;
  const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid >> 1, wn = wid & 1, r32 = lane & 31, g = lane >> 5;
  const uint32_t lds0 = lds_addr(smem);

  // A tile's rows of a panel (plane) are one run of bytes: the descriptors end with it, and rows past it load as zeros.
  // E4M3: wavefronts 0 and 1 load the stage's first panel, 2 and 3 its second
  i32x4 ra = descriptor(a.q + (A8 ? (wid >> 1) * a.panel : 0), mr * 64), rb = descriptor(b.q, nc * 64);
  const uint64_t step_a = (uint64_t)(T::NPA * a.panel), step_b = (uint64_t)b.panel;
  const uint32_t chunk = (lane >> 2) * 64 + ((lane & 3) ^ ((lane >> 4) & 3)) * 16;
  const uint32_t va = (A8 ? (wid & 1) : wid) * T::NLA * 1024 + chunk, vb = wid * T::NLB * 1024 + chunk;
  i32x4 rs[T::NS];
  uint64_t step_s[T::NS];
  uint32_t vs[T::NS];
#pragma unroll
  for (int i = 0; i < T::NS; ++i) {
    const int j = wid + 4 * i;  // rows 64 j of A, then of B
    const bool of_a = j < BM / 64;
    rs[i] = descriptor(of_a ? a.s : b.s, j < T::NSC ? (of_a ? mr : nc) * 4 : 0);
    step_s[i] = (uint64_t)(of_a ? a.plane : b.plane);
    vs[i] = ((of_a ? j : j - BM / 64) * 64 + lane) * 4;
  }
  // Load i of L of the next stage into the slot at st.
  auto load = [&](auto i_, uint32_t st) {
    constexpr int i = decltype(i_)::value;
    if constexpr (i < T::NLA)
      load_run<i>(ra, va, st + wid * T::NLA * 1024);
    else if constexpr (i < T::NLA + T::NLB)
      load_run<i - T::NLA>(rb, vb, st + T::B_OFF + wid * T::NLB * 1024);
    else
      buffer_to_lds4(rs[i - T::NLA - T::NLB], vs[i - T::NLA - T::NLB], st + T::S_OFF + (wid + 4 * (i - T::NLA - T::NLB)) * 256);
  };
  auto none = [&]() {  // past the last stage: loads of nothing, so that every stage counts alike
    ra[2] = rb[2] = 0;
#pragma unroll
    for (int i = 0; i < T::NS; ++i) rs[i][2] = 0;
  };
  auto advance = [&]() {
    move_on(ra, step_a);
    move_on(rb, step_b);
#pragma unroll
    for (int i = 0; i < T::NS; ++i) move_on(rs[i], step_s[i]);
  };
  const int ma = wm * (BM / 2) + r32, nb = wn * (BN / 2) + r32;
  // Fragment reads of half ks of the stage at st, one by one: A's (E4M3: two each), then B's.
  constexpr int RA = A8 ? 2 : 1, NR = FM * RA + FN;
  uint32_t rd_a[2][RA], rd_b[2];  // their places in slot 0
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
    for (int h = 0; h < RA; ++h) {
      const int c = A8 ? 2 * h + g : 2 * ks + g;
      rd_a[ks][h] = lds0 + (A8 ? ks * BM * 64 : 0) + ma * 64 + ((c ^ ((ma >> 2) & 3)) << 4);
    }
    rd_b[ks] = lds0 + T::B_OFF + nb * 64 + (((2 * ks + g) ^ ((nb >> 2) & 3)) << 4);
  }
  const uint32_t rd_sa = lds0 + T::S_OFF + ma * 4, rd_sb = lds0 + T::S_OFF + BM * 4 + nb * 4;
  i32x8 fa[2][FM], fb[2][FN];
  auto read = [&](int r, int ks, uint32_t st) {
    if (r < FM * RA) {
      const int i = r / RA, h = r % RA;
      const u32x4_t v = lds16_at(rd_a[ks][h] + st)[i * 128];
#pragma unroll
      for (int q = 0; q < 4; ++q) fa[ks][i][4 * h + q] = (int)v[q];
    } else {
      const int j = r - FM * RA;
      const u32x4_t v = lds16_at(rd_b[ks] + st)[j * 128];
#pragma unroll
      for (int q = 0; q < 4; ++q) fb[ks][j][q] = (int)v[q];
    }
  };
  typedef __attribute__((address_space(3))) const uint32_t lds_u32;
  uint32_t sa[FM], sb[FN], na[FM], nsb[FN];
  auto read_scale = [&](int r, uint32_t st) {
    if (r < FM)
      na[r] = ((lds_u32*)(uintptr_t)(rd_sa + st))[32 * r];
    else
      nsb[r - FM] = ((lds_u32*)(uintptr_t)(rd_sb + st))[32 * (r - FM)];
  };
  auto take_scales = [&]() {  // bytes 0 and 2 of the words are then the lane's groups of the two halves
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = na[i] >> (8 * g);
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = nsb[j] >> (8 * g);
  };

  f32x16 acc[FM][FN];
  // the operands swap places: a lane holds one output row and, in runs of four accumulators, four neighbouring columns
  // E4M3: per fragment of A all products with its large codes, beside which the small ones are made, then those with the small ones,
  // beside which the next fragment's large ones are (always after the product, which would wait for them). LIVE: fragments
  // that have rows.
  constexpr int PARTS = A8 ? 2 : 1;
  // the order as written, but for E4M3 on 128 x 128 tiles, few of which have a second wavefront to fill the gaps (one expert, 256 rows of
  // 8192 x 8192 43.8 us against 49.4; on 128 x 256 tiles 208 against 203 at 24576 x 2816 x 2048)
  constexpr bool FIXED = !(A8 && FN == 2);
  i32x8 part[2];
  auto multiply = [&](auto m_, auto ks_, auto live_) {
    constexpr int m = decltype(m_)::value, ks = decltype(ks_)::value, LIVE = decltype(live_)::value;
    constexpr int i = m / (PARTS * FN), h = m / FN % PARTS, j = m % FN;
    if constexpr (i < LIVE) {
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[ks][j], A8 ? part[h] : fa[ks][i], acc[i][j], 4, A8 ? 0 : 4, 2 * ks,
                                                                  (int)sb[j], 2 * ks, (int)sa[i]);
      if constexpr (A8) {
        if (FIXED) __builtin_amdgcn_sched_barrier(0);
        constexpr int n = (i + 1) % LIVE;
#pragma unroll
        for (int q = 8 * j / FN; q < 8 * (j + 1) / FN; ++q) {
          if (h)
            part[0][q] = large_codes(fa[n ? ks : 1 - ks][n][q]);
          else
            part[1][q] = fa[ks][i][q] ^ part[0][q];
        }
      }
    }
  };
  using K0 = std::integral_constant<int, 0>;
  using K1 = std::integral_constant<int, 1>;
  constexpr int NM = PARTS * FM * FN;
  if (KT == 0) none();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    each<T::L>([&](auto i) { load(i, lds0 + s * T::STAGE); });
    advance();
    if (s + 1 >= KT) none();
  }
  constexpr int LH = T::L / 2;  // loads in the second half of a stage, the others in the first half of the next
  each<LH>([&](auto i) { load(i, lds0 + (S - 1) * T::STAGE); });
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
  uint32_t slot = 0;
  auto after = [](uint32_t st) { return st == (S - 1) * T::STAGE ? 0u : st + (uint32_t)T::STAGE; };
  if (KT > 0) {
    wait_vmcnt<(S - 2) * T::L + LH>();
    __syncthreads();
#pragma unroll
    for (int r = 0; r < FM + FN; ++r) read_scale(r, 0);
#pragma unroll
    for (int r = 0; r < NR; ++r) read(r, 0, 0);
    take_scales();
    if constexpr (A8) {
#pragma unroll
      for (int q = 0; q < 8; ++q) part[0][q] = large_codes(fa[0][0][q]);
    }
    uint32_t last = (S - 1) * T::STAGE;
    const auto stages = [&](auto live) {
#pragma unroll 1
      for (int kt = 0; kt < KT; ++kt) {
        // first half, beside the reads of the second and the rest of the loads of stage kt + S - 1
        each<NM>([&](auto m_) {
          constexpr int m = decltype(m_)::value, l0 = LH + m * (T::L - LH) / NM, l1 = LH + (m + 1) * (T::L - LH) / NM;
          multiply(m_, K0(), live);
#pragma unroll
          for (int r = m * NR * 2 / NM; r < (m + 1) * NR * 2 / NM && r < NR; ++r) read(r, 1, slot);
          each<l1 - l0>([&](auto i) { load(std::integral_constant<int, l0 + decltype(i)::value>(), lds0 + last); });
          if (FIXED) __builtin_amdgcn_sched_barrier(0);
        });
        advance();
        if (kt + S >= KT) none();
        wait_vmcnt<(S - 2) * T::L>();  // the next stage has landed
        __syncthreads();               // for every wavefront, and all have read this one, whose slot stage kt + S takes
        const uint32_t next = after(slot);
        // second half, beside the reads of the next stage's first and the first loads of stage kt + S
        each<NM>([&](auto m_) {
          constexpr int m = decltype(m_)::value, l0 = m * LH / NM, l1 = (m + 1) * LH / NM, NRS = NR + FM + FN;
          multiply(m_, K1(), live);
#pragma unroll
          for (int r = m * NRS * 2 / NM; r < (m + 1) * NRS * 2 / NM && r < NRS; ++r) {
            if (r < FM + FN)
              read_scale(r, next);
            else
              read(r - FM - FN, 0, next);
          }
          each<l1 - l0>([&](auto i) { load(std::integral_constant<int, l0 + decltype(i)::value>(), lds0 + slot); });
          if (FIXED) __builtin_amdgcn_sched_barrier(0);
        });
        take_scales();
        last = slot;
        slot = next;
      }
    };
    using F = std::integral_constant<int, FM>;
    if constexpr (A8 && FN == 2) {  // (a wavefront's rows may end in its first fragment, or before; all pass the same barriers)
      static_assert(FM == 2);
      const int live = (mr - wm * (BM / 2) + 31) >> 5;
      if (live <= 0)
        stages(std::integral_constant<int, 0>());
      else if (live < FM)
        stages(std::integral_constant<int, 1>());
      else
        stages(F());
    } else {
      stages(F());
    }
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
template <int BM, int BN, bool A8, bool F32, int S, int OCC>
__global__ __launch_bounds__(256, OCC) void grouped_mx_rows_kernel(GroupedMxParams p, int col_tiles) {
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

// ------------------------------------------------------------------ long lists of tiles

// E2M1 x E2M1 where the chip's tiles take several rounds: one block per compute unit walks its share of 256 x 256 tiles without
// a break. The stages of all its tiles are one stream through the ring of four, so the loads of the next tile's first stages run
// under the last ones of this; the results (BF16) are packed into 128 registers and stored under the next tile's first
// stages, where a tile that stores at its end leaves the matrix cores idle for the time that 131 KB per compute unit take
// at the memory's rate. Stores are whole 128-byte lines past the caches (64-byte halves or cached lines: 97 us for 85 below), two to
// each of 16 stages, or four to each of 8 where a tile has fewer than 16.
//
// 24576 x 2816 x 2048, 16 experts, 83-86 us (3.3 PFLOP/s; tiles one by one 90, compute 40 at the instructions' rate): a tile is 16
// stages, the chip stores 138 MB at the same time, and the matrix cores are busy 40% of the cycles. 16384 x 4096 x 7168, 8 experts,
// 230-237 us (4.1 PFLOP/s), 8192^3 231 (4.7): busy 58% and 66% of the cycles. These run at 1.7 GHz, as the instructions alone do (2.4
// without load), so what is left is cycles without a matrix instruction: one wavefront to a SIMD waits, at barriers and for LDS, 20%
// of its time, and nothing else can issue meanwhile.
constexpr int kStreamTiles = 1024;  // of a block: its list is in LDS

struct StreamTile {
  int e, m0, mr, n0;
};

// Lanes with bit 3 of x exchanged with lanes without it of y.
__device__ __forceinline__ void swap_eights(u32x4_t& x, u32x4_t& y) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {  // (a row of 16 lanes turned by 8, and half of it taken)
    const uint32_t t = x[q];
    x[q] = (uint32_t)__builtin_amdgcn_update_dpp((int)t, (int)y[q], 0x128, 0xF, 0xC, false);
    y[q] = (uint32_t)__builtin_amdgcn_update_dpp((int)y[q], (int)t, 0x128, 0xF, 0x3, false);
  }
}

__device__ __forceinline__ void store16_bounded(u32x4_t v, i32x4 rsrc, uint32_t voff) {
  const __amdgpu_buffer_rsrc_t r =
      __builtin_amdgcn_make_buffer_rsrc((void*)((uint64_t)(uint32_t)rsrc[1] << 32 | (uint32_t)rsrc[0]), 0, rsrc[2], 0x00020000);
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(i32x4, v), r, voff, 0, 2);  // (non-temporal)
}

template <int PRE>
__device__ __forceinline__ void stream_tiles(const GroupedMxParams& p, uint8_t* smem, const StreamTile* list, int n) {
  using T = MxTile<256, 256, false, 4>;
  constexpr int S = 4, FM = 4, FN = 4, NM = 16, NR = 8, LH = T::L / 2;
  constexpr int ST = 32 / PRE;  // stores of each of the PRE stages that have some
  const int tid = threadIdx.x, lane = tid & 63, wid = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wid >> 1, wn = wid & 1, r32 = lane & 31, g = lane >> 5;
  const uint32_t lds0 = lds_addr(smem);
  const int KT = (int)((p.K + 127) >> 7);
  const uint64_t step_a = (uint64_t)p.M * 64, step_b = (uint64_t)p.N * 64;
  const uint32_t va = wid * 4096 + (lane >> 2) * 64 + ((lane & 3) ^ ((lane >> 4) & 3)) * 16, vs = (wid * 64 + lane) * 4;

  // the loads' place in the stream: tile, stages left of it
  i32x4 ra, rb, rsa, rsb;
  int lt = 0, ll = 0;
  auto next_tile = [&]() {  // the descriptors of tile lt, or of nothing past the last
    const int i = min(lt, n - 1);
    const StreamTile t = {__builtin_amdgcn_readfirstlane(list[i].e), __builtin_amdgcn_readfirstlane(list[i].m0),
                          __builtin_amdgcn_readfirstlane(list[i].mr), __builtin_amdgcn_readfirstlane(list[i].n0)};
    const int mr = lt < n ? t.mr : 0, nc = lt < n ? (int)min(p.N - t.n0, (int64_t)256) : 0;
    const int64_t w0 = (int64_t)t.e * KT * p.N + t.n0;
    ra = descriptor(p.a + (int64_t)t.m0 * 64, mr * 64);
    rb = descriptor(p.b + w0 * 64, nc * 64);
    rsa = descriptor(p.as + (int64_t)t.m0 * 4, mr * 4);
    rsb = descriptor(p.bs + w0 * 4, nc * 4);
    ll = KT;
    ++lt;
  };
  auto advance = [&]() {
    if (--ll == 0) {
      next_tile();
    } else {
      move_on(ra, step_a);
      move_on(rb, step_b);
      move_on(rsa, step_a / 16);
      move_on(rsb, step_b / 16);
    }
  };
  auto load = [&](auto i_, uint32_t st) {
    constexpr int i = decltype(i_)::value;
    if constexpr (i < 4)
      load_run<i>(ra, va, st + wid * 4096);
    else if constexpr (i < 8)
      load_run<i - 4>(rb, va, st + T::B_OFF + wid * 4096);
    else
      buffer_to_lds4(i == 8 ? rsa : rsb, vs, st + T::S_OFF + (i == 8 ? 0 : 1024) + wid * 256);
  };
  const int ma = wm * 128 + r32, nb = wn * 128 + r32;
  uint32_t rd_a[2], rd_b[2];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    rd_a[ks] = lds0 + ma * 64 + (((2 * ks + g) ^ ((ma >> 2) & 3)) << 4);
    rd_b[ks] = lds0 + T::B_OFF + nb * 64 + (((2 * ks + g) ^ ((nb >> 2) & 3)) << 4);
  }
  const uint32_t rd_sa = lds0 + T::S_OFF + ma * 4, rd_sb = lds0 + T::S_OFF + 1024 + nb * 4;
  i32x8 fa[2][FM], fb[2][FN];
  auto read = [&](int r, int ks, uint32_t st) {
    const u32x4_t v = r < FM ? lds16_at(rd_a[ks] + st)[r * 128] : lds16_at(rd_b[ks] + st)[(r - FM) * 128];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (r < FM)
        fa[ks][r][q] = (int)v[q];
      else
        fb[ks][r - FM][q] = (int)v[q];
    }
  };
  typedef __attribute__((address_space(3))) const uint32_t lds_u32;
  uint32_t sa[FM], sb[FN], na[FM], nsb[FN];
  auto read_scale = [&](int r, uint32_t st) {
    if (r < FM)
      na[r] = ((lds_u32*)(uintptr_t)(rd_sa + st))[32 * r];
    else
      nsb[r - FM] = ((lds_u32*)(uintptr_t)(rd_sb + st))[32 * (r - FM)];
  };
  auto take_scales = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i) sa[i] = na[i] >> (8 * g);
#pragma unroll
    for (int j = 0; j < FN; ++j) sb[j] = nsb[j] >> (8 * g);
  };
  f32x16 acc[FM][FN];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
  };

  // the finished tile: packed results, and where they go. Fragments (i, 2 j) and (i, 2 j + 1) are four pieces of 16 bytes per lane: piece
  // (u, h) is 8 rows of 128 bytes, row 32 i + 16 h + 8 u + lane % 8, columns 64 j + col and the next seven
  u32x4_t done[NM][2];
#pragma unroll
  for (int m = 0; m < NM; ++m) done[m][0] = done[m][1] = (u32x4_t){0, 0, 0, 0};
  i32x4 ro = {0, 0, 0, 0x00020000};  // (nothing to store yet)
  uint32_t vo[2] = {kNoElement, kNoElement};  // columns col and 64 + col of the lane's first row
  const int col = wn * 128 + 8 * g + 16 * ((lane >> 4) & 1) + 32 * ((lane >> 3) & 1);
  const uint32_t eight_rows = (uint32_t)p.ldc * 16;
  auto store = [&](auto k_) {
    constexpr int k = decltype(k_)::value, m = k / 2, h = k % 2;
    // (rows past the tile's are found by the whole offset: an instruction's scalar offset need not be part of the bounds check)
    store16_bounded(done[m][h], ro, vo[m % FN / 2] + (m / FN * 4 + h * 2 + m % 2) * eight_rows);
  };

  auto pin = [&]() {  // (else the compiler moves the matrix instructions of a half past the branches after it)
#pragma unroll
    for (int m = 0; m < NM; ++m) asm volatile("" : "+a"(acc[m / FN][m % FN]));
  };
  auto stage = [&](auto pre_, uint32_t& slot, uint32_t& last) {
    constexpr int pre = decltype(pre_)::value;  // the stores' share of this stage, -1 none
    // first half, beside the reads of the second, the rest of the loads of the stage that took the last slot, and stores
    each<NM>([&](auto m_) {
      constexpr int m = decltype(m_)::value, l0 = LH + m * (T::L - LH) / NM, l1 = LH + (m + 1) * (T::L - LH) / NM;
      acc[m / FN][m % FN] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[0][m % FN], fa[0][m / FN], acc[m / FN][m % FN], 4, 4, 0,
                                                                            (int)sb[m % FN], 0, (int)sa[m / FN]);
#pragma unroll
      for (int r = m * NR * 2 / NM; r < (m + 1) * NR * 2 / NM && r < NR; ++r) read(r, 1, slot);
      each<l1 - l0>([&](auto i) { load(std::integral_constant<int, l0 + decltype(i)::value>(), lds0 + last); });
      if constexpr (pre >= 0 && m % (2 * NM / ST) == NM / ST) store(std::integral_constant<int, pre * ST + m / (2 * NM / ST)>());
      __builtin_amdgcn_sched_barrier(0);
    });
    pin();
    advance();
    // the next stage has landed: at most two stages' loads may be in flight, and the stores among them
    constexpr int HS = ST / 2;
    constexpr int between = pre < 0 ? 0 : pre == 0 ? HS : pre == 1 ? 3 * HS : 4 * HS;
    wait_vmcnt<(S - 2) * T::L + between>();
    __syncthreads();
    const uint32_t next = slot == (S - 1) * T::STAGE ? 0u : slot + (uint32_t)T::STAGE;
    each<NM>([&](auto m_) {
      constexpr int m = decltype(m_)::value, l0 = m * LH / NM, l1 = (m + 1) * LH / NM, NRS = NR + FM + FN;
      acc[m / FN][m % FN] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(fb[1][m % FN], fa[1][m / FN], acc[m / FN][m % FN], 4, 4, 2,
                                                                            (int)sb[m % FN], 2, (int)sa[m / FN]);
#pragma unroll
      for (int r = m * NRS * 2 / NM; r < (m + 1) * NRS * 2 / NM && r < NRS; ++r) {
        if (r < FM + FN)
          read_scale(r, next);
        else
          read(r - FM - FN, 0, next);
      }
      each<l1 - l0>([&](auto i) { load(std::integral_constant<int, l0 + decltype(i)::value>(), lds0 + slot); });
      if constexpr (pre >= 0 && m % (2 * NM / ST) == NM / ST)
        store(std::integral_constant<int, pre * ST + ST / 2 + m / (2 * NM / ST)>());
      __builtin_amdgcn_sched_barrier(0);
    });
    pin();
    take_scales();
    last = slot;
    slot = next;
  };

  next_tile();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    each<T::L>([&](auto i) { load(i, lds0 + s * T::STAGE); });
    advance();
  }
  each<LH>([&](auto i) { load(i, lds0 + (S - 1) * T::STAGE); });
  clear();
  wait_vmcnt<(S - 2) * T::L + LH>();
  __syncthreads();
#pragma unroll
  for (int r = 0; r < FM + FN; ++r) read_scale(r, 0);
#pragma unroll
  for (int r = 0; r < NR; ++r) read(r, 0, 0);
  take_scales();
  uint32_t slot = 0, last = (S - 1) * T::STAGE;
#pragma unroll 1
  for (int t = 0; t < n; ++t) {
    each<PRE>([&](auto k) { stage(k, slot, last); });
#pragma unroll 1
    for (int kt = PRE; kt < KT; ++kt) stage(std::integral_constant<int, -1>(), slot, last);
    // pack: accumulators 4 c .. 4 c + 3 are row r32, columns 8 c + 4 g and the next three; the halves of the wavefront exchange so
    // that a lane has eight columns in a row, then its quarters (64 bytes of 16 rows), then eights of neighbouring fragments: a
    // store has 128 bytes of 8 rows
    const int m0 = __builtin_amdgcn_readfirstlane(list[t].m0), mr = __builtin_amdgcn_readfirstlane(list[t].mr),
              n0 = __builtin_amdgcn_readfirstlane(list[t].n0);
    const int nc = (int)min(p.N - n0, (int64_t)256);
    // (the descriptor ends with the tile's last row: rows past it are not stored)
    ro = descriptor(reinterpret_cast<uint16_t*>(p.c) + (int64_t)m0 * p.ldc + n0, (int)((mr - 1) * p.ldc + nc) * 2);
#pragma unroll
    for (int c = 0; c < 2; ++c)  // (no column: past the descriptor's end whatever rows are added)
      vo[c] = 64 * c < nc - col ? (uint32_t)(wm * 128 + (lane & 7)) * (uint32_t)(p.ldc * 2) + (64 * c + col) * 2 : kNoElement;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      f32x16& v = acc[m / FN][m % FN];
      asm volatile("" : "+a"(v));  // fragments leave the AGPRs one at a time
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t x0 = bf16x2_bits(v[8 * h], v[8 * h + 1]), x1 = bf16x2_bits(v[8 * h + 2], v[8 * h + 3]);
        const uint32_t y0 = bf16x2_bits(v[8 * h + 4], v[8 * h + 5]), y1 = bf16x2_bits(v[8 * h + 6], v[8 * h + 7]);
        const auto u0 = __builtin_amdgcn_permlane32_swap(x0, y0, false, false);
        const auto u1 = __builtin_amdgcn_permlane32_swap(x1, y1, false, false);
        done[m][h] = (u32x4_t){u0[0], u1[0], u0[1], u1[1]};
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const auto u = __builtin_amdgcn_permlane16_swap(done[m][0][q], done[m][1][q], false, false);
        done[m][0][q] = u[0];
        done[m][1][q] = u[1];
      }
      if (m & 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h) swap_eights(done[m - 1][h], done[m][h]);
      }
#pragma unroll
      for (int q = 0; q < 16; ++q) v[q] = 0.0f;
      asm volatile("" : "+a"(v));
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  each<32>([&](auto k) { store(k); });
  wait_vmcnt<0>();  // no load may still target LDS
}

// The tiles that do not fill a round of an XCD's compute units are split into four quarters or two halves of the rows, where that
// many fit, and come last, by themselves.
template <int PRE>
__global__ __launch_bounds__(256, 1) void grouped_mx_stream_kernel(GroupedMxParams p, int col_tiles) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[4 * MxTile<256, 256, false, 4>::STAGE];
  __shared__ StreamTile list[kStreamTiles];
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // a block's tile i is position first + j0 + i * per_xcd of the order, blocks b, b + 8, ... share an XCD
  const uint32_t per_xcd = gridDim.x / 8, j0 = blockIdx.x / 8, xcd = blockIdx.x % 8;
  const auto place = [&](const RowTiles& rt, uint32_t pos) {
    constexpr uint32_t GM = 4;
    const uint32_t per = GM * (uint32_t)col_tiles, grp = pos / per, in = pos - grp * per;
    const uint32_t rows = min(GM, (uint32_t)rt.tiles - grp * GM);
    const RowTile r = find_row_tile(rt, p.offs, p.E, 256, (int)(grp * GM + in % rows));
    return StreamTile{r.e, r.m0, r.m1 - r.m0, (int)(in / rows) * 256};
  };
  uint32_t first, whole, rest, split;
  int n;
  {
    const RowTiles rt = count_row_tiles(p.offs, p.E, p.M, 256);
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) *p.status = rt.ok ? 0 : 1;
    if (!rt.ok) return;
    const uint32_t total = (uint32_t)rt.tiles * (uint32_t)col_tiles, q = total / 8, r = total % 8;
    first = xcd < r ? xcd * (q + 1) : r * (q + 1) + (xcd - r) * q;
    const uint32_t mine = q + (xcd < r ? 1 : 0);
    rest = mine % per_xcd;
    whole = mine - rest;
    split = 4 * rest <= per_xcd ? 4 : 2 * rest <= per_xcd ? 2 : 1;
    n = (int)(whole / per_xcd) + (split == 1 && j0 < rest ? 1 : 0);
    for (int i = wid; i < n; i += 4) {
      const StreamTile t = place(rt, first + j0 + i * per_xcd);
      if (lane == 0) list[i] = t;
    }
  }
  __syncthreads();
  if (n > 0) stream_tiles<PRE>(p, smem, list, n);
  if (split == 1 || j0 >= rest * split) return;
  __syncthreads();
  const StreamTile t = place(count_row_tiles(p.offs, p.E, p.M, 256), first + whole + j0 / split);
  const uint32_t part = j0 % split;
  const int m0 = t.m0 + (int)(part >> (split == 4)) * 128, mr = min(t.m0 + t.mr - m0, 128);
  const int64_t n0 = t.n0 + (split == 4 ? (part & 1) * 128 : 0), P = (p.K + 127) >> 7;
  if (mr <= 0 || n0 >= p.N) return;
  const MxOperand a = {p.a + (int64_t)m0 * 64, p.as + (int64_t)m0 * 4, p.M * 64, p.M * 4};
  const MxOperand b = {p.b + (t.e * P * p.N + n0) * 64, p.bs + (t.e * P * p.N + n0) * 4, p.N * 64, p.N * 4};
  void* out = out_at<false>(p.c, m0 * p.ldc + n0);
  if (split == 4)
    mx_tile<128, 128, false, false, 4>(smem, a, b, mr, (int)min(p.N - n0, (int64_t)128), (int)P, out, p.ldc, false);
  else
    mx_tile<128, 256, false, false, 4>(smem, a, b, mr, (int)min(p.N - n0, (int64_t)256), (int)P, out, p.ldc, false);
}

// The contract of the weight gradient's offsets: as ragged_ok, and multiples of 128.
__device__ __forceinline__ bool panels_ok(const int32_t* offs, int E, int64_t M) {
  bool bad = false;
  for (int i = threadIdx.x & 63; i < E; i += 64) bad = bad || (offs[i + 1] & 127) != 0;
  return ragged_ok(offs, E, M) && !__any(bad);
}

// Weight gradient: one grid of output tiles per expert, experts with the most rows first.
template <int BM, int BN, bool A8, bool F32, int S, int OCC>
__global__ __launch_bounds__(256, OCC) void grouped_mx_dw_kernel(GroupedMxParams p, int row_tiles, int col_tiles) {
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

// ------------------------------------------------------------------ few rows

// Forward where experts have few rows (serving): bound by the weights' bytes, each read once. A block owns 32 columns of one
// expert and up to 32 of its rows; its eight wavefronts share the panels out and add up in LDS in index order. Codes go from memory
// straight to the registers of v_mfma_scale_f32_16x16x128_f8f6f4, whose lane l = r + 16 g holds row r's codes [32 g, 32 g + 32) and
// their scale: 16 rows of a panel are one contiguous kilobyte, one load. (E4M3: codes [16 g, 16 g + 16) and 64 further.)
constexpr int FR = 32, FC = 32, FW = 8;  // rows, columns, wavefronts of a block
typedef float f32x4 __attribute__((ext_vector_type(4)));

template <bool A8>
__device__ __forceinline__ void few_rows(float* red, const MxOperand& a, const MxOperand& b, int mr, int nc, int P) {
  constexpr int U = 2, MT = FR / 16, NT = FC / 16;  // panels in flight
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r16 = lane & 15, g = lane >> 4;
  const int each_wave = (P + FW - 1) / FW, p0 = wave * each_wave, p1 = min(P, p0 + each_wave);
  const uint8_t *aq[MT], *as[MT], *bq[NT], *bs[NT];  // (rows past the end: the last one, not stored)
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = min(16 * i + r16, mr - 1);
    aq[i] = a.q + r * 64 + g * 16;
    as[i] = a.s + r * 4;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int r = min(16 * j + r16, nc - 1);
    bq[j] = b.q + r * 64 + g * 16;
    bs[j] = b.s + r * 4;
  }
  const bool both = mr > 16;
  f32x4 acc[MT][NT] = {};
  for (int p = p0; p < p1; p += U) {
    u32x4_t fb[U][NT], fa[U][MT][A8 ? 2 : 1];
    uint32_t sb[U][NT], sa[U][MT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t k = min(p + u, p1 - 1);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        fb[u][j] = *reinterpret_cast<const u32x4_t*>(bq[j] + k * b.panel);
        sb[u][j] = *reinterpret_cast<const uint32_t*>(bs[j] + k * b.plane);
      }
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (i && !both) continue;
#pragma unroll
        for (int h = 0; h < (A8 ? 2 : 1); ++h)
          fa[u][i][h] = *reinterpret_cast<const u32x4_t*>(aq[i] + (A8 ? 2 * k + h : k) * a.panel);
        sa[u][i] = *reinterpret_cast<const uint32_t*>(as[i] + k * a.plane);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (p + u >= p1) break;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        if (i && !both) continue;
        i32x8 codes = {};
#pragma unroll
        for (int q = 0; q < (A8 ? 8 : 4); ++q) codes[q] = (int)fa[u][i][q / 4][q % 4];
#pragma unroll
        for (int h = 0; h < (A8 ? 2 : 1); ++h) {
          i32x8 va = codes;
#pragma unroll
          for (int q = 0; A8 && q < 8; ++q) va[q] = h ? codes[q] ^ large_codes(codes[q]) : large_codes(codes[q]);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            i32x8 vb = {};
#pragma unroll
            for (int q = 0; q < 4; ++q) vb[q] = (int)fb[u][j][q];
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, acc[i][j], A8 ? 0 : 4, 4, 0, (int)(sa[u][i] >> (8 * g)),
                                                                         0, (int)(sb[u][j] >> (8 * g)));
          }
        }
      }
    }
  }
  // accumulator: lane l holds column l % 16 and rows 4 (l / 16) + q of a 16 x 16 block
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) red[(wave * FR + i * 16 + 4 * g + q) * (FC + 1) + j * 16 + r16] = acc[i][j][q];
}

template <bool A8>
__global__ __launch_bounds__(64 * FW, 2) void grouped_mx_few_rows_kernel(GroupedMxParams p, int col_tiles) {
  __shared__ float red[FW * FR * (FC + 1)];
  const RowTiles rt = count_row_tiles(p.offs, p.E, p.M, FR);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) *p.status = rt.ok ? 0 : 1;
  if (!rt.ok) return;
  const RowTile r = find_row_tile(rt, p.offs, p.E, FR, (int)(blockIdx.x / (uint32_t)col_tiles));
  if (r.e < 0) return;
  const int64_t n0 = (int64_t)(blockIdx.x % (uint32_t)col_tiles) * FC, P = (p.K + 127) >> 7;
  const int mr = r.m1 - r.m0, nc = (int)min(p.N - n0, (int64_t)FC);
  const MxOperand a = {p.a + (int64_t)r.m0 * 64, p.as + (int64_t)r.m0 * 4, p.M * 64, p.M * 4};
  const MxOperand b = {p.b + (r.e * P * p.N + n0) * 64, p.bs + (r.e * P * p.N + n0) * 4, p.N * 64, p.N * 4};
  few_rows<A8>(red, a, b, mr, nc, (int)P);
  __syncthreads();
  for (int i = threadIdx.x; i < mr * FC; i += 64 * FW) {
    const int m = i / FC, n = i % FC;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < FW; ++k) v += red[(k * FR + m) * (FC + 1) + n];
    if (n < nc) {
      const int64_t o = (r.m0 + m) * p.ldc + n0 + n;
      if (p.out_f32)
        reinterpret_cast<float*>(p.c)[o] = v;
      else
        reinterpret_cast<uint16_t*>(p.c)[o] = (uint16_t)bf16_bits(v);
    }
  }
}

}  // namespace mxf

namespace {

using namespace mxf;

template <int BM, int BN, bool A8, bool F32, int S, int OCC>
hipError_t launch_tiles(bool wgrad, const GroupedMxParams& p, hipStream_t st) {
  if (wgrad) {
    const int64_t rt = (p.N + BM - 1) / BM, ct = (p.K + BN - 1) / BN;
    hipLaunchKernelGGL((grouped_mx_dw_kernel<BM, BN, A8, F32, S, OCC>), dim3((unsigned)(p.E * rt * ct)), dim3(256), 0, st, p,
                       (int)rt, (int)ct);
    return hipGetLastError();
  }
  const int64_t ct = (p.N + BN - 1) / BN;
  int64_t rt = p.M / BM + (p.E < p.M ? p.E : p.M);  // every expert may end inside a tile
  if (rt == 0) rt = 1;                              // (one block looks at the offsets)
  hipLaunchKernelGGL((grouped_mx_rows_kernel<BM, BN, A8, F32, S, OCC>), dim3((unsigned)(rt * ct)), dim3(256), 0, st, p, (int)ct);
  return hipGetLastError();
}
template <bool A8, bool F32>
hipError_t launch(bool wgrad, const GroupedMxParams& p, int ncu, hipStream_t st) {
  const int64_t met = p.E < p.M ? p.E : p.M;  // experts that can have rows, each of which may end inside a tile
  // Few rows where even 128 x 128 tiles would leave a quarter of the chip idle: a tile's wavefronts walk the whole contraction, these
  // share it (us, in tiles): one row 4096 x 4096 4.0, 10.1; 4 experts of 4096 x 4096, 8 rows each 8.4, 10.6; one expert of 1024
  // x 8192, 200 rows 7.3, 17.1; 32 experts of 300 x 7168, 3 rows each 10.8, 15.5. With more blocks a strip's own cost weighs more: 16
  // experts of 2816 x 2048, 32 rows each 13.8, 12.2; 256 experts, 1 row each 212, 161.
  // E4M3 rows, whose instructions cost twice as much, share a long contraction out further (us, in tiles): 16 experts of 2816 x 2048, 3
  // rows each 12.6, 14.4, 32 rows each 18.0, 14.6; 256 rows of 4096 x 4096 16.3, 26.7, of 8192 x 8192 58, 44; and with few rows to an
  // expert still further: 64 experts, 3 rows each 45.8, 67, 16 rows each 68.7, 68.4; 2048 x 1408, 4 rows each 28.5, 32.2, of 1024
  // x 512 11.6, 10.5; but 256 experts of 2048 x 1408 with 2 rows each 157, 81, as blocks without rows cost too.
  const int64_t fct = (p.N + FC - 1) / FC, frt = p.M / FR + met, fs = frt * ((p.N + 127) / 128);
  if (!wgrad && (fs <= 3 * ncu / 4 || (A8 && p.K > 1024 && (fs <= 7 * ncu / 4 || (p.M <= 8 * met && fs <= 8 * ncu))))) {
    hipLaunchKernelGGL(grouped_mx_few_rows_kernel<A8>, dim3((unsigned)(frt ? frt * fct : 1)), dim3(64 * FW), 0, st, p, (int)fct);
    return hipGetLastError();
  }
  // One block per compute unit on a list of 256 x 256 tiles where the lists or the contractions are long (us, with 128 x 256 tiles, two
  // blocks to a compute unit): 24576 x 2816 x 2048 of 16 experts 86, 90; 8192^3 232, 259; 8192 rows of 8 experts, 2048 x 7168
  // 71, 80; two experts, 3000 x 3200 x 8192 49, 54; but 8192 x 2816 x 2048 36, 32 and 24576 x 2048 x 1408 59, 56.
  if constexpr (!A8 && !F32) {
    const int64_t ct = (p.N + 255) / 256, tiles = (2 * (p.M / 256) + met) * ct / 2;
    const bool rows16 = p.N % 8 == 0 && p.ldc % 8 == 0 && ((uintptr_t)p.c & 15) == 0 && p.ldc < (1 << 21);
    const bool lists = ncu % 8 == 0 && (p.M / 256 + p.E) * ct <= (int64_t)(kStreamTiles - 1) * ncu;
    if (!wgrad && rows16 && lists && ((p.K > 7 * 128 && tiles >= 4 * ncu) || (p.K >= 4096 && 2 * tiles >= ncu))) {
      const auto kernel = p.K > 15 * 128 ? grouped_mx_stream_kernel<16> : grouped_mx_stream_kernel<8>;
      hipLaunchKernelGGL(kernel, dim3(ncu), dim3(256), 0, st, p, (int)ct);
      return hipGetLastError();
    }
  }
  // 128 x 256 tiles where 128 x 128 ones, two to a compute unit, would take a second round (us, with those): 2048 x 2048 x 2048 12.0,
  // 9.1; 4096 x 2048 x 2048 14.5, 14.4; 2048 rows of 8 experts, 2816 x 2048 13.0, 14.0; 4096^2 x 2048 22.9, 25.9.
  const int64_t strips = ((wgrad ? p.K : p.N) + 127) / 128, tiles = (wgrad ? p.E * ((p.N + 127) / 128) : p.M / 128 + met) * strips;
  if (tiles > 2 * ncu) return launch_tiles<128, 256, A8, F32, A8 ? 2 : 3, 2>(wgrad, p, st);
  // (E2M1: a ring of three stages leaves room for a third block: 64 experts of 2816 x 2048, 192 rows 39.7 against 40.9 us, 256 of
  // 2048 x 1024, 512 rows 73, 84; one expert of 8192^2, 128 rows 19.7, 17.5)
  return launch_tiles<128, 128, A8, F32, 3, A8 ? 2 : 3>(wgrad, p, st);
}

}  // namespace

hipError_t mxf_launch_grouped_mx(bool wgrad, const GroupedMxParams& p, bool a8, int ncu, hipStream_t st) {
  if (a8) return p.out_f32 ? launch<true, true>(wgrad, p, ncu, st) : launch<true, false>(wgrad, p, ncu, st);
  return p.out_f32 ? launch<false, true>(wgrad, p, ncu, st) : launch<false, false>(wgrad, p, ncu, st);
}
