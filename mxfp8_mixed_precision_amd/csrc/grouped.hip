// Expert products in BF16 over ragged row segments: expert e owns rows [offs[e], offs[e+1]) of any
// count, with no padding between experts.
//
//   OP 0   y[r, n] = sum_k x[r, k] w[e, n, k]
//   OP 1   dx[r, k] = sum_n dy[r, n] w[e, n, k]
//   OP 2   dw[e, n, k] = sum_{r of e} dy[r, n] x[r, k]        (x BF16, or MXFP8 codes and scales)
//
// BF16 operands, FP32 accumulation in the matrix cores, one rounding at the store. A code of the
// MXFP8 checkpoint has four significant bits, so its product with the scale is a BF16 number and
// enters the same matrix instruction unrounded, for scales from 2^-117 on: below (groups whose largest value is under
// 2^-109) the smallest codes leave BF16's normal range.
//
// Measured, 16 experts ragged, 24576 x 2816 x 2048: forward 262 us (1080 TFLOP/s), weight gradient 274 into BF16, 295
// into FP32; 8 experts ragged, 16384 rows, input gradient from 7168 to 2048 columns 444 (1083), even 398; 8192^3: 781,
// 825, 850. The matrix cores are busy 57% of the first (53% input gradient, 47% weight gradient): a tile has a compute
// unit to itself, so nothing multiplies during its first loads and its stores, and a long main loop (8192^3: 71-75%) waits
// for operands a tenth of its time (732 us without any loads). Rows without 16-byte alignment take about twice the time.
#include <type_traits>

#include "chunk.h"
#include "kernels.h"
#include "mx_device.h"

namespace mxf {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// The contract of offs (offs[0] = 0, non-decreasing, offs[E] <= M), the number of row tiles of all
// experts, and the expert and rows of row tile t. Whole wavefronts, the same answer in every lane:
// lane i looks at expert 64 j + i, tiles are counted in expert order. Offsets that break the contract may
// leave any counts behind; the caller stops on ok = false before it uses them.
struct RowTile {
  int e;       // -1: past the last tile
  int m0, m1;  // rows of the tile
};
struct RowTiles {
  bool ok;
  int tiles;
  int lo, hi, first, n;  // of the lane's last expert looked at (E <= 64: its only one)
};
__device__ __forceinline__ void scan_experts(const int32_t* offs, int E, int bm, int base, RowTiles& r) {
  const int lane = threadIdx.x & 63, i = base + lane;
  r.lo = i < E ? offs[i] : 0;
  r.hi = i < E ? offs[i + 1] : 0;
  r.n = r.hi > r.lo ? (int)(((uint32_t)r.hi - (uint32_t)r.lo + bm - 1) / bm) : 0;
  int pre = r.n;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(pre, o);
    if (lane >= o) pre += v;
  }
  r.first = r.tiles + pre - r.n;
  r.tiles += __builtin_amdgcn_readlane(pre, 63);
}
__device__ __forceinline__ RowTiles count_row_tiles(const int32_t* offs, int E, int64_t M, int bm) {
  RowTiles r = {true, 0, 0, 0, 0, 0};
  bool bad = false;
  for (int base = 0; base < E; base += 64) {
    scan_experts(offs, E, bm, base, r);
    bad = bad || r.lo > r.hi || r.lo < 0 || r.hi > M || (base == 0 && (threadIdx.x & 63) == 0 && r.lo != 0);
  }
  r.ok = !__any(bad);
  return r;
}
__device__ __forceinline__ RowTile find_row_tile(RowTiles r, const int32_t* offs, int E, int bm, int t) {
  if (E > 64) r.tiles = 0;
  for (int base = 0; base < E; base += 64) {
    if (E > 64) scan_experts(offs, E, bm, base, r);
    const uint64_t hit = __ballot(r.n > 0 && t >= r.first && t < r.first + r.n);
    if (hit) {
      const int l = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)hit) - 1);
      const int m0 = __builtin_amdgcn_readlane(r.lo, l) + (t - __builtin_amdgcn_readlane(r.first, l)) * bm;
      return {base + l, m0, min(m0 + bm, __builtin_amdgcn_readlane(r.hi, l))};
    }
  }
  return {-1, 0, 0};
}

// The contract alone.
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

// ------------------------------------------------------------------ pipelined tiles

// Block tile BM x BN, four wavefronts in a 2 x 2 grid, each owning a (BM/2) x (BN/2) tile of 32 x 32
// matrix-core fragments (256 x 256: all 256 accumulators of a lane in AGPRs, one block per CU).
//
// The contraction advances 64 at a time (128-byte rows: whole cache lines). A stage's share of one
// operand is a unit; five units fill the LDS, which direct global->LDS loads of 1 KB fill in the order
// A0 B0 A1 B1 A2 B2 ... A stage is four 16-deep quarters; the matrix instructions of one run beside the
// LDS reads of the next. Before the last quarter one wait and one barrier make the next stage visible and
// this stage's two units free: B of stage + 2 and A of stage + 3 follow into them, one load per four matrix
// instructions over the next four quarters, so the vector-memory pipe never takes a burst. Loads past
// the last stage ask for no element (below), which keeps every stage the same.
//
// An operand is stored in LDS as it lies in memory:
//   contraction-contiguous (x and dy of OP 0, 1; w of OP 0): rows of 64 elements (128 bytes), fragments
//     read with ds_read_b128. 16-byte chunk c of row r sits at c ^ ((r / 2) % 8): 16 consecutive rows
//     at one chunk index then hit 16 different 16-byte bank groups.
//   contraction-slow (w of OP 1, both of OP 2): rows of BM or BN elements, one per contraction index,
//     fragments read with the transposing ds_read_b64_tr_b16, which gives each of 16 lanes one
//     column of four rows. Chunk c of row k sits at c ^ 4 (k % 4): the four rows of a read, 32 bytes
//     each, and the two 16-column halves of a fragment hit eight different 32-byte bank groups.
//
// Operands whose rows are not 16-byte aligned, and the MXFP8 codes of OP 2, cannot go to LDS as they are:
// they are fetched into registers two quarters ahead (16 bytes per load, at any alignment; element by
// element at a ragged end), decoded if they are codes, and written to the same places of the same units.
//
// Bounds: the direct loads are buffer loads against a descriptor that ends at 2 GB from the tile's first
// element; a lane whose row or column does not exist asks for an offset past it and gets zeros in
// LDS. So ragged segment ends, odd tile ends and the last contraction stage need no other path, rows of
// another expert are never read, and 64-bit offsets live in the descriptor's base.
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr uint32_t kNoElement = 0x80000000u;  // = the descriptors' size

__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)v) |
         ((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32);
}
// 16 bytes per lane into LDS [lds, lds + 1024) in lane order. The loads have no destination registers;
// the kernel waits for them with vmcnt. (One wait state between a write of M0 and its use.)
__device__ __forceinline__ void buffer_to_lds(i32x4 rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
// One operand of a tile: R rows or columns of the output, contraction-contiguous (KC) or not.
template <bool KC, int R>
struct Operand {
  static constexpr int NLOAD = R / 32;         // 1 KB loads per wavefront and stage
  static constexpr int CPR = R / 8;            // contraction-slow: 16-byte chunks per row
  static constexpr int RPL = 64 / CPR;         // and rows per load
  static constexpr int NR = KC ? 1 : 2;        // LDS reads per fragment
  i32x4 rsrc;         // from the first element of the stage to load next
  uint64_t step;      // bytes between stages
  uint32_t voff[NLOAD];
  uint32_t k_lane;    // contraction index of the lane's first element: KC: of even loads, else of load 0
  uint32_t rd[4];     // LDS read addresses in slot 0: KC: per quarter, else per fragment

  // origin: the tile's first element; ld: elements between rows; `valid`: rows or columns that exist; w0:
  // this wavefront's first row or column; lds: the operand's place in slot 0
  __device__ __forceinline__ void init(const uint16_t* origin, int64_t ld, int valid, int wid, int w0, uint32_t lds) {
    const int l = threadIdx.x & 63;
    const uint64_t base = uniform64((uint64_t)origin);
    rsrc = (i32x4){(int)(uint32_t)base, (int)(uint32_t)(base >> 32), (int)kNoElement, 0x00020000};
    step = KC ? 128 : (uint64_t)ld * 128;
    const uint32_t ldb = (uint32_t)ld * 2;
#pragma unroll
    for (int i = 0; i < NLOAD; ++i) {
      const int q = wid * NLOAD + i;
      if constexpr (KC) {
        const int r = 8 * q + (l >> 3), c = (l & 7) ^ ((r >> 1) & 7);
        voff[i] = r < valid ? (uint32_t)r * ldb + c * 16 : kNoElement;
      } else {
        const int k = RPL * q + l / CPR, c = (l % CPR) ^ (4 * (k & 3));
        voff[i] = c * 8 < valid ? (uint32_t)k * ldb + c * 16 : kNoElement;
      }
    }
    k_lane = KC ? ((l & 7) ^ ((l >> 4) & 7)) * 8 : RPL * NLOAD * wid + l / CPR;
    init_reads(w0, lds);
  }
  __device__ __forceinline__ void init_reads(int w0, uint32_t lds) {
    const int l = threadIdx.x & 63;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (KC) {
        const int r = w0 + (l & 31), c = (2 * j + (l >> 5)) ^ ((r >> 1) & 7);
        rd[j] = lds + r * 128 + c * 16;
      } else {
        const int k = 8 * (l >> 5) + ((l & 15) >> 2), c32 = (w0 >> 4) + 2 * j + ((l >> 4) & 1);
        rd[j] = lds + k * (R * 2) + ((c32 ^ (2 * (k & 3))) << 5) + (l & 3) * 8;
      }
    }
  }
  // Load i of the stage at `rsrc`, of which `left` contraction indexes exist, into LDS.
  __device__ __forceinline__ void load(int i, int left, uint32_t lds) const {
    // odd loads of a contraction-contiguous operand start four rows further, which flips chunk bit 2
    const int k = KC ? (int)(k_lane ^ (32 * (i & 1))) : (int)k_lane + RPL * i;
    buffer_to_lds(rsrc, k < left ? voff[i] : kNoElement, lds + i * 1024);
  }
  __device__ __forceinline__ void advance() {
    const uint64_t b = ((uint64_t)(uint32_t)rsrc[1] << 32 | (uint32_t)rsrc[0]) + step;  // (48-bit addresses: no stride bits)
    rsrc[0] = (int)(uint32_t)b;
    rsrc[1] = (int)(uint32_t)(b >> 32);
  }
  // Part h of fragment i in quarter s.
  __device__ __forceinline__ void read(u32x4_t& f, int i, int h, int s, uint32_t slot) const {
    if constexpr (KC) {
      f = lds16_at(rd[s] + slot)[i * 256];
    } else {
      const s16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
          (lds_s16x4*)(uintptr_t)(rd[i] + slot + (16 * s + 4 * h) * (R * 2)));
      const uint2 u = __builtin_bit_cast(uint2, v);
      f[2 * h] = u.x;
      f[2 * h + 1] = u.y;
    }
  }
};

// 16 bytes from any address.
__device__ __forceinline__ u32x4_t load16_any(const void* p) {
  u32x4_t v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ uint32_t bf16_of_fp8(uint32_t w, bool hi, float scale) {
  return __builtin_bit_cast(uint32_t, hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, true)
                                         : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, scale, false));
}

// An operand that passes through registers: BF16 at any alignment, or (X8, contraction-slow) codes with
// their scales. LDS layout and reads are Operand's.
//
// A fetch is 16 bytes of a row. The one in which a row ends is loaded from its end backwards (into elements
// that its neighbour holds) and shifted when it is used, and a lane with nothing to fetch loads the tile's
// first piece and drops it: no branch between the loads. Rows shorter than a fetch go element by element.
template <bool KC, int R, bool X8>
struct StagedOperand : Operand<KC, R> {
  using Base = Operand<KC, R>;
  static constexpr int PER = X8 ? 16 : 8;            // elements per fetch
  static constexpr int BITS = 128 / PER;             // and of an element
  static constexpr int NF = R * 64 / PER / 256;      // fetches per thread and stage
  static constexpr int PPR = (KC ? 64 : R) / PER;    // fetches per row
  static constexpr int RPT = 256 / PPR;              // rows per round of the block's fetches
  const uint8_t* src;   // the tile's first element of the stage to fetch next
  const uint8_t* scl;   // X8: its row's first scale of this tile
  int64_t ldb, lds_;    // bytes between rows, scales between rows
  int valid;
  bool tiny;            // rows of fewer than PER elements
  u32x4_t v[NF];
  uint32_t sc[X8 ? NF : 1];
  uint32_t have, shift;  // of the fetch in registers: which pieces exist, bits to drop

  __device__ __forceinline__ void init(const void* origin, const uint8_t* scales, int64_t ld, int64_t ld_scales,
                                       int64_t row_length, int valid_, int w0, uint32_t lds) {
    Base::init_reads(w0, lds);
    src = reinterpret_cast<const uint8_t*>(origin);
    scl = scales;
    ldb = X8 ? ld : 2 * ld;
    lds_ = ld_scales;
    valid = valid_;
    tiny = row_length < PER;
  }
  __device__ __forceinline__ void fetch(int left) {
    const int r0 = (int)threadIdx.x / PPR, c = (int)threadIdx.x % PPR * PER;
    const int rows = KC ? valid : left, width = KC ? left : valid;  // that exist
    have = 0;
    shift = 0;
    if (tiny) {
#pragma unroll
      for (int t = 0; t < NF; ++t) {
        const int r = r0 + t * RPT;
        const uint8_t* p = src + r * ldb;
        v[t] = (u32x4_t){0, 0, 0, 0};
        if (X8) sc[t] = r < rows && c < width ? scl[r * lds_ + (c >> 5)] : 0u;
#pragma unroll 1
        for (int e = 0; e < PER; ++e) {  // the next element enters at the top
          uint32_t x = 0;
          if (r < rows && c + e < width) x = X8 ? p[c + e] : reinterpret_cast<const uint16_t*>(p)[c + e];
          v[t] = shr128(v[t], BITS);
          v[t][3] |= x << (32 - BITS);
        }
      }
      have = (1u << NF) - 1;
    } else if (rows > 0 && width > 0) {
      const int cc = c < width ? c : 0, back = max(0, PER - (width - cc));
      shift = (uint32_t)(back * BITS);
      const uint8_t* p = src + (X8 ? cc - back : 2 * (cc - back));
#pragma unroll
      for (int t = 0; t < NF; ++t) {
        const int r = r0 + t * RPT, rr = r < rows ? r : 0;
        v[t] = load16_any(p + rr * ldb);
        if (X8) sc[t] = scl[rr * lds_ + (cc >> 5)];
        have |= (r < rows && c < width ? 1u : 0u) << t;
      }
    }
    src += KC ? 128 : 64 * ldb;
    if (X8) scl += 64 * lds_;
  }
  __device__ __forceinline__ void put(uint8_t* unit) const {
    const int r0 = (int)threadIdx.x / PPR, c = (int)threadIdx.x % PPR * (PER / 8);  // row, 16-byte chunk
    const bool cut = __any(shift != 0);
#pragma unroll
    for (int t = 0; t < NF; ++t) {
      const int r = r0 + t * RPT;
      u32x4_t x = v[t];
      if (cut) x = shr128(x, shift);
      const bool in = (have >> t) & 1;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = in ? x[i] : 0u;
      uint8_t* row = unit + r * (KC ? 128 : R * 2);
      if constexpr (X8) {
        const float s = e8m0_value(in ? sc[t] : 0u);
        u32x4_t lo, hi;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          lo[2 * i] = bf16_of_fp8(x[i], false, s);
          lo[2 * i + 1] = bf16_of_fp8(x[i], true, s);
          hi[2 * i] = bf16_of_fp8(x[2 + i], false, s);
          hi[2 * i + 1] = bf16_of_fp8(x[2 + i], true, s);
        }
        *reinterpret_cast<u32x4_t*>(row + ((c ^ (4 * (r & 3))) << 4)) = lo;
        *reinterpret_cast<u32x4_t*>(row + (((c + 1) ^ (4 * (r & 3))) << 4)) = hi;
      } else {
        *reinterpret_cast<u32x4_t*>(row + ((c ^ (KC ? (r >> 1) & 7 : 4 * (r & 3))) << 4)) = x;
      }
    }
  }
};

// Codes whose rows are multiples of 16 bytes: the same through bounded buffer loads (codes past the stage's
// rows or the tile's columns read as zero), with so few instructions that a piece fits between matrix
// instructions: piece by piece, all in quarter 0: a piece of the next stage is decoded and the same piece of the stage after it fetched
// into its registers. These fetches come before A's loads of quarter 1, so the stage's wait for all but those loads
// covers them too. Weight gradient of 16 experts,
// 24576 x 2816 x 2048: 298 us against 370 with the general fetch between the quarters (274 from BF16).
template <int R>
struct CodesOperand : Operand<false, R> {
  using Base = Operand<false, R>;
  static constexpr int NF = R * 64 / 16 / 256;  // pieces (16 codes) per thread and stage
  static constexpr int PPR = R / 16, RPT = 256 / PPR;
  uint64_t src, scl;     // the tile's first code and scale of the stage to fetch next
  uint32_t ldb, lds_;    // bytes between rows, scales between rows
  uint32_t voff, soff;   // the lane's first piece: offsets from src and scl
  int r0, left;
  uint32_t put0;         // its place in a unit
  u32x4_t v[NF];
  uint32_t sc[NF];

  __device__ __forceinline__ void init(const void* origin, const uint8_t* scales, int64_t ld, int64_t ld_scales, int64_t,
                                       int valid, int w0, uint32_t lds) {
    Base::init_reads(w0, lds);
    src = uniform64((uint64_t)origin);
    scl = uniform64((uint64_t)scales);
    ldb = (uint32_t)ld;
    lds_ = (uint32_t)ld_scales;
    const int tid = (int)threadIdx.x, c = tid % PPR;
    r0 = tid / PPR;
    const bool in = c * 16 < valid;
    voff = in ? (uint32_t)r0 * ldb + c * 16 : kNoElement;
    soff = in ? (uint32_t)r0 * lds_ + (c >> 1) : kNoElement;
    // a lane's two 16-byte halves go in two writes; lanes 4-11 of 16 write the upper half first, so that 8 and 16
    // neighbouring lanes of a write hit different bank groups
    put0 = r0 * (R * 2) + (((2 * c + upper()) ^ (4 * (r0 & 3))) << 4);
  }
  static __device__ __forceinline__ int upper() { return ((threadIdx.x >> 2) ^ (threadIdx.x >> 3)) & 1; }
  __device__ __forceinline__ void begin(int l) { left = l; }
  __device__ __forceinline__ void piece(int t) {
    const __amdgpu_buffer_rsrc_t q = __builtin_amdgcn_make_buffer_rsrc((void*)src, 0, kNoElement, 0x00020000);
    const __amdgpu_buffer_rsrc_t s = __builtin_amdgcn_make_buffer_rsrc((void*)scl, 0, kNoElement, 0x00020000);
    const bool in = r0 + t * RPT < left;
    v[t] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(q, in ? voff + t * RPT * ldb : kNoElement, 0, 0));
    sc[t] = __builtin_amdgcn_raw_buffer_load_b8(s, in ? soff + t * RPT * lds_ : kNoElement, 0, 0);
  }
  __device__ __forceinline__ void end() {
    src += 64 * (uint64_t)ldb;
    scl += 64 * (uint64_t)lds_;
  }
  __device__ __forceinline__ void fetch(int l) {
    begin(l);
#pragma unroll
    for (int t = 0; t < NF; ++t) piece(t);
    end();
  }
  __device__ __forceinline__ void put(uint8_t* unit, int t) const {
    const float s = e8m0_value(sc[t]);
    const bool up = upper();
    u32x4_t lo, hi, a, b;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      lo[2 * i] = bf16_of_fp8(v[t][i], false, s);
      lo[2 * i + 1] = bf16_of_fp8(v[t][i], true, s);
      hi[2 * i] = bf16_of_fp8(v[t][2 + i], false, s);
      hi[2 * i + 1] = bf16_of_fp8(v[t][2 + i], true, s);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = up ? hi[i] : lo[i];
      b[i] = up ? lo[i] : hi[i];
    }
    // (RPT rows further r % 4 is the same)
    *reinterpret_cast<u32x4_t*>(unit + put0 + t * RPT * (R * 2)) = a;
    *reinterpret_cast<u32x4_t*>(unit + (put0 ^ 16) + t * RPT * (R * 2)) = b;
  }
  __device__ __forceinline__ void put(uint8_t* unit) const {
#pragma unroll
    for (int t = 0; t < NF; ++t) put(unit, t);
  }
};
// A codes operand's share of matrix instruction m of nm: a piece decoded into its unit, and the same piece
// of the next stage fetched into its registers (other operands have none).
template <class O>
__device__ __forceinline__ void next_piece(O&, uint8_t*, int, int) {}
template <int R>
__device__ __forceinline__ void next_piece(CodesOperand<R>& o, uint8_t* unit, int m, int nm) {
#pragma unroll
  for (int t = m * CodesOperand<R>::NF / nm; t < (m + 1) * CodesOperand<R>::NF / nm; ++t) {
    o.put(unit, t);
    o.piece(t);
  }
}

template <int BM, int BN, int UNITS>
struct TileSize {
  static constexpr int FM = BM / 64, FN = BN / 64;
  static constexpr int UNIT = (BM > BN ? BM : BN) * 128;  // bytes of an operand's stage
  static constexpr int PITCH16 = BN + 8, PITCH32 = BN + 4;  // epilogue staging rows (elements)
  static constexpr int EPI16 = BM * PITCH16 * 2, EPI32 = BM / 2 * PITCH32 * 4;
  static constexpr int max3(int a, int b, int c) { return a > b ? (a > c ? a : c) : (b > c ? b : c); }
  static constexpr int LDS = max3(UNITS * UNIT, EPI16, EPI32);
};

// 16 bytes past the caches' retention (outputs are not read again by this launch), or to any address.
template <bool ANY>
__device__ __forceinline__ void store16(void* p, uint4 v) {
  if constexpr (ANY)
    __builtin_memcpy(p, &v, 16);
  else
    store16_nt(p, v);
}

enum Feed { DIRECT, STAGED, STAGED_CODES, CODES };  // how an operand gets to LDS

// mr rows and nc columns of output at c_base; contraction length kc; a and b: the operands' first elements of
// the tile. RING: the pipeline above; otherwise two units and no lookahead: a stage is loaded, awaited and
// multiplied, and the CU's other blocks fill the waits.
template <int OP, int BM, int BN, bool F32, Feed FA, Feed FB, bool RING = true>
__device__ __forceinline__ void grouped_tile(const GroupedParams& p, uint8_t* smem, const uint16_t* a, const void* b,
                                             const uint8_t* b_scales, int64_t ldb, int64_t c_base, int mr, int nc,
                                             int kc) {
  using S = TileSize<BM, BN, RING ? 5 : 2>;
  constexpr int FM = S::FM, FN = S::FN;
  using OA = std::conditional_t<FA == DIRECT, Operand<OP != 2, BM>, StagedOperand<OP != 2, BM, false>>;
  using OB = std::conditional_t<
      FB == DIRECT, Operand<OP == 0, BN>,
      std::conditional_t<FB == CODES, CodesOperand<BN>, StagedOperand<OP == 0, BN, FB == STAGED_CODES>>>;
  constexpr bool SA = FA != DIRECT, SB = FB != DIRECT;
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int wid_u = __builtin_amdgcn_readfirstlane(wid);
  const int wm = wid >> 1, wn = wid & 1;
  const uint32_t lds0 = lds_addr(smem);
  OA oa;
  OB ob;
  if constexpr (SA)
    oa.init(a, nullptr, p.lda, 0, OP == 0 ? p.K : p.N, mr, wm * (BM / 2), lds0);
  else
    oa.init(a, p.lda, mr, wid, wm * (BM / 2), lds0);
  if constexpr (SB)
    ob.init(b, b_scales, ldb, (p.K + 31) / 32, p.K, nc, wn * (BN / 2), lds0);
  else
    ob.init(reinterpret_cast<const uint16_t*>(b), ldb, nc, wid, wn * (BN / 2), lds0);
  constexpr int NLA = SA ? 0 : OA::NLOAD, NLB = SB ? 0 : OB::NLOAD;  // direct loads of a unit per wavefront
  const uint32_t lds_a = lds0 + wid_u * NLA * 1024, lds_b = lds0 + wid_u * NLB * 1024;  // its part of unit 0
  const int KT = (kc + 63) >> 6;

  f32x16 acc[FM][FN];
  u32x4_t fa[2][FM], fb[2][FN];
  constexpr int NRA = FM * OA::NR, NR = NRA + FN * OB::NR;  // LDS reads of a quarter
  auto read = [&](int r, int s, int set, uint32_t ua, uint32_t ub) {
    if (r < NRA)
      oa.read(fa[set][r / OA::NR], r / OA::NR, r % OA::NR, s, ua);
    else
      ob.read(fb[set][(r - NRA) / OB::NR], (r - NRA) / OB::NR, (r - NRA) % OB::NR, s, ub);
  };
  // Matrix instructions of quarter s (register set s % 2), interleaved with the reads of the next quarter
  // (units ua, ub) and with half a unit of loads: quarter 3: B's first, 0: B's second, 1 and 2: A's halves.
  // The operands swap places, so a lane holds one output row and, in runs of four accumulators, four
  // neighbouring columns.
  auto quarter = [&](auto s_, uint32_t ua, uint32_t ub, int left, uint32_t ld, uint32_t nb) {
    constexpr int s = decltype(s_)::value, set = s & 1;
    constexpr int NM = FM * FN, NH = NM / 2, NQ = FB == CODES ? (s == 1 ? NLA : 0) : (s == 0 || s == 3 ? NLB : NLA) / 2;
    constexpr int L0 = (s == 0 || s == 2) ? NQ : 0;
#pragma unroll
    for (int m = 0; m < NM; ++m) {
      acc[m / FN][m % FN] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
          __builtin_bit_cast(bf16x8, fb[set][m % FN]), __builtin_bit_cast(bf16x8, fa[set][m / FN]), acc[m / FN][m % FN],
          0, 0, 0);
      if (m < NH) {
#pragma unroll
        for (int r = m * NR / NH; r < (m + 1) * NR / NH; ++r) read(r, (s + 1) & 3, 1 - set, ua, ub);
      }
#pragma unroll
      for (int i = L0 + m * NQ / NM; i < L0 + (m + 1) * NQ / NM; ++i) {
        if constexpr (s == 3 || s == 0) {
          if constexpr (!SB) ob.load(i, left, ld);
        } else {
          if constexpr (!SA) oa.load(i, left, ld);
        }
      }
      if (s == 0) next_piece(ob, smem + nb, m, NM);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  using Q0 = std::integral_constant<int, 0>;
  using Q1 = std::integral_constant<int, 1>;
  using Q2 = std::integral_constant<int, 2>;
  using Q3 = std::integral_constant<int, 3>;
  constexpr uint32_t U = S::UNIT;

  if (RING && KT > 0) {  // A0 B0 A1 and half of B1; of staged operands A0 and B0 into registers
    if constexpr (SA) {
      oa.fetch(kc);
    } else {
#pragma unroll
      for (int i = 0; i < NLA; ++i) oa.load(i, kc, lds_a);
      oa.advance();
    }
    if constexpr (SB) {
      ob.fetch(kc);
    } else {
#pragma unroll
      for (int i = 0; i < NLB; ++i) ob.load(i, kc, lds_b + U);
      ob.advance();
    }
    if constexpr (!SA) {
#pragma unroll
      for (int i = 0; i < NLA; ++i) oa.load(i, kc - 64, lds_a + 2 * U);
      oa.advance();
    }
    if constexpr (!SB) {
#pragma unroll
      for (int i = 0; i < NLB / 2; ++i) ob.load(i, kc - 64, lds_b + 3 * U);
    }
  }
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int q = 0; q < 16; ++q) acc[i][j][q] = 0.0f;
  if constexpr (!RING) {
#pragma unroll 1
    for (int left = kc; left > 0; left -= 64) {
#pragma unroll
      for (int i = 0; i < NLA; ++i) oa.load(i, left, lds_a);
      oa.advance();
      if constexpr (SB) {
        ob.fetch(left);
        ob.put(smem + U);
      } else {
#pragma unroll
        for (int i = 0; i < NLB; ++i) ob.load(i, left, lds_b + U);
        ob.advance();
      }
      wait_vmcnt<0>();
      __syncthreads();
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if (16 * s >= left) break;
#pragma unroll
        for (int r = 0; r < NR; ++r) read(r, s, 0, 0, U);
#pragma unroll
        for (int m = 0; m < FM * FN; ++m)
          acc[m / FN][m % FN] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
              __builtin_bit_cast(bf16x8, fb[0][m % FN]), __builtin_bit_cast(bf16x8, fa[0][m / FN]), acc[m / FN][m % FN],
              0, 0, 0);
      }
      if (left > 64) __syncthreads();  // all have read the units
    }
  }
  if (RING && KT > 0) {
    if constexpr (SA) oa.put(smem);
    if constexpr (SB) ob.put(smem + U);
    wait_vmcnt<NLA + NLB / 2>();  // stage 0 has landed
    __syncthreads();
    if constexpr (SA) oa.fetch(kc - 64);
    if constexpr (SB) ob.fetch(kc - 64);
#pragma unroll
    for (int r = 0; r < NR; ++r) read(r, 0, 0, 0, U);
    uint32_t ua = 0, ub = U;                          // units of stage kt
    uint32_t pa = lds_b + 3 * U, pb = lds_a + 4 * U;  // where B of stage kt + 1 and A of stage kt + 2 go
    int left = kc - 64;
#pragma unroll 1
    for (int kt = 0; kt < KT; ++kt) {
      const uint32_t na = ua >= 3 * U ? ua - 3 * U : ua + 2 * U;  // units of stage kt + 1
      const uint32_t nb = ub >= 3 * U ? ub - 3 * U : ub + 2 * U;
      if constexpr (FB == CODES) ob.begin(left - 64);  // stage kt + 2
      quarter(Q0(), ua, ub, left, pa, nb);
      if constexpr (FB == CODES) ob.end();
      if constexpr (SA) oa.put(smem + na);
      if constexpr (SB && FB != CODES) ob.put(smem + nb);
      if constexpr (!SB) ob.advance();
      left -= 64;
      quarter(Q1(), ua, ub, left, pb, 0);
      quarter(Q2(), ua, ub, left, pb, 0);
      if constexpr (!SA) oa.advance();
      wait_vmcnt<NLA>();  // all but A of stage kt + 2 has landed
      __syncthreads();    // for every wavefront, and none reads this stage's units any more
      if constexpr (SA) oa.fetch(left);  // stage kt + 2
      if constexpr (SB && FB != CODES) ob.fetch(left);
      pa = lds_b + ua;
      pb = lds_a + ub;
      ua = na;
      ub = nb;
      quarter(Q3(), ua, ub, left, pa, 0);
    }
    wait_vmcnt<0>();  // no load may still target LDS
  }
  __syncthreads();  // the slots become the epilogue's staging

  // Epilogue: the tile goes through LDS so that stores are 16-byte runs along output rows.
  constexpr bool ANY = SA || FB == STAGED;  // (the launcher stages operands where the output is unaligned too)
  const int r32 = lane & 31, g = lane >> 5;
  if constexpr (!F32) {
    uint16_t* cs = reinterpret_cast<uint16_t*>(smem);
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if constexpr (RING) asm volatile("" : "+a"(acc[i][j]));  // fragments leave the AGPRs one at a time
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint2*>(cs + (wm * (BM / 2) + i * 32 + r32) * S::PITCH16 + wn * (BN / 2) + j * 32 + 8 * c + 4 * g) =
              make_uint2(bf16x2_bits(acc[i][j][4 * c], acc[i][j][4 * c + 1]),
                         bf16x2_bits(acc[i][j][4 * c + 2], acc[i][j][4 * c + 3]));
      }
    __syncthreads();
    constexpr int CPR = BN / 8;
#pragma unroll 2
    for (int t = tid; t < BM * CPR; t += 256) {
      const int r = t / CPR, c = t % CPR * 8;
      if (r < mr && c < nc) {
        uint16_t* o = reinterpret_cast<uint16_t*>(p.c) + c_base + (int64_t)r * p.ldc + c;
        if (!ANY || c + 8 <= nc) {
          store16<ANY>(o, *reinterpret_cast<const uint4*>(cs + r * S::PITCH16 + c));
        } else {
          for (int e = 0; c + e < nc; ++e) o[e] = cs[r * S::PITCH16 + c + e];
        }
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
        for (int j = 0; j < FN; ++j) {
          if constexpr (RING) asm volatile("" : "+a"(acc[i][j]));
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<float4*>(cs + (i * 32 + r32) * S::PITCH32 + wn * (BN / 2) + j * 32 + 8 * c + 4 * g) =
                make_float4(acc[i][j][4 * c], acc[i][j][4 * c + 1], acc[i][j][4 * c + 2], acc[i][j][4 * c + 3]);
        }
    }
    __syncthreads();
    constexpr int CPR = BN / 4;
#pragma unroll 2
    for (int t = tid; t < BM / 2 * CPR; t += 256) {
      const int r = t / CPR, c = t % CPR * 4, row = half * (BM / 2) + r;
      if (row < mr && c < nc) {
        float4 v = *reinterpret_cast<const float4*>(cs + r * S::PITCH32 + c);
        float* o = reinterpret_cast<float*>(p.c) + c_base + (int64_t)row * p.ldc + c;
        if (!ANY || c + 4 <= nc) {
          if (p.accum) {
            const float4 u = __builtin_bit_cast(float4, load16_any(o));
            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
          }
          store16<ANY>(o, __builtin_bit_cast(uint4, v));
        } else {
          const float* s = cs + r * S::PITCH32 + c;
          for (int e = 0; c + e < nc; ++e) o[e] = p.accum ? o[e] + s[e] : s[e];
        }
      }
    }
  }
}

// Position of block b of n (a contiguous run of positions per XCD: blocks go to the 8 XCDs in turn).
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t n) {
  const uint32_t q = n / 8, r = n % 8, x = b % 8;
  return (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + b / 8;
}

// OP 0 and 1: row tiles in groups of GM, all column tiles of a group before the next, so that the tiles
// in flight on an XCD share rows of x and columns of w in its L2.
//
// Of T tiles on C compute units the last T mod C would leave most of the chip idle for a whole tile's time:
// they are split into four quarters, or two halves of the rows, where that many fit the chip at once. Their
// blocks come first (lowest ids). A tile whose expert ends within its first 128 rows runs as a half.
template <int OP, int BM, int BN, bool F32, Feed F>
__global__ __launch_bounds__(256, BM == 256 ? 1 : 2) void grouped_rows_kernel(GroupedParams p, int col_tiles, int ncu) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[TileSize<BM, BN, 5>::LDS];
  const RowTiles rt = count_row_tiles(p.offs, p.E, p.M, BM);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) *p.status = rt.ok ? 0 : 1;
  if (!rt.ok) return;
  const uint32_t total = (uint32_t)rt.tiles * (uint32_t)col_tiles;
  uint32_t pos, part = 0, split = 1;
  if constexpr (BM == 256) {
    const uint32_t rem = total % (uint32_t)ncu, full = total - rem;
    split = 4 * rem <= (uint32_t)ncu ? 4 : 2 * rem <= (uint32_t)ncu ? 2 : 1;
    const uint32_t first = split == 1 ? 0 : (rem * split + 7) & ~7u;  // (a multiple of 8 keeps block id % 8 the XCD)
    if (blockIdx.x < first) {
      if (blockIdx.x >= rem * split) return;
      pos = full + blockIdx.x / split;
      part = blockIdx.x % split;
    } else {
      const uint32_t n = split == 1 ? total : full;
      if (blockIdx.x - first >= n) return;
      pos = xcd_run(blockIdx.x - first, n);
      split = 1;
    }
  } else {
    if (blockIdx.x >= total) return;
    pos = xcd_run(blockIdx.x, total);
  }
  constexpr uint32_t GM = 4;
  const uint32_t per = GM * (uint32_t)col_tiles, grp = pos / per, in = pos - grp * per;
  const uint32_t rows = min(GM, (uint32_t)rt.tiles - grp * GM);
  const RowTile r = find_row_tile(rt, p.offs, p.E, BM, (int)(grp * GM + in % rows));
  int64_t n0 = (int64_t)(in / rows) * BN;
  const int64_t on = OP == 0 ? p.N : p.K, kc = OP == 0 ? p.K : p.N;
  const uint16_t* w = p.b + (int64_t)r.e * p.N * p.K;
  int m0 = r.m0, mr = r.m1 - r.m0;
  if constexpr (BM == 256) {
    if (split > 1) {
      m0 += (int)(part >> (split == 4)) * 128;
      mr = min(r.m1 - m0, 128);
      if (split == 4) n0 += (part & 1) * 128;
      if (mr <= 0 || n0 >= on) return;
    }
    if (split == 4) {
      grouped_tile<OP, 128, 128, F32, F, F>(p, smem, p.a + m0 * p.lda, OP == 0 ? w + n0 * p.K : w + n0, nullptr, p.K,
          m0 * p.ldc + n0, mr, (int)min(on - n0, (int64_t)128), (int)kc);
      return;
    }
    if (mr <= 128) {
      grouped_tile<OP, 128, 256, F32, F, F>(p, smem, p.a + m0 * p.lda, OP == 0 ? w + n0 * p.K : w + n0, nullptr, p.K,
          m0 * p.ldc + n0, mr, (int)min(on - n0, (int64_t)256), (int)kc);
      return;
    }
  }
  grouped_tile<OP, BM, BN, F32, F, F>(p, smem, p.a + m0 * p.lda, OP == 0 ? w + n0 * p.K : w + n0, nullptr, p.K,
          m0 * p.ldc + n0, mr,
                                (int)min(on - n0, (int64_t)BN), (int)kc);
}

// OP 2: one grid of output tiles per expert, experts with the most rows first (their blocks run longest),
// in index order past 64 experts.
//
// With few rows per expert a tile is a stage or two and its time is latency and the epilogue's stores. Without
// the ring four blocks share a CU and fill each other's waits (`few_rows_each` in the launcher).
template <int BM, int BN, bool F32, Feed FA, Feed FB, bool RING>
__global__ __launch_bounds__(256, !RING ? 4 : BM == 256 ? 1 : 2) void grouped_dw_kernel(GroupedParams p, int row_tiles, int col_tiles) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[TileSize<BM, BN, RING ? 5 : 2>::LDS];
  const bool ok = ragged_ok(p.offs, p.E, p.M);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) *p.status = ok ? 0 : 1;
  if (!ok) return;
  const uint32_t per = (uint32_t)row_tiles * (uint32_t)col_tiles;
  const int place = (int)(blockIdx.x / per);
  int e = __builtin_amdgcn_readfirstlane(place), c0, c1;
  if (p.E <= 64) {
    const int lane = threadIdx.x & 63;
    const int lo = lane < p.E ? p.offs[lane] : 0, hi = lane < p.E ? p.offs[lane + 1] : -1, n = hi - lo;
    int rank = 0;
    for (int j = 0; j < p.E; ++j) {
      const int nj = __builtin_amdgcn_readlane(n, j);
      rank += nj > n || (nj == n && j < lane);
    }
    e = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(lane < p.E && rank == place)) - 1);
    c0 = __builtin_amdgcn_readlane(lo, e);
    c1 = __builtin_amdgcn_readlane(hi, e);
  } else {
    c0 = p.offs[e];
    c1 = p.offs[e + 1];
  }
  const uint32_t pos = xcd_run(blockIdx.x % per, per);
  // (row tiles in groups, as above)
  constexpr uint32_t GM = 4;
  const uint32_t grp = pos / (GM * (uint32_t)col_tiles), in = pos - grp * (GM * (uint32_t)col_tiles);
  const uint32_t rows = min(GM, (uint32_t)row_tiles - grp * GM);
  const int64_t m0 = (int64_t)(grp * GM + in % rows) * BM, n0 = (int64_t)(in / rows) * BN;
  if (p.accum && c1 == c0) return;  // nothing to add
  const void* b = p.b + (int64_t)c0 * p.ldb + n0;
  const uint8_t* scales = nullptr;
  int64_t ldb = p.ldb;
  if constexpr (FB == STAGED_CODES || FB == CODES) {
    b = p.bq + (int64_t)c0 * p.K + n0;
    scales = p.bs + (int64_t)c0 * ((p.K + 31) / 32) + (n0 >> 5);
    ldb = p.K;
  }
  grouped_tile<2, BM, BN, F32, FA, FB, RING>(p, smem, p.a + (int64_t)c0 * p.lda + m0, b, scales, ldb,
                                             (int64_t)e * p.N * p.K + m0 * p.ldc + n0,
                                             (int)min(p.N - m0, (int64_t)BM), (int)min(p.K - n0, (int64_t)BN), c1 - c0);
}

// ------------------------------------------------------------------ few rows

// OP 0 where experts have few rows (serving): bound by the weights' bytes, each read once. A block owns 32
// columns of one expert and up to 32 of its rows; its eight wavefronts split the contraction and add up in LDS
// in index order. Weights go from memory straight to the matrix instruction's registers (16 bytes per lane;
// 16 columns x 32 contraction indexes are one operand of the 16 x 16 x 32 instruction), the few rows of x
// from the L2 cache. Blocks of this size put a whole CU's loads behind every strip: one row against one
// 4096 x 4096 expert takes 12.5 us (35 in 128 x 128 tiles), 48 rows and 16 experts of 2816 x 2048, weights from memory,
// 40 us (45), 64 experts and 192 rows 127 us (156; 5.6 TB/s). Non-temporal loads fetch a line's halves twice (+20%); 16 or 64
// rows per block measured alike and 10% slower.
constexpr int FR = 32, FN_COLS = 32, FW = 8;  // rows, columns, wavefronts of a block

template <bool ANY>
__device__ __forceinline__ u32x4_t load16(const uint16_t* p) {
  if constexpr (ANY)
    return load16_any(p);
  else
    return *reinterpret_cast<const u32x4_t*>(p);
}
template <bool ANY>
__device__ __forceinline__ void few_rows(const GroupedParams& p, float* red, const uint16_t* x, const uint16_t* w, int mr,
                                         int nc) {
  constexpr int MT = FR / 16;
  constexpr int U = 4;  // steps of 32 in flight
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, kg = (lane >> 4) * 8, K = (int)p.K;
  const int steps = (K + 31) >> 5, each = (steps + FW - 1) / FW;
  const int s0 = wave * each, s1 = min(steps, s0 + each);
  const uint16_t* wp[2];
  const uint16_t* xp[MT];
#pragma unroll
  for (int j = 0; j < 2; ++j) wp[j] = w + (int64_t)min(j * 16 + r16, nc - 1) * p.K;  // (past the end: the last, not stored)
#pragma unroll
  for (int i = 0; i < MT; ++i) xp[i] = x + (int64_t)min(i * 16 + r16, mr - 1) * p.lda;
  f32x4 acc[MT][2] = {};
  for (int s = s0; s < s1; s += U) {
    u32x4_t fw[U][2], fx[U][MT];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (s + u) * 32 + kg;
      in[u] = s + u < s1 && k < K;
      const int kk = in[u] ? (ANY ? min(k, K - 8) : k) : 0;  // (the last eight of a row, shifted below)
#pragma unroll
      for (int j = 0; j < 2; ++j) fw[u][j] = load16<ANY>(wp[j] + kk);
#pragma unroll
      for (int i = 0; i < MT; ++i) fx[u][i] = load16<ANY>(xp[i] + kk);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const u32x4_t zero = {0, 0, 0, 0};
      if constexpr (ANY) {
        const int over = (s + u) * 32 + kg + 8 - K;  // elements of the lane's eight past the row's end
        if (over > 0 && over < 8) {
#pragma unroll
          for (int j = 0; j < 2; ++j) fw[u][j] = shr128(fw[u][j], 16 * over);
#pragma unroll
          for (int i = 0; i < MT; ++i) fx[u][i] = shr128(fx[u][i], 16 * over);
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) fw[u][j] = in[u] ? fw[u][j] : zero;
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        fx[u][i] = in[u] ? fx[u][i] : zero;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fx[u][i]),
                                                              __builtin_bit_cast(bf16x8, fw[u][j]), acc[i][j], 0, 0, 0);
      }
    }
  }
  // accumulator: lane l holds column l % 16 and rows 4 (l / 16) + q of a 16 x 16 block
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        red[(wave * FR + i * 16 + 4 * (lane >> 4) + q) * (FN_COLS + 1) + j * 16 + r16] = acc[i][j][q];
}

template <bool ANY>
__global__ __launch_bounds__(64 * FW, 2) void grouped_few_rows_kernel(GroupedParams p, int col_tiles) {
  __shared__ float red[FW * FR * (FN_COLS + 1)];
  const RowTiles rt = count_row_tiles(p.offs, p.E, p.M, FR);
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.status) *p.status = rt.ok ? 0 : 1;
  if (!rt.ok) return;
  const RowTile r = find_row_tile(rt, p.offs, p.E, FR, (int)(blockIdx.x / (uint32_t)col_tiles));
  if (r.e < 0) return;
  const int64_t n0 = (int64_t)(blockIdx.x % (uint32_t)col_tiles) * FN_COLS;
  const int mr = r.m1 - r.m0, nc = (int)min(p.N - n0, (int64_t)FN_COLS);
  const uint16_t* w = p.b + ((int64_t)r.e * p.N + n0) * p.K;
  const uint16_t* x = p.a + r.m0 * p.lda;
  few_rows<ANY>(p, red, x, w, mr, nc);
  __syncthreads();
  for (int i = threadIdx.x; i < mr * FN_COLS; i += 64 * FW) {
    const int m = i / FN_COLS, n = i % FN_COLS;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < FW; ++k) v += red[(k * FR + m) * (FN_COLS + 1) + n];
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

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

template <int OP, int B, bool F32, mxf::Feed FA, mxf::Feed FB, bool RING = true>
hipError_t launch_tiles_as(const mxf::GroupedParams& p, int ncu, hipStream_t st) {
  const int64_t on = OP == 0 ? p.N : p.K, ct = (on + B - 1) / B;
  if constexpr (OP == 2) {
    const int64_t rt = (p.N + B - 1) / B;
    hipLaunchKernelGGL((mxf::grouped_dw_kernel<B, B, F32, FA, FB, RING>), dim3((unsigned)(p.E * rt * ct)), dim3(256), 0, st, p,
                       (int)rt, (int)ct);
  } else {
    int64_t rt = p.M / B + (p.E < p.M ? p.E : p.M);  // every expert may end inside a tile
    if (rt == 0) rt = 1;                             // (one block looks at the offsets)
    hipLaunchKernelGGL((mxf::grouped_rows_kernel<OP, B, B, F32, FA>),
                       dim3((unsigned)(rt * ct + (B == 256 ? ncu + 8 : 0))), dim3(256), 0, st, p, (int)ct, ncu);
  }  // (ncu + 8 more: the blocks of split tiles)
  return hipGetLastError();
}
template <int OP, mxf::Feed FA, mxf::Feed FB>
hipError_t launch_tiles(const mxf::GroupedParams& p, bool big, int ncu, hipStream_t st) {
  if (big)
    return p.out_f32 ? launch_tiles_as<OP, 256, true, FA, FB>(p, ncu, st)
                     : launch_tiles_as<OP, 256, false, FA, FB>(p, ncu, st);
  return p.out_f32 ? launch_tiles_as<OP, 128, true, FA, FB>(p, ncu, st)
                   : launch_tiles_as<OP, 128, false, FA, FB>(p, ncu, st);
}

template <mxf::Feed FB>
hipError_t launch_few_rows_each(const mxf::GroupedParams& p, int ncu, hipStream_t st) {
  return p.out_f32 ? launch_tiles_as<2, 128, true, mxf::DIRECT, FB, false>(p, ncu, st)
                   : launch_tiles_as<2, 128, false, mxf::DIRECT, FB, false>(p, ncu, st);
}

}  // namespace

hipError_t mxf_launch_grouped(int op, const mxf::GroupedParams& p, int ncu, hipStream_t st) {
  using namespace mxf;
  const int64_t om = op == 2 ? p.N : p.M, on = op == 0 ? p.N : p.K;
  // 16-byte rows, and offsets inside a tile that a descriptor covers (256 rows of ld elements < 2 GB)
  const bool aligned = p.N % 8 == 0 && p.K % 8 == 0 && p.lda % 8 == 0 && p.ldb % 8 == 0 &&
                       p.ldc % (p.out_f32 ? 4 : 8) == 0 && a16(p.a) && a16(p.b) && a16(p.c) && p.lda < (1 << 22) &&
                       p.ldb < (1 << 22);
  // Few rows: up to 96, or eight per expert, unless the weights have many strips of 128 columns. A block's own cost (the
  // look at the offsets, 64 experts at a time, and the sum in LDS) weighs more the shorter K is, while 128 x 128
  // tiles gain from a full chip; without 16-byte alignment they are slower, so a short K may have more strips. Us in these
  // blocks, in tiles: one row per expert, 2816 x 2048, 16 experts 27, 33; 64 experts 88, 106; 256 experts 450, 331;
  // four, 2048 x 1024, 16 experts 17, 19; 64 experts 58, 51; 2048 x 1408, 16 experts 26, 25; 32 experts 48, 34; 7168 x 512,
  // 2 experts 9.1, 9.1; 8 experts 27, 16; unaligned, 2048 x 1022, 16 experts 21, 30; 64 experts 68, 66. One block per
  // compute unit is always better: 8 rows, 1024 experts of 1024 x 1024 18, 22. The average does not see a router that
  // sends every row to one expert: 512 rows and 64 experts of 2816 x 2048 then take 52, 20 in tiles.
  // Rows that are 4-byte aligned will do (16 experts of 2816 x 2044, 64 rows: 45, 57); 16-byte loads at odd
  // elements take several times as long (2816 x 2047, 48 rows: 67, 53).
  const auto a4 = [](const void* q) { return (reinterpret_cast<uintptr_t>(q) & 3u) == 0; };
  const int64_t strips = (p.E < p.M ? p.E : p.M) * ((p.N + 127) / 128);
  // strips per 1024 compute units; twice as many up to one row per expert, when many experts have none
  const int64_t most = (p.K >= 2000 ? 7 * 1024 : aligned ? p.K : 3 * p.K) * (p.M <= p.E ? 2 : 1);
  const bool short_grid = 4 * strips <= ncu || strips * ((p.E + 63) / 64) * 1024 <= most * ncu;
  if (op == 0 && p.K >= 8 && p.K % 2 == 0 && p.lda % 2 == 0 && a4(p.a) && a4(p.b) && (p.M <= 96 || p.M <= 8 * p.E) &&
      short_grid) {
    const bool any = p.K % 8 || p.lda % 8 || !a16(p.a) || !a16(p.b);
    const int64_t ct = (p.N + FN_COLS - 1) / FN_COLS, rt = p.M / FR + (p.E < p.M ? p.E : p.M);
    hipLaunchKernelGGL(any ? grouped_few_rows_kernel<true> : grouped_few_rows_kernel<false>,
                       dim3((unsigned)(rt ? rt * ct : 1)), dim3(64 * FW), 0, st, p, (int)ct);
    return hipGetLastError();
  }
  // 256 x 256 tiles where they fill the chip (forward of 24576 x 2816 x 2048, 64 experts: 335 us against 390 on
  // 128 x 128), or where, half a tile of every expert's end counted, they take one round of the chip and the smaller
  // ones, two to a compute unit, would take a second: forward of 8 experts, 4096 x 7168, 2816 rows 276 on 128, 186 on
  // 256; one expert, 4096 x 4096, 2304 rows 91, 73; but 3 experts of 6000 x 2048, 1000 rows (one round of either) 32, 44;
  // 16 experts of 2816 x 2048, 4096 rows (a second round of either) 57, 67. In the weight gradient they fill it twice
  // over, since the experts' tiles differ in length (8192 rows of 4 experts, 2048 x 2048, 256 tiles: 73, 126).
  const int64_t ct = (on + 255) / 256, tiles = (om + 255) / 256 * ct;
  const bool one_round = (om + 128 * (int64_t)p.E) * ct <= 256 * ncu &&
                         (om + 64 * (int64_t)p.E) * ((on + 127) / 128) > 128 * 2 * ncu;
  const bool big = op == 2 ? p.E * tiles >= 2 * ncu : tiles >= ncu || one_round;
  if (op == 0)
    return aligned ? launch_tiles<0, DIRECT, DIRECT>(p, big, ncu, st) : launch_tiles<0, STAGED, STAGED>(p, big, ncu, st);
  if (op == 1)
    return aligned ? launch_tiles<1, DIRECT, DIRECT>(p, big, ncu, st) : launch_tiles<1, STAGED, STAGED>(p, big, ncu, st);
  // Weight gradient without the ring where experts average few rows and tiles abound (us with it, without), also
  // where one of them has all the rows (64 experts of 1408 x 2048, 24576 rows: 477, 392). 64
  // experts of 1408 x 2048: 6144 rows 164, 120 (from codes 168, 111), 24576 rows 244, 215; 256 experts, 8192 rows
  // 397, 255 (5.8 TB/s of output); 16 experts of 2816 x 2048: 128 rows each 71, 51, 512 124, 110, 768 156, 158.
  // 1024 tiles are too few: 4 experts of 2048 x 2048, 512 rows 13.6, 15.1. Staged operands need too many registers
  // (64 experts of 1407 x 2047, 24576 rows: 418, 488).
  const bool few_rows_each = p.M <= 512 * p.E && p.E * ((om + 127) / 128) * ((on + 127) / 128) >= 8 * ncu;
  if (p.bq) {
    if (!aligned || p.K % 16 != 0 || !a16(p.bq)) return launch_tiles<2, STAGED, STAGED_CODES>(p, big, ncu, st);
    return few_rows_each ? launch_few_rows_each<CODES>(p, ncu, st) : launch_tiles<2, DIRECT, CODES>(p, big, ncu, st);
  }
  if (!aligned) return launch_tiles<2, STAGED, STAGED>(p, big, ncu, st);
  return few_rows_each ? launch_few_rows_each<DIRECT>(p, ncu, st) : launch_tiles<2, DIRECT, DIRECT>(p, big, ncu, st);
}
