// Row segments of experts on the device, bounded loads into LDS and the order of tiles: what the BF16 and the MXFP4
// expert products share.
#pragma once
#include "mx_device.h"

namespace mxf {

typedef int i32x4 __attribute__((ext_vector_type(4)));

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

// The place-th segment in falling order of rows (to 64 rows; then in any order); in index order past 64 experts. Valid offsets.
struct Segment {
  int e, lo, hi;
};
__device__ __forceinline__ Segment by_length(const int32_t* offs, int E, int place) {
  if (E > 64) {
    const int e = __builtin_amdgcn_readfirstlane(place);
    return {e, offs[e], offs[e + 1]};
  }
  const int lane = threadIdx.x & 63;
  const int lo = lane < E ? offs[lane] : 0, hi = lane < E ? offs[lane + 1] : -1, n = hi - lo;
  const int key = n < 0 ? -1 : (n >> 6) << 6 | (63 - lane);  // (unique; experts of nearly equal lengths come in any order)
  int rank = 0;
  for (int j = 0; j < E; ++j) rank += __builtin_amdgcn_readlane(key, j) > key;
  const int e = __builtin_amdgcn_readfirstlane(__ffsll((unsigned long long)__ballot(lane < E && rank == place)) - 1);
  return {e, __builtin_amdgcn_readlane(lo, e), __builtin_amdgcn_readlane(hi, e)};
}

__device__ __forceinline__ float e8m0_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

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
// The same with OFF (a constant) more on both sides, and 4 bytes per lane into LDS [lds, lds + 256).
template <int OFF>
__device__ __forceinline__ void buffer_to_lds_off(i32x4 rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen offset:%3 lds" ::"s"(lds), "v"(voff),
               "s"(rsrc), "i"(OFF)
               : "memory", "m0");
}
__device__ __forceinline__ void buffer_to_lds4(i32x4 rsrc, uint32_t voff, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(lds), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
// A descriptor of [p, p + bytes), and the same moved on. (48-bit addresses: no stride bits.)
__device__ __forceinline__ i32x4 descriptor(const void* p, int bytes = (int)kNoElement) {
  const uint64_t base = uniform64((uint64_t)p);
  return (i32x4){(int)(uint32_t)base, (int)(uint32_t)(base >> 32), __builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}
__device__ __forceinline__ void move_on(i32x4& rsrc, uint64_t bytes) {
  const uint64_t b = ((uint64_t)(uint32_t)rsrc[1] << 32 | (uint32_t)rsrc[0]) + bytes;
  rsrc[0] = (int)(uint32_t)b;
  rsrc[1] = (int)(uint32_t)(b >> 32);
}
// Position of block b of n (a contiguous run of positions per XCD: blocks go to the 8 XCDs in turn).
__device__ __forceinline__ uint32_t xcd_run(uint32_t b, uint32_t n) {
  const uint32_t q = n / 8, r = n % 8, x = b % 8;
  return (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + b / 8;
}

}  // namespace mxf
