// SwiGLU whose inputs are kept for the backward pass in MXFP8.
//
//   forward   h = BF16(g sigmoid(g) u), and the gate and up rows of [rows, 2F] as MXFP8 rows:
//             q [rows, 2, F], s [rows, 2, ceil(F / 32)]
//   backward  from the decoded g', u': dg = dh u' s (1 + g' (1 - s)), du = dh g' s, s = sigmoid(g'),
//             and h' = g' s u', which the next product's weight gradient needs and which is
//             computed again here instead of being kept
//
// Bound: HBM (8.06 bytes per element of h forward, 10.06 backward with h'): 24576 x 1408 takes 42 us and 53 (6.6
// TB/s). h of the forward comes
// from the unrounded g and u; only what is kept is rounded to 8 bits. All arithmetic is FP32 with
// one rounding to BF16 per result.
//
// A thread owns eight consecutive columns of one row, of g and of u, and a 32-group is four neighbouring
// lanes, so its maximum takes two lane exchanges. EXACT: F is a multiple of 8, so that no chunk is short: 16-byte loads
// and stores at any alignment. Other widths are loaded element by element and take 1.8 times as long forward, 1.4
// times backward (8192 x 1411: 27.7 us, 26.2; 8192 x 1408: 15.3, 18.5).
#include "chunk.h"
#include "kernels.h"
#include "mx_device.h"

namespace mxf {

// n / d for n < 2^31 as a product with m = ceil(2^p / d), p = 31 + ceil(log2 d): the product's error,
// n (m d - 2^p) / (d 2^p) < n / 2^p * 1 <= 1 / d, never reaches the next quotient.
struct FastDiv {
  uint32_t d, m, p;
};
static FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while (((uint64_t)1 << l) < d) ++l;
  const uint64_t two_p = (uint64_t)1 << (31 + l);
  return {d, (uint32_t)((two_p + d - 1) / d), 31 + l};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv& f) { return (uint32_t)(((uint64_t)n * f.m) >> f.p); }

struct SwigluParams {
  const uint16_t* gu;  // forward: [rows, 2F], row stride ldgu
  const uint16_t* dh;  // backward: [rows, F]
  uint16_t* dgu;       // backward: [rows, 2F]
  uint16_t* h;         // [rows, F]; backward: may be null
  uint8_t* q;          // [rows, 2, F]
  uint8_t* s;          // [rows, 2, G]
  int64_t row0, rows, F, G, ldgu, lddh, lddgu, ldh;
  FastDiv per_row;     // chunks in a row, forward: up to a whole group
  uint32_t units;      // of this launch: at most 2^31 - 1
};

// Eight codes to or from q, of which the first n exist.
template <bool EXACT>
__device__ __forceinline__ void store_codes(uint8_t* q, uint2 k, int n) {
  if (EXACT || n >= 8) {
    __builtin_memcpy(q, &k, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) q[i] = (uint8_t)((i < 4 ? k.x : k.y) >> (8 * (i % 4)));
  }
}
template <bool EXACT>
__device__ __forceinline__ void load_codes(const uint8_t* q, uint32_t* k, int n) {
  if (EXACT || n >= 8) {
    __builtin_memcpy(k, q, 8);
  } else {
    k[0] = k[1] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) k[i / 4] |= (uint32_t)q[i] << (8 * (i % 4));
  }
}

// Eight BF16 values, of which the first n exist. (Past the caches' retention, as dgu, h and h' are larger than
// the caches when it matters: backward 24576 x 1408 55.5 against 60.4 us, forward alike.)
template <bool EXACT>
__device__ __forceinline__ void store_words(uint16_t* p, u32x4_t v, int n) {
  if (EXACT || n >= 8) {
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)(v[i / 2] >> (16 * (i % 2)));
  }
}

// Codes and scale of one lane's eight values, n of which exist (the others are zero); the group is four
// neighbouring lanes, and all four call this.
template <bool EXACT>
__device__ __forceinline__ void quant8(u32x4_t v, int n, uint8_t* q, uint8_t* s, bool first) {
  uint32_t m = pk_max_u16(pk_max_u16(mag2(v[0]), mag2(v[1])), pk_max_u16(mag2(v[2]), mag2(v[3])));
  m = max(m & 0xFFFFu, m >> 16);
  m = max(m, dpp_xor1(m));
  m = max(m, dpp_xor2(m));
  const Scale sc = scale_from_amax(m);
  if (n > 0) {
    store_codes<EXACT>(q, make_uint2(cvt4(v[0], v[1], sc), cvt4(v[2], v[3], sc)), n);
    if (first) *s = (uint8_t)sc.byte;
  }
}

template <bool EXACT>
__global__ __launch_bounds__(256) void swiglu_fwd_kernel(SwigluParams p) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= p.units) return;  // whole groups: units is a multiple of four
  const uint32_t r = div_by(i, p.per_row);
  const uint32_t ch = i - r * p.per_row.d;
  const int64_t row = p.row0 + r;
  const int F = (int)p.F, c = (int)ch * 8, n = F - c;
  u32x4_t g = {0, 0, 0, 0}, u = g;
  if (n > 0) {
    const uint16_t* src = p.gu + row * p.ldgu;
    g = load_chunk<uint16_t, EXACT ? Ends::EXACT : TINY>(src, c, F);
    u = load_chunk<uint16_t, EXACT ? Ends::EXACT : TINY>(src + F, c, F);
    const u32x4_t h = {swiglu_h2(g[0], u[0]), swiglu_h2(g[1], u[1]), swiglu_h2(g[2], u[2]), swiglu_h2(g[3], u[3])};
    store_words<EXACT>(p.h + row * p.ldh + c, h, n);
  }
  uint8_t* q = p.q + row * 2 * p.F + c;
  uint8_t* s = p.s + row * 2 * p.G + (ch >> 2);
  quant8<EXACT>(g, n, q, s, (ch & 3) == 0);
  quant8<EXACT>(u, n, q + F, s + p.G, (ch & 3) == 0);
}

template <bool EXACT>
__global__ __launch_bounds__(256) void swiglu_bwd_kernel(SwigluParams p) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= p.units) return;
  const uint32_t r = div_by(i, p.per_row);
  const uint32_t ch = i - r * p.per_row.d;
  const int64_t row = p.row0 + r;
  const int F = (int)p.F, c = (int)ch * 8, n = F - c;
  const uint8_t* q = p.q + row * 2 * p.F + c;
  const uint8_t* s = p.s + row * 2 * p.G + (ch >> 2);
  const u32x4_t d = load_chunk<uint16_t, EXACT ? Ends::EXACT : TINY>(p.dh + row * p.lddh, c, F);
  uint32_t qg[2], qu[2];
  load_codes<EXACT>(q, qg, n);
  load_codes<EXACT>(q + F, qu, n);
  const float sg = ckpt_scale(s[0]), su = ckpt_scale(s[p.G]);
  float dh[8], g[8], u[8], dg[8], du[8];
  Elem<uint16_t>::unpack(d, dh);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    g[k] = ckpt_value(qg, k, sg);
    u[k] = ckpt_value(qu, k, su);
    dswiglu_f(dh[k], g[k], u[k], dg[k], du[k]);
  }
  uint16_t* o = p.dgu + row * p.lddgu + c;
  store_words<EXACT>(o, Elem<uint16_t>::pack(dg), n);
  store_words<EXACT>(o + F, Elem<uint16_t>::pack(du), n);
  if (p.h) {
#pragma unroll
    for (int k = 0; k < 8; ++k) g[k] = silu_mul(g[k], u[k]);
    store_words<EXACT>(p.h + row * p.ldh + c, Elem<uint16_t>::pack(g), n);
  }
}

// Launches the kernel over all rows, in slabs of rows whose chunks a 31-bit index covers.
static hipError_t swiglu_slabs(SwigluParams p, int64_t per_row, void (*kernel)(SwigluParams), hipStream_t st) {
  const int64_t slab = 0x7FFFFF00 / per_row;
  p.per_row = fast_div((uint32_t)per_row);
  for (p.row0 = 0; p.row0 < p.rows; p.row0 += slab) {
    const int64_t n = p.rows - p.row0 < slab ? p.rows - p.row0 : slab;
    p.units = (uint32_t)(n * per_row);
    hipLaunchKernelGGL(kernel, dim3((p.units + 255) / 256), dim3(256), 0, st, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace mxf

hipError_t mxf_launch_swiglu_ckpt_fwd(const void* gu, int64_t rows, int64_t F, int64_t ldgu, int64_t ldh, void* h,
                                      void* q, void* s, hipStream_t st) {
  mxf::SwigluParams p = {};
  p.gu = (const uint16_t*)gu;
  p.h = (uint16_t*)h;
  p.q = (uint8_t*)q;
  p.s = (uint8_t*)s;
  p.rows = rows; p.F = F; p.G = (F + 31) / 32; p.ldgu = ldgu; p.ldh = ldh;
  return mxf::swiglu_slabs(p, 4 * p.G, F % 8 ? mxf::swiglu_fwd_kernel<false> : mxf::swiglu_fwd_kernel<true>, st);
}

hipError_t mxf_launch_swiglu_ckpt_bwd(const void* dh, const void* q, const void* s, int64_t rows, int64_t F,
                                      int64_t lddh, int64_t lddgu, int64_t ldh, void* dgu, void* h, hipStream_t st) {
  mxf::SwigluParams p = {};
  p.dh = (const uint16_t*)dh;
  p.q = (uint8_t*)const_cast<void*>(q);
  p.s = (uint8_t*)const_cast<void*>(s);
  p.dgu = (uint16_t*)dgu;
  p.h = (uint16_t*)h;
  p.rows = rows; p.F = F; p.G = (F + 31) / 32; p.lddh = lddh; p.lddgu = lddgu; p.ldh = ldh;
  return mxf::swiglu_slabs(p, (F + 7) / 8, F % 8 ? mxf::swiglu_bwd_kernel<false> : mxf::swiglu_bwd_kernel<true>, st);
}
