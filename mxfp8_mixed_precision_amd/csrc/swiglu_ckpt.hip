// SwiGLU whose inputs are kept for the backward pass in MXFP8.
//
//   forward   h = BF16(g sigmoid(g) u), and the gate and up rows of [rows, 2F] as MXFP8 rows:
//             q [rows, 2, F], s [rows, 2, ceil(F / 32)]
//   backward  from the decoded g', u': dg = dh u' s (1 + g' (1 - s)), du = dh g' s, s = sigmoid(g'),
//             and h' = g' s u', which the next product's weight gradient needs and which is
//             computed again here instead of being kept
//
// Bound: HBM (8.06 bytes per element of h forward, 10.06 backward with h'). h of the forward comes
// from the unrounded g and u; only what is kept is rounded to 8 bits. All arithmetic is FP32 with
// one rounding to BF16 per result.
//
// A thread owns eight consecutive columns of one row, of g and of u: 16-byte loads and stores, and a
// 32-group is four neighbouring lanes, so its maximum takes two lane exchanges. Rows that are not
// 16-byte aligned take one column per thread instead, with a group in 32 lanes.
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
  FastDiv per_row;     // units (chunks or groups) in a row
  uint32_t units;      // of this launch: at most 2^31 - 1
};

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Codes and scale of one lane's eight values; the group is four neighbouring lanes. `on`: they exist.
__device__ __forceinline__ void quant8(uint4 v, bool on, uint8_t* q, uint8_t* s, bool first) {
  uint32_t m = pk_max_u16(pk_max_u16(mag2(v.x), mag2(v.y)), pk_max_u16(mag2(v.z), mag2(v.w)));
  m = max(m & 0xFFFFu, m >> 16);
  m = max(m, dpp_xor1(m));
  m = max(m, dpp_xor2(m));
  const Scale sc = scale_from_amax(m);
  if (on) {
    *reinterpret_cast<uint2*>(q) = make_uint2(cvt4(v.x, v.y, sc), cvt4(v.z, v.w, sc));
    if (first) *s = (uint8_t)sc.byte;
  }
}

__global__ __launch_bounds__(256) void swiglu_fwd_kernel(SwigluParams p) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= p.units) return;  // whole groups: units is a multiple of four
  const uint32_t r = div_by(i, p.per_row);
  const uint32_t ch = i - r * p.per_row.d;
  const int64_t row = p.row0 + r, c = (int64_t)ch * 8;
  const bool on = c < p.F;
  uint4 g = make_uint4(0, 0, 0, 0), u = g;
  if (on) {
    const uint16_t* src = p.gu + row * p.ldgu + c;
    g = *reinterpret_cast<const uint4*>(src);
    u = *reinterpret_cast<const uint4*>(src + p.F);
    *reinterpret_cast<uint4*>(p.h + row * p.ldh + c) =
        make_uint4(swiglu_h2(g.x, u.x), swiglu_h2(g.y, u.y), swiglu_h2(g.z, u.z), swiglu_h2(g.w, u.w));
  }
  uint8_t* q = p.q + row * 2 * p.F + c;
  uint8_t* s = p.s + row * 2 * p.G + (ch >> 2);
  quant8(g, on, q, s, (ch & 3) == 0);
  quant8(u, on, q + p.F, s + p.G, (ch & 3) == 0);
}

// Any alignment: 32 lanes per group, one column each.
__global__ __launch_bounds__(256) void swiglu_fwd_any_kernel(SwigluParams p) {
  const uint32_t i = blockIdx.x * 8u + (threadIdx.x >> 5);
  if (i >= p.units) return;  // 32 lanes agree
  const uint32_t r = div_by(i, p.per_row);
  const uint32_t grp = i - r * p.per_row.d;
  const int64_t row = p.row0 + r, c = (int64_t)grp * 32 + (threadIdx.x & 31);
  const bool on = c < p.F;
  const uint16_t* src = p.gu + row * p.ldgu + c;
  const uint32_t v[2] = {on ? (uint32_t)src[0] : 0u, on ? (uint32_t)src[p.F] : 0u};
  if (on) p.h[row * p.ldh + c] = (uint16_t)swiglu_h2(v[0], v[1]);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t m = v[k] & 0x7FFFu;
#pragma unroll
    for (int o = 16; o; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o, 32));
    const Scale sc = scale_from_amax(m);
    const uint32_t code = cvt2<false>(0u, v[k], sc) | sc.nanmask;
    if (on) p.q[(row * 2 + k) * p.F + c] = (uint8_t)code;
    if (on && (threadIdx.x & 31) == 0) p.s[(row * 2 + k) * p.G + grp] = (uint8_t)sc.byte;
  }
}

__device__ __forceinline__ void decode4(uint32_t w, float sc, float* f) {
  f[0] = __builtin_amdgcn_cvt_f32_fp8((int)w, 0) * sc;
  f[1] = __builtin_amdgcn_cvt_f32_fp8((int)w, 1) * sc;
  f[2] = __builtin_amdgcn_cvt_f32_fp8((int)w, 2) * sc;
  f[3] = __builtin_amdgcn_cvt_f32_fp8((int)w, 3) * sc;
}

__global__ __launch_bounds__(256) void swiglu_bwd_kernel(SwigluParams p) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= p.units) return;
  const uint32_t r = div_by(i, p.per_row);
  const uint32_t ch = i - r * p.per_row.d;
  const int64_t row = p.row0 + r, c = (int64_t)ch * 8;
  const uint8_t* q = p.q + row * 2 * p.F + c;
  const uint8_t* s = p.s + row * 2 * p.G + (ch >> 2);
  const uint4 d = *reinterpret_cast<const uint4*>(p.dh + row * p.lddh + c);
  const uint2 qg = *reinterpret_cast<const uint2*>(q), qu = *reinterpret_cast<const uint2*>(q + p.F);
  const float sg = scale_value(s[0]), su = scale_value(s[p.G]);
  float g[8], u[8], dg[8], du[8];
  decode4(qg.x, sg, g);
  decode4(qg.y, sg, g + 4);
  decode4(qu.x, su, u);
  decode4(qu.y, su, u + 4);
  const uint32_t dw[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
  for (int k = 0; k < 8; ++k) dswiglu_f((k & 1) ? bf16_hi(dw[k / 2]) : bf16_lo(dw[k / 2]), g[k], u[k], dg[k], du[k]);
  uint16_t* o = p.dgu + row * p.lddgu + c;
  *reinterpret_cast<uint4*>(o) = make_uint4(bf16x2_bits(dg[0], dg[1]), bf16x2_bits(dg[2], dg[3]),
                                            bf16x2_bits(dg[4], dg[5]), bf16x2_bits(dg[6], dg[7]));
  *reinterpret_cast<uint4*>(o + p.F) = make_uint4(bf16x2_bits(du[0], du[1]), bf16x2_bits(du[2], du[3]),
                                                  bf16x2_bits(du[4], du[5]), bf16x2_bits(du[6], du[7]));
  if (p.h) {
    float hv[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) hv[k] = silu_mul(g[k], u[k]);
    *reinterpret_cast<uint4*>(p.h + row * p.ldh + c) =
        make_uint4(bf16x2_bits(hv[0], hv[1]), bf16x2_bits(hv[2], hv[3]), bf16x2_bits(hv[4], hv[5]),
                   bf16x2_bits(hv[6], hv[7]));
  }
}

__global__ __launch_bounds__(256) void swiglu_bwd_any_kernel(SwigluParams p) {
  const uint32_t i = blockIdx.x * 8u + (threadIdx.x >> 5);
  if (i >= p.units) return;
  const uint32_t r = div_by(i, p.per_row);
  const uint32_t grp = i - r * p.per_row.d;
  const int64_t row = p.row0 + r, c = (int64_t)grp * 32 + (threadIdx.x & 31);
  if (c >= p.F) return;
  const uint8_t* q = p.q + row * 2 * p.F + c;
  const uint8_t* s = p.s + row * 2 * p.G + grp;
  const float g = __builtin_amdgcn_cvt_f32_fp8((int)q[0], 0) * scale_value(s[0]);
  const float u = __builtin_amdgcn_cvt_f32_fp8((int)q[p.F], 0) * scale_value(s[p.G]);
  float dg, du;
  dswiglu_f(bf16_lo(p.dh[row * p.lddh + c]), g, u, dg, du);
  uint16_t* o = p.dgu + row * p.lddgu + c;
  o[0] = (uint16_t)bf16_bits(dg);
  o[p.F] = (uint16_t)bf16_bits(du);
  if (p.h) p.h[row * p.ldh + c] = (uint16_t)bf16_bits(silu_mul(g, u));
}

// Launches `vec` or `any` over all rows, in slabs of rows whose units a 31-bit index covers.
template <class K>
static hipError_t swiglu_slabs(SwigluParams p, bool vec, int64_t rows, K vec_kernel, K any_kernel, hipStream_t st) {
  const int64_t per_row = vec ? (vec_kernel == swiglu_fwd_kernel ? 4 * p.G : p.F / 8) : p.G;
  // a launch has fewer than 2^32 threads: one per chunk, or 32 per group
  const int64_t slab = (vec ? 0x7FFFFF00 : 0x07FFFF00) / per_row;
  p.per_row = fast_div((uint32_t)per_row);
  for (p.row0 = 0; p.row0 < rows; p.row0 += slab) {
    const int64_t n = rows - p.row0 < slab ? rows - p.row0 : slab;
    p.units = (uint32_t)(n * per_row);
    const uint32_t per_block = vec ? 256 : 8;
    hipLaunchKernelGGL(vec ? vec_kernel : any_kernel, dim3((p.units + per_block - 1) / per_block), dim3(256), 0, st, p);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace mxf

hipError_t mxf_launch_swiglu_ckpt_fwd(const void* gu, int64_t rows, int64_t F, int64_t ldgu, int64_t ldh, void* h,
                                      void* q, void* s, hipStream_t st) {
  mxf::SwigluParams p = {};
  p.gu = (const uint16_t*)gu;
  p.h = (uint16_t*)h;
  p.q = (uint8_t*)q;
  p.s = (uint8_t*)s;
  p.rows = rows; p.F = F; p.G = (F + 31) / 32; p.ldgu = ldgu; p.ldh = ldh;
  const bool vec = F % 8 == 0 && ldgu % 8 == 0 && ldh % 8 == 0 && mxf::al16(gu) && mxf::al16(h) && mxf::al16(q);
  return mxf::swiglu_slabs(p, vec, rows, mxf::swiglu_fwd_kernel, mxf::swiglu_fwd_any_kernel, st);
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
  const bool vec = F % 8 == 0 && lddh % 8 == 0 && lddgu % 8 == 0 && (!h || ldh % 8 == 0) && mxf::al16(dh) &&
                   mxf::al16(q) && mxf::al16(dgu) && mxf::al16(h);
  return mxf::swiglu_slabs(p, vec, rows, mxf::swiglu_bwd_kernel, mxf::swiglu_bwd_any_kernel, st);
}
