// Layer norm, forward and backward, with an optional MXFP8 checkpoint of the normalised rows.
//
//   forward   mean = sum x / C, var = sum (x - mean)^2 / C, rstd = 1 / sqrt(var + eps),
//             xh = (x - mean) rstd, y = xh w + b
//   backward  g = dy w, c1 = sum g / C, c2 = sum g xh / C, dx = rstd (g - c1 - xh c2),
//             dw = sum_rows dy xh, db = sum_rows dy
//
// Bound: HBM. A row is read once and stays in registers as FP32 while its two sums are formed, so
// the variance is the second, centred pass over the same registers (no cancellation of
// sum x^2 - mean^2) at no memory cost. TPR threads share a row (a wavefront, or a block with one
// LDS exchange per sum) and NE elements of it live in each thread; the column a register holds
// is fixed, so a block that walks rows keeps w and b (and in the backward its share of dw and db)
// in registers for all of them.
//
// The backward's column sums have no atomics: block p leaves one partial row of dw and of db in the
// workspace and a second launch adds the partial rows in index order, so equal inputs give equal
// bits.
//
// Checkpoint: xh is rounded to BF16 and quantized by the library's rule (groups of 32 along the
// row), i.e. the codes equal those of mxfp8_quantize on the BF16 tensor. The rounding to BF16 (2^-9)
// is far below the codes' own (2^-4) and makes the two routes agree bit for bit. Keeping xh
// rather than x means that a row's mean, however large, costs no code precision and that the
// backward needs no mean.
#include "kernels.h"
#include "mx_device.h"

namespace mxf {

template <class T>
struct Elem;
template <>
struct Elem<uint16_t> {  // BF16 bit patterns
  static __device__ __forceinline__ float get(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t put(float f) { return (uint16_t)bf16_bits(f); }
};
template <>
struct Elem<float> {
  static __device__ __forceinline__ float get(float v) { return v; }
  static __device__ __forceinline__ float put(float f) { return f; }
};

// VEC consecutive elements (16 bytes, or one element) as FP32.
template <class T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float* f) {
  if constexpr (VEC == 1) {
    f[0] = Elem<T>::get(*p);
  } else if constexpr (VEC == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
  } else {
    const float4 v = *reinterpret_cast<const float4*>(p);
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  }
}
template <class T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float* f) {
  if constexpr (VEC == 1) {
    *p = Elem<T>::put(f[0]);
  } else if constexpr (VEC == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_bits(f[0], f[1]), bf16x2_bits(f[2], f[3]),
                                              bf16x2_bits(f[4], f[5]), bf16x2_bits(f[6], f[7]));
  } else {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
}

// Element c of a weight vector that is FP32, BF16 or absent (then `none`).
__device__ __forceinline__ float weight_at(const void* w, bool f32, int64_t c, float none) {
  if (!w) return none;
  return f32 ? reinterpret_cast<const float*>(w)[c] : Elem<uint16_t>::get(reinterpret_cast<const uint16_t*>(w)[c]);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Sum of a pair over the TPR threads of a row. TPR 64 is one wavefront; more is the whole block, with
// one barrier: the slots alternate, so the next call's writes cannot meet this call's reads.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& a, float& b, float2* red, int& phase) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    float2* slot = red + phase * NW;
    phase ^= 1;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = make_float2(a, b);
    __syncthreads();
    a = 0.0f;
    b = 0.0f;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const float2 v = slot[i];
      a += v.x;
      b += v.y;
    }
  }
}
template <int TPR>
__device__ __forceinline__ float row_sum(float a, float2* red, int& phase) {
  float b = 0.0f;
  row_sum2<TPR>(a, b, red, phase);
  return a;
}

// Largest magnitude (BF16 bits) over the 32-group that the lane's VEC elements belong to: 32 / VEC
// consecutive lanes.
template <int VEC>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
  m = max(m, dpp_xor1(m));
  m = max(m, dpp_xor2(m));
  if constexpr (VEC < 8) m = max(m, (uint32_t)__shfl_xor((int)m, 4));
  if constexpr (VEC < 4) {
    m = max(m, (uint32_t)__shfl_xor((int)m, 8));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  }
  return m;
}

// Quantize VEC normalised values (zeros where the lane is past the row's end) and store codes and
// the group's scale. `on`: the lane's elements exist. Every lane of the group calls this.
template <int VEC>
__device__ __forceinline__ void put_codes(const float* xh, bool on, int64_t c, uint8_t* q, uint8_t* s) {
  if constexpr (VEC == 1) {
    const uint32_t v = bf16_bits(xh[0]);
    const Scale sc = scale_from_amax(group_max<1>(v & 0x7FFFu));
    const uint32_t code = cvt2<false>(0u, v, sc) | sc.nanmask;
    if (on) q[c] = (uint8_t)code;
    if (on && (c & 31) == 0) s[c >> 5] = (uint8_t)sc.byte;
  } else {
    uint32_t w[VEC / 2];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      w[i] = bf16x2_bits(xh[2 * i], xh[2 * i + 1]);
      m = pk_max_u16(m, mag2(w[i]));
    }
    const Scale sc = scale_from_amax(group_max<VEC>(max(m & 0xFFFFu, m >> 16)));
    if (on) {
      if constexpr (VEC == 8)
        *reinterpret_cast<uint2*>(q + c) = make_uint2(cvt4(w[0], w[1], sc), cvt4(w[2], w[3], sc));
      else
        *reinterpret_cast<uint32_t*>(q + c) = cvt4(w[0], w[1], sc);
      if ((c & 31) == 0) s[c >> 5] = (uint8_t)sc.byte;
    }
  }
}

// VEC checkpointed values decoded to FP32 (exact: a code has four significant bits).
template <int VEC>
__device__ __forceinline__ void get_codes(const uint8_t* q, const uint8_t* s, int64_t c, float* xh) {
  const uint32_t byte = s[c >> 5];
  const float sc = byte == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte ? byte << 23 : 0x00400000u);
  if constexpr (VEC == 1) {
    xh[0] = __builtin_amdgcn_cvt_f32_fp8((int)q[c], 0) * sc;
  } else {
    uint32_t w[2];
    if constexpr (VEC == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(q + c);
      w[0] = v.x;
      w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(q + c);
    }
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) {
      xh[4 * i + 0] = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 0) * sc;
      xh[4 * i + 1] = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 1) * sc;
      xh[4 * i + 2] = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 2) * sc;
      xh[4 * i + 3] = __builtin_amdgcn_cvt_f32_fp8((int)w[i], 3) * sc;
    }
  }
}

// ------------------------------------------------------------------ forward

template <class T, int VEC, int TPR, int NE>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_fwd_kernel(NormParams p) {
  constexpr int BLK = TPR > 256 ? TPR : 256;
  constexpr int RPB = BLK / TPR;  // rows in flight per block
  constexpr int NC = NE / VEC;    // chunks per thread
  static_assert(TPR == 64 || TPR == BLK, "a row belongs to one wavefront or to the whole block");
  __shared__ float2 red[TPR > 64 ? 2 * (TPR / 64) : 1];
  int phase = 0;
  const int t = threadIdx.x % TPR;
  const float n = (float)p.cols;  // divided by, so that a constant row's mean is exact
  float w[NE], b[NE];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int64_t c = (int64_t)(j * TPR + t) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      const bool in = c < p.cols;
      w[j * VEC + i] = in ? weight_at(p.w, p.w_f32, c + i, 1.0f) : 0.0f;
      b[j * VEC + i] = in ? weight_at(p.b, p.w_f32, c + i, 0.0f) : 0.0f;
    }
  }
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < p.rows; row += (int64_t)gridDim.x * RPB) {
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
    T* y = reinterpret_cast<T*>(p.y) + row * p.ldy;
    float v[NE];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int64_t c = (int64_t)(j * TPR + t) * VEC;
      if (c < p.cols) {
        load_vec<T, VEC>(x + c, v + j * VEC);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j * VEC + i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum += v[j * VEC + i];
    }
    const float mean = row_sum<TPR>(sum, red, phase) / n;
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const bool in = (int64_t)(j * TPR + t) * VEC < p.cols;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        v[j * VEC + i] = in ? v[j * VEC + i] - mean : 0.0f;
        ss += v[j * VEC + i] * v[j * VEC + i];
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<TPR>(ss, red, phase) / n + p.eps);
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int64_t c = (int64_t)(j * TPR + t) * VEC;
      const bool in = c < p.cols;
      float xh[VEC], o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        xh[i] = v[j * VEC + i] * rstd;
        o[i] = xh[i] * w[j * VEC + i] + b[j * VEC + i];
      }
      if (in) store_vec<T, VEC>(y + c, o);
      // a lane past the end still takes part in its group's maximum; its xh is NaN in a row whose
      // rstd is, as is every other of that row
      if (p.q) put_codes<VEC>(xh, in, c, p.q + row * p.cols, p.s + row * ((p.cols + 31) / 32));
    }
  }
}

// Rows too long for registers: one block per row, three passes over memory (the later two mostly from
// the L2 cache).
template <class T>
__global__ __launch_bounds__(1024) void norm_fwd_long_kernel(NormParams p) {
  __shared__ float2 red[32];
  int phase = 0;
  const int t = threadIdx.x;
  const float n = (float)p.cols;  // divided by, so that a constant row's mean is exact
  const int64_t ceil32 = (p.cols + 31) / 32 * 32;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
    T* y = reinterpret_cast<T*>(p.y) + row * p.ldy;
    float sum = 0.0f;
    for (int64_t c = t; c < p.cols; c += 1024) sum += Elem<T>::get(x[c]);
    const float mean = row_sum<1024>(sum, red, phase) / n;
    float ss = 0.0f;
    for (int64_t c = t; c < p.cols; c += 1024) {
      const float d = Elem<T>::get(x[c]) - mean;
      ss += d * d;
    }
    const float rstd = 1.0f / sqrtf(row_sum<1024>(ss, red, phase) / n + p.eps);
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
    for (int64_t c = t; c < ceil32; c += 1024) {  // whole groups: 32 lanes agree on the condition
      const bool in = c < p.cols;
      const float xh = in ? (Elem<T>::get(x[c]) - mean) * rstd : 0.0f;
      if (in) y[c] = Elem<T>::put(xh * weight_at(p.w, p.w_f32, c, 1.0f) + weight_at(p.b, p.w_f32, c, 0.0f));
      if (p.q) put_codes<1>(&xh, in, c, p.q + row * p.cols, p.s + row * (ceil32 / 32));
    }
  }
}

// ------------------------------------------------------------------ backward

// One pass: dx, and this block's partial dw and db in row blockIdx.x of the workspace.
template <class T, int VEC, int TPR, int NE, bool CK>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_bwd_kernel(NormParams p) {
  constexpr int BLK = TPR > 256 ? TPR : 256;
  constexpr int RPB = BLK / TPR;
  constexpr int NC = NE / VEC;
  __shared__ float2 red[TPR > 64 ? 2 * (TPR / 64) : 1];
  int phase = 0;
  const int t = threadIdx.x % TPR;
  const float inv = 1.0f / (float)p.cols;
  float w[NE], dw[NE], db[NE];
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int64_t c = (int64_t)(j * TPR + t) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      w[j * VEC + i] = c < p.cols ? weight_at(p.w, p.w_f32, c + i, 1.0f) : 0.0f;
      dw[j * VEC + i] = 0.0f;
      db[j * VEC + i] = 0.0f;
    }
  }
  for (int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR; row < p.rows; row += (int64_t)gridDim.x * RPB) {
    const T* dy = reinterpret_cast<const T*>(p.dy) + row * p.ldy;
    const T* x = CK ? nullptr : reinterpret_cast<const T*>(p.x) + row * p.ldx;
    const uint8_t* q = CK ? p.q + row * p.cols : nullptr;
    const uint8_t* s = CK ? p.s + row * ((p.cols + 31) / 32) : nullptr;
    T* dx = reinterpret_cast<T*>(p.dx) + row * p.lddx;
    const float mean = CK ? 0.0f : p.mean[row];
    const float rstd = p.rstd[row];
    float g[NE], xh[NE];
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int64_t c = (int64_t)(j * TPR + t) * VEC;
      if (c < p.cols) {
        load_vec<T, VEC>(dy + c, g + j * VEC);
        if constexpr (CK)
          get_codes<VEC>(q, s, c, xh + j * VEC);
        else
          load_vec<T, VEC>(x + c, xh + j * VEC);
#pragma unroll
        for (int i = j * VEC; i < (j + 1) * VEC; ++i) {
          if (!CK) xh[i] = (xh[i] - mean) * rstd;
          dw[i] += g[i] * xh[i];
          db[i] += g[i];
          g[i] *= w[i];
          c1 += g[i];
          c2 += g[i] * xh[i];
        }
      }
    }
    row_sum2<TPR>(c1, c2, red, phase);
    c1 *= inv;
    c2 *= inv;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int64_t c = (int64_t)(j * TPR + t) * VEC;
      if (c < p.cols) {
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = rstd * (g[j * VEC + i] - c1 - xh[j * VEC + i] * c2);
        store_vec<T, VEC>(dx + c, o);
      }
    }
  }
  if (!p.part) return;
  // The wavefronts of a block that each walked their own rows add up in LDS, one after another.
  float* pw = p.part + (int64_t)blockIdx.x * 2 * p.cols;
  if constexpr (RPB > 1) {
    __shared__ float acc[2][TPR * NE];
    for (int k = 0; k < RPB; ++k) {
      if (threadIdx.x / TPR == k) {
#pragma unroll
        for (int i = 0; i < NE; ++i) {
          acc[0][i * TPR + t] = k ? acc[0][i * TPR + t] + dw[i] : dw[i];
          acc[1][i * TPR + t] = k ? acc[1][i * TPR + t] + db[i] : db[i];
        }
      }
      __syncthreads();
    }
    if (threadIdx.x >= TPR) return;
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      dw[i] = acc[0][i * TPR + t];
      db[i] = acc[1][i * TPR + t];
    }
  }
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    const int64_t c = (int64_t)(j * TPR + t) * VEC;
    if (c < p.cols) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        pw[c + i] = dw[j * VEC + i];
        pw[p.cols + c + i] = db[j * VEC + i];
      }
    }
  }
}

// Rows too long for registers: dx alone (two passes over a row), and the column sums by a second
// kernel in which a thread owns a column.
template <class T, bool CK>
__device__ __forceinline__ float xhat_at(const NormParams& p, int64_t row, int64_t c, float mean, float rstd) {
  if constexpr (CK) {
    float v;
    get_codes<1>(p.q + row * p.cols, p.s + row * ((p.cols + 31) / 32), c, &v);
    return v;
  } else {
    return (Elem<T>::get(reinterpret_cast<const T*>(p.x)[row * p.ldx + c]) - mean) * rstd;
  }
}
template <class T, bool CK>
__global__ __launch_bounds__(1024) void norm_bwd_long_kernel(NormParams p) {
  __shared__ float2 red[32];
  int phase = 0;
  const float inv = 1.0f / (float)p.cols;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* dy = reinterpret_cast<const T*>(p.dy) + row * p.ldy;
    T* dx = reinterpret_cast<T*>(p.dx) + row * p.lddx;
    const float mean = CK ? 0.0f : p.mean[row];
    const float rstd = p.rstd[row];
    float c1 = 0.0f, c2 = 0.0f;
    for (int64_t c = threadIdx.x; c < p.cols; c += 1024) {
      const float g = Elem<T>::get(dy[c]) * weight_at(p.w, p.w_f32, c, 1.0f);
      c1 += g;
      c2 += g * xhat_at<T, CK>(p, row, c, mean, rstd);
    }
    row_sum2<1024>(c1, c2, red, phase);
    c1 *= inv;
    c2 *= inv;
    for (int64_t c = threadIdx.x; c < p.cols; c += 1024) {
      const float g = Elem<T>::get(dy[c]) * weight_at(p.w, p.w_f32, c, 1.0f);
      dx[c] = Elem<T>::put(rstd * (g - c1 - xhat_at<T, CK>(p, row, c, mean, rstd) * c2));
    }
  }
}
// Columns blockIdx.x * 256 + thread over rows y, y + parts, ...: partial row y. Runs before
// norm_bwd_long_kernel, which may write dx over dy.
template <class T, bool CK>
__global__ __launch_bounds__(256) void norm_bwd_cols_kernel(NormParams p) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= p.cols) return;
  float dw = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
    const float d = Elem<T>::get(reinterpret_cast<const T*>(p.dy)[row * p.ldy + c]);
    dw += d * xhat_at<T, CK>(p, row, c, CK ? 0.0f : p.mean[row], p.rstd[row]);
    db += d;
  }
  float* pw = p.part + (int64_t)blockIdx.y * 2 * p.cols;
  pw[c] = dw;
  pw[p.cols + c] = db;
}

// dw and db as the sum of `parts` partial rows, 64 columns a block and 16 rows at a time; the order of
// the additions depends on `parts` alone.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* part, int parts, int64_t cols, float* dw,
                                                           float* db) {
  __shared__ float acc[16][64];
  const int64_t c = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);  // over dw's columns, then db's
  const int r = threadIdx.x >> 6;
  float v = 0.0f;
  if (c < 2 * cols)
    for (int i = r; i < parts; i += 16) v += part[(int64_t)i * 2 * cols + c];
  acc[r][threadIdx.x & 63] = v;
  __syncthreads();
  if (r == 0 && c < 2 * cols) {
    for (int i = 1; i < 16; ++i) v += acc[i][threadIdx.x];
    float* out = c < cols ? dw : db;
    if (out) out[c < cols ? c : c - cols] = v;
  }
}

}  // namespace mxf

// ------------------------------------------------------------------ launch

namespace {

using mxf::NormParams;

bool a16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Threads per row and elements per thread for a width; {0, 0}: longer than registers hold.
struct NormShape {
  int tpr, ne;
};
NormShape norm_shape(int64_t cols) {
  if (cols <= 512) return {64, 8};
  if (cols <= 1024) return {64, 16};
  if (cols <= 2048) return {64, 32};
  if (cols <= 4096) return {256, 16};
  if (cols <= 8192) return {256, 32};
  if (cols <= 16384) return {1024, 16};
  return {0, 0};
}

bool norm_vec(const NormParams& p, int esz) {
  const int64_t v = 16 / esz;
  bool ok = p.cols % v == 0;
  if (p.x) ok = ok && a16(p.x) && p.ldx % v == 0;
  if (p.y) ok = ok && a16(p.y) && p.ldy % v == 0;
  if (p.dy) ok = ok && a16(p.dy) && p.ldy % v == 0;
  if (p.dx) ok = ok && a16(p.dx) && p.lddx % v == 0;
  if (p.q) ok = ok && a16(p.q);
  return ok;
}

template <int TPR, int NE>
void launch_fwd(const NormParams& p, bool f32, bool vec, int64_t blocks, hipStream_t st) {
  const dim3 g((unsigned)blocks), b(TPR > 256 ? TPR : 256);
  if (f32)
    hipLaunchKernelGGL((vec ? mxf::norm_fwd_kernel<float, 4, TPR, NE>
             : mxf::norm_fwd_kernel<float, 1, TPR, NE>),
        g, b, 0, st, p);
  else
    hipLaunchKernelGGL((vec ? mxf::norm_fwd_kernel<uint16_t, 8, TPR, NE>
             : mxf::norm_fwd_kernel<uint16_t, 1, TPR, NE>),
        g, b, 0, st, p);
}

template <int TPR, int NE, bool CK>
void launch_bwd(const NormParams& p, bool f32, bool vec, int64_t blocks, hipStream_t st) {
  const dim3 g((unsigned)blocks), b(TPR > 256 ? TPR : 256);
  if (f32)
    hipLaunchKernelGGL((vec ? mxf::norm_bwd_kernel<float, 4, TPR, NE, CK>
             : mxf::norm_bwd_kernel<float, 1, TPR, NE, CK>),
        g, b, 0, st, p);
  else
    hipLaunchKernelGGL((vec ? mxf::norm_bwd_kernel<uint16_t, 8, TPR, NE, CK>
             : mxf::norm_bwd_kernel<uint16_t, 1, TPR, NE, CK>),
        g, b, 0, st, p);
}

template <bool CK>
hipError_t norm_bwd_any(const NormParams& p, bool f32, bool vec, int64_t blocks, int parts, hipStream_t st) {
  const NormShape s = norm_shape(p.cols);
  switch (s.tpr * 100 + s.ne) {
    case 6408: launch_bwd<64, 8, CK>(p, f32, vec, blocks, st); break;
    case 6416: launch_bwd<64, 16, CK>(p, f32, vec, blocks, st); break;
    case 6432: launch_bwd<64, 32, CK>(p, f32, vec, blocks, st); break;
    case 25616: launch_bwd<256, 16, CK>(p, f32, vec, blocks, st); break;
    case 25632: launch_bwd<256, 32, CK>(p, f32, vec, blocks, st); break;
    case 102416:
      if (vec) {
        const dim3 g((unsigned)blocks);
        if (f32)
          hipLaunchKernelGGL((mxf::norm_bwd_kernel<float, 4, 1024, 16, CK>), g, dim3(1024), 0, st, p);
        else
          hipLaunchKernelGGL((mxf::norm_bwd_kernel<uint16_t, 8, 1024, 16, CK>), g, dim3(1024), 0, st, p);
        break;
      }
      [[fallthrough]];  // one element per load needs more registers than 1024 threads have
    default: {
      const dim3 cg((unsigned)((p.cols + 255) / 256), (unsigned)parts);
      if (p.part) {
        if (f32)
          hipLaunchKernelGGL((mxf::norm_bwd_cols_kernel<float, CK>), cg, dim3(256), 0, st, p);
        else
          hipLaunchKernelGGL((mxf::norm_bwd_cols_kernel<uint16_t, CK>), cg, dim3(256), 0, st, p);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
      }
      const dim3 rg((unsigned)(p.rows < 4096 ? p.rows : 4096));
      if (f32)
        hipLaunchKernelGGL((mxf::norm_bwd_long_kernel<float, CK>), rg, dim3(1024), 0, st, p);
      else
        hipLaunchKernelGGL((mxf::norm_bwd_long_kernel<uint16_t, CK>), rg, dim3(1024), 0, st, p);
    }
  }
  return hipGetLastError();
}

}  // namespace

// Blocks of the backward, which is also the number of partial rows.
int mxf_norm_parts(int64_t rows, int64_t cols) {
  const NormShape s = norm_shape(cols);
  if (!s.tpr) return (int)(rows < 32 ? rows : 32);
  const int64_t need = s.tpr == 64 ? (rows + 3) / 4 : rows;
  return (int)(need < 512 ? need : 512);
}

hipError_t mxf_launch_norm_fwd(const NormParams& p, bool f32, hipStream_t st) {
  const NormShape s = norm_shape(p.cols);
  const bool vec = norm_vec(p, f32 ? 4 : 2);
  const int64_t need = s.tpr == 64 ? (p.rows + 3) / 4 : p.rows;
  const int64_t blocks = need < 2048 ? need : 2048;
  switch (s.tpr * 100 + s.ne) {
    case 6408: launch_fwd<64, 8>(p, f32, vec, blocks, st); break;
    case 6416: launch_fwd<64, 16>(p, f32, vec, blocks, st); break;
    case 6432: launch_fwd<64, 32>(p, f32, vec, blocks, st); break;
    case 25616: launch_fwd<256, 16>(p, f32, vec, blocks, st); break;
    case 25632: launch_fwd<256, 32>(p, f32, vec, blocks, st); break;
    case 102416: launch_fwd<1024, 16>(p, f32, vec, blocks, st); break;
    default:
      if (f32)
        hipLaunchKernelGGL(mxf::norm_fwd_long_kernel<float>, dim3((unsigned)blocks), dim3(1024), 0, st, p);
      else
        hipLaunchKernelGGL(mxf::norm_fwd_long_kernel<uint16_t>, dim3((unsigned)blocks), dim3(1024), 0, st, p);
  }
  return hipGetLastError();
}

// p.part: the workspace, or null where neither dw nor db is wanted.
hipError_t mxf_launch_norm_bwd(const NormParams& p, bool f32, hipStream_t st) {
  const bool vec = norm_vec(p, f32 ? 4 : 2);
  const int parts = mxf_norm_parts(p.rows, p.cols);
  if (p.rows > 0) {
    hipError_t e = p.q ? norm_bwd_any<true>(p, f32, vec, parts, parts, st)
                       : norm_bwd_any<false>(p, f32, vec, parts, parts, st);
    if (e != hipSuccess) return e;
  }
  if (!p.part) return hipSuccess;
  hipLaunchKernelGGL(mxf::norm_reduce_kernel, dim3((unsigned)((2 * p.cols + 63) / 64)), dim3(1024), 0, st, p.part,
                     parts, p.cols, p.dw, p.db);
  return hipGetLastError();
}
