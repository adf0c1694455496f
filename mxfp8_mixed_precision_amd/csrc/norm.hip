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
// LDS exchange per sum) and NE elements of it live in each thread, in chunks of 16 bytes; the column a
// register holds is fixed, so a block that walks rows keeps w and b (and in the backward its share of
// dw and db) in registers for all of them. The next row's loads are issued before this row's sums are
// formed: without them a block waits out a full memory latency per row. Chunks are loaded and stored
// whole at any alignment; only the stores of the chunk in which a row ends go element by element.
//
// The backward's column sums have no atomics: block p leaves one partial row of dw and of db in the
// workspace and a second launch adds the partial rows in index order, so equal inputs give equal
// bits.
//
// Measured: forward of 8192 x 7168 BF16 with a checkpoint 55.6 us (5.3 TB/s), 16384 x 2048 without 22.6 (5.9);
// backward of 16384 x 2048 from a checkpoint 29 (6.0) and 4 for the second launch, 8192 x 7168 from x 71 (5.0). FP32, 8192 x
// 4096: forward 44 (6.1), with a checkpoint 55, backward from it 58.
//
// Checkpoint: xh is rounded to BF16 and quantized by the library's rule (groups of 32 along the
// row), i.e. the codes equal those of mxfp8_quantize on the BF16 tensor. The rounding to BF16 (2^-9)
// is far below the codes' own (2^-4) and makes the two routes agree bit for bit. Keeping xh
// rather than x means that a row's mean, however large, costs no code precision and that the
// backward needs no mean.
#include "chunk.h"
#include "kernels.h"
#include "mx_device.h"

namespace mxf {

// Element c of a weight vector that is FP32, BF16 or absent (then `none`).
__device__ __forceinline__ float weight_at(const void* w, bool f32, int64_t c, float none) {
  if (!w) return none;
  return f32 ? reinterpret_cast<const float*>(w)[c] : Elem<uint16_t>::get(reinterpret_cast<const uint16_t*>(w)[c]);
}

// NE weights of this thread's columns as FP32 (FP32, BF16 or absent: then `none`), once per block.
template <int VEC, int TPR, int NE>
__device__ __forceinline__ void load_weights(const void* w, bool f32, int t, int cols, float none, float* f) {
#pragma unroll
  for (int j = 0; j < NE / VEC; ++j) {
    const int c = (j * TPR + t) * VEC;
    if (w && c + VEC <= cols) {
      if (f32) {
        __builtin_memcpy(f + j * VEC, reinterpret_cast<const float*>(w) + c, VEC * 4);
      } else {
        uint32_t k[VEC / 2];
        __builtin_memcpy(k, reinterpret_cast<const uint16_t*>(w) + c, VEC * 2);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[j * VEC + i] = i % 2 ? bf16_hi(k[i / 2]) : bf16_lo(k[i / 2]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[j * VEC + i] = c + i < cols ? weight_at(w, f32, c + i, none) : 0.0f;
    }
  }
}

// Lane exchanges on the vector ALU (DPP), a few cycles each; through the LDS crossbar a row's six steps
// took longer than everything else between its loads and its stores. CTRL: 0xB1 lane ^ 1, 0x4E lane ^ 2,
// 0x141 mirror in 8 (once 4 lanes agree: the other 4), 0x140 mirror in 16, 0x142 / 0x143 the last lane
// of row 0, 2 / of lane 31 to the rows above.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), CTRL, ROWS, 0xF, false));
}
template <int N>  // sum over N lanes (a power of two, at most 16), in all of them
__device__ __forceinline__ float lanes_sum(float v) {
  if (N >= 2) v = dpp_add<0xB1>(v);
  if (N >= 4) v = dpp_add<0x4E>(v);
  if (N >= 8) v = dpp_add<0x141>(v);
  if (N >= 16) v = dpp_add<0x140>(v);
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
  v = lanes_sum<16>(v);
  v = dpp_add<0x142, 0xA>(v);
  v = dpp_add<0x143, 0xC>(v);
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}

// s / n with the product's error taken out, so that a constant row's mean is exact (inv = 1 / n rounded).
__device__ __forceinline__ float exact_mean(float s, float n, float inv) {
  const float m = s * inv;
  return fmaf(fmaf(-m, n, s), inv, m);
}

// Sum of NW wavefronts' values v[0..NW).
template <int NW>
__device__ __forceinline__ float2 waves_sum2(const float2* v) {
  if constexpr ((NW & (NW - 1)) == 0) {
    const float2 u = v[threadIdx.x & (NW - 1)];
    return make_float2(lanes_sum<NW>(u.x), lanes_sum<NW>(u.y));
  } else {
    float2 s = v[0];
#pragma unroll
    for (int i = 1; i < NW; ++i) {
      s.x += v[i].x;
      s.y += v[i].y;
    }
    return s;
  }
}

// Sum of a pair over the TPR threads of a row; a block of BLK threads holds BLK / TPR rows. TPR 64 is one
// wavefront; more takes one barrier of the block: the slots alternate, so the next call's writes
// cannot meet this call's reads. `red`: 2 * BLK / 64 slots.
template <int TPR, int BLK>
__device__ __forceinline__ void row_sum2(float& a, float& b, float2* red, int& phase) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    float2* slot = red + phase * (BLK / 64);
    phase ^= 1;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = make_float2(a, b);
    __syncthreads();
    const float2 v = waves_sum2<NW>(slot + threadIdx.x / TPR * NW);
    a = v.x;
    b = v.y;
  }
}
template <int TPR, int BLK>
__device__ __forceinline__ float row_sum(float a, float2* red, int& phase) {
  a = wave_sum(a);
  if constexpr (TPR > 64) {
    constexpr int NW = TPR / 64;
    float2* slot = red + phase * (BLK / 64);
    phase ^= 1;
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6].x = a;
    __syncthreads();
    a = lanes_sum<NW>(slot[threadIdx.x / TPR * NW + (threadIdx.x & (NW - 1))].x);
  }
  return a;
}

// Largest magnitude (BF16 bits) over the 32-group that the lane's VEC elements belong to: 32 / VEC
// consecutive lanes.
template <int VEC>
__device__ __forceinline__ uint32_t group_max(uint32_t m) {
  m = max(m, dpp_xor1(m));
  m = max(m, dpp_xor2(m));
  if constexpr (VEC < 8) m = max(m, dpp_half_mirror(m));
  if constexpr (VEC < 4) {
    m = max(m, (uint32_t)__shfl_xor((int)m, 8));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  }
  return m;
}

// Quantize VEC normalised values, of which the first n exist (the others are zero), and store codes and the
// group's scale at column c. Every lane of the group calls this.
template <int VEC, Ends E>
__device__ __forceinline__ void put_codes(const float* xh, int n, int c, uint8_t* q, uint8_t* s) {
  if constexpr (VEC == 1) {
    const uint32_t v = bf16_bits(xh[0]);
    const Scale sc = scale_from_amax(group_max<1>(v & 0x7FFFu));
    const uint32_t code = cvt2<false>(0u, v, sc) | sc.nanmask;
    if (n > 0) q[c] = (uint8_t)code;
    if (n > 0 && (c & 31) == 0) s[c >> 5] = (uint8_t)sc.byte;
  } else {
    uint32_t w[VEC / 2], k[VEC / 4];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < VEC / 2; ++i) {
      w[i] = bf16x2_bits(xh[2 * i], xh[2 * i + 1]);
      m = pk_max_u16(m, mag2(w[i]));
    }
    const Scale sc = scale_from_amax(group_max<VEC>(max(m & 0xFFFFu, m >> 16)));
#pragma unroll
    for (int i = 0; i < VEC / 4; ++i) k[i] = cvt4(w[2 * i], w[2 * i + 1], sc);
    if (E == EXACT ? n > 0 : n >= VEC) {
      __builtin_memcpy(q + c, k, VEC);
    } else if (E != EXACT) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (i < n) q[c + i] = (uint8_t)(k[i / 4] >> (8 * (i % 4)));
    }
    if (n > 0 && (c & 31) == 0) s[c >> 5] = (uint8_t)sc.byte;
  }
}

// ------------------------------------------------------------------ forward

template <class T, int TPR, int NE, Ends E>
__global__ __launch_bounds__(TPR > 256 ? TPR : 256) void norm_fwd_kernel(NormParams p) {
  constexpr int BLK = TPR > 256 ? TPR : 256, RPB = BLK / TPR;  // rows in flight per block
  static_assert(TPR == 64 || RPB == 1, "rows of several wavefronts have a block of their own");
  constexpr int VEC = Elem<T>::VEC, NC = NE / VEC;             // chunks per thread
  __shared__ float2 red[2 * (BLK / 64)];
  int phase = 0;
  const int t = threadIdx.x % TPR, cols = (int)p.cols, G = (cols + 31) >> 5;
  const float n = (float)cols, inv = 1.0f / n;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  if (TPR == 64 && row >= p.rows) return;
  u32x4_t x0[NC], x1[NC];  // this row and the next, in turn
  auto fetch = [&](int64_t r, u32x4_t* x) {  // (past the last row: the last)
    const T* src = reinterpret_cast<const T*>(p.x) + (r < p.rows ? r : p.rows - 1) * p.ldx;
#pragma unroll
    for (int j = 0; j < NC; ++j) x[j] = load_chunk<T, E>(src, (j * TPR + t) * VEC, cols);
  };
  float w[NE], b[NE];
  fetch(row, x0);
  fetch(row + step, x1);
  load_weights<VEC, TPR, NE>(p.w, p.w_f32, t, cols, 1.0f, w);
  load_weights<VEC, TPR, NE>(p.b, p.w_f32, t, cols, 0.0f, b);
  auto one_row = [&](u32x4_t* x, u32x4_t* next) {
    float v[NE];
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      if (E == EXACT && (j * TPR + t) * VEC >= cols) continue;
      Elem<T>::unpack(chunk_of<T, E>(x[j], cols - (j * TPR + t) * VEC), v + j * VEC);
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum += v[j * VEC + i];
    }
    fetch(row + 2 * step, x);
    const float mean = exact_mean(row_sum<TPR, BLK>(sum, red, phase), n, inv);
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int m = cols - (j * TPR + t) * VEC;
      if (E == EXACT && m <= 0) continue;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        float& d = v[j * VEC + i];
        d = E == EXACT || i < m ? d - mean : 0.0f;
        ss += d * d;
      }
    }
    const float rstd = rsqrtf(row_sum<TPR, BLK>(ss, red, phase) * inv + p.eps);
    // The next row's loads end here, before this row's stores are issued: loads and stores are counted in
    // order, so a wait for the loads after them would wait for the stores as well.
#pragma unroll
    for (int j = 0; j < NC; ++j) asm volatile("" : "+v"(next[j]));
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
    T* y = reinterpret_cast<T*>(p.y) + row * p.ldy;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = (j * TPR + t) * VEC;
      if (E != EXACT || c < cols) {
        float o[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          float& xh = v[j * VEC + i];
          xh *= rstd;
          o[i] = xh * w[j * VEC + i] + b[j * VEC + i];
        }
        store_chunk<T, E>(y + c, o, cols - c);
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j * VEC + i] = 0.0f;
      }
      // All lanes of a group take part, those past the row's end with zeros (or with NaN in a row whose rstd is, as
      // is every other of that row): a lane that is left out also passes nothing on, and of three lanes the
      // second would not see the third's maximum.
      if (p.q && (E != EXACT || c < 32 * G)) put_codes<VEC, E>(v + j * VEC, cols - c, c, p.q + row * cols, p.s + row * G);
    }
    row += step;
  };
#pragma unroll
  for (int j = 0; j < NC; ++j) asm volatile("" : "+v"(x0[j]));
  while (row < p.rows) {
    one_row(x0, x1);
    if (row < p.rows) one_row(x1, x0);
  }
}

// Rows too long for registers: one block per row, three passes over memory (the later two mostly from
// the L2 cache), an element per load. 4096 x 14336 FP32: 181 us (2.6 TB/s), 212 with a checkpoint.
template <class T>
__global__ __launch_bounds__(1024) void norm_fwd_long_kernel(NormParams p) {
  __shared__ float2 red[32];
  int phase = 0;
  const int t = threadIdx.x, cols = (int)p.cols, G = (cols + 31) >> 5;
  const float n = (float)cols, inv = 1.0f / n;
  for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
    const T* x = reinterpret_cast<const T*>(p.x) + row * p.ldx;
    T* y = reinterpret_cast<T*>(p.y) + row * p.ldy;
    float sum = 0.0f;
    for (int c = t; c < cols; c += 1024) sum += Elem<T>::get(x[c]);
    const float mean = exact_mean(row_sum<1024, 1024>(sum, red, phase), n, inv);
    float ss = 0.0f;
    for (int c = t; c < cols; c += 1024) {
      const float d = Elem<T>::get(x[c]) - mean;
      ss += d * d;
    }
    const float rstd = rsqrtf(row_sum<1024, 1024>(ss, red, phase) * inv + p.eps);
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
    for (int c = t; c < 32 * G; c += 1024) {  // whole groups: 32 lanes agree on the condition
      const bool in = c < cols;
      const float xh = in ? (Elem<T>::get(x[c]) - mean) * rstd : 0.0f;
      if (in) y[c] = Elem<T>::put(xh * weight_at(p.w, p.w_f32, c, 1.0f) + weight_at(p.b, p.w_f32, c, 0.0f));
      if (p.q) put_codes<1, INSIDE>(&xh, cols - c, c, p.q + row * cols, p.s + row * G);
    }
  }
}

// ------------------------------------------------------------------ backward

// chunk_of for VEC codes.
template <int VEC>
__device__ __forceinline__ void codes_of(uint32_t* k, int n) {
  if (n >= VEC) return;
  uint64_t v = VEC == 8 ? (uint64_t)k[VEC / 4 - 1] << 32 | k[0] : k[0];
  v = n > 0 ? v >> (8 * (VEC - n)) : 0;
  k[0] = (uint32_t)v;
  if (VEC == 8) k[VEC / 4 - 1] = (uint32_t)(v >> 32);
}

// One pass: dx, and (SUMS) this block's partial dw and db in row blockIdx.x of the workspace. Blocks of up to 1024
// threads hold 1024 / TPR rows, so that one block per CU keeps enough loads in flight and leaves one partial
// row: 256 partial rows cost 1/32 of the traffic of 8192 rows.
template <class T, int TPR, int NE, bool CK, bool SUMS, Ends E>
__global__ __launch_bounds__(1024 / TPR * TPR) void norm_bwd_kernel(NormParams p) {
  constexpr int RPB = 1024 / TPR, BLK = RPB * TPR;
  constexpr int VEC = Elem<T>::VEC, NC = NE / VEC;
  __shared__ float2 red[2 * (BLK / 64)];
  int phase = 0;
  const int t = threadIdx.x % TPR, cols = (int)p.cols, G = (cols + 31) >> 5;
  const float inv = 1.0f / (float)cols;
  const int64_t step = (int64_t)gridDim.x * RPB;
  int64_t row0 = (int64_t)blockIdx.x * RPB;  // the block's first row; all its threads walk together
  const int sub = threadIdx.x / TPR;
  struct Row {  // dy, x or its codes and scales, mean, rstd
    u32x4_t dy[NC], x[CK ? 1 : NC];
    uint32_t k[CK ? NC : 1][VEC / 4], s[CK ? NC : 1];
    float mean, rstd;
  };
  Row r0, r1;  // this row and the next, in turn
  auto fetch = [&](int64_t r, Row& o) {
    r = r < p.rows ? r : p.rows - 1;
    const T* dy = reinterpret_cast<const T*>(p.dy) + r * p.ldy;
    const T* x = CK ? nullptr : reinterpret_cast<const T*>(p.x) + r * p.ldx;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = (j * TPR + t) * VEC, m = cols - c;
      o.dy[j] = load_chunk<T, E>(dy, c, cols);
      if constexpr (CK) {
        const uint8_t* q = p.q + r * cols;
#pragma unroll
        for (int i = 0; i < VEC / 4; ++i) o.k[j][i] = 0;
        if constexpr (E != TINY) {
          __builtin_memcpy(o.k[j], q + (E == INSIDE ? min(c, cols - VEC) : m > 0 ? c : 0), VEC);
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            if (i < m) o.k[j][i / 4] |= (uint32_t)q[c + i] << (8 * (i % 4));
        }
        o.s[j] = p.s[r * G + (m > 0 ? c >> 5 : 0)];
      } else {
        o.x[j] = load_chunk<T, E>(x, c, cols);
      }
    }
    o.mean = CK ? 0.0f : p.mean[r];
    o.rstd = p.rstd[r];
  };
  float w[NE], dw[SUMS ? NE : 1], db[SUMS ? NE : 1];
  fetch(row0 + sub, r0);
  fetch(row0 + sub + step, r1);
  load_weights<VEC, TPR, NE>(p.w, p.w_f32, t, cols, 1.0f, w);
#pragma unroll
  for (int i = 0; i < (SUMS ? NE : 1); ++i) dw[i] = db[i] = 0.0f;
  auto one_row = [&](Row& r, Row& next) {
    const int64_t row = row0 + sub;
    const bool on = row < p.rows;  // (whole wavefronts; the others hold the last row again and drop it)
    float g[NE], xh[NE];
    float c1 = 0.0f, c2 = 0.0f;
    const float rs = r.rstd;
#pragma unroll
    for (int j = 0; j < NC; ++j) {  // (elements past the row's end have dy = 0 and add nothing)
      if (!on || (E == EXACT && (j * TPR + t) * VEC >= cols)) continue;
      float xf[VEC];
      const int m = cols - (j * TPR + t) * VEC;
      Elem<T>::unpack(chunk_of<T, E>(r.dy[j], m), g + j * VEC);
      if (!CK) Elem<T>::unpack(chunk_of<T, E>(r.x[CK ? 0 : j], m), xf);
      if (CK && E == INSIDE) codes_of<VEC>(r.k[j], m);
      const float sc = CK ? ckpt_scale(r.s[j]) : 0.0f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int k = j * VEC + i;
        xh[k] = CK ? ckpt_value(r.k[j], i, sc) : (xf[i] - r.mean) * rs;
        if constexpr (SUMS) {
          dw[k] += g[k] * xh[k];
          db[k] += g[k];
        }
        g[k] *= w[k];
        c1 += g[k];
        c2 += g[k] * xh[k];
      }
    }
    fetch(row + 2 * step, r);
    row_sum2<TPR, BLK>(c1, c2, red, phase);
    c1 *= inv;
    c2 *= inv;
    // (the next row's loads end before this row's stores are issued, as in the forward)
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      asm volatile("" : "+v"(next.dy[j]));
      if constexpr (CK) {
        asm volatile("" : "+v"(next.k[j][0]), "+v"(next.s[j]));
        if constexpr (VEC == 8) asm volatile("" : "+v"(next.k[j][1]));
      } else {
        asm volatile("" : "+v"(next.x[j]));
      }
    }
    row0 += step;
    if (!on) return;
    T* dx = reinterpret_cast<T*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int c = (j * TPR + t) * VEC;
      if (E == EXACT && c >= cols) continue;
      float o[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[i] = rs * (g[j * VEC + i] - c1 - xh[j * VEC + i] * c2);
      store_chunk<T, E>(dx + c, o, cols - c);
    }
  };
#pragma unroll
  for (int j = 0; j < NC; ++j) {
    asm volatile("" : "+v"(r0.dy[j]));
    if constexpr (CK)
      asm volatile("" : "+v"(r0.k[j][0]), "+v"(r0.k[j][VEC / 4 - 1]), "+v"(r0.s[j]));
    else
      asm volatile("" : "+v"(r0.x[j]));
  }
  while (row0 < p.rows) {
    one_row(r0, r1);
    if (row0 < p.rows) one_row(r1, r0);
  }
  if constexpr (SUMS) {
    if (!p.part) return;
    // The rows of a block add up in LDS, one after another.
    float* pw = p.part + (int64_t)blockIdx.x * 2 * cols;
    if constexpr (RPB > 1) {
      __shared__ float acc[2][TPR * NE];
      for (int k = 0; k < RPB; ++k) {
        if (sub == k) {
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
      const int c = (j * TPR + t) * VEC;
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        store_chunk<float, INSIDE>(pw + c + i, dw + j * VEC + i, cols - c - i);
        store_chunk<float, INSIDE>(pw + cols + c + i, db + j * VEC + i, cols - c - i);
      }
    }
  }
}

// Rows too long for registers: dx alone (two passes over a row, an element per load). Past 8192 columns dw and db no longer
// fit beside a row, and a second kernel reads everything again for the column sums. 4096 x 14336 FP32: 286 us from x, 249
// from a checkpoint.
template <class T, bool CK>
__device__ __forceinline__ float xhat_at(const NormParams& p, int64_t row, int64_t c, float mean, float rstd) {
  if constexpr (CK) {
    return __builtin_amdgcn_cvt_f32_fp8((int)p.q[row * p.cols + c], 0) *
           ckpt_scale(p.s[row * ((p.cols + 31) / 32) + (c >> 5)]);
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
    row_sum2<1024, 1024>(c1, c2, red, phase);
    c1 *= inv;
    c2 *= inv;
    for (int64_t c = threadIdx.x; c < p.cols; c += 1024) {
      const float g = Elem<T>::get(dy[c]) * weight_at(p.w, p.w_f32, c, 1.0f);
      dx[c] = Elem<T>::put(rstd * (g - c1 - xhat_at<T, CK>(p, row, c, mean, rstd) * c2));
    }
  }
}
// A thread's 16 bytes of columns over rows y, y + parts, ..., four rows' loads in flight: partial row y. Runs
// before dx is written, which may be over dy. (4096 BF16 rows of 14336 from a checkpoint, the whole backward: 88 us;
// 132 with a column per thread.)
template <class T, bool CK, Ends E>
__global__ __launch_bounds__(256) void norm_bwd_cols_kernel(NormParams p) {
  constexpr int VEC = Elem<T>::VEC, U = 4;
  const int cols = (int)p.cols, c = (int)(blockIdx.x * 256 + threadIdx.x) * VEC, n = cols - c;
  if (n <= 0) return;
  const int64_t G = (p.cols + 31) >> 5, step = gridDim.y;
  float dw[VEC], db[VEC];
#pragma unroll
  for (int i = 0; i < VEC; ++i) dw[i] = db[i] = 0.0f;
  for (int64_t row = blockIdx.y; row < p.rows; row += U * step) {
    u32x4_t dy[U], x[U];
    uint32_t k[U][VEC / 4], s[U];
    float mean[U], rstd[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t r = min(row + u * step, p.rows - 1);  // (past the last row: the last, not added)
      dy[u] = load_chunk<T, E>(reinterpret_cast<const T*>(p.dy) + r * p.ldy, c, cols);
      if constexpr (CK) {
        __builtin_memcpy(k[u], p.q + r * p.cols + (E == INSIDE ? min(c, cols - VEC) : c), VEC);
        s[u] = p.s[r * G + (c >> 5)];
      } else {
        x[u] = load_chunk<T, E>(reinterpret_cast<const T*>(p.x) + r * p.ldx, c, cols);
        mean[u] = p.mean[r];
        rstd[u] = p.rstd[r];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (row + u * step >= p.rows) break;
      float d[VEC], xf[VEC];
      Elem<T>::unpack(chunk_of<T, E>(dy[u], n), d);
      if constexpr (CK) {
        if (E == INSIDE) codes_of<VEC>(k[u], n);
      } else {
        Elem<T>::unpack(chunk_of<T, E>(x[u], n), xf);
      }
      const float sc = CK ? ckpt_scale(s[u]) : 0.0f;
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        dw[i] += d[i] * (CK ? ckpt_value(k[u], i, sc) : (xf[i] - mean[u]) * rstd[u]);
        db[i] += d[i];
      }
    }
  }
  float* pw = p.part + (int64_t)blockIdx.y * 2 * p.cols + c;
#pragma unroll
  for (int i = 0; i < VEC; i += 4) {
    store_chunk<float, INSIDE>(pw + i, dw + i, n - i);
    store_chunk<float, INSIDE>(pw + p.cols + i, db + i, n - i);
  }
}

// dw and db as the sum of `parts` partial rows, 32 columns a block and 32 rows at a time; the order of
// the additions depends on `parts` alone.
__global__ __launch_bounds__(1024) void norm_reduce_kernel(const float* part, int parts, int64_t cols, float* dw,
                                                           float* db) {
  __shared__ float acc[32][33];
  const int64_t c = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);  // over dw's columns, then db's
  const int r = threadIdx.x >> 5;
  float v = 0.0f;
  if (c < 2 * cols) {
#pragma unroll 8
    for (int i = r; i < parts; i += 32) v += part[(int64_t)i * 2 * cols + c];
  }
  acc[r][threadIdx.x & 31] = v;
  __syncthreads();
  if (r == 0 && c < 2 * cols) {
#pragma unroll
    for (int i = 1; i < 32; ++i) v += acc[i][threadIdx.x];
    float* out = c < cols ? dw : db;
    if (out) out[c < cols ? c : c - cols] = v;
  }
}

}  // namespace mxf

// ------------------------------------------------------------------ launch

namespace {

using mxf::NormParams;

// Threads per row and elements per thread for a width; {0, 0}: longer than registers hold.
struct NormShape {
  int tpr, ne;
  int key() const { return tpr * 100 + ne; }
};
// Eight elements per thread up to 8192 columns: the next row's loads in flight and enough wavefronts per CU;
// with 32 per thread (a wavefront per row of 2048, four per row of 7168) the registers left two wavefronts
// per SIMD and the forward of 8192 x 7168 with a checkpoint took 87 us, not 56.
NormShape norm_shape(int64_t cols, bool f32) {
  if (cols <= 512) return {64, 8};
  if (cols <= 1024) return {128, 8};
  if (cols <= 2048) return {256, 8};
  if (cols <= 4096) return {512, 8};
  if (cols <= 8192) return {1024, 8};
  if (cols <= 16384 && !f32) return {1024, 16};  // (FP32: a row and the next no longer fit)
  return {0, 0};
}

// In the backward a row's idle lanes hold a block's registers and loads: widths between powers of two have
// shapes of their own (8192 BF16 rows with a checkpoint, 2560 columns: 30.2 us in 512 threads, 24.2 in 320;
// 2816: 31.3, 26.5 in 384; 1411: 31.1, 28.4 in 192; 5120: 46.2 in 1024, 46.5 in 640, not kept). In the forward, with
// a row per block, they gained nothing (2560: 20.9, 20.4; 5120: 35.6, 41.2).
NormShape bwd_shape(int64_t cols, bool f32) {
  NormShape s = norm_shape(cols, f32);
  if (s.ne == 8)
    for (int tpr : {192, 320, 384})
      if (cols <= tpr * 8 && tpr < s.tpr) return {tpr, 8};
  return s;
}

template <class T, mxf::Ends E>
void launch_fwd(const NormParams& p, hipStream_t st) {
  NormShape s = norm_shape(p.cols, sizeof(T) == 4);
  if (s.tpr == 128) s.tpr = 256;  // one row per block, half of its lanes idle at most
  const int blk = s.tpr > 256 ? s.tpr : s.tpr ? 256 : 1024;
  const int64_t rpb = s.tpr == 64 ? 4 : 1, need = (p.rows + rpb - 1) / rpb, most = 256 * 2048 / blk;
  const dim3 g((unsigned)(need < most ? need : most)), b(blk);
  switch (s.key()) {
    case 6408: hipLaunchKernelGGL((mxf::norm_fwd_kernel<T, 64, 8, E>), g, b, 0, st, p); break;
    case 25608: hipLaunchKernelGGL((mxf::norm_fwd_kernel<T, 256, 8, E>), g, b, 0, st, p); break;
    case 51208: hipLaunchKernelGGL((mxf::norm_fwd_kernel<T, 512, 8, E>), g, b, 0, st, p); break;
    case 102408: hipLaunchKernelGGL((mxf::norm_fwd_kernel<T, 1024, 8, E>), g, b, 0, st, p); break;
    case 102416:
      if constexpr (sizeof(T) == 2) hipLaunchKernelGGL((mxf::norm_fwd_kernel<T, 1024, 16, E>), g, b, 0, st, p);
      break;
    default: hipLaunchKernelGGL((mxf::norm_fwd_long_kernel<T>), g, b, 0, st, p);
  }
}

template <class T, bool CK, mxf::Ends E>
hipError_t launch_bwd(const NormParams& p, int parts, hipStream_t st) {
  const NormShape s = bwd_shape(p.cols, sizeof(T) == 4);
  const dim3 g((unsigned)parts), b(s.tpr ? 1024 / s.tpr * s.tpr : 1024);
  switch (s.key()) {
    case 6408: hipLaunchKernelGGL((mxf::norm_bwd_kernel<T, 64, 8, CK, true, E>), g, b, 0, st, p); break;
    case 12808: hipLaunchKernelGGL((mxf::norm_bwd_kernel<T, 128, 8, CK, true, E>), g, b, 0, st, p); break;
    case 19208: hipLaunchKernelGGL((mxf::norm_bwd_kernel<T, 192, 8, CK, true, E>), g, b, 0, st, p); break;
    case 25608: hipLaunchKernelGGL((mxf::norm_bwd_kernel<T, 256, 8, CK, true, E>), g, b, 0, st, p); break;
    case 32008: hipLaunchKernelGGL((mxf::norm_bwd_kernel<T, 320, 8, CK, true, E>), g, b, 0, st, p); break;
    case 38408: hipLaunchKernelGGL((mxf::norm_bwd_kernel<T, 384, 8, CK, true, E>), g, b, 0, st, p); break;
    case 51208: hipLaunchKernelGGL((mxf::norm_bwd_kernel<T, 512, 8, CK, true, E>), g, b, 0, st, p); break;
    case 102408: hipLaunchKernelGGL((mxf::norm_bwd_kernel<T, 1024, 8, CK, true, E>), g, b, 0, st, p); break;
    default: {
      if (p.part) {
        constexpr int per = 256 * mxf::Elem<T>::VEC;
        hipLaunchKernelGGL((mxf::norm_bwd_cols_kernel<T, CK, E>), dim3((unsigned)((p.cols + per - 1) / per), (unsigned)parts),
                           dim3(256), 0, st, p);
        hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
      }
      const dim3 rg((unsigned)(p.rows < 512 ? p.rows : 512));
      if constexpr (sizeof(T) == 2) {
        if (s.tpr) {
          hipLaunchKernelGGL((mxf::norm_bwd_kernel<T, 1024, 16, CK, false, E>), rg, b, 0, st, p);
          break;
        }
      }
      hipLaunchKernelGGL((mxf::norm_bwd_long_kernel<T, CK>), rg, b, 0, st, p);
    }
  }
  return hipGetLastError();
}
// How rows end is the width's: 8192 BF16 rows of 2815 took 39 us forward and 55 backward with the last chunk
// element by element (a branch, after which all loads are awaited), 26 and 33 without.
template <class T>
void launch_fwd_any(const NormParams& p, hipStream_t st) {
  constexpr int VEC = mxf::Elem<T>::VEC;
  if (p.cols < VEC) {
    const int64_t need = (p.rows + 3) / 4;
    hipLaunchKernelGGL((mxf::norm_fwd_kernel<T, 64, 8, mxf::TINY>), dim3((unsigned)(need < 2048 ? need : 2048)), dim3(256),
                       0, st, p);
  } else {
    p.cols % VEC ? launch_fwd<T, mxf::INSIDE>(p, st) : launch_fwd<T, mxf::EXACT>(p, st);
  }
}
template <class T, bool CK>
hipError_t launch_bwd_any(const NormParams& p, int parts, hipStream_t st) {
  constexpr int VEC = mxf::Elem<T>::VEC;
  if (p.cols < VEC) {
    hipLaunchKernelGGL((mxf::norm_bwd_kernel<T, 64, 8, CK, true, mxf::TINY>), dim3((unsigned)parts), dim3(1024), 0, st, p);
    return hipGetLastError();
  }
  return p.cols % VEC ? launch_bwd<T, CK, mxf::INSIDE>(p, parts, st) : launch_bwd<T, CK, mxf::EXACT>(p, parts, st);
}

}  // namespace

// Blocks of the backward, which is also the number of partial rows.
int mxf_norm_parts(int64_t rows, int64_t cols) {
  const NormShape s = bwd_shape(cols, false);
  const bool one = s.ne == 8;  // dx and the column sums in one kernel
  const int64_t need = one ? (rows + 1024 / s.tpr - 1) / (1024 / s.tpr) : rows;
  const int64_t most = one ? 256 : 128;
  return (int)(need < most ? need : most);
}

hipError_t mxf_launch_norm_fwd(const NormParams& p, bool f32, hipStream_t st) {
  f32 ? launch_fwd_any<float>(p, st) : launch_fwd_any<uint16_t>(p, st);
  return hipGetLastError();
}

// p.part: the workspace, or null where neither dw nor db is wanted.
hipError_t mxf_launch_norm_bwd(const NormParams& p, bool f32, hipStream_t st) {
  const int parts = mxf_norm_parts(p.rows, p.cols);
  if (p.rows > 0) {
    hipError_t e = f32 ? (p.q ? launch_bwd_any<float, true>(p, parts, st) : launch_bwd_any<float, false>(p, parts, st))
                       : (p.q ? launch_bwd_any<uint16_t, true>(p, parts, st) : launch_bwd_any<uint16_t, false>(p, parts, st));
    if (e != hipSuccess) return e;
  }
  if (!p.part) return hipSuccess;
  hipLaunchKernelGGL(mxf::norm_reduce_kernel, dim3((unsigned)((2 * p.cols + 31) / 32)), dim3(1024), 0, st, p.part,
                     parts, p.cols, p.dw, p.db);
  return hipGetLastError();
}
