// Token rows copied to their experts' rows and back, with the router's weights, and the gradients of both.
//
//   dispatch      xe[r] = x[a_r / topk], a_r = row_assign[r]; zeros for a pad row (a_r = -1)
//   combine       y[t] = (residual[t] +) sum_k w[t, k] h[row(t, k)], row = assign_row; dropped assignments (-1) add nothing
//   its gradient  dh[r] = w[a_r] dy[a_r / topk] (zeros for a pad row), dw[t, k] = <dy[t], h[row(t, k)]>
//
// combine with all weights 1 is dispatch's gradient. Sums are FP32 in the order of k, rounded once; dw is FP32.
//
// All three go by tokens, read a token's row once and touch the topk rows of its assignments with all loads in flight, where
// going by rows would read it topk times. 8, 16, 32 or 64 lanes (the fewest that hold it in 16-byte chunks) own a
// span of 64 chunks of a token's row in dispatch and combine, a whole token in the gradient, whose dot products run along
// it; there a row past one 16-byte chunk for each of 256 threads takes a block. Pad rows are found by blocks of the same launch, 16 rows
// of row_assign to a wavefront, and in dispatch and the gradient these come first.
//
// Bound by HBM (copy: 6.1 TB/s; BF16): dispatch of 4096 tokens to 24576 rows of 2048 and the padding 20.6 us (127 MB, 5.9 TB/s;
// by whole tokens 25.7); combine back 18.2 (119 MB, 6.1 TB/s); gradient of 4096 tokens, 32768 rows of 7168 and the padding 191
// (1057 MB, 5.5 TB/s; h through the caches 206, with 64 lanes per token, which hold a row's chunks one after the other, 220).
// Dispatch's gradient of 4096 tokens of 6 rows of 2048 18.1 (119 MB), of 8 of 7168 97 (531 MB, 5.5 TB/s).
// Combine of 8 tokens: 3.9.
//
// A row's last chunk is taken from its end backwards, over elements that its neighbour has too: both store the same
// values (the dot products skip them), so any width and alignment goes without a branch. Rows shorter than a chunk
// go element by element.
#include "chunk.h"
#include "kernels.h"

namespace mxf {

constexpr int kPadRows = 16;  // rows of row_assign per wavefront
constexpr int kRowsInFlight = 8;

// (rows of a grid of more than one are equally long)
__device__ __forceinline__ unsigned block_of_grid() { return blockIdx.y * gridDim.x + blockIdx.x; }

// The expert row of assignment a, -1 if it has none.
__device__ __forceinline__ int64_t row_of(const RouteParams& p, int64_t a) {
  const int32_t r = p.assign_row[a];
  return r >= 0 && r < p.rows ? r : -1;
}

__device__ __forceinline__ u32x4_t load_any(const void* p) {
  u32x4_t v;
  __builtin_memcpy(&v, p, 16);
  return v;
}
__device__ __forceinline__ u32x4_t load_once(const void* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_any*>(p));
}
__device__ __forceinline__ void store_any(void* p, u32x4_t v) {
  __builtin_nontemporal_store(v, reinterpret_cast<u32x4_any*>(p));
}

// Zeros into the pad rows of [first, first + kPadRows); rows of `bytes` bytes, `pitch` apart.
__device__ __forceinline__ void zero_pads(const RouteParams& p, uint8_t* out, int64_t bytes, int64_t pitch, int64_t first) {
  const int lane = threadIdx.x & 63;
  const int64_t end = min<int64_t>(p.offs[p.E], p.rows), n = p.tokens * p.topk;
  const int64_t r = first + lane;
  bool pad = false;
  if (lane < kPadRows && r < end) {
    const int32_t a = p.row_assign[r];
    pad = a < 0 || a >= n;
  }
  const u32x4_t zero = {0, 0, 0, 0};
  for (uint64_t m = __ballot(pad); m; m &= m - 1) {
    uint8_t* o = out + (first + __ffsll((unsigned long long)m) - 1) * pitch;
    if (bytes >= 16) {
      for (int64_t c = lane * 16; c < bytes; c += 1024) store_any(o + min<int64_t>(c, bytes - 16), zero);
    } else if (lane < bytes) {
      o[lane] = 0;
    }
  }
}

// LPT lanes per token; with 64 a wavefront takes one span of 64 chunks of it. (combine, ONCE: h is read past the caches.)
template <int LPT>
__global__ __launch_bounds__(256) void dispatch_kernel(RouteParams p, unsigned pad_blocks, int spans) {
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned block = block_of_grid();
  uint8_t* out = reinterpret_cast<uint8_t*>(p.h);
  if (block < pad_blocks) {
    zero_pads(p, out, p.D, p.ldh, ((int64_t)block * 4 + w) * kPadRows);
    return;
  }
  const int64_t wave = (int64_t)(block - pad_blocks) * 4 + w;
  const int64_t t = LPT == 64 ? wave / spans : wave * (64 / LPT) + lane / LPT;
  if (t >= p.tokens) return;
  const uint8_t* x = reinterpret_cast<const uint8_t*>(p.x) + t * p.ldx;
  const int64_t a0 = t * p.topk, c = LPT == 64 ? (wave % spans) * 1024 + lane * 16 : lane % LPT * 16;
  if (p.D < 16) {
    for (int k = 0; k < p.topk; ++k) {
      const int64_t r = row_of(p, a0 + k);
      for (int64_t i = c / 16; r >= 0 && i < p.D; i += LPT) out[r * p.ldh + i] = x[i];
    }
    return;
  }
  if (c >= p.D) return;
  const int64_t cc = min<int64_t>(c, p.D - 16);
  const u32x4_t v = load_any(x + cc);
  for (int k0 = 0; k0 < p.topk; k0 += kRowsInFlight) {
    int64_t row[kRowsInFlight];
#pragma unroll
    for (int k = 0; k < kRowsInFlight; ++k) row[k] = k0 + k < p.topk ? row_of(p, a0 + k0 + k) : -1;
#pragma unroll
    for (int k = 0; k < kRowsInFlight; ++k)
      if (row[k] >= 0) store_any(out + row[k] * p.ldh + cc, v);
  }
}

__device__ __forceinline__ float weight_of(const RouteParams& p, int64_t a) {
  return p.w_f32 ? reinterpret_cast<const float*>(p.w)[a] : Elem<uint16_t>::get(reinterpret_cast<const uint16_t*>(p.w)[a]);
}

template <class T, int LPT, bool W, bool ONCE>
__global__ __launch_bounds__(256) void combine_kernel(RouteParams p, int spans) {
  constexpr int VEC = Elem<T>::VEC;
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)block_of_grid() * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t t = LPT == 64 ? wave / spans : wave * (64 / LPT) + lane / LPT;
  if (t >= p.tokens) return;
  const T* h = reinterpret_cast<const T*>(p.h);
  T* y = reinterpret_cast<T*>(p.y) + t * p.ldx;
  const T* res = p.residual ? reinterpret_cast<const T*>(p.residual) + t * p.ldr : nullptr;
  const int64_t a0 = t * p.topk;
  const int64_t c0 = LPT == 64 ? (wave % spans) * 64 * VEC + lane * VEC : (lane % LPT) * VEC;
  if (p.D < VEC) {
    const int64_t c = c0 / VEC;
    if (c < p.D) {
      float s = res ? Elem<T>::get(res[c]) : 0.0f;
      for (int k = 0; k < p.topk; ++k) {
        const int64_t r = row_of(p, a0 + k);
        if (r >= 0) s += (W ? weight_of(p, a0 + k) : 1.0f) * Elem<T>::get(h[r * p.ldh + c]);
      }
      y[c] = Elem<T>::put(s);
    }
    return;
  }
  if (c0 >= p.D) return;
  const int64_t c = min<int64_t>(c0, p.D - VEC);
  float sum[VEC] = {};
  if (res) Elem<T>::unpack(load_any(res + c), sum);
  for (int k0 = 0; k0 < p.topk; k0 += kRowsInFlight) {
    u32x4_t v[kRowsInFlight];
    float w[kRowsInFlight];
    bool in[kRowsInFlight];
#pragma unroll
    for (int k = 0; k < kRowsInFlight; ++k) {
      const int64_t a = a0 + min(k0 + k, p.topk - 1);
      const int64_t r = row_of(p, a);
      in[k] = k0 + k < p.topk && r >= 0;
      w[k] = W ? weight_of(p, a) : 1.0f;
      v[k] = (u32x4_t){0, 0, 0, 0};
      if (in[k]) v[k] = ONCE ? load_once(h + r * p.ldh + c) : load_any(h + r * p.ldh + c);
    }
#pragma unroll
    for (int k = 0; k < kRowsInFlight; ++k) {
      if (!in[k]) continue;
      float f[VEC];
      Elem<T>::unpack(v[k], f);
#pragma unroll
      for (int i = 0; i < VEC; ++i) sum[i] = W ? fmaf(w[k], f[i], sum[i]) : sum[i] + f[i];
    }
  }
  store_any(y + c, Elem<T>::pack(sum));
}

// DOT: the weights' gradient too; without it h is not read. LPT past 64: wavefronts of a block share a token. ONCE: h is read past the
// caches.
template <class T, int LPT, bool DOT, bool ONCE>
__global__ __launch_bounds__(256) void combine_bwd_kernel(RouteParams p, unsigned pad_blocks) {
  constexpr int VEC = Elem<T>::VEC, TPB = 256 / LPT, WPT = LPT / 64;
  __shared__ float red[DOT && WPT > 1 ? 4 * kRowsInFlight : 1];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const unsigned block = block_of_grid();
  if (block < pad_blocks) {
    zero_pads(p, reinterpret_cast<uint8_t*>(p.dh), p.D * sizeof(T), p.lddh * sizeof(T),
              ((int64_t)block * 4 + wave) * kPadRows);
    return;
  }
  int64_t t = (int64_t)(block - pad_blocks) * TPB;
  if (t >= p.tokens) return;
  if constexpr (WPT > 0)
    t += wave / WPT;
  else
    t += threadIdx.x / LPT;
  const bool live = t < p.tokens;
  if (WPT == 1 && !live) return;
  const int l = (int)threadIdx.x % LPT;
  const T* dy = reinterpret_cast<const T*>(p.dy) + (live ? t : 0) * p.ldx;
  const T* h = reinterpret_cast<const T*>(p.h);
  T* dh = reinterpret_cast<T*>(p.dh);
  const int64_t a0 = t * p.topk;
  for (int k0 = 0; k0 < p.topk; k0 += kRowsInFlight) {
    float w[kRowsInFlight], dot[kRowsInFlight];
    int64_t row[kRowsInFlight];
#pragma unroll
    for (int k = 0; k < kRowsInFlight; ++k) {
      const bool in = live && k0 + k < p.topk;
      row[k] = in ? row_of(p, a0 + k0 + k) : -1;
      w[k] = row[k] >= 0 ? weight_of(p, a0 + k0 + k) : 0.0f;
      dot[k] = 0.0f;
    }
    if (p.D < VEC) {
      for (int64_t c = l; c < p.D; c += LPT) {
        const float g = Elem<T>::get(dy[c]);
#pragma unroll
        for (int k = 0; k < kRowsInFlight; ++k)
          if (row[k] >= 0) {
            if (DOT) dot[k] = fmaf(g, Elem<T>::get(h[row[k] * p.ldh + c]), dot[k]);
            dh[row[k] * p.lddh + c] = Elem<T>::put(w[k] * g);
          }
      }
    } else {
      for (int64_t c0 = l * VEC; c0 < p.D; c0 += LPT * VEC) {
        const int64_t c = min<int64_t>(c0, p.D - VEC);
        const int skip = (int)(c0 - c);  // elements that the chunk before has too
        const u32x4_t gv = load_any(dy + c);
        u32x4_t v[kRowsInFlight];
#pragma unroll
        for (int k = 0; k < kRowsInFlight; ++k)
          if (DOT && row[k] >= 0) v[k] = ONCE ? load_once(h + row[k] * p.ldh + c) : load_any(h + row[k] * p.ldh + c);
        float g[VEC];
        Elem<T>::unpack(gv, g);
#pragma unroll
        for (int k = 0; k < kRowsInFlight; ++k) {
          if (row[k] < 0) continue;
          float f[VEC], o[VEC];
          if (DOT) Elem<T>::unpack(v[k], f);
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            o[i] = w[k] * g[i];
            if (DOT) dot[k] = i < skip ? dot[k] : fmaf(g[i], f[i], dot[k]);
          }
          store_any(dh + row[k] * p.lddh + c, Elem<T>::pack(o));
        }
      }
    }
    if constexpr (!DOT) continue;
#pragma unroll
    for (int k = 0; k < kRowsInFlight; ++k) {
#pragma unroll
      for (int o = (LPT < 64 ? LPT : 64) / 2; o; o >>= 1) dot[k] += __shfl_xor(dot[k], o);
    }
    if constexpr (WPT > 1) {
      if (k0) __syncthreads();
#pragma unroll
      for (int k = 0; k < kRowsInFlight; ++k)
        if (lane == 0) red[wave * kRowsInFlight + k] = dot[k];
      __syncthreads();
      if (l < kRowsInFlight && live && k0 + l < p.topk) {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < WPT; ++i) s += red[(wave + i) * kRowsInFlight + l];
        p.dw[a0 + k0 + l] = s;
      }
    } else {
#pragma unroll
      for (int k = 0; k < kRowsInFlight; ++k)
        if (l == 0 && live && k0 + k < p.topk) p.dw[a0 + k0 + k] = dot[k];
    }
  }
}

}  // namespace mxf

namespace {

// Lanes that hold a row of `chunks` 16-byte chunks: a power of two from 8 to 64.
int lanes_per_token(int64_t chunks) { return chunks <= 8 ? 8 : chunks <= 16 ? 16 : chunks <= 32 ? 32 : 64; }
int64_t blocks_of(int64_t waves) { return (waves + 3) / 4; }
int64_t blocks_of_pads(int64_t rows) { return blocks_of((rows + mxf::kPadRows - 1) / mxf::kPadRows); }
// A row of a grid holds fewer than 2^24 blocks of 256 threads; the blocks of the last row that are too many find no token.
dim3 grid_of(int64_t blocks) {
  constexpr int64_t kRow = 0xFFFFFF;
  return blocks <= kRow ? dim3((unsigned)blocks) : dim3((unsigned)kRow, (unsigned)((blocks + kRow - 1) / kRow));
}

// Whether h (`copies` 2: and dh) fills most of the 256 MB last-level cache, so that none of it is still there: it is read past the caches
// then, where its rows are whole 128-byte lines (a line that two instructions share would come twice).
bool read_once(const mxf::RouteParams& p, int64_t size, int64_t copies) {
  return p.ldh * size % 128 == 0 && ((uintptr_t)p.h & 127) == 0 && copies * p.tokens * p.topk * p.D * size >= ((int64_t)192 << 20);
}

template <class Fn>
hipError_t with_lanes(int64_t chunks, Fn&& fn) {
  switch (lanes_per_token(chunks)) {
    case 8: return fn(std::integral_constant<int, 8>());
    case 16: return fn(std::integral_constant<int, 16>());
    case 32: return fn(std::integral_constant<int, 32>());
    default: return fn(std::integral_constant<int, 64>());
  }
}

template <class T, bool W, bool ONCE>
hipError_t launch_combine(const mxf::RouteParams& p, hipStream_t st) {
  const int64_t chunks = (p.D + mxf::Elem<T>::VEC - 1) / mxf::Elem<T>::VEC;
  const int64_t spans = (chunks + 63) / 64;
  return with_lanes(chunks, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    const int64_t waves = L == 64 ? p.tokens * spans : (p.tokens + 64 / L - 1) / (64 / L);
    hipLaunchKernelGGL((mxf::combine_kernel<T, L, W, ONCE>), grid_of(blocks_of(waves)), dim3(256), 0, st, p, (int)spans);
    return hipGetLastError();
  });
}

template <class T, bool DOT, bool ONCE>
hipError_t launch_combine_bwd(const mxf::RouteParams& p, hipStream_t st) {
  const int64_t chunks = (p.D + mxf::Elem<T>::VEC - 1) / mxf::Elem<T>::VEC;
  const auto go = [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    const int64_t tb = (p.tokens + 256 / L - 1) / (256 / L), pads = blocks_of_pads(p.rows);
    hipLaunchKernelGGL((mxf::combine_bwd_kernel<T, L, DOT, ONCE>), grid_of(pads + tb), dim3(256), 0, st, p, (unsigned)pads);
    return hipGetLastError();
  };
  // A block per token for long rows, or few tokens (us with a wavefront per token): 4096 tokens of 8 rows of 7168 BF16 207, 215; of 6
  // rows of 2048 47, 54; 8 tokens of 6 rows of 2048 5.0, 7.6; but 4096 tokens of 2 rows of 1411 20, 13.
  if (chunks >= 256 || (chunks > 64 && p.tokens <= 1024)) return go(std::integral_constant<int, 256>());
  return with_lanes(chunks, go);
}

}  // namespace

// D, ldx and ldh in bytes.
hipError_t mxf_launch_dispatch(const mxf::RouteParams& p, hipStream_t st) {
  const int64_t chunks = (p.D + 15) / 16, spans = (chunks + 63) / 64;
  return with_lanes(chunks, [&](auto lanes) {
    constexpr int L = decltype(lanes)::value;
    const int64_t tb = blocks_of(L == 64 ? p.tokens * spans : (p.tokens + 64 / L - 1) / (64 / L)), pads = blocks_of_pads(p.rows);
    if (pads + tb == 0) return hipSuccess;
    hipLaunchKernelGGL((mxf::dispatch_kernel<L>), grid_of(pads + tb), dim3(256), 0, st, p, (unsigned)pads, (int)spans);
    return hipGetLastError();
  });
}

hipError_t mxf_launch_combine(const mxf::RouteParams& p, bool f32, hipStream_t st) {
  // (us, through the caches): 4096 tokens of 8 rows of 7168 BF16 89, 96; of 6 rows of 2048 FP32 40, 43.5; but 8192 tokens of 4
  // rows of 1411 BF16 21.5, 20. Without weights (dispatch's gradient) h goes through the caches; the other way was not measured.
  if (p.w && read_once(p, f32 ? 4 : 2, 1))
    return f32 ? launch_combine<float, true, true>(p, st) : launch_combine<uint16_t, true, true>(p, st);
  if (p.w) return f32 ? launch_combine<float, true, false>(p, st) : launch_combine<uint16_t, true, false>(p, st);
  return f32 ? launch_combine<float, false, false>(p, st) : launch_combine<uint16_t, false, false>(p, st);
}

hipError_t mxf_launch_combine_bwd(const mxf::RouteParams& p, bool f32, hipStream_t st) {
  if (!p.dw) return f32 ? launch_combine_bwd<float, false, false>(p, st) : launch_combine_bwd<uint16_t, false, false>(p, st);
  // (us, through the caches): 4096 tokens of 8 rows of 7168 BF16 191, 206; of 2 rows of 4096 FP32 62, 71; of 6 rows of 2048 BF16
  // 46, 49; but 8192 tokens of 8 rows of 512 BF16, 134 MB of which a part is still there, 31.5, 26.3; 512 tokens of 8 rows of 5120 20, 18.
  if (read_once(p, f32 ? 4 : 2, 2))
    return f32 ? launch_combine_bwd<float, true, true>(p, st) : launch_combine_bwd<uint16_t, true, true>(p, st);
  return f32 ? launch_combine_bwd<float, true, false>(p, st) : launch_combine_bwd<uint16_t, true, false>(p, st);
}
