// Rotary positions, and the append of new tokens to a paged KV cache with the rotation folded
// into it.
//
// Each pair (x1, x2) of a head's first rot_dim channels is turned by a = p f_i:
//   y1 = s (x1 cos a - x2 sin a),  y2 = s (x2 cos a + x1 sin a);   the gradient turns by -a.
// Every element is read once and written once, so the kernels are bound by HBM. The angles are
// shared by all heads of a token: a workgroup forms the sines and cosines of its tokens once, in
// fp64 turns reduced to [-1/2, 1/2] (an fp32 product p f would be off by up to 2^-24 p f radians,
// 0.06 at p f = 10^6), keeps them in LDS as fp32, and then streams the heads: one unit is two
// 16-byte loads and stores of one head.
// Measured: 16384 tokens of 32 + 8 heads of 128, bf16, either pairing: 336 MB in 49 to 54 us, 6.2 to 6.9 TB/s (fp32, 8192
// tokens: 50 us; with 16 channels in a row per lane fp32 took 65, heads of 256 up to 113 where they take 39). The append of 20 chunks of 64 to
// 2048 tokens (213 MB): 34 to 35 us, 6.2 TB/s; of 256 single tokens (6 MB): 4.5 us, launch and latency.
#include "kda_device.h"
#include "kda_paged_int.h"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 512;

// Channels of 16 bytes, as fp32, and back with one rounding each.
template <typename T>
constexpr int kWide = 16 / (int)sizeof(T);
__device__ __forceinline__ void load(const bf16* p, float (&x)[8]) {
  const bf16x8 v = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
}
__device__ __forceinline__ void load(const float* p, float (&x)[4]) {
  const f32x4 v = *reinterpret_cast<const f32x4*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = v[i];
}
template <bool STREAM>
__device__ __forceinline__ void store(bf16* p, const float (&x)[8]) {
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (bf16)x[i];
  if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<bf16x8*>(p));
  else *reinterpret_cast<bf16x8*>(p) = v;
}
template <bool STREAM>
__device__ __forceinline__ void store(float* p, const float (&x)[4]) {
  const f32x4 v = {x[0], x[1], x[2], x[3]};
  if constexpr (STREAM) __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(p));
  else *reinterpret_cast<f32x4*>(p) = v;
}

// Sine and cosine of p * f (radians) times scale. The angle is formed in turns, f / (2 pi) and its
// product with p each as a sum of two doubles: at p = 2^31 one double alone would leave 6e-7
// radians. What is left of it after whole turns are dropped is exact to fp32.
__device__ __forceinline__ f32x2 turn(int p, double f, float scale, bool inverse) {
  constexpr double kHi = 0.15915494309189535, kLo = -9.839338337591243e-18;  // 1 / (2 pi)
  const double g = f * kHi, gl = fma(f, kHi, -g) + f * kLo;
  const double t = (double)p * g, tl = fma((double)p, g, -t) + (double)p * gl;
  float s, c;
  sincospif(2.f * (float)((t - rint(t)) + tl), &s, &c);
  return f32x2{scale * c, inverse ? -scale * s : scale * s};
}

// One unit: twice 16 bytes of one head at src to dst (either may be the other), half of the turned channels (or of the
// others) apart, so that what the lanes of a wave load or store at once lies side by side. c: the unit's index in the
// head, the turning ones first.
template <typename T, bool INTER, bool STREAM>
__device__ __forceinline__ void unit(const T* src, T* dst, int c, int dim, int rot, const f32x2* cs) {
  constexpr int W = kWide<T>;
  float x[W], y[W];
  if (2 * W * c < rot) {
    const int a = W * c, b = rot / 2 + W * c;
    load(src + a, x);
    load(src + b, y);
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < W / 2; ++i) {
        const f32x2 u = cs[a / 2 + i], w = cs[b / 2 + i];
        const float x1 = x[2 * i], x2 = x[2 * i + 1], y1 = y[2 * i], y2 = y[2 * i + 1];
        x[2 * i] = x1 * u[0] - x2 * u[1];
        x[2 * i + 1] = x2 * u[0] + x1 * u[1];
        y[2 * i] = y1 * w[0] - y2 * w[1];
        y[2 * i + 1] = y2 * w[0] + y1 * w[1];
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const f32x2 u = cs[a + i];
        const float x1 = x[i], x2 = y[i];
        x[i] = x1 * u[0] - x2 * u[1];
        y[i] = x2 * u[0] + x1 * u[1];
      }
    }
    store<STREAM>(dst + a, x);
    store<STREAM>(dst + b, y);
  } else if (dst != src) {
    const int a = rot / 2 + W * c, b = a + (dim - rot) / 2;
    load(src + a, x);
    load(src + b, y);
    store<STREAM>(dst + a, x);
    store<STREAM>(dst + b, y);
  }
}

// This workgroup's token: a grid holds 2^32 threads in one dimension, so many tokens take two.
constexpr int kGridTokens = 1 << 22;
__device__ __forceinline__ int64_t token() { return (int64_t)blockIdx.y * kGridTokens + blockIdx.x; }

// One token per workgroup.
template <typename T, bool INTER, bool STREAM>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a) {
  __shared__ f32x2 cs[kMaxDim / 2];
  const int64_t t = token();
  if (t >= a.b.total_tokens) return;
  const int half = a.rot_dim / 2;
  for (int j = threadIdx.x; j < half; j += kThreads) cs[j] = turn(a.positions[t], a.inv_freq[j], a.scale, a.inverse);
  __syncthreads();
  const int C = a.head_dim / (2 * kWide<T>), heads = a.num_q_heads + a.num_k_heads;
  for (int u = threadIdx.x; u < heads * C; u += kThreads) {
    const int h = u / C, c = u - h * C;
    const bool isq = h < a.num_q_heads;
    const int hh = isq ? h : h - a.num_q_heads;
    const T* src = (const T*)(isq ? a.q : a.k) + t * (isq ? a.q_stride : a.k_stride) + hh * a.head_dim;
    T* dst = (T*)(isq ? a.q_out : a.k_out) + t * (isq ? a.q_out_stride : a.k_out_stride) + hh * a.head_dim;
    unit<T, INTER, STREAM>(src, dst, c, a.head_dim, a.rot_dim, cs);
  }
}

// First row of sequence n's new tokens (n = num_seqs: one past the last), clamped to the rows.
__device__ __forceinline__ int64_t first_row(const PagedBatch& b, int n) {
  if (!b.cu_seqlens) return b.total_tokens / b.num_seqs * n;
  const int64_t c = b.cu_seqlens[n];
  return c < 0 ? 0 : c > b.total_tokens ? b.total_tokens : c;
}

// The append: q's heads are turned, k's turned and stored in their pages, v's stored. The
// workgroup finds its token's sequence by counting the boundaries at or below the token, one
// boundary per thread: one round of loads where a binary search would wait for log2 N of them.
template <typename T, bool INTER, bool STREAM>
__global__ __launch_bounds__(kThreads) void append_kernel(RopeArgs a) {
  __shared__ f32x2 cs[kMaxDim / 2];
  __shared__ int seq, pos, page;
  const int64_t t = token();
  if (t >= a.b.total_tokens) return;
  if (threadIdx.x == 0) seq = a.b.cu_seqlens ? 0 : (int)(t / (a.b.total_tokens / a.b.num_seqs));
  __syncthreads();
  if (a.b.cu_seqlens) {
    int count = 0;
    for (int n = threadIdx.x; n < a.b.num_seqs; n += kThreads) count += first_row(a.b, n + 1) <= t;
    if (count) atomicAdd(&seq, count);
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    const int n = seq;
    int p = -1, pg = -1;
    if (n < a.b.num_seqs && t >= first_row(a.b, 0)) {
      p = (int)(a.b.seq_lens[n] - (first_row(a.b, n + 1) - t));
      if (p >= 0 && p / a.b.page_size < a.b.max_pages) {
        pg = a.b.block_table[n * a.b.table_stride + p / a.b.page_size];
        if ((unsigned)pg >= (unsigned)a.b.num_pages) pg = -1;
      }
    } else {
      seq = -1;  // behind the last sequence
    }
    pos = p;
    page = pg;
  }
  __syncthreads();
  if (seq < 0) return;
  if (a.inv_freq) {
    for (int j = threadIdx.x; j < a.rot_dim / 2; j += kThreads) cs[j] = turn(pos, a.inv_freq[j], a.scale, false);
    __syncthreads();
  }
  const int D = a.head_dim, C = D / (2 * kWide<T>), ps = a.b.page_size;
  const int rot = a.inv_freq ? a.rot_dim : 0;
  const int nq = a.q ? a.num_q_heads : 0, nk = a.num_k_heads, heads = nq + 2 * nk;
  for (int u = threadIdx.x; u < heads * C; u += kThreads) {
    const int h = u / C, c = u - h * C;
    if (h < nq) {
      unit<T, INTER, STREAM>((const T*)a.q + t * a.q_stride + h * D, (T*)a.q_out + t * a.q_out_stride + h * D, c, D, rot, cs);
      continue;
    }
    if (page < 0) continue;
    const bool isk = h < nq + nk;
    const int hh = isk ? h - nq : h - nq - nk;
    const int64_t at = ((int64_t)hh * ps + pos % ps) * D;
    if (isk)
      unit<T, INTER, STREAM>((const T*)a.k + t * a.k_stride + hh * D, (T*)a.k_pages + page * a.k_page_stride + at, c, D,
                             rot, cs);
    else
      unit<T, INTER, STREAM>((const T*)a.v + t * a.v_stride + hh * D, (T*)a.v_pages + page * a.v_page_stride + at, c, D, 0,
                             cs);
  }
}

// What is more than the L2s hold (32 MB) passes them by: 16384 tokens of 40 heads turn in 57 us where they
// took 65 us through the caches (5.9 TB/s). Less is left in them for the next kernel.
constexpr int64_t kStreamBytes = 32 << 20;

template <typename T, bool INTER>
void rope_launch(const RopeArgs& a, bool append) {
  const int64_t tokens = a.b.total_tokens;
  const dim3 grid((unsigned)(tokens < kGridTokens ? tokens : kGridTokens),
                  (unsigned)((tokens + kGridTokens - 1) / kGridTokens));
  const int64_t heads = a.num_q_heads + (append ? 2 : 1) * a.num_k_heads;
  const bool stream = a.b.total_tokens * heads * a.head_dim * (int64_t)sizeof(T) > kStreamBytes;
  if (append) {
    if (stream)
      append_kernel<T, INTER, true><<<grid, kThreads, 0, a.stream>>>(a);
    else
      append_kernel<T, INTER, false><<<grid, kThreads, 0, a.stream>>>(a);
  } else {
    if (stream)
      rope_kernel<T, INTER, true><<<grid, kThreads, 0, a.stream>>>(a);
    else
      rope_kernel<T, INTER, false><<<grid, kThreads, 0, a.stream>>>(a);
  }
}

hipError_t launch(const RopeArgs& a, bool append) {
  if (a.b.total_tokens == 0) return hipSuccess;
  if (a.dtype_bf16)
    a.interleaved ? rope_launch<bf16, true>(a, append) : rope_launch<bf16, false>(a, append);
  else
    a.interleaved ? rope_launch<float, true>(a, append) : rope_launch<float, false>(a, append);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a) { return launch(a, false); }
hipError_t launch_append(const RopeArgs& a) { return launch(a, true); }

}  // namespace kda
