// Rotary positions, and the append of new tokens to a paged KV cache with the rotation folded
// into it.
//
// Each pair (x1, x2) of a head's first rot_dim channels is turned by a = p f_i:
//   y1 = s (x1 cos a - x2 sin a),  y2 = s (x2 cos a + x1 sin a);   the gradient turns by -a.
// Every element is read once and written once, so the kernels are bound by HBM. The angles are
// shared by all heads of a token: a workgroup forms the sines and cosines of its tokens once, in
// fp64 turns reduced to [-1/2, 1/2] (an fp32 product p f would be off by up to 2^-24 p f radians,
// 0.06 at p f = 10^6), keeps them in LDS as fp32, and then streams the heads: one unit is 16 channels
// (8 pairs) of one head, two 16-byte loads and stores in bf16.
#include "kda_device.h"
#include "kda_paged_int.h"

namespace kda {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxDim = 512;

// 8 consecutive channels as fp32, and back with one rounding each.
__device__ __forceinline__ void load8(const bf16* p, float (&x)[8]) {
  const bf16x8 v = *reinterpret_cast<const bf16x8*>(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (float)v[i];
}
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = a[i], x[4 + i] = b[i];
}
__device__ __forceinline__ void store8(bf16* p, const float (&x)[8]) {
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (bf16)x[i];
  *reinterpret_cast<bf16x8*>(p) = v;
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
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

// One unit: channels of one head at src to dst (either may be the other). c: the unit's index
// in the head; units below rot / 16 turn 8 pairs, the others copy 16 channels.
template <typename T, bool INTER>
__device__ __forceinline__ void unit(const T* src, T* dst, int c, int rot, const f32x2* cs) {
  float x[8], y[8];
  if (16 * c < rot) {
    const int a = INTER ? 16 * c : 8 * c, b = INTER ? 16 * c + 8 : rot / 2 + 8 * c;
    load8(src + a, x);
    load8(src + b, y);
    const f32x2* t = cs + 8 * c;
    if constexpr (INTER) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 u = t[i], w = t[4 + i];
        const float x1 = x[2 * i], x2 = x[2 * i + 1], y1 = y[2 * i], y2 = y[2 * i + 1];
        x[2 * i] = x1 * u[0] - x2 * u[1];
        x[2 * i + 1] = x2 * u[0] + x1 * u[1];
        y[2 * i] = y1 * w[0] - y2 * w[1];
        y[2 * i + 1] = y2 * w[0] + y1 * w[1];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const f32x2 u = t[i];
        const float x1 = x[i], x2 = y[i];
        x[i] = x1 * u[0] - x2 * u[1];
        y[i] = x2 * u[0] + x1 * u[1];
      }
    }
    store8(dst + a, x);
    store8(dst + b, y);
  } else if (dst != src) {
    load8(src + 16 * c, x);
    load8(src + 16 * c + 8, y);
    store8(dst + 16 * c, x);
    store8(dst + 16 * c + 8, y);
  }
}

// TB tokens per workgroup.
template <typename T, bool INTER, int TB>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a) {
  __shared__ f32x2 cs[TB][kMaxDim / 2];
  const int64_t t0 = (int64_t)blockIdx.x * TB;
  const int nt = (int)min((int64_t)TB, a.b.total_tokens - t0), half = a.rot_dim / 2;
  for (int i = threadIdx.x; i < nt * half; i += kThreads) {
    const int t = i / half, j = i - t * half;
    cs[t][j] = turn(a.positions[t0 + t], a.inv_freq[j], a.scale, a.inverse);
  }
  __syncthreads();
  const int C = a.head_dim / 16, heads = a.num_q_heads + a.num_k_heads;
  for (int u = threadIdx.x; u < nt * heads * C; u += kThreads) {
    const int hc = u / C, c = u - hc * C, t = hc / heads, h = hc - t * heads;
    const bool isq = h < a.num_q_heads;
    const int hh = isq ? h : h - a.num_q_heads;
    const T* src = (const T*)(isq ? a.q : a.k) + (t0 + t) * (isq ? a.q_stride : a.k_stride) + hh * a.head_dim;
    T* dst = (T*)(isq ? a.q_out : a.k_out) + (t0 + t) * (isq ? a.q_out_stride : a.k_out_stride) + hh * a.head_dim;
    unit<T, INTER>(src, dst, c, a.rot_dim, cs[t]);
  }
}

// First row of sequence n's new tokens (n = num_seqs: one past the last), clamped to the rows.
__device__ __forceinline__ int64_t first_row(const PagedBatch& b, int n) {
  if (!b.cu_seqlens) return b.total_tokens / b.num_seqs * n;
  const int64_t c = b.cu_seqlens[n];
  return c < 0 ? 0 : c > b.total_tokens ? b.total_tokens : c;
}

// The append: q's heads are turned, k's turned and stored in their pages, v's stored. The
// workgroup finds its tokens' sequences by counting the boundaries at or below each token, one
// boundary per thread: one round of loads where a binary search would wait for log2 N of them.
template <typename T, bool INTER, int TB>
__global__ __launch_bounds__(kThreads) void append_kernel(RopeArgs a) {
  __shared__ f32x2 cs[TB][kMaxDim / 2];
  __shared__ int seq[TB], pos[TB], page[TB];
  const int64_t t0 = (int64_t)blockIdx.x * TB;
  const int nt = (int)min((int64_t)TB, a.b.total_tokens - t0);
  if (threadIdx.x < TB) seq[threadIdx.x] = 0;
  __syncthreads();
  if (a.b.cu_seqlens) {
    int cnt[TB] = {};
    for (int n = threadIdx.x; n < a.b.num_seqs; n += kThreads) {
      const int64_t e = first_row(a.b, n + 1);
#pragma unroll
      for (int t = 0; t < TB; ++t) cnt[t] += e <= t0 + t;
    }
#pragma unroll
    for (int t = 0; t < TB; ++t)
      if (cnt[t]) atomicAdd(&seq[t], cnt[t]);
  } else if (threadIdx.x < nt) {
    seq[threadIdx.x] = (int)((t0 + threadIdx.x) / (a.b.total_tokens / a.b.num_seqs));
  }
  __syncthreads();
  if (threadIdx.x < nt) {
    const int t = threadIdx.x, n = seq[t];
    int p = -1, pg = -1;
    if (n < a.b.num_seqs && t0 + t >= first_row(a.b, 0)) {
      p = (int)(a.b.seq_lens[n] - (first_row(a.b, n + 1) - (t0 + t)));
      if (p >= 0 && p / a.b.page_size < a.b.max_pages) {
        pg = a.b.block_table[n * a.b.table_stride + p / a.b.page_size];
        if ((unsigned)pg >= (unsigned)a.b.num_pages) pg = -1;
      }
    } else {
      seq[t] = -1;  // behind the last sequence
    }
    pos[t] = p;
    page[t] = pg;
  }
  __syncthreads();
  if (a.inv_freq) {
    const int half = a.rot_dim / 2;
    for (int i = threadIdx.x; i < nt * half; i += kThreads) {
      const int t = i / half, j = i - t * half;
      cs[t][j] = turn(pos[t], a.inv_freq[j], a.scale, false);
    }
    __syncthreads();
  }
  const int D = a.head_dim, C = D / 16, ps = a.b.page_size;
  const int rot = a.inv_freq ? a.rot_dim : 0;
  const int nq = a.q ? a.num_q_heads : 0, nk = a.num_k_heads, heads = nq + 2 * nk;
  for (int u = threadIdx.x; u < nt * heads * C; u += kThreads) {
    const int hc = u / C, c = u - hc * C, t = hc / heads, h = hc - t * heads;
    if (seq[t] < 0) continue;
    if (h < nq) {
      unit<T, INTER>((const T*)a.q + (t0 + t) * a.q_stride + h * D, (T*)a.q_out + (t0 + t) * a.q_out_stride + h * D,
                     c, rot, cs[t]);
      continue;
    }
    if (page[t] < 0) continue;
    const bool isk = h < nq + nk;
    const int hh = isk ? h - nq : h - nq - nk;
    const int64_t at = ((int64_t)hh * ps + pos[t] % ps) * D;
    if (isk)
      unit<T, INTER>((const T*)a.k + (t0 + t) * a.k_stride + hh * D,
                     (T*)a.k_pages + page[t] * a.k_page_stride + at, c, rot, cs[t]);
    else
      unit<T, INTER>((const T*)a.v + (t0 + t) * a.v_stride + hh * D,
                     (T*)a.v_pages + page[t] * a.v_page_stride + at, c, 0, cs[t]);
  }
}

// Tokens per workgroup: enough units for every thread, and enough workgroups for the chip.
int tokens_per_group(int64_t tokens) { return tokens >= 4096 ? 4 : 1; }

template <typename T, bool INTER>
void rope_launch(const RopeArgs& a, bool append) {
  const int tb = tokens_per_group(a.b.total_tokens);
  const dim3 grid((unsigned)((a.b.total_tokens + tb - 1) / tb));
  if (append) {
    if (tb == 4)
      append_kernel<T, INTER, 4><<<grid, kThreads, 0, a.stream>>>(a);
    else
      append_kernel<T, INTER, 1><<<grid, kThreads, 0, a.stream>>>(a);
  } else {
    if (tb == 4)
      rope_kernel<T, INTER, 4><<<grid, kThreads, 0, a.stream>>>(a);
    else
      rope_kernel<T, INTER, 1><<<grid, kThreads, 0, a.stream>>>(a);
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
