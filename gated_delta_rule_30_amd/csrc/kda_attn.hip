// Causal attention of new tokens over a paged KV cache (include/kda_paged.h).
#include "kda_device.h"
#include "kda_paged_int.h"

namespace kda {

namespace {

__device__ __forceinline__ int64_t first_row(const PagedBatch& b, int n) {
  if (!b.cu_seqlens) return b.total_tokens / b.num_seqs * n;
  const int64_t c = b.cu_seqlens[n];
  return c < 0 ? 0 : c > b.total_tokens ? b.total_tokens : c;
}

// One wave per (token, query head): D / 64 channels per lane, one key at a time.
template <typename T, int D>
__global__ __launch_bounds__(64) void attn_kernel(AttnArgs a) {
  constexpr int E = D / 64;
  const int64_t t = blockIdx.x / a.num_q_heads;
  const int hq = (int)(blockIdx.x - t * a.num_q_heads), h = hq / (a.num_q_heads / a.num_kv_heads);
  int n = 0;
  while (n < a.b.num_seqs && first_row(a.b, n + 1) <= t) ++n;
  if (n == a.b.num_seqs || t < first_row(a.b, 0)) return;
  const int ps = a.b.page_size;
  const int64_t p = a.b.seq_lens[n] - (first_row(a.b, n + 1) - t);
  const int64_t lo = a.window ? max((int64_t)0, p - a.window + 1) : 0;
  const int64_t hi = min(p, (int64_t)a.b.max_pages * ps - 1);
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e)
    q[e] = to_f32<T>(((const T*)a.q)[t * a.q_stride + hq * D + e * 64 + threadIdx.x]) * a.scale;
  for (int64_t j = lo; j <= hi; ++j) {
    const int pg = a.b.block_table[n * a.b.table_stride + j / ps];
    if ((unsigned)pg >= (unsigned)a.b.num_pages) continue;
    const int64_t at = ((int64_t)h * ps + j % ps) * D + threadIdx.x;
    const T* k = (const T*)a.k_pages + pg * a.k_page_stride + at;
    const T* v = (const T*)a.v_pages + pg * a.v_page_stride + at;
    float s = 0.f;
    for (int e = 0; e < E; ++e) s += q[e] * to_f32<T>(k[e * 64]);
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    if (s == -INFINITY) continue;
    const float mn = fmaxf(m, s), al = expf(m - mn), w = expf(s - mn);
    l = l * al + w;
    for (int e = 0; e < E; ++e) o[e] = o[e] * al + w * to_f32<T>(v[e * 64]);
    m = mn;
  }
  for (int e = 0; e < E; ++e)
    ((T*)a.o)[(t * a.num_q_heads + hq) * D + e * 64 + threadIdx.x] = from_f32<T>(l > 0.f ? o[e] / l : l);
  if (a.lse && threadIdx.x == 0) a.lse[t * a.num_q_heads + hq] = m + logf(l);
}

}  // namespace

size_t attn_workspace_bytes(int, int64_t, int, int, int, bool) { return 256; }

hipError_t launch_attn(const AttnArgs& a) {
  const unsigned g = (unsigned)(a.b.total_tokens * a.num_q_heads);
  if (g == 0) return hipSuccess;
  if (a.dtype_bf16) {
    if (a.head_dim == 64) attn_kernel<bf16, 64><<<g, 64, 0, a.stream>>>(a);
    if (a.head_dim == 128) attn_kernel<bf16, 128><<<g, 64, 0, a.stream>>>(a);
    if (a.head_dim == 256) attn_kernel<bf16, 256><<<g, 64, 0, a.stream>>>(a);
  } else {
    if (a.head_dim == 64) attn_kernel<float, 64><<<g, 64, 0, a.stream>>>(a);
    if (a.head_dim == 128) attn_kernel<float, 128><<<g, 64, 0, a.stream>>>(a);
    if (a.head_dim == 256) attn_kernel<float, 256><<<g, 64, 0, a.stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace kda
