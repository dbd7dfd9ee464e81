// Device helpers shared by the attention kernels over a paged cache.
#pragma once

#include "kda_device.h"
#include "kda_paged_int.h"

namespace kda {

// First row of sequence n's new tokens (n = num_seqs: one past the last), clamped to the rows.
__device__ __forceinline__ int64_t first_row(const PagedBatch& b, int n) {
  if (!b.cu_seqlens) return b.total_tokens / b.num_seqs * n;
  const int64_t c = b.cu_seqlens[n];
  return c < 0 ? 0 : c > b.total_tokens ? b.total_tokens : c;
}

// One sequence of a batch as the attention kernels see it. Its rows are the pairs (new token i,
// query head g of the G that share a K/V head), row i * G + g: all of them read the same keys.
struct Seq {
  int64_t row0;   // its first new token
  int rows;       // new tokens * G
  int p0;         // position of its first new token (may be negative)
  int lo, hi;     // keys lo .. hi - 1 are seen by some row (lo a multiple of the caller's unit)
};
__device__ __forceinline__ Seq seq_at(const AttnArgs& a, int n, int G, int unit) {
  Seq s;
  s.row0 = first_row(a.b, n);
  const int64_t m = max((int64_t)0, first_row(a.b, n + 1) - s.row0);
  const int64_t len = a.b.seq_lens[n], cap = (int64_t)a.b.max_pages * a.b.page_size;
  s.rows = (int)(m * G);
  s.p0 = (int)max(len - m, (int64_t)INT32_MIN);
  s.hi = (int)max((int64_t)0, min(min(len, cap), (int64_t)INT32_MAX - 4096));
  const int64_t lo = a.window ? (int64_t)s.p0 - a.window + 1 : 0;
  s.lo = lo > 0 ? (int)(lo / unit) * unit : 0;
  if (m == 0 || s.lo >= s.hi) s.lo = s.hi = 0;
  return s;
}

// Max / sum over the lanes l, l ^ 16, l ^ 32, l ^ 48, and l, l ^ 32 (v_permlane*_swap: swapping a register with a
// copy of itself leaves each lane one of the pair in each).
template <typename F>
__device__ __forceinline__ float across32(float x, F f) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return f(__builtin_bit_cast(float, (unsigned)r[0]), __builtin_bit_cast(float, (unsigned)r[1]));
}
template <typename F>
__device__ __forceinline__ float across16(float x, F f) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  return f(__builtin_bit_cast(float, (unsigned)r[0]), __builtin_bit_cast(float, (unsigned)r[1]));
}
struct MaxOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};
struct SumOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// A page's first element of one K/V head; entry < 0 or past the pool names no page, and page 0
// stands in for it, whose rows are then masked.
__device__ __forceinline__ bool page_ok(int entry, int num_pages) { return (unsigned)entry < (unsigned)num_pages; }

// Whether any of the elements in 16 bytes is an infinity or NaN.
template <typename T> __device__ __forceinline__ bool any_nonfinite(v4u32 x);
template <> __device__ __forceinline__ bool any_nonfinite<float>(v4u32 x) {
  bool r = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= (x[i] & 0x7f800000u) == 0x7f800000u;
  return r;
}
template <> __device__ __forceinline__ bool any_nonfinite<bf16>(v4u32 x) {
  bool r = false;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r |= (x[i] & 0x7f80u) == 0x7f80u || (x[i] & 0x7f800000u) == 0x7f800000u;
  return r;
}
__device__ __forceinline__ bool nonfinite(float x) {
  return (__builtin_bit_cast(unsigned, x) & 0x7f800000u) == 0x7f800000u;
}

constexpr float LN2 = 0.6931471805599453f;


}  // namespace kda
