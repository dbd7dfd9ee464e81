// Device helpers shared by the attention kernels over a paged cache.
#pragma once

#include "kda_device.h"
#include "kda_paged_int.h"

namespace kda {

// An item (the rows of one tile, over all their keys) that is cut between workgroups: its number of
// units and the first one's place among all. The workgroup that has its first part writes this, or n = -1 if
// there is none; every part leaves its sums in the workspace, and the join kernel adds them up.
struct Cut {
  int64_t at, per;  // per: units per workgroup
  int32_t n, h, tile, units;
};
// Part of workgroup w of an item that starts at `at`, in shares of `per` units: a workgroup leaves at most
// two, of the item that it starts with and of the one it ends with.
__host__ __device__ inline int64_t part_of(int64_t w, int64_t at, int64_t per) { return 2 * w + (at > w * per); }

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
  // (the kernels look a few thousand keys ahead of the last one, which 32 bits still have to hold)
  s.hi = (int)max((int64_t)0, min(min(len, cap), (int64_t)INT32_MAX - 65535));
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
// Largest of three, NaN if one is (v_maximum3_f32; fmaxf would first quiet each operand's NaN).
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}
__device__ __forceinline__ float across32_max(float x) {
  const unsigned u = __builtin_bit_cast(unsigned, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const float a = __builtin_bit_cast(float, (unsigned)r[0]), b = __builtin_bit_cast(float, (unsigned)r[1]);
  return max3(a, b, b);
}
struct SumOp {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};

// A float that was stored as part of 16 bytes of unsigned words.
typedef float __attribute__((may_alias)) lds_float;

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
  // an exponent of all ones carries into the sign's place
  unsigned r = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) r |= (x[i] & 0x7f807f80u) + 0x00800080u;
  return (r & 0x80008000u) != 0;
}

// 16 bytes of elements, infinities and NaN as 0.
template <typename T> __device__ __forceinline__ v4u32 finite_part(v4u32 x);
template <> __device__ __forceinline__ v4u32 finite_part<float>(v4u32 x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = (x[i] & 0x7f800000u) == 0x7f800000u ? 0u : x[i];
  return x;
}
template <> __device__ __forceinline__ v4u32 finite_part<bf16>(v4u32 x) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] &= ((x[i] & 0x7f80u) == 0x7f80u ? 0u : 0xffffu) | ((x[i] & 0x7f800000u) == 0x7f800000u ? 0u : 0xffff0000u);
  return x;
}
// PART 0: x, an infinity or NaN as 0; 1: 1 for +inf or NaN, else 0; 2: 1 for -inf or NaN, else 0.
template <int PART>
__device__ __forceinline__ float odd_part(float x) {
  const bool odd = (__builtin_bit_cast(unsigned, x) & 0x7f800000u) == 0x7f800000u;
  if constexpr (PART == 0) return odd ? 0.f : x;
  return odd && x != (PART == 1 ? -INFINITY : INFINITY) ? 1.f : 0.f;
}
template <int PART>
__device__ __forceinline__ bf16x8 odd_part(bf16x8 x) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = (bf16)odd_part<PART>((float)x[i]);
  return x;
}
template <int PART>
__device__ __forceinline__ f32x4 odd_part(f32x4 x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = odd_part<PART>(x[i]);
  return x;
}

// ------------------------------------------------------------------ the tile kernel's plan
// Sequences of more than row_limit rows go to the tile kernel (kda_attn_tile.hip), in tiles of
// tile_rows rows. The plan numbers the tiles of all sequences, sequence n's from seq[n].tile,
// and adds up what they cost for one K/V head: pre[i] is that of the tiles before tile i, seq[n].cost that of
// the sequences before n. A tile costs its units (32 keys) and kTileLead more: what is done before its
// first step and after its last takes about as long as that many steps (measured on a batch of short
// sequences: 50 us without the lead, when one workgroup in a batch got many tiles of one unit). All
// heads' tiles are laid end to end by (sequence, head, tile), each one's lead before its units.
constexpr int kTileUnit = 32;
constexpr int kTileLead = 4;

// A workgroup's waves (of 32 rows each), the waves per SIMD that its registers allow,
// and the workgroups: as many as the chip holds at once.
template <int D, bool BF16>
struct TileShape {
  static constexpr int WAVES = BF16 && D <= 128 ? 8 : 4, PER_SIMD = D <= 128 ? 2 : 1;
  static constexpr int ROWS = 32 * WAVES, GROUPS = 256 * 4 * PER_SIMD / WAVES;
};
template <typename F>
constexpr int attn_tile_shape(int D, bool bf16, F f) {
  return D == 64    ? (bf16 ? f(TileShape<64, true>()) : f(TileShape<64, false>()))
         : D == 128 ? (bf16 ? f(TileShape<128, true>()) : f(TileShape<128, false>()))
                    : (bf16 ? f(TileShape<256, true>()) : f(TileShape<256, false>()));
}
constexpr int attn_tile_rows(int D, bool bf16) {
  return attn_tile_shape(D, bf16, [](auto s) { return decltype(s)::ROWS; });
}
constexpr int attn_tile_groups(int D, bool bf16) {
  return attn_tile_shape(D, bf16, [](auto s) { return decltype(s)::GROUPS; });
}

struct SeqFirst {
  int64_t tile, cost;
};
struct TilePlan {
  int64_t* pre;
  SeqFirst* seq;
  Cut* cut;     // of each workgroup
  float* part;  // two partial results per workgroup: tile_rows rows of D sums, then m and l of each
};
__host__ __device__ inline int64_t max_tiles(int num_seqs, int64_t total_tokens, int G, int tile_rows) {
  return total_tokens * G / tile_rows + num_seqs;
}
constexpr int kMaxTileGroups = 512;
__host__ __device__ inline size_t tile_plan_bytes(int num_seqs, int64_t tiles) {
  return (sizeof(Cut) * kMaxTileGroups + (size_t)(tiles + 1) * 8 + sizeof(SeqFirst) * (num_seqs + 1) + 255) / 256 * 256;
}
__host__ __device__ inline TilePlan tile_plan_at(char* ws, int num_seqs, int64_t tiles) {
  TilePlan p;
  p.cut = reinterpret_cast<Cut*>(ws);
  p.seq = reinterpret_cast<SeqFirst*>(p.cut + kMaxTileGroups);
  p.pre = reinterpret_cast<int64_t*>(p.seq + num_seqs + 1);
  p.part = reinterpret_cast<float*>(ws + tile_plan_bytes(num_seqs, tiles));
  return p;
}
__host__ __device__ constexpr int64_t tile_part_floats(int rows, int D) { return (int64_t)rows * D + 2 * rows; }

// Keys lo .. hi - 1 that some row of a sequence's tile sees (lo a multiple of the unit).
struct TileKeys {
  int lo, hi, units;
};
__device__ __forceinline__ TileKeys tile_keys(const AttnArgs& a, const Seq& s, int tile, int G) {
  const int i0 = (int)((int64_t)tile * a.tile_rows / G);
  const int i1 = (int)((min((int64_t)(tile + 1) * a.tile_rows, (int64_t)s.rows) - 1) / G);
  TileKeys k;
  k.hi = (int)min((int64_t)s.hi, (int64_t)s.p0 + i1 + 1);
  const int64_t lo = a.window ? (int64_t)s.p0 + i0 - a.window + 1 : 0;
  k.lo = lo > 0 ? (int)(min(lo, (int64_t)INT32_MAX) / kTileUnit) * kTileUnit : 0;
  // a tile without keys is computed all the same: one unit that nobody sees
  k.units = k.hi > k.lo ? (k.hi - k.lo + kTileUnit - 1) / kTileUnit : 1;
  return k;
}

// The plan, by one workgroup of kPlanThreads threads.
constexpr int kPlanThreads = 256;
struct PlanLds {
  int64_t sums[kPlanThreads / 64];
};
__device__ __forceinline__ void make_tile_plan(const AttnArgs& a, PlanLds& lds) {
  constexpr int kWaves = kPlanThreads / 64;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, N = a.b.num_seqs;
  const int G = a.num_q_heads / a.num_kv_heads;
  const int64_t most = max_tiles(N, a.b.total_tokens, G, a.tile_rows);
  const TilePlan pl = tile_plan_at(a.tile_ws, N, most);
  auto scan = [&](int64_t x, int64_t* total) {  // inclusive, in thread order
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 63) lds.sums[wave] = x;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) x += lds.sums[w];
      all += lds.sums[w];
    }
    *total = all;
    return x;
  };
  int64_t carry = 0, total;
  for (int n0 = 0; n0 < N; n0 += kPlanThreads) {
    const int n = n0 + tid;
    int64_t tiles = 0;
    if (n < N) {
      const Seq s = seq_at(a, n, G, kTileUnit);
      if (s.rows > a.row_limit) tiles = (s.rows + a.tile_rows - 1) / a.tile_rows;
    }
    const int64_t x = carry + scan(tiles, &total);
    if (n < N) pl.seq[n].tile = min(most, x - tiles);
    carry = min(most, carry + total);
  }
  if (tid == 0) pl.seq[N].tile = carry;
  __syncthreads();
  const int64_t tiles = carry;
  carry = 0;
  for (int64_t i0 = 0; i0 < tiles; i0 += kPlanThreads) {
    const int64_t i = i0 + tid;
    int64_t units = 0;
    if (i < tiles) {
      int lo = 0, hi = N - 1;  // the last sequence that starts at or before tile i
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (pl.seq[mid].tile <= i) lo = mid;
        else hi = mid - 1;
      }
      units = tile_keys(a, seq_at(a, lo, G, kTileUnit), (int)(i - pl.seq[lo].tile), G).units + kTileLead;
    }
    const int64_t x = carry + scan(units, &total);
    if (i < tiles) pl.pre[i] = x - units;
    carry += total;
  }
  if (tid == 0) pl.pre[tiles] = carry;
  __syncthreads();
  for (int n = tid; n <= N; n += kPlanThreads) pl.seq[n].cost = pl.pre[pl.seq[n].tile];
}

// plan: whether the plan has to be made first (else the row kernel's launch has made it)
void launch_attn_tile(const AttnArgs& a, bool plan);
size_t attn_tile_bytes(int num_seqs, int64_t total_tokens, int G, int head_dim, bool bf16);

}  // namespace kda
