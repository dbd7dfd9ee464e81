// Causal attention of many new tokens over a paged KV cache: prompts and their chunks
// (kda_attn.hip takes the sequences of few rows).
//
// The formulas and the one pass with a running maximum are those of kda_attn.hip. Bound by the
// matrix cores: 4 D flops per (row, key). A workgroup of four waves takes a tile of 256 (or 128)
// rows of one sequence and K/V head, each wave 64 (32) of them, and walks over the keys 32 at a
// time, staged through LDS for all four.
//  - Scores are formed transposed, S^T = K Q^T, in 32 x 32 tiles: a lane holds 16 scores of one
//    row, so that the softmax is register work and one lane exchange, and the weights are already laid
//    out as the second operand of O^T = V^T P^T. The order of keys within an operand is free as long as
//    both operands share it, so no weight moves between lanes.
//  - 64 rows per wave halve the LDS reads per flop: with 32, four waves read 128 bytes per clock
//    at the full matrix rate, all that LDS gives.
//  - One wave per SIMD has nothing else to hide behind, so three steps run side by side: the scores of the
//    next 32 keys and the output of the last 32 on the matrix cores, the softmax of these 32 on the
//    vector units.
//  - The output is rescaled only when a maximum grows by more than 2^8: weights up to 2^8 cost
//    neither the fp32 sums nor the bf16 weights any relative accuracy.
//  - The tiles' keys are laid end to end and cut into equal shares, one per workgroup; a tile
//    that is cut leaves partial (o, m, l), joined with those of the row kernel.
#include "kda_attn.h"

namespace kda {

namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int SUB = kTileUnit;  // keys of a step

typedef __attribute__((ext_vector_type(16))) float f32x16;

template <typename MT, int D>
struct Tile {
  static constexpr int ES = sizeof(MT), RC = D * ES / 16;  // 16-byte parts of a row
  static constexpr int BYTES = SUB * D * ES;               // one step's keys (or values)
  static constexpr int NL = BYTES / 16 / kThreads;         // 16-byte loads per thread of them
  static constexpr int SF = RC / 2;                        // operand fragments of a score
  static constexpr int NC = D / 32;                        // 32-channel tiles of the output
  // PIPE: scores of step i + 1 beside the softmax of i and the output of i - 1, with keys i .. i + 2 and
  // values i - 1 .. i + 1 in LDS. fp32 heads of 256 channels have no room for that: keys and values of
  // steps i and i + 1.
  static constexpr bool PIPE = BYTES < 32768;
  static constexpr int AHEAD = PIPE ? 2 : 1, KSLOTS = AHEAD + 1, VSLOTS = PIPE ? 3 : 2;
  static constexpr int LDS = (KSLOTS + VSLOTS) * BYTES;
};

// The parts of a row are permuted in LDS: a key fragment is the same part of 32 rows, a transposed value
// fragment two parts of four rows (fp32: 32 channels of two rows), each without bank conflicts.
template <typename MT, int D>
__device__ __forceinline__ int k_at(int row, int part) {
  return row * (D * (int)sizeof(MT)) + (part ^ (row & 7)) * 16;
}
template <typename MT, int D>
__device__ __forceinline__ int v_at(int row, int part) {
  const int sw = sizeof(MT) == 2 ? (row & 3) << 1 : ((row >> 2) & 1) << 3;
  return row * (D * (int)sizeof(MT)) + (part ^ sw) * 16;
}

// Lane l is (m = l % 32, h = l / 32). In a 32 x 32 result it holds column m, rows
// 8 (r / 4) + 4 h + r % 4 for r = 0 .. 15. A 16-byte fragment holds 8 (fp32: 4) reduction
// indices of each half h; scores take part 2 s + h of a row as fragment s on both sides.
template <typename MT> struct Op;
template <> struct Op<bf16> {
  typedef struct { bf16x8 f[2]; } weights;
  __device__ __forceinline__ static f32x16 score(v4u32 k, v4u32 q, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, k), __builtin_bit_cast(bf16x8, q), c, 0, 0, 0);
  }
  __device__ __forceinline__ static weights pack(const f32x16& s) {
    weights w;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) w.f[i][e] = (bf16)s[8 * i + e];
    return w;
  }
  static constexpr int NF = 2;  // fragments of a step's weights
  __device__ __forceinline__ static f32x16 value(bf16x8 v, const weights& w, int i, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, w.f[i], c, 0, 0, 0);
  }
};
template <> struct Op<float> {
  typedef struct { f32x16 f; } weights;
  __device__ __forceinline__ static f32x16 score(v4u32 k, v4u32 q, f32x16 c) {
    const f32x4 x = __builtin_bit_cast(f32x4, k), y = __builtin_bit_cast(f32x4, q);
#pragma unroll
    for (int e = 0; e < 4; ++e) c = __builtin_amdgcn_mfma_f32_32x32x2f32(x[e], y[e], c, 0, 0, 0);
    return c;
  }
  __device__ __forceinline__ static weights pack(const f32x16& s) { return {s}; }
  static constexpr int NF = 16;
  __device__ __forceinline__ static f32x16 value(float v, const weights& w, int i, f32x16 c) {
    return __builtin_amdgcn_mfma_f32_32x32x2f32(v, w.f[i], c, 0, 0, 0);
  }
};

// Fragment i of the step's values for channels 32 c .. + 31, as the first operand of O^T = V^T P^T.
template <int D>
__device__ __forceinline__ bf16x8 value_frag(const char* v, int lane, int i, int c, bf16) {
  const int h = lane >> 5, half = (lane >> 4) & 1, row = 16 * i + 4 * h + ((lane & 15) >> 2);
  const int part = 4 * c + 2 * half + ((lane & 3) >> 1);
  const bf16x4 lo = ds_read_tr4((const bf16*)(v + v_at<bf16, D>(row, part) + 8 * (lane & 1)));
  const bf16x4 hi = ds_read_tr4((const bf16*)(v + v_at<bf16, D>(row + 8, part) + 8 * (lane & 1)));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <int D>
__device__ __forceinline__ float value_frag(const char* v, int lane, int i, int c, float) {
  const int h = lane >> 5, m = lane & 31;
  return *(const lds_float*)(v + v_at<float, D>(8 * (i / 4) + 4 * h + i % 4, 8 * c + (m >> 2)) + 4 * (m & 3));
}

// O^T += V^T P^T
template <typename MT, int D, int NQ>
__device__ __forceinline__ void add_values(const char* v, int lane, const typename Op<MT>::weights (&p)[NQ],
                                           f32x16 (&acc)[NQ][D / 32]) {
#pragma unroll
  for (int i = 0; i < Op<MT>::NF; ++i)
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const auto f = value_frag<D>(v, lane, i, c, MT());
#pragma unroll
      for (int q = 0; q < NQ; ++q) acc[q][c] = Op<MT>::value(f, p[q], i, acc[q][c]);
    }
}
// ------------------------------------------------------------------ the plan
constexpr int kPlan = 1024;
__global__ __launch_bounds__(kPlan) void tile_plan_kernel(AttnArgs a) {
  __shared__ int64_t lds[kPlan / 64];
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
    if (lane == 63) lds[wave] = x;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < kPlan / 64; ++w) {
      if (w < wave) x += lds[w];
      all += lds[w];
    }
    *total = all;
    return x;
  };
  int64_t carry = 0, total;
  for (int n0 = 0; n0 < N; n0 += kPlan) {
    const int n = n0 + tid;
    int64_t tiles = 0;
    if (n < N) {
      const Seq s = seq_at(a, n, G, SUB);
      if (s.rows > a.row_limit) tiles = (s.rows + a.tile_rows - 1) / a.tile_rows;
    }
    const int64_t x = carry + scan(tiles, &total);
    if (n < N) pl.tile_first[n] = min(most, x - tiles);
    carry = min(most, carry + total);
  }
  if (tid == 0) pl.tile_first[N] = carry;
  __syncthreads();
  const int64_t tiles = carry;
  carry = 0;
  for (int64_t i0 = 0; i0 < tiles; i0 += kPlan) {
    const int64_t i = i0 + tid;
    int64_t units = 0;
    if (i < tiles) {
      int lo = 0, hi = N - 1;  // the last sequence that starts at or before tile i
      while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (pl.tile_first[mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      units = tile_keys(a, seq_at(a, lo, G, SUB), (int)(i - pl.tile_first[lo]), G).units;
    }
    const int64_t x = carry + scan(units, &total);
    if (i < tiles) pl.pre[i] = x - units;
    carry += total;
  }
  if (tid == 0) pl.pre[tiles] = carry;
}

// ------------------------------------------------------------------ the kernel
template <typename MT, int D, int NQ>
__global__ __launch_bounds__(kThreads, 1) void tile_kernel(AttnArgs a) {
  typedef Tile<MT, D> T;
  typedef typename Op<MT>::weights weights;
  constexpr int RC = T::RC, NL = T::NL, SF = T::SF, NC = T::NC, ROWS = 128 * NQ;
  constexpr int KSLOTS = T::KSLOTS, VSLOTS = T::VSLOTS, AHEAD = T::AHEAD;
  __shared__ __align__(16) char lds[T::LDS];
  __shared__ int odd_at[VSLOTS][kWaves], counts[kWaves];
  char* const kl = lds;
  char* const vl = lds + KSLOTS * T::BYTES;
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 31, h2 = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.b.num_seqs, Hk = a.num_kv_heads, G = a.num_q_heads / Hk, ps = a.b.page_size,
            shift = __builtin_ctz(ps);
  const TilePlan pl = tile_plan_at(a.tile_ws, N, max_tiles(N, a.b.total_tokens, G, ROWS));

  // --- this workgroup's share of all units. The shares of the workgroups of one XCD (every
  // eighth) lie side by side, so that they read the same heads' keys through one L2.
  const int64_t total = Hk * pl.pre[pl.tile_first[N]], per = max((int64_t)1, (total + kTileGroups - 1) / kTileGroups);
  const int share = (blockIdx.x % 8) * (kTileGroups / 8) + blockIdx.x / 8;
  int64_t at = share * per;
  const int64_t begin = at, end = min(total, at + per);
  if (at >= end) return;
  // the entries of a sorted array that are at most x, counted over the threads
  auto count = [&](const int64_t* v, int64_t n, auto value, int64_t x) {
    int c = 0;
    for (int64_t i = tid; i < n; i += kThreads) c += value(v[i]) <= x;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) c += __shfl_xor(c, d);
    __syncthreads();
    if (lane == 0) counts[wave] = c;
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(counts[0] + counts[1] + counts[2] + counts[3]);
  };
  int n = count(pl.tile_first + 1, N, [&](int64_t f) { return Hk * pl.pre[f]; }, at);
  int64_t t0 = pl.tile_first[n], nt = pl.tile_first[n + 1] - t0;
  int64_t per_head = pl.pre[t0 + nt] - pl.pre[t0];
  int h = (int)((at - Hk * pl.pre[t0]) / per_head);
  int64_t off = at - Hk * pl.pre[t0] - h * per_head;  // unit within the (sequence, head)
  int tile = count(pl.pre + t0 + 1, nt, [&](int64_t f) { return f - pl.pre[t0]; }, off);
  off -= pl.pre[t0 + tile] - pl.pre[t0];              // unit within the tile

  const float c = a.scale * LOG2E, slack = 8.f / c;
  while (at < end) {
    if (tile == nt) {
      tile = 0;
      if (++h == Hk) {
        h = 0;
        do ++n, t0 += nt, nt = pl.tile_first[n + 1] - t0;
        while (nt == 0);
      }
      off = 0;
    }
    const Seq s = seq_at(a, n, G, SUB);
    const TileKeys tk = tile_keys(a, s, tile, G);
    const int u0 = (int)off, u1 = (int)min((int64_t)tk.units, u0 + (end - at));
    if (tk.units == 0) {
      ++tile;
      off = 0;
      continue;
    }

    // --- the wave's rows: lane m's queries and their visible keys; the ranges that some row
    // (any) and every row (full) sees, of the wave and of the workgroup
    int plo[NQ], phi[NQ];
    v4u32 qf[NQ][SF];
    int any_lo = INT32_MAX, any_hi = -1, full_lo = 0, full_hi = INT32_MAX;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int row = tile * ROWS + (wave * NQ + q) * 32 + m;
      const bool has = row < s.rows;
      const int tok = has ? row / G : 0, hq = h * G + (has ? row - tok * G : 0), p = s.p0 + tok;
      phi[q] = has ? min(p, s.hi - 1) : -1;
      plo[q] = a.window ? max(0, p - a.window + 1) : 0;
      const MT* src = (const MT*)a.q + (s.row0 + tok) * a.q_stride + hq * D;
#pragma unroll
      for (int i = 0; i < SF; ++i) {
        qf[q][i] = *reinterpret_cast<const v4u32*>((const char*)src + (2 * i + h2) * 16);
        if (!has) qf[q][i] = v4u32{0, 0, 0, 0};
      }
      any_lo = min(any_lo, has ? plo[q] : INT32_MAX);
      any_hi = max(any_hi, phi[q]);
      full_lo = max(full_lo, has ? plo[q] : 0);
      full_hi = min(full_hi, has ? phi[q] : INT32_MAX);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      any_lo = min(any_lo, __shfl_xor(any_lo, d));
      any_hi = max(any_hi, __shfl_xor(any_hi, d));
      full_lo = max(full_lo, __shfl_xor(full_lo, d));
      full_hi = min(full_hi, __shfl_xor(full_hi, d));
    }
    any_lo = __builtin_amdgcn_readfirstlane(any_lo);
    any_hi = __builtin_amdgcn_readfirstlane(any_hi);
    full_lo = __builtin_amdgcn_readfirstlane(full_lo);
    full_hi = __builtin_amdgcn_readfirstlane(full_hi);
    // rows of the tile run over consecutive tokens, so its ranges follow from the first and last
    const int last = (int)((min((int64_t)(tile + 1) * ROWS, (int64_t)s.rows) - 1) / G);
    const int pf = s.p0 + (int)((int64_t)tile * ROWS / G), pe = s.p0 + last;
    const int w_any_hi = min(pe, s.hi - 1), w_full_hi = min(pf, s.hi - 1);
    const int w_any_lo = a.window ? max(0, pf - a.window + 1) : 0, w_full_lo = a.window ? max(0, pe - a.window + 1) : 0;

    const int32_t* table = a.b.block_table + n * a.b.table_stride;
    const int64_t head = (int64_t)h * ps * D;
    const int key0 = tk.lo + u0 * SUB, nb = u1 - u0;

    // --- staging: step i's keys and values, thread by thread in 16-byte parts
    auto entries = [&](int i, int (&e)[2]) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int key = key0 + i * SUB + 16 * t;
        int x = -1;
        if (i < nb && key < s.hi) x = table[key >> shift];
        x = __builtin_amdgcn_readfirstlane(x);
        e[t] = page_ok(x, a.b.num_pages) ? x : -1;
      }
    };
    auto fetch = [&](const char* pages, int64_t stride, int i, const int (&e)[2], v4u32 (&r)[NL]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int grp = (j * kThreads + wave * 64) / RC / 16;  // 16-key group of the wave's rows
        const int key = key0 + i * SUB + 16 * grp;
        const MT* src = (const MT*)pages + max(grp ? e[1] : e[0], 0) * stride + head + (key & (ps - 1)) * D;
        r[j] = *reinterpret_cast<const v4u32*>((const char*)src + (j * kThreads + tid - grp * 16 * RC) * 16);
      }
    };
    auto put_k = [&](int i, const v4u32 (&r)[NL]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int x = j * kThreads + tid;
        *reinterpret_cast<v4u32*>(kl + (i % KSLOTS) * T::BYTES + k_at<MT, D>(x / RC, x % RC)) = r[j];
      }
    };
    // whether a step is seen whole by every row of the range, and none of its pages is missing
    auto whole = [&](int i, const int (&e)[2], int lo, int hi) __attribute__((always_inline)) {
      const int kb = key0 + i * SUB;
      return kb >= lo && kb + SUB - 1 <= hi && e[0] >= 0 && e[1] >= 0;
    };
    // Values that no row sees become 0. So does an infinity or NaN where some row does not see it, since a
    // weight of 0 would not hide it; the step is then marked, and the rows that do see it get it
    // from `add`.
    auto put_v = [&](int i, const int (&e)[2], v4u32 (&r)[NL]) __attribute__((always_inline)) {
      if (!whole(i, e, w_full_lo, w_full_hi)) {
        bool odd = false;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
          const int x = (j * kThreads + tid) / RC, key = key0 + i * SUB + x;
          if (key < w_any_lo || key > w_any_hi || (x < 16 ? e[0] : e[1]) < 0) r[j] = v4u32{0, 0, 0, 0};
          odd |= any_nonfinite<MT>(r[j]);
          r[j] = finite_part<MT>(r[j]);
        }
        if (lane == 0) odd_at[i % VSLOTS][wave] = 0;
        if (odd) odd_at[i % VSLOTS][wave] = 1;
      }
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        const int x = j * kThreads + tid;
        *reinterpret_cast<v4u32*>(vl + (i % VSLOTS) * T::BYTES + v_at<MT, D>(x / RC, x % RC)) = r[j];
      }
    };
    auto scores = [&](int i, f32x16 (&st)[NQ]) __attribute__((always_inline)) {
      const char* k = kl + (i % KSLOTS) * T::BYTES;
#pragma unroll
      for (int q = 0; q < NQ; ++q) st[q] = f32x16{};
#pragma unroll
      for (int f = 0; f < SF; ++f) {
        const v4u32 kf = *reinterpret_cast<const v4u32*>(k + k_at<MT, D>(m, 2 * f + h2));
#pragma unroll
        for (int q = 0; q < NQ; ++q) st[q] = Op<MT>::score(kf, qf[q][f], st[q]);
      }
    };

    f32x16 acc[NQ][NC] = {};
    float mx[NQ], sum[NQ];
#pragma unroll
    for (int q = 0; q < NQ; ++q) mx[q] = -INFINITY, sum[q] = 0.f;

    auto mask = [&](int i, const int (&e)[2], f32x16 (&st)[NQ]) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int key = key0 + i * SUB + 8 * (r / 4) + 4 * h2 + r % 4;
          if (key < plo[q] || key > phi[q] || e[r / 8] < 0) st[q][r] = -INFINITY;
        }
    };
    // softmax of one step: weights, running maximum and sum, and the factors for the output
    auto softmax = [&](f32x16 (&st)[NQ], weights (&p)[NQ], float (&al)[NQ]) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        float tm = st[q][0];
#pragma unroll
        for (int r = 1; r < 16; ++r) tm = fmaxf(tm, st[q][r]);
        tm = across32(tm, MaxOp());
        const float mn = tm > mx[q] + slack ? tm : mx[q], mu = mn == -INFINITY ? 0.f : mn, mc = mu * c;
        al[q] = exp2_f(mx[q] * c - mc);
        mx[q] = mn;
        float t = 0.f;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          st[q][r] = exp2_f(fmaf(st[q][r], c, -mc));
          t += st[q][r];
        }
        sum[q] = sum[q] * al[q] + t;
        p[q] = Op<MT>::pack(st[q]);
      }
    };
    auto rescale = [&](const float (&al)[NQ]) __attribute__((always_inline)) {
      bool any = false;
#pragma unroll
      for (int q = 0; q < NQ; ++q) any |= al[q] != 1.f;
      if (__any(any)) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int x = 0; x < NC; ++x) acc[q][x] *= al[q];
      }
    };
    auto add = [&](int i, const int (&e)[2], const weights (&p)[NQ]) __attribute__((always_inline)) {
      add_values<MT, D, NQ>(vl + ((i + VSLOTS) % VSLOTS) * T::BYTES, lane, p, acc);
      if (i >= 0 && !whole(i, e, w_full_lo, w_full_hi)) {
        bool odd = false;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) odd |= odd_at[i % VSLOTS][w] != 0;
        if (__any(odd)) {
#pragma unroll 1
          for (int x = 0; x < SUB; ++x) {
            const int key = key0 + i * SUB + x, pg = x < 16 ? e[0] : e[1];
            if (key > w_any_hi || pg < 0) continue;
            const MT* v = (const MT*)a.v_pages + pg * a.v_page_stride + head + (key & (ps - 1)) * D;
#pragma unroll
            for (int y = 0; y < NC * 16; ++y) {
              const float f = (float)v[32 * (y / 16) + 8 * (y / 4 % 4) + 4 * h2 + y % 4];
              if (f - f != 0.f)
#pragma unroll
                for (int q = 0; q < NQ; ++q)
                  if (key >= plo[q] && key <= phi[q]) acc[q][y / 16][y % 16] += f;
            }
          }
        }
      }
    };

    // --- the steps. During step i the keys of i + AHEAD and the values of i + 1 are fetched, and put
    // in LDS at its end.
    v4u32 kr[NL], vr[NL];
    int ep[2] = {-1, -1}, e0[2], e1[2], e2[2], e3[2];  // pages of steps i - 1 .. i + 3
    entries(0, e0);
    entries(1, e1);
    entries(2, e2);
    __syncthreads();  // LDS is free of the last tile's use
    fetch(a.k_pages, a.k_page_stride, 0, e0, kr);
    fetch(a.v_pages, a.v_page_stride, 0, e0, vr);
    put_k(0, kr);
    put_v(0, e0, vr);
    if (T::PIPE) {
      // "step -1", whose weights are 0
#pragma unroll
      for (int j = 0; j < NL; ++j)
        *reinterpret_cast<v4u32*>(vl + (VSLOTS - 1) * T::BYTES + (j * kThreads + tid) * 16) = v4u32{0, 0, 0, 0};
      if (nb > 1) {
        fetch(a.k_pages, a.k_page_stride, 1, e1, kr);
        put_k(1, kr);
      }
    }
    __syncthreads();
    weights p[NQ] = {}, pn[NQ];
    f32x16 cur[NQ], nxt[NQ];
    float al[NQ];
    if (T::PIPE) scores(0, cur);
#pragma unroll 1
    for (int i = 0; i < nb; ++i) {
      if (i + AHEAD < nb) fetch(a.k_pages, a.k_page_stride, i + AHEAD, AHEAD == 2 ? e2 : e1, kr);
      if (i + 1 < nb) fetch(a.v_pages, a.v_page_stride, i + 1, e1, vr);
      entries(i + 3, e3);
      // (behind the last step, the scores of what lies in LDS, which nobody reads)
      scores(T::PIPE ? i + 1 : i, T::PIPE ? nxt : cur);
      if (!whole(i, e0, full_lo, full_hi)) mask(i, e0, cur);
      softmax(cur, pn, al);
      if (T::PIPE) add(i - 1, ep, p);
      rescale(al);
      if (!T::PIPE) add(i, e0, pn);
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        p[q] = pn[q];
        if (T::PIPE) cur[q] = nxt[q];
      }
      if (i + AHEAD < nb) put_k(i + AHEAD, kr);
      if (i + 1 < nb) put_v(i + 1, e1, vr);
#pragma unroll
      for (int t = 0; t < 2; ++t) ep[t] = e0[t], e0[t] = e1[t], e1[t] = e2[t], e2[t] = e3[t];
      lds_barrier();
    }
    if (T::PIPE) add(nb - 1, ep, p);

    // --- out
    const bool done = u0 == 0 && u1 == tk.units;
    float* part = pl.part + (2 * (int64_t)share + (at == begin ? 0 : 1)) * tile_part_floats(ROWS, D);
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int r = (wave * NQ + q) * 32 + m, row = tile * ROWS + r;
      const float l = across32(sum[q], SumOp());
      if (row >= s.rows) continue;
      if (done) {
        const int tok = row / G;
        const int64_t out = (s.row0 + tok) * a.num_q_heads + h * G + row - tok * G;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        MT* dst = (MT*)a.o + out * D + 4 * h2;
#pragma unroll
        for (int x = 0; x < NC; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y)
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[32 * x + 8 * y + e] = from_f32<MT>(acc[q][x][4 * y + e] * inv);
        if (a.lse && h2 == 0) a.lse[out] = mx[q] * a.scale + (l == 0.f ? 0.f : logf(l));
      } else {
#pragma unroll
        for (int x = 0; x < NC; ++x)
#pragma unroll
          for (int y = 0; y < 4; ++y)
            *reinterpret_cast<f32x4*>(part + (int64_t)r * D + 32 * x + 8 * y + 4 * h2) =
                f32x4{acc[q][x][4 * y], acc[q][x][4 * y + 1], acc[q][x][4 * y + 2], acc[q][x][4 * y + 3]};
        if (h2 == 0) part[ROWS * D + 2 * r] = mx[q], part[ROWS * D + 2 * r + 1] = l;
      }
    }
    at += u1 - u0;
    off = 0;
    ++tile;
  }
}

template <typename MT, int D>
void launch(const AttnArgs& a) {
  if constexpr (attn_tile_rows(D, sizeof(MT) == 2) == 256)
    tile_kernel<MT, D, 2><<<kTileGroups, kThreads, 0, a.stream>>>(a);
  else
    tile_kernel<MT, D, 1><<<kTileGroups, kThreads, 0, a.stream>>>(a);
}

}  // namespace

void launch_attn_tile(const AttnArgs& a) {
  tile_plan_kernel<<<1, kPlan, 0, a.stream>>>(a);
  if (a.dtype_bf16) {
    if (a.head_dim == 64) launch<bf16, 64>(a);
    if (a.head_dim == 128) launch<bf16, 128>(a);
    if (a.head_dim == 256) launch<bf16, 256>(a);
  } else {
    if (a.head_dim == 64) launch<float, 64>(a);
    if (a.head_dim == 128) launch<float, 128>(a);
    if (a.head_dim == 256) launch<float, 256>(a);
  }
}

size_t attn_tile_bytes(int num_seqs, int64_t total_tokens, int G, int head_dim, int tile_rows) {
  return tile_plan_bytes(num_seqs, max_tiles(num_seqs, total_tokens, G, tile_rows)) +
         (size_t)(2 * kTileGroups * tile_part_floats(tile_rows, head_dim)) * 4;
}

}  // namespace kda
