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

constexpr int SUB = kTileUnit;  // keys of a step

typedef __attribute__((ext_vector_type(16))) float f32x16;

template <typename MT, int D>
struct Tile {
  typedef TileShape<D, sizeof(MT) == 2> S;
  static constexpr int ES = sizeof(MT), RC = D * ES / 16;  // 16-byte parts of a row
  static constexpr int WAVES = S::WAVES, THREADS = 64 * WAVES, ROWS = S::ROWS;
  static constexpr int BYTES = SUB * D * ES;               // one step's keys (or values)
  static constexpr int PARTS = BYTES / 16;
  static constexpr int NL = (PARTS + THREADS - 1) / THREADS;  // 16-byte loads per thread of them
  static constexpr int SF = RC / 2;                        // operand fragments of a score
  static constexpr int NC = D / 32;                        // 32-channel tiles of the output
  // PIPE: scores of step i + 1 beside the softmax of i and the output of i - 1, with keys i .. i + 2 and
  // values i - 1 .. i + 1 in LDS; otherwise keys and values of steps i and i + 1. In fp32 the products take
  // 25 times as long as the softmax, so there is nothing to gain.
  static constexpr bool PIPE = ES == 2;
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
  __device__ __forceinline__ static void hold(weights& w) { asm volatile("" : "+v"(w.f[0]), "+v"(w.f[1])); }
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
  __device__ __forceinline__ static void hold(weights& w) { asm volatile("" : "+v"(w.f)); }
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
template <typename MT, int D>
__device__ __forceinline__ void add_values(const char* v, int lane, const typename Op<MT>::weights& p,
                                           f32x16 (&acc)[D / 32]) {
#pragma unroll
  for (int i = 0; i < Op<MT>::NF; ++i)
#pragma unroll
    for (int c = 0; c < D / 32; ++c) acc[c] = Op<MT>::value(value_frag<D>(v, lane, i, c, MT()), p, i, acc[c]);
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
// Where a workgroup is in its share: kept in LDS between tiles, and the arguments read again
// where they are needed, so that the steps' loop holds no scalar registers that it does not use.
struct Walk {
  int64_t at, end, begin, t0, nt;  // units; the sequence's tiles t0 .. t0 + nt - 1
  int n, h, tile, off;             // off: units of the tile that are done
};
__device__ __forceinline__ AttnArgs fresh_args() {
  auto p = (const __attribute__((address_space(4))) char*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttnArgs*)(const void*)p;
}

template <typename MT, int D>
__global__ __launch_bounds__((Tile<MT, D>::THREADS), (Tile<MT, D>::S::PER_SIMD)) void tile_kernel(AttnArgs) {
  typedef Tile<MT, D> T;
  typedef typename Op<MT>::weights weights;
  constexpr int kThreads = T::THREADS, kWaves = T::WAVES, kGroups = T::S::GROUPS, ROWS = T::ROWS;
  constexpr int RC = T::RC, NL = T::NL, SF = T::SF, NC = T::NC, ES = T::ES, BYTES = T::BYTES;
  constexpr int KSLOTS = T::KSLOTS, VSLOTS = T::VSLOTS, AHEAD = T::AHEAD;
  __shared__ __align__(16) char lds[T::LDS];
  __shared__ int odd_at[VSLOTS][kWaves], counts[kWaves];
  __shared__ Walk walk;
  char* const kl = lds;
  char* const vl = lds + KSLOTS * BYTES;
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 31, h2 = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int share = (blockIdx.x % 8) * (kGroups / 8) + blockIdx.x / 8;

  // --- this workgroup's share of all units. The shares of the workgroups of one XCD (every
  // eighth) lie side by side, so that they read the same heads' keys through one L2.
  {
    const AttnArgs a = fresh_args();
    const int N = a.b.num_seqs, Hk = a.num_kv_heads, G = a.num_q_heads / Hk;
    const TilePlan pl = tile_plan_at(a.tile_ws, N, max_tiles(N, a.b.total_tokens, G, ROWS));
    const int64_t total = Hk * pl.pre[pl.tile_first[N]], per = max((int64_t)1, (total + kGroups - 1) / kGroups);
    const int64_t at = share * per;
    if (at >= total) return;
    // the entries of a sorted array that are at most x, counted over the threads
    auto count = [&](int64_t n, auto entry, int64_t x) {
      int c = 0;
      for (int64_t i = tid; i < n; i += kThreads) c += entry(i) <= x;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) c += __shfl_xor(c, d);
      __syncthreads();
      if (lane == 0) counts[wave] = c;
      __syncthreads();
      int all = 0;
      for (int w = 0; w < kWaves; ++w) all += counts[w];
      return all;
    };
    const int n = count(N, [&](int64_t i) { return Hk * pl.pre[pl.tile_first[i + 1]]; }, at);
    const int64_t t0 = pl.tile_first[n], nt = pl.tile_first[n + 1] - t0, u0 = pl.pre[t0];
    const int64_t per_head = pl.pre[t0 + nt] - u0;
    const int h = (int)((at - Hk * u0) / per_head);
    const int64_t off = at - Hk * u0 - h * per_head;
    const int tile = count(nt, [&](int64_t i) { return pl.pre[t0 + i + 1] - u0; }, off);
    if (tid == 0) walk = {at, min(total, at + per), at, t0, nt, n, h, tile, (int)(off - (pl.pre[t0 + tile] - u0))};
  }
  for (;;) {
    __syncthreads();  // `walk` is up to date, and LDS free of the last tile's use
    if (walk.at >= walk.end) return;
    if (walk.tile == walk.nt) {
      __syncthreads();
      if (tid == 0) {
        const AttnArgs a = fresh_args();
        const int G = a.num_q_heads / a.num_kv_heads;
        const TilePlan pl = tile_plan_at(a.tile_ws, a.b.num_seqs, max_tiles(a.b.num_seqs, a.b.total_tokens, G, ROWS));
        walk.tile = 0;
        if (++walk.h == a.num_kv_heads) {
          walk.h = 0;
          do ++walk.n, walk.t0 += walk.nt, walk.nt = pl.tile_first[walk.n + 1] - walk.t0;
          while (walk.nt == 0);
        }
      }
      continue;
    }
    const AttnArgs a = fresh_args();
    const int n = __builtin_amdgcn_readfirstlane(walk.n), h = __builtin_amdgcn_readfirstlane(walk.h),
              tile = __builtin_amdgcn_readfirstlane(walk.tile), off = __builtin_amdgcn_readfirstlane(walk.off);
    const int left = __builtin_amdgcn_readfirstlane((int)min(walk.end - walk.at, (int64_t)INT32_MAX));
    const int G = a.num_q_heads / a.num_kv_heads, ps1 = a.b.page_size - 1, shift = __builtin_ctz(a.b.page_size);
    const Seq s = seq_at(a, n, G, SUB);
    const TileKeys tk = tile_keys(a, s, tile, G);
    const int nb = min(tk.units - off, left);  // steps
    if (nb <= 0) {                             // a tile without keys
      __syncthreads();
      if (tid == 0) ++walk.tile, walk.off = 0;
      continue;
    }

    // --- the wave's rows: lane m's query and its visible keys plo .. phi; the ranges that every row of the
    // wave sees (full), and that some (any) and every row of the workgroup sees
    const int row = tile * ROWS + wave * 32 + m;
    const bool has = row < s.rows;
    int plo, phi;
    v4u32 qf[SF];
    {
      const int tok = has ? row / G : 0, hq = h * G + (has ? row - tok * G : 0), p = s.p0 + tok;
      phi = has ? min(p, s.hi - 1) : -1;
      plo = a.window ? max(0, p - a.window + 1) : 0;
      const char* src = (const char*)((const MT*)a.q + (s.row0 + tok) * a.q_stride + hq * D) + h2 * 16;
#pragma unroll
      for (int i = 0; i < SF; ++i) qf[i] = *reinterpret_cast<const v4u32*>(src + 32 * i);
    }
    int full_lo = has ? plo : 0, full_hi = has ? phi : INT32_MAX;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      full_lo = max(full_lo, __shfl_xor(full_lo, d));
      full_hi = min(full_hi, __shfl_xor(full_hi, d));
    }
    full_lo = __builtin_amdgcn_readfirstlane(full_lo);
    full_hi = __builtin_amdgcn_readfirstlane(full_hi);
    // rows of the tile run over consecutive tokens, so its ranges follow from the first and last
    const int last = (int)((min((int64_t)(tile + 1) * ROWS, (int64_t)s.rows) - 1) / G);
    const int pf = s.p0 + (int)((int64_t)tile * ROWS / G), pe = s.p0 + last;
    const int w_any_hi = min(pe, s.hi - 1), w_full_hi = min(pf, s.hi - 1);
    const int w_any_lo = a.window ? max(0, pf - a.window + 1) : 0, w_full_lo = a.window ? max(0, pe - a.window + 1) : 0;

    const int32_t* table = a.b.block_table + n * a.b.table_stride;
    const int num_pages = a.b.num_pages;
    const int key0 = tk.lo + off * SUB, hi_key = min(s.hi, key0 + nb * SUB);
    const int64_t kstride = a.k_page_stride * ES, vstride = a.v_page_stride * ES;
    const char* const kbase = a.k_pages + (int64_t)h * (ps1 + 1) * D * ES;
    const char* const vbase = a.v_pages + (int64_t)h * (ps1 + 1) * D * ES;
    const float c = a.scale * LOG2E, slack = 8.f / c;

    // --- staging: a step's keys and values, thread by thread in 16-byte parts. A wave's parts lie in
    // one 16-key group of the step, or (GRPS 2) half of them in each; a group lies in one page.
    // The table is read for 64 steps at once, a step per lane, 64 steps ahead: where a step's
    // keys and values start is a lane of kat, vat, and whether its pages exist a bit of `pages`.
    constexpr int GRPS = NL > 1 ? 2 : 1;
    const int grp0 = GRPS == 2 ? 0 : wave * 64 / RC / 16;
    int64_t kat[GRPS], vat[GRPS];
    uint64_t pages[2];
    int ahead[2];
    auto read_table = [&](int block) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int key = key0 + (block * 64 + lane) * SUB + 16 * t;
        ahead[t] = key < hi_key ? table[key >> shift] : -1;
      }
    };
    auto take_table = [&](int block) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 2; ++t) pages[t] = __ballot(page_ok(ahead[t], num_pages));
#pragma unroll
      for (int g = 0; g < GRPS; ++g) {
        const int t = GRPS == 2 ? g : grp0, key = key0 + (block * 64 + lane) * SUB + 16 * t;
        const int x = t ? ahead[1] : ahead[0];
        const int64_t page = page_ok(x, num_pages) ? x : 0, in = (key & ps1) * (D * ES);
        kat[g] = page * kstride + in;
        vat[g] = page * vstride + in;
      }
    };
    auto lane64 = [&](int64_t x, int l) __attribute__((always_inline)) {
      const unsigned lo = __builtin_amdgcn_readlane((unsigned)x, l), hi = __builtin_amdgcn_readlane((unsigned)(x >> 32), l);
      return (int64_t)((uint64_t)hi << 32 | lo);
    };
    struct Step {
      int64_t k[GRPS], v[GRPS];
      int ok;  // bit t: the page of group t exists
    };
    // where step i lies (called for i = 0, 1, 2, ..)
    auto look_up = [&](int i, Step& x) __attribute__((always_inline)) {
      const int l = i & 63;
      if (l == 0) {
        take_table(i >> 6);
        read_table((i >> 6) + 1);
      }
#pragma unroll
      for (int g = 0; g < GRPS; ++g) x.k[g] = lane64(kat[g], l), x.v[g] = lane64(vat[g], l);
      x.ok = (int)(pages[0] >> l & 1) | (int)(pages[1] >> l & 1) << 1;
    };
    auto fetch = [&](const char* base, const int64_t (&at)[GRPS], v4u32 (&r)[NL]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        if (T::PARTS < kThreads && wave * 64 >= T::PARTS) break;
        const int part = j * kThreads + wave * 64, g = GRPS == 2 ? part / RC / 16 : 0;  // (j alone decides it)
        const char* src = base + (GRPS == 2 && g ? at[GRPS - 1] : at[0]) + (part - (GRPS == 2 ? g : grp0) * 16 * RC) * 16;
        r[j] = *reinterpret_cast<const v4u32*>(src + (unsigned)lane * 16u);
      }
    };
    auto put_k = [&](int slot, const v4u32 (&r)[NL]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        if (T::PARTS < kThreads && wave * 64 >= T::PARTS) break;
        const int x = j * kThreads + tid;
        *reinterpret_cast<v4u32*>(kl + slot + k_at<MT, D>(x / RC, x % RC)) = r[j];
      }
    };
    // whether a step's keys are all in the range, and none of its pages is missing
    auto whole = [&](int i, int ok, int lo, int hi) __attribute__((always_inline)) {
      const int kb = key0 + i * SUB;
      return kb >= lo && kb + SUB - 1 <= hi && ok == 3;
    };
    // Values that no row sees become 0. So does an infinity or NaN where some row does not see it, since a
    // weight of 0 would not hide it; the step is then marked, and the rows that do see it get it
    // from add_odd.
    auto put_v = [&](int i, int slot, int ok, v4u32 (&r)[NL]) __attribute__((always_inline)) {
      if (!whole(i, ok, w_full_lo, w_full_hi)) {
        bool odd = false;
#pragma unroll
        for (int j = 0; j < NL; ++j) {
          if (T::PARTS < kThreads && wave * 64 >= T::PARTS) break;
          const int x = (j * kThreads + tid) / RC, key = key0 + i * SUB + x;
          if (key < w_any_lo || key > w_any_hi || !(ok >> (x / 16) & 1)) r[j] = v4u32{0, 0, 0, 0};
          odd |= any_nonfinite<MT>(r[j]);
          r[j] = finite_part<MT>(r[j]);
        }
        if (lane == 0) odd_at[i % VSLOTS][wave] = 0;
        if (odd) odd_at[i % VSLOTS][wave] = 1;
      }
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        if (T::PARTS < kThreads && wave * 64 >= T::PARTS) break;
        const int x = j * kThreads + tid;
        *reinterpret_cast<v4u32*>(vl + slot + v_at<MT, D>(x / RC, x % RC)) = r[j];
      }
    };

    f32x16 acc[NC] = {};
    float mx = -INFINITY, sum = 0.f;
    auto scores = [&](int slot, f32x16& st) __attribute__((always_inline)) {
      st = f32x16{};
#pragma unroll
      for (int f = 0; f < SF; ++f)
        st = Op<MT>::score(*reinterpret_cast<const v4u32*>(kl + slot + k_at<MT, D>(m, 2 * f + h2)), qf[f], st);
    };
    auto mask = [&](int i, int ok, f32x16& st) __attribute__((always_inline)) {
      const int kb = key0 + i * SUB + 4 * h2;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int key = kb + 8 * (r / 4) + r % 4;
        if ((key < plo) | (key > phi) | !(ok >> (r / 8) & 1)) st[r] = -INFINITY;
      }
    };
    // softmax of one step: weights, running maximum and sum, and the factor for the output
    auto softmax = [&](f32x16& st, weights& p, float& al) __attribute__((always_inline)) {
      float tm = max3(st[0], st[1], st[2]);
#pragma unroll
      for (int r = 3; r < 15; r += 2) tm = max3(tm, st[r], st[r + 1]);
      tm = max3(tm, st[15], st[15]);
      tm = across32_max(tm);
      const bool up = tm > mx + slack;
      const float mn = up ? tm : mx, mc = mn == -INFINITY ? 0.f : mn * c;
      al = up ? exp2_f(fmaf(mx, c, -mc)) : 1.f;
      mx = mn;
      float t[4];
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        st[r] = exp2_f(fmaf(st[r], c, -mc));
        t[r % 4] = r < 4 ? st[r] : t[r % 4] + st[r];
      }
      sum = fmaf(sum, al, (t[0] + t[1]) + (t[2] + t[3]));
      p = Op<MT>::pack(st);
      // (held here, or they would be sunk to where they are used, a step later)
      Op<MT>::hold(p);
      asm volatile("" : "+v"(sum));
    };
    auto rescale = [&](float al) __attribute__((always_inline)) {
      if (__any(al != 1.f)) {
#pragma unroll
        for (int x = 0; x < NC; ++x) acc[x] *= al;
      }
    };
    auto add_odd = [&](int i, int ok) __attribute__((always_inline)) {
      if (i >= 0 && !whole(i, ok, w_full_lo, w_full_hi)) {
        bool odd = false;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) odd |= odd_at[i % VSLOTS][w] != 0;
        if (__any(odd)) {
#pragma unroll 1
          for (int x = 0; x < SUB; ++x) {
            const int key = key0 + i * SUB + x;
            if (key > w_any_hi || !(ok >> (x / 16) & 1)) continue;
            const MT* v = (const MT*)(vbase + table[key >> shift] * vstride) + (key & ps1) * D;
#pragma unroll
            for (int y = 0; y < NC * 16; ++y) {
              const float f = (float)v[32 * (y / 16) + 8 * (y / 4 % 4) + 4 * h2 + y % 4];
              if (f - f != 0.f && key >= plo && key <= phi) acc[y / 16][y % 16] += f;
            }
          }
        }
      }
    };

    // --- the steps. During step i the keys of i + AHEAD and the values of i + 1 are fetched, and put
    // in LDS at its end. (Behind the last step the fetches read page 0, and the scores are of what lies in
    // LDS: nobody reads either.)
    v4u32 kr[NL], vr[NL];
    Step x0, x1, x2;   // steps i, i + 1, i + 2
    int okp = 0;       // x.ok of step i - 1
    read_table(0);
    look_up(0, x0);
    look_up(1, x1);
    fetch(kbase, x0.k, kr);
    fetch(vbase, x0.v, vr);
    put_k(0, kr);
    put_v(0, 0, x0.ok, vr);
    if (T::PIPE) {
      // "step -1", whose weights are 0
      for (int x = tid; x < T::PARTS; x += kThreads)
        *reinterpret_cast<v4u32*>(vl + (VSLOTS - 1) * BYTES + x * 16) = v4u32{0, 0, 0, 0};
      fetch(kbase, x1.k, kr);
      put_k(BYTES, kr);
    }
    __syncthreads();
    weights pa = {}, pb;
    f32x16 sa, sb;
    // slots: of the next step's scores or (not PIPE) this one's, of what is put, of the values
    int kread = T::PIPE ? BYTES : 0, kput = AHEAD % KSLOTS * BYTES, vread = T::PIPE ? (VSLOTS - 1) * BYTES : 0, vput = BYTES;
    auto next = [](int slot, int slots) { return slot == (slots - 1) * BYTES ? 0 : slot + BYTES; };
    if (T::PIPE) scores(0, sa);
    auto step = [&](int i, f32x16& cur, f32x16& nxt, weights& p, weights& pn) __attribute__((always_inline)) {
      look_up(i + 2, x2);
      fetch(kbase, AHEAD == 2 ? x2.k : x1.k, kr);
      fetch(vbase, x1.v, vr);
      float al;
      if (!T::PIPE) scores(kread, cur);
      if (!whole(i, x0.ok, full_lo, full_hi)) mask(i, x0.ok, cur);
      if (T::PIPE) {
        scores(kread, nxt);
        softmax(cur, pn, al);
        add_values<MT, D>(vl + vread, lane, p, acc);
        add_odd(i - 1, okp);
        rescale(al);
      } else {
        softmax(cur, pn, al);
        rescale(al);
        add_values<MT, D>(vl + vread, lane, pn, acc);
        add_odd(i, x0.ok);
      }
      put_k(kput, kr);
      put_v(i + 1, vput, x1.ok, vr);
      kread = next(kread, KSLOTS), kput = next(kput, KSLOTS), vread = next(vread, VSLOTS), vput = next(vput, VSLOTS);
      okp = x0.ok, x0 = x1, x1 = x2;
      lds_barrier();
    };
    if constexpr (T::PIPE) {
      int i = 0;
#pragma unroll 1
      for (; i + 1 < nb; i += 2) {
        step(i, sa, sb, pa, pb);
        step(i + 1, sb, sa, pb, pa);
      }
      if (i < nb) {
        step(i, sa, sb, pa, pb);
        pa = pb;
      }
      add_values<MT, D>(vl + vread, lane, pa, acc);
      add_odd(nb - 1, okp);
    } else {
#pragma unroll 1
      for (int i = 0; i < nb; ++i) step(i, sa, sa, pa, pa);
    }

    // --- out
    {
      const AttnArgs a = fresh_args();
      const int N = a.b.num_seqs, G = a.num_q_heads / a.num_kv_heads;
      const int n = walk.n, h = walk.h, tile = walk.tile, off = walk.off;
      const Seq s = seq_at(a, n, G, SUB);
      const TileKeys tk = tile_keys(a, s, tile, G);
      const bool done = off == 0 && nb == tk.units;
      const int r = wave * 32 + m, row = tile * ROWS + r;
      const float l = across32(sum, SumOp());
      if (row < s.rows) {
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
              for (int e = 0; e < 4; ++e) dst[32 * x + 8 * y + e] = from_f32<MT>(acc[x][4 * y + e] * inv);
          if (a.lse && h2 == 0) a.lse[out] = mx * a.scale + (l == 0.f ? 0.f : logf(l));
        } else {
          const TilePlan pl = tile_plan_at(a.tile_ws, N, max_tiles(N, a.b.total_tokens, G, ROWS));
          float* part = pl.part + (2 * (int64_t)share + (walk.at == walk.begin ? 0 : 1)) * tile_part_floats(ROWS, D);
#pragma unroll
          for (int x = 0; x < NC; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              *reinterpret_cast<f32x4*>(part + (int64_t)r * D + 32 * x + 8 * y + 4 * h2) =
                  f32x4{acc[x][4 * y], acc[x][4 * y + 1], acc[x][4 * y + 2], acc[x][4 * y + 3]};
          if (h2 == 0) part[ROWS * D + 2 * r] = mx, part[ROWS * D + 2 * r + 1] = l;
        }
      }
    }
    __syncthreads();
    if (tid == 0) walk.at += nb, ++walk.tile, walk.off = 0;
  }
}

template <typename MT, int D>
void launch(const AttnArgs& a) {
  tile_kernel<MT, D><<<Tile<MT, D>::S::GROUPS, Tile<MT, D>::THREADS, 0, a.stream>>>(a);
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

size_t attn_tile_bytes(int num_seqs, int64_t total_tokens, int G, int head_dim, bool bf16) {
  const int rows = attn_tile_rows(head_dim, bf16), groups = attn_tile_groups(head_dim, bf16);
  return tile_plan_bytes(num_seqs, max_tiles(num_seqs, total_tokens, G, rows)) +
         (size_t)(2 * groups * tile_part_floats(rows, head_dim)) * 4;
}

}  // namespace kda
