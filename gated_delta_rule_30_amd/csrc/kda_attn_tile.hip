// Causal attention of many new tokens over a paged KV cache: prompts and their chunks
// (kda_attn.hip takes the sequences of few rows).
//
// The formulas and the one pass with a running maximum are those of kda_attn.hip. Bound by the
// matrix cores: 4 D flops per (row, key). A workgroup takes a tile of one sequence and K/V head, 32 rows
// per wave (8 waves; fp32 and D = 256: 4, for whose registers there is no more room), and walks over the
// keys 32 at a time, staged through LDS for all of its waves.
//  - Scores are formed transposed, S^T = K Q^T, in 32 x 32 tiles: a lane holds 16 scores of one
//    row, so that the softmax is register work and one lane exchange, and the weights are already laid
//    out as the second operand of O^T = V^T P^T. The order of keys within an operand is free as long as
//    both operands share it, so no weight moves between lanes.
//  - With 8 waves the two waves of a SIMD take turns, one in its products while the other is in its softmax. A
//    step of a wave is 512 clocks of products and about 400 of vector work; left to themselves the waves
//    drift into the same phase (the case below, when this was built: 1.69 ms without turns, 1.34 with).
//  - Loads are made two steps ahead: a step takes 1.1 us, about as long as
//    a key is on its way from HBM (on one card one step ahead 1370 us, two 1285).
//  - The output is rescaled only when a maximum grows by more than 2^8: weights up to 2^8 cost
//    neither the fp32 sums nor the bf16 weights any relative accuracy.
//  - The tiles' keys are laid end to end and cut into equal shares, one per workgroup; a tile
//    that is cut leaves partial (o, m, l), joined with those of the row kernel.
// Measured: 4096 new tokens behind 16384, 32 query heads over 8, D = 128, bf16: 1257 to 1310 us by
// card, 945 to 984 TFLOP/s (a library product of 16384^3 bf16 reaches 1381; the clock is held down by power in both). fp32: 3
// sequences, 432 new tokens over 5392, 16 heads: 106 us; 9.7 GFLOP with the rows that pad the last tiles, at 92 of
// the 154 TFLOP/s of a library product.
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
  // keys and values of two steps each
  static constexpr int LDS = 4 * BYTES;
};

// The parts of a row are permuted in LDS so that what is read at once lies in different banks
// (64 of 4 bytes): a key fragment is the same part of 16 rows, a transposed value fragment four parts of four
// rows (fp32: consecutive parts of a row, left in place).
template <typename MT, int D>
__device__ __forceinline__ int k_at(int row, int part) {
  constexpr int RC = D * (int)sizeof(MT) / 16;
  return row * (RC * 16) + (part ^ (RC >= 16 ? row & 15 : (row >> 1) & 7)) * 16;
}
template <typename MT, int D>
__device__ __forceinline__ int v_at(int row, int part) {
  constexpr int RC = D * (int)sizeof(MT) / 16;
  const int sw = sizeof(MT) == 4 ? 0 : RC >= 16 ? (row & 3) << 2 : ((row >> 1) & 1) << 2;
  return row * (RC * 16) + (part ^ sw) * 16;
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
  static constexpr int together(int D) { return D >= 128 ? 4 : 2; }  // output tiles whose values lie side by side
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
// O^T += V^T P^T
template <typename MT, int D>
__device__ __forceinline__ void add_values(const char* v, int lane, const typename Op<MT>::weights& p,
                                           f32x16 (&acc)[D / 32]) {
  if constexpr (sizeof(MT) == 2) {
#pragma unroll
    for (int i = 0; i < Op<MT>::NF; ++i)
#pragma unroll
      for (int c = 0; c < D / 32; ++c) acc[c] = Op<MT>::value(value_frag<D>(v, lane, i, c, MT()), p, i, acc[c]);
  } else {
    // One product takes one float per lane, of one key and channel: the channels of V of tile c are so
    // chosen (channel_of) that a lane reads those of all tiles of a key at once.
    constexpr int W = Op<float>::together(D);
    typedef __attribute__((ext_vector_type(W), may_alias)) float vec;
    const int h = lane >> 5, m = lane & 31;
#pragma unroll
    for (int i = 0; i < Op<MT>::NF; ++i)
#pragma unroll
      for (int g = 0; g < D / 32 / W; ++g) {
        const vec f = *(const vec*)(v + (8 * (i / 4) + 4 * h + i % 4) * (D * 4) + (32 * g + m) * (W * 4));
#pragma unroll
        for (int x = 0; x < W; ++x) acc[W * g + x] = Op<MT>::value(f[x], p, i, acc[W * g + x]);
      }
  }
}
// Channel of row `row` of output tile c.
template <typename MT, int D>
__device__ __forceinline__ int channel_of(int c, int row) {
  if constexpr (sizeof(MT) == 2) return 32 * c + row;
  constexpr int W = Op<float>::together(D);
  return W * (32 * (c / W) + row) + c % W;
}

__global__ __launch_bounds__(kPlanThreads) void tile_plan_kernel(AttnArgs a) {
  __shared__ PlanLds lds;
  make_tile_plan(a, lds);
}

// ------------------------------------------------------------------ the kernel
// Where a workgroup is in its share: kept in LDS between tiles, and the arguments read again
// where they are needed, so that the steps' loop holds no scalar registers that it does not use.
struct Walk {
  int64_t at, end, per, t0, nt;  // (costs); the sequence's tiles are t0 .. t0 + nt - 1
  int n, h, tile;
  int64_t off;  // what of the tile, its lead first, is done
};
// The keys that some row of the tile sees, and the first and last step that has an infinity or NaN among
// their values.
struct Odd {
  int seen_lo, seen_hi, first, last;
};
__device__ __forceinline__ AttnArgs fresh_args() {
  auto p = (const __attribute__((address_space(4))) char*)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(p));
  return *(const AttnArgs*)(const void*)p;
}

// x in scalar registers of its own: a value that is a part of loaded arguments keeps all of the registers
// that they were loaded to.
template <typename X>
__device__ __forceinline__ X own(X x) {
  static_assert(sizeof(X) == 4 || sizeof(X) == 8, "");
  if constexpr (sizeof(X) == 4) {
    return __builtin_bit_cast(X, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, x)));
  } else {
    const uint64_t u = __builtin_bit_cast(uint64_t, x);
    const unsigned lo = __builtin_amdgcn_readfirstlane((unsigned)u), hi = __builtin_amdgcn_readfirstlane((unsigned)(u >> 32));
    return __builtin_bit_cast(X, (uint64_t)hi << 32 | lo);
  }
}

// A pointer to global memory (that has been through `own`, it would be taken for one to any).
template <typename X>
__device__ __forceinline__ const __attribute__((address_space(1))) X* global(const void* p) {
  return (const __attribute__((address_space(1))) X*)p;
}

template <typename MT, int D>
__global__ __launch_bounds__((Tile<MT, D>::THREADS), (Tile<MT, D>::S::PER_SIMD)) void tile_kernel(AttnArgs) {
  typedef Tile<MT, D> T;
  typedef typename Op<MT>::weights weights;
  constexpr int kThreads = T::THREADS, kWaves = T::WAVES, kGroups = T::S::GROUPS, ROWS = T::ROWS;
  constexpr int RC = T::RC, NL = T::NL, SF = T::SF, NC = T::NC, ES = T::ES, BYTES = T::BYTES;
  constexpr bool TURNS = kWaves == 8;  // two waves per SIMD of this workgroup
  __shared__ __align__(16) char lds[T::LDS];
  __shared__ Odd odd;
  __shared__ Walk walk;
  char* const kl = lds;
  char* const vl = lds + 2 * BYTES;
  const int tid = threadIdx.x, lane = tid & 63, m = lane & 31, h2 = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int share = (blockIdx.x % 8) * (kGroups / 8) + blockIdx.x / 8;

  // --- this workgroup's share of all units. The shares of the workgroups of one XCD (every
  // eighth) lie side by side, so that they read the same heads' keys through one L2.
  {
    const AttnArgs a = fresh_args();
    const int N = a.b.num_seqs, Hk = a.num_kv_heads, G = a.num_q_heads / Hk;
    const TilePlan pl = tile_plan_at(a.tile_ws, N, max_tiles(N, a.b.total_tokens, G, ROWS));
    const int64_t total = Hk * pl.seq[N].cost, per = max((int64_t)1, (total + kGroups - 1) / kGroups);
    const int64_t at = share * per;
    if (tid == 0) pl.cut[share].n = -1;
    if (at >= total) return;
    // the sequence that `at` lies in, and the tile: whichever thread has it tells the others
    for (int n = tid; n < N; n += kThreads) {
      const SeqFirst s = pl.seq[n], e = pl.seq[n + 1];
      if (Hk * s.cost <= at && at < Hk * e.cost) {
        const int64_t in = at - Hk * s.cost, per_head = e.cost - s.cost;
        walk = {at, min(total, at + per), per, s.tile, e.tile - s.tile, n, (int)(in / per_head), 0, in % per_head};
      }
    }
    __syncthreads();
    const int64_t t0 = walk.t0, nt = walk.nt, u0 = pl.pre[t0], off = walk.off;
    __syncthreads();
    for (int64_t i = tid; i < nt; i += kThreads) {
      const int64_t s = pl.pre[t0 + i] - u0, e = pl.pre[t0 + i + 1] - u0;
      if (s <= off && off < e) walk.tile = (int)i, walk.off = off - s;
    }
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
          do ++walk.n, walk.t0 += walk.nt, walk.nt = pl.seq[walk.n + 1].tile - walk.t0;
          while (walk.nt == 0);
        }
      }
      continue;
    }
    if (walk.off < kTileLead) {
      __syncthreads();
      if (tid == 0) walk.at += kTileLead - walk.off, walk.off = kTileLead;
      continue;
    }
    const AttnArgs a = fresh_args();
    const int n = __builtin_amdgcn_readfirstlane(walk.n), h = __builtin_amdgcn_readfirstlane(walk.h),
              tile = __builtin_amdgcn_readfirstlane(walk.tile),
              off = __builtin_amdgcn_readfirstlane((int)walk.off - kTileLead);
    const int left = __builtin_amdgcn_readfirstlane((int)min(walk.end - walk.at, (int64_t)INT32_MAX));
    const int G = a.num_q_heads / a.num_kv_heads;
    const Seq s = seq_at(a, n, G, SUB);
    const TileKeys tk = tile_keys(a, s, tile, G);
    const int nb = min(tk.units - off, left);  // steps

    if (tid == 0) {  // (read behind the next barrier, and last read before the one above)
      const int last = (int)((min((int64_t)(tile + 1) * ROWS, (int64_t)s.rows) - 1) / G);
      const int pf = s.p0 + (int)((int64_t)tile * ROWS / G);
      odd = {a.window ? max(0, pf - a.window + 1) : 0, min(s.p0 + last, s.hi - 1), INT32_MAX, -1};
    }
    // --- the wave's rows: lane m's query and its visible keys vlo .. vlo + span; and the steps full_lo ..
    // full_lo + full_n - 1 that every row of the wave sees whole, and those (some) that some row sees a part of
    const int key0 = tk.lo + off * SUB, hi_key = own(min(s.hi, key0 + nb * SUB));
    int vlo, span, full_lo, full_n, some_lo, some_n;
    v4u32 qf[SF];
    {
      const int row = tile * ROWS + wave * 32 + m;
      const bool has = row < s.rows;
      const int tok = has ? row / G : 0, hq = h * G + (has ? row - tok * G : 0), p = s.p0 + tok;
      const int phi = has ? min(p, s.hi - 1) : -1, plo = a.window ? max(0, p - a.window + 1) : 0;
      const char* src = (const char*)((const MT*)a.q + (s.row0 + tok) * a.q_stride + hq * D) + h2 * 16;
#pragma unroll
      for (int i = 0; i < SF; ++i) qf[i] = *reinterpret_cast<const v4u32*>(src + 32 * i);
      vlo = phi >= plo ? plo : INT32_MAX;  // (nothing: no key is at or above that)
      span = max(0, phi - plo);
      int lo = has ? plo : 0, hi = has ? phi : INT32_MAX, slo = phi >= plo ? plo : INT32_MAX, shi = phi >= plo ? phi : -1;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        lo = max(lo, __shfl_xor(lo, d));
        hi = min(hi, __shfl_xor(hi, d));
        slo = min(slo, __shfl_xor(slo, d));
        shi = max(shi, __shfl_xor(shi, d));
      }
      slo = max(0, slo - key0) / SUB;
      some_lo = own(slo);
      some_n = own(shi >= key0 ? max(0, (shi - key0) / SUB + 1 - slo) : 0);
      lo = max(0, lo - key0 + SUB - 1) / SUB;
      hi = hi >= key0 ? (int)(((int64_t)hi - key0 + 1) / SUB) : 0;
      full_lo = own(lo);
      full_n = own(max(0, hi - lo));
    }
    const char* const kbase = own(a.k_pages + (int64_t)h * a.b.page_size * D * ES);
    const char* const vbase = own(a.v_pages + (int64_t)h * a.b.page_size * D * ES);
    const float c = own(a.scale * LOG2E), slack = fminf(8.f / c, 1e30f);  // (finite: -inf + slack is -inf)

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
      const AttnArgs a = fresh_args();
      const int32_t* table = a.b.block_table + walk.n * a.b.table_stride;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int key = key0 + (block * 64 + lane) * SUB + 16 * t;
        ahead[t] = key < hi_key ? table[key >> __builtin_ctz(a.b.page_size)] : -1;
      }
    };
    auto take_table = [&](int block) __attribute__((always_inline)) {
      const AttnArgs a = fresh_args();
#pragma unroll
      for (int t = 0; t < 2; ++t) pages[t] = __ballot(page_ok(ahead[t], a.b.num_pages));
#pragma unroll
      for (int g = 0; g < GRPS; ++g) {
        const int t = GRPS == 2 ? g : grp0, key = key0 + (block * 64 + lane) * SUB + 16 * t;
        const int x = t ? ahead[1] : ahead[0];
        const int64_t page = page_ok(x, a.b.num_pages) ? x : 0, in = (key & (a.b.page_size - 1)) * D;
        kat[g] = (page * a.k_page_stride + in) * ES;
        vat[g] = (page * a.v_page_stride + in) * ES;
      }
    };
    auto lane64 = [&](int64_t x, int l) __attribute__((always_inline)) {
      const unsigned lo = __builtin_amdgcn_readlane((unsigned)x, l), hi = __builtin_amdgcn_readlane((unsigned)(x >> 32), l);
      return (int64_t)((uint64_t)hi << 32 | lo);
    };
    // where step i lies, and into `ok` (two bits a step, the latest lowest) whether its pages exist; called for
    // i = 0, 1, 2, ..
    unsigned ok = 0;
    auto look_up = [&](int i, int64_t (&k)[GRPS], int64_t (&v)[GRPS]) __attribute__((always_inline)) {
      const int l = i & 63;
      if (l == 0) {
        take_table(i >> 6);
        read_table((i >> 6) + 1);
      }
#pragma unroll
      for (int g = 0; g < GRPS; ++g) k[g] = lane64(kat[g], l), v[g] = lane64(vat[g], l);
      ok = ok << 2 | (unsigned)(pages[0] >> l & 1) | (unsigned)(pages[1] >> l & 1) << 1;
    };
    auto fetch = [&](const char* base, const int64_t (&at)[GRPS], v4u32 (&r)[NL]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        if (T::PARTS < kThreads && wave * 64 >= T::PARTS) break;
        const int part = j * kThreads + wave * 64, g = GRPS == 2 ? part / RC / 16 : 0;  // (j alone decides it)
        const char* src = base + (GRPS == 2 && g ? at[GRPS - 1] : at[0]) + (part - (GRPS == 2 ? g : grp0) * 16 * RC) * 16;
        r[j] = *global<v4u32>(src + (unsigned)lane * 16u);
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
    // An infinity or NaN is put as 0: it may lie where some row does not look, and a weight of 0 would not hide it.
    // If some row does see its key, the step is noted, and those rows get it at the end.
    auto put_v = [&](int i, unsigned ok, int slot, v4u32 (&r)[NL]) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < NL; ++j) {
        if (T::PARTS < kThreads && wave * 64 >= T::PARTS) break;
        const int x = j * kThreads + tid;
        if (__any(any_nonfinite<MT>(r[j]))) {
          const int key = key0 + i * SUB + x / RC;
          if (any_nonfinite<MT>(r[j]) && key >= odd.seen_lo && key <= odd.seen_hi && (ok >> (x / RC / 16) & 1)) {
            atomicMin(&odd.first, i);
            atomicMax(&odd.last, i);
          }
          r[j] = finite_part<MT>(r[j]);
        }
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
    auto mask = [&](int i, unsigned ok, f32x16& st) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const unsigned at = ok >> t & 1 ? (unsigned)(key0 + i * SUB + 4 * h2 + 16 * t - vlo) : 0xc0000000u;
#pragma unroll
        for (int r = 0; r < 8; ++r)
          if (at + (unsigned)(8 * (r / 4) + r % 4) > (unsigned)span) st[8 * t + r] = -INFINITY;
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
    auto masked = [&](int i, unsigned ok) __attribute__((always_inline)) {
      return (unsigned)(i - full_lo) >= (unsigned)full_n || (ok & 3) != 3;
    };
    weights p = {};
    if constexpr (TURNS) {
      // --- the steps. Scores of step i and values of step i - 1 are one phase, the softmax of i the next. Of
      // the two waves on a SIMD one is a phase behind the other: one has the matrix core while the
      // other has the vector unit. Keys of step i + 1 and values of step i come to LDS while the first wave is in
      // its softmax of i and the second in its products of i; they were fetched two steps before. (Behind the
      // last step the fetches read page 0, which nobody uses.)
      v4u32 k0[NL], v0[NL], k1[NL], v1[NL];
      int64_t xk[GRPS], xv[GRPS], yv[GRPS], zv[GRPS];  // where keys and values of the latest steps lie
      read_table(0);
      look_up(0, xk, zv);
      fetch(kbase, xk, k0);
      put_k(0, k0);
      look_up(1, xk, yv);
      fetch(kbase, xk, k0);
      fetch(vbase, zv, v0);
      look_up(2, xk, xv);
      fetch(kbase, xk, k1);
      fetch(vbase, yv, v1);
      // "step -1", whose weights are 0
      for (int x = tid; x < T::PARTS; x += kThreads) *reinterpret_cast<v4u32*>(vl + BYTES + x * 16) = v4u32{0, 0, 0, 0};
      lds_barrier();
      // (each role has a loop of its own: in a shared one, where both could put, the compiler would wait for the
      // loads just made)
      auto run = [&](auto SECOND) __attribute__((always_inline)) {
        constexpr bool second = decltype(SECOND)::value;
        if constexpr (second) lds_barrier();
        // ODD: i & 1
        auto step = [&](int i, auto ODD, v4u32 (&kf)[NL], v4u32 (&vf)[NL]) __attribute__((always_inline)) {
          constexpr int par = decltype(ODD)::value;
  #pragma unroll
          for (int g = 0; g < GRPS; ++g) yv[g] = xv[g];
          look_up(i + 3, xk, xv);  // `ok` ends at step i + 3 from here on
          auto put = [&]() __attribute__((always_inline)) {
            put_k((1 - par) * BYTES, kf);
            put_v(i, ok >> 6, par * BYTES, vf);
            fetch(kbase, xk, kf);
            fetch(vbase, yv, vf);
          };
          // all of the phase's fragments are on their way before its first product: waiting for each in
          // turn costs more than the products
          f32x16 st = {};
          bf16x8 vfr[Op<MT>::NF][NC];
          v4u32 kfr[SF];
  #pragma unroll
          for (int f = 0; f < Op<MT>::NF; ++f)
  #pragma unroll
            for (int x = 0; x < NC; ++x) vfr[f][x] = value_frag<D>(vl + (1 - par) * BYTES, lane, f, x, MT());
  #pragma unroll
          for (int f = 0; f < SF / 2; ++f) kfr[f] = *reinterpret_cast<const v4u32*>(kl + par * BYTES + k_at<MT, D>(m, 2 * f + h2));
          __builtin_amdgcn_sched_barrier(0);
  #pragma unroll
          for (int f = SF / 2; f < SF; ++f) kfr[f] = *reinterpret_cast<const v4u32*>(kl + par * BYTES + k_at<MT, D>(m, 2 * f + h2));
  #pragma unroll
          for (int f = 0; f < Op<MT>::NF; ++f)
  #pragma unroll
            for (int x = 0; x < NC; ++x) acc[x] = Op<MT>::value(vfr[f][x], p, f, acc[x]);
  #pragma unroll
          for (int f = 0; f < SF; ++f) st = Op<MT>::score(kfr[f], qf[f], st);
          if constexpr (second) put();
          lds_barrier();
          if (masked(i, ok >> 6)) mask(i, ok >> 6, st);
          float al;
          softmax(st, p, al);
          rescale(al);
          if constexpr (!second) put();
          lds_barrier();
        };
        int i = 0;
  #pragma unroll 1
        for (; i + 1 < nb; i += 2) {
          step(i, std::integral_constant<int, 0>(), k0, v0);
          step(i + 1, std::integral_constant<int, 1>(), k1, v1);
        }
        if (i < nb) step(i, std::integral_constant<int, 0>(), k0, v0);
        if constexpr (!second) lds_barrier();
      };
      if (wave >= kWaves / 2) run(std::true_type());
      else run(std::false_type());
      add_values<MT, D>(vl + ((nb - 1) & 1) * BYTES, lane, p, acc);
    } else {
      // --- the steps, one wave per SIMD of this workgroup: step i's products and softmax in turn, the next step's
      // keys and values fetched meanwhile and put in LDS at the end
      v4u32 staged[NL];
      int64_t xk[GRPS], xv[GRPS];
      read_table(0);
      look_up(0, xk, xv);
      fetch(kbase, xk, staged);
      put_k(0, staged);
      fetch(vbase, xv, staged);
      lds_barrier();
      put_v(0, ok, 0, staged);
      lds_barrier();
#pragma unroll 1
      for (int i = 0; i < nb; ++i) {
        const int slot = (i & 1) * BYTES;
        look_up(i + 1, xk, xv);
        // one register set serves both: the keys come during the scores, the values during the output
        fetch(kbase, xk, staged);
        const bool some = (unsigned)(i - some_lo) < (unsigned)some_n;
        if (some) {
          f32x16 st;
          float al;
          scores(slot, st);
          if (masked(i, ok >> 2)) mask(i, ok >> 2, st);
          softmax(st, p, al);
          rescale(al);
        }
        put_k(BYTES - slot, staged);
        fetch(vbase, xv, staged);
        if (some) add_values<MT, D>(vl + slot, lane, p, acc);
        put_v(i + 1, ok, BYTES - slot, staged);
        lds_barrier();
      }
    }

    // --- the rows that see an infinity or NaN among the values gain it
    if (odd.first <= odd.last) {
      const AttnArgs a = fresh_args();
      const int32_t* table = a.b.block_table + walk.n * a.b.table_stride;
      const int ps = a.b.page_size, end = min(hi_key, key0 + (odd.last + 1) * SUB);
#pragma unroll 1
      for (int key = key0 + odd.first * SUB; key < end; ++key) {
        const int pg = table[key / ps];
        if (!page_ok(pg, a.b.num_pages) || (unsigned)(key - vlo) > (unsigned)span) continue;
        const MT* v = (const MT*)a.v_pages + pg * a.v_page_stride + ((int64_t)walk.h * ps + key % ps) * D;
#pragma unroll
        for (int y = 0; y < NC * 16; ++y) {
          const float f = (float)v[channel_of<MT, D>(y / 16, 8 * (y / 4 % 4) + 4 * h2 + y % 4)];
          if (f - f != 0.f) acc[y / 16][y % 16] += f;
        }
      }
    }

    // --- out
    {
      const AttnArgs a = fresh_args();
      const int N = a.b.num_seqs, G = a.num_q_heads / a.num_kv_heads;
      const int n = walk.n, h = walk.h, tile = walk.tile, off = (int)walk.off - kTileLead;
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
          MT* dst = (MT*)a.o + out * D;
#pragma unroll
          for (int x = 0; x < NC; ++x)
#pragma unroll
            for (int y = 0; y < 16; ++y)
              dst[channel_of<MT, D>(x, 8 * (y / 4) + 4 * h2 + y % 4)] = from_f32<MT>(acc[x][y] * inv);
          if (a.lse && h2 == 0) a.lse[out] = mx * a.scale + (l == 0.f ? 0.f : logf(l));
        } else {
          const TilePlan pl = tile_plan_at(a.tile_ws, N, max_tiles(N, a.b.total_tokens, G, ROWS));
          float* part = pl.part + part_of(share, walk.at, walk.per) * tile_part_floats(ROWS, D);
          if (tid == 0 && off == 0) pl.cut[share] = {walk.at, walk.per, n, h, tile, tk.units};
#pragma unroll
          for (int x = 0; x < NC; ++x)
#pragma unroll
            for (int y = 0; y < 16; ++y)
              part[(int64_t)r * D + channel_of<MT, D>(x, 8 * (y / 4) + 4 * h2 + y % 4)] = acc[x][y];
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

void launch_attn_tile(const AttnArgs& a, bool plan) {
  if (plan) tile_plan_kernel<<<1, kPlanThreads, 0, a.stream>>>(a);
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
