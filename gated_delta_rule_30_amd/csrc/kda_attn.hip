// Causal attention of few new tokens over a paged KV cache: the decode step, speculative and
// short chunks (kda_attn_tile.hip takes the long ones).
//
//   o_t = sum_j softmax_j(scale q_t . k_j) v_j,  one pass over the keys with a running maximum m
//   and sum l: o <- o e^{m - m'} + sum_j e^{s_j - m'} v_j,  l likewise, o / l at the end.
//
// Bound by HBM: every key and value is read once for the G query heads (times new tokens) that
// share it, 4 G flops per byte of bf16. So the work is laid out for bytes in flight:
//  - The keys of all (sequence, K/V head, 16-row tile) items are laid end to end in units of 128
//    (fp32: 64) keys and cut into equal shares, one per workgroup, wherever the borders fall: a
//    ragged batch loads every compute unit alike. An item that is cut leaves partial (o, m, l) in the
//    workspace, which a second launch joins.
//  - A unit is four blocks of 32 (fp32: 16) keys, one per wave; the waves run on their own, with
//    the next block's keys and values in flight in registers while one is computed, and meet at
//    the item's end.
// Scores are formed transposed, S^T = K Q^T, so that a lane holds scores of one row: the maximum
// and sum are register loops and two lane exchanges, and the weights are already laid out as the
// second operand of O^T = V^T P^T. K goes from memory straight to the operand registers; V
// passes through LDS, where it is read transposed.
// Measured: 64 sequences of 1024 to 32768 keys, 32 query heads over 8, D = 128, bf16: 2.38 GB in 404 to 414 us, 5.8
// TB/s (neg over 1 GiB reaches 6.2 read + write). 4 sequences of up to 1000 keys: 8.2 us and 4.7 us to join,
// both latency (launch, table, keys, sums in turn).
#include "kda_attn.h"

namespace kda {

namespace {

constexpr int kThreads = 256, kWaves = 4;
constexpr int kGroups = 512;  // workgroups of the row kernel: two per compute unit

template <typename MT, int D>
struct Row {
  typedef typename Mma<MT>::frag frag;
  static constexpr int ES = sizeof(MT), KS = Mma<MT>::KS, EPL = Mma<MT>::EPL;
  static constexpr int UNIT = kWaves * KS;      // keys of a unit
  static constexpr int NG = KS / 16;            // 16-key groups of a block
  static constexpr int SK = D / KS;             // reduction steps of a score
  static constexpr int NC = D / 16;             // 16-channel tiles of the output
  static constexpr int RC = D * ES / 16;        // 16-byte parts of a row
  static constexpr int RPI = 64 / RC;           // rows that one wave-wide load covers
  static constexpr int VL = KS / RPI;           // such loads of a block
  static constexpr int TILE = KS * D * ES;      // bytes of a block's values in LDS
  static constexpr int OBYTES = 16 * D * 4;     // bytes of one wave's output tile
  static constexpr int LDS = kWaves * (TILE > OBYTES ? TILE : OBYTES);
};

// Byte offset of 16-byte part `part` of row `row` of a block's values in LDS. Parts are permuted
// within a row so that what is read at once lies in different banks (64 of 4 bytes): two parts of eight
// rows (fp32: four parts of four rows, four apart).
template <typename MT, int D>
__device__ __forceinline__ int v_at(int row, int part) {
  constexpr int RC = D * (int)sizeof(MT) / 16;
  const int sw = sizeof(MT) == 4 ? ((row >> 2) & 3) << 2 : RC >= 16 ? (row & 7) << 1 : ((row >> 1) & 3) << 1;
  return row * (RC * 16) + (part ^ sw) * 16;
}

// Fragment of V^T: channels 16 c .. + 15, the block's keys.
template <int D>
__device__ __forceinline__ bf16x8 v_frag(const char* v, int c, int m, int g, bf16) {
  const int part = 2 * c + ((m & 3) >> 1), row = 4 * g + (m >> 2);
  const bf16x4 lo = ds_read_tr4((const bf16*)(v + v_at<bf16, D>(row, part) + 8 * (m & 1)));
  const bf16x4 hi = ds_read_tr4((const bf16*)(v + v_at<bf16, D>(row + 16, part) + 8 * (m & 1)));
  return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}
template <int D>
__device__ __forceinline__ f32x4 v_frag(const char* v, int c, int m, int g, float) {
  f32x4 r;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    r[e] = *(const lds_float*)(v + v_at<float, D>(4 * g + e, 4 * c + (m >> 2)) + 4 * (m & 3));
  return r;
}
__device__ __forceinline__ bf16x8 p_frag(const f32x4 (&s)[2], bf16) { return frag_from_acc(s[0], s[1], bf16()); }
__device__ __forceinline__ f32x4 p_frag(const f32x4 (&s)[1], float) { return s[0]; }

// Workspace: each workgroup's cut item, and its two partial results, each 16 rows
// of D sums, then m and l of each row.
struct Ws {
  Cut* cut;
  float* part;
};
__host__ __device__ inline Ws ws_at(char* ws) {
  return {reinterpret_cast<Cut*>(ws), reinterpret_cast<float*>(ws + sizeof(Cut) * kGroups)};
}
constexpr int part_floats(int D) { return 16 * D + 32; }

// Units of one of a sequence's items (a tile without keys is computed all the same: one unit that nobody
// sees), and of all of them; none if the tile kernel takes the sequence.
__device__ __forceinline__ int item_units(const Seq& s, int unit) { return max(1, (s.hi - s.lo + unit - 1) / unit); }
__device__ __forceinline__ int64_t seq_units(const AttnArgs& a, const Seq& s, int Hk, int unit) {
  return s.rows > a.row_limit ? 0 : (int64_t)((s.rows + 15) / 16) * Hk * item_units(s, unit);
}

template <typename MT, int D>
__global__ __launch_bounds__(kThreads, D == 256 ? 1 : 2) void row_kernel(AttnArgs a) {
  typedef Row<MT, D> R;
  typedef typename R::frag frag;
  constexpr int KS = R::KS, NG = R::NG, SK = R::SK, NC = R::NC, UNIT = R::UNIT;
  __shared__ __align__(16) char lds[R::LDS];
  __shared__ float ml[kWaves][16][2];
  __shared__ int64_t scan[kWaves], found[2];
  __shared__ PlanLds plan;
  if (blockIdx.x == kGroups) {  // one workgroup more, where the tile kernel is to follow
    make_tile_plan(a, plan);
    return;
  }
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, m = lane & 15, g = lane >> 4;
  const int N = a.b.num_seqs, Hk = a.num_kv_heads, G = a.num_q_heads / Hk, ps = a.b.page_size,
            shift = __builtin_ctz(ps);
  const Ws ws = ws_at(a.workspace);

  // --- this workgroup's share [at, end) of all units: each thread adds up a run of sequences
  const int run = (N + kThreads - 1) / kThreads, n0 = min(N, tid * run), n1 = min(N, n0 + run);
  int64_t mine = 0;
  for (int n = n0; n < n1; ++n) mine += seq_units(a, seq_at(a, n, G, UNIT), Hk, UNIT);
  int64_t incl = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t y = __shfl_up(incl, d);
    if (lane >= d) incl += y;
  }
  if (lane == 63) scan[wave] = incl;
  __syncthreads();
  int64_t total = 0, before = incl - mine;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += w < wave ? scan[w] : 0;
    total += scan[w];
  }
  const int64_t per = max((int64_t)1, (total + kGroups - 1) / kGroups);
  if (tid == 0) ws.cut[blockIdx.x].n = -1;
  int64_t at = (int64_t)blockIdx.x * per;
  const int64_t end = min(total, at + per);
  if (at >= end) return;
  if (before <= at && at < before + mine) {
    int64_t f = before;
    int n = n0;
    for (;; ++n) {
      const int64_t u = seq_units(a, seq_at(a, n, G, UNIT), Hk, UNIT);
      if (at < f + u) break;
      f += u;
    }
    found[0] = n;
    found[1] = f;
  }
  __syncthreads();
  int n = (int)found[0];
  int64_t first = found[1];  // first unit of sequence n

  const float c = a.scale * LOG2E;
  while (at < end) {
    const Seq s = seq_at(a, n, G, UNIT);
    const int units = item_units(s, UNIT), tiles = (s.rows + 15) / 16;
    const int64_t all = seq_units(a, s, Hk, UNIT);
    if (at >= first + all) {
      first += all;
      ++n;
      continue;
    }
    const int item = (int)((at - first) / units), u0 = (int)((at - first) - (int64_t)item * units);
    const int u1 = (int)min((int64_t)units, u0 + (end - at));
    const int h = item / tiles, tile = item - h * tiles;

    // --- the tile's rows: lane m's query, its visible keys
    const int row = tile * 16 + m;
    const bool has = row < s.rows;
    const int tok = has ? row / G : 0, hq = h * G + (has ? row - tok * G : 0);
    const int p = s.p0 + tok, phi = has ? min(p, s.hi - 1) : -1,
              plo = a.window ? max(0, p - a.window + 1) : 0;
    const MT* q = (const MT*)a.q + (s.row0 + tok) * a.q_stride + hq * D;
    frag qf[SK];
#pragma unroll
    for (int i = 0; i < SK; ++i) {
      qf[i] = *reinterpret_cast<const frag*>(q + KS * i + R::EPL * g);
      if (!has) qf[i] = frag{};
    }
    // keys any_lo .. any_hi are seen by some row, full_lo .. full_hi by every row
    int any_lo = has ? plo : INT32_MAX, any_hi = phi, full_lo = has ? plo : 0, full_hi = has ? phi : INT32_MAX;
#pragma unroll
    for (int d = 1; d < 16; d <<= 1) {
      any_lo = min(any_lo, __shfl_xor(any_lo, d));
      any_hi = max(any_hi, __shfl_xor(any_hi, d));
      full_lo = max(full_lo, __shfl_xor(full_lo, d));
      full_hi = min(full_hi, __shfl_xor(full_hi, d));
    }
    any_lo = __builtin_amdgcn_readfirstlane(any_lo);
    any_hi = __builtin_amdgcn_readfirstlane(any_hi);
    full_lo = __builtin_amdgcn_readfirstlane(full_lo);
    full_hi = __builtin_amdgcn_readfirstlane(full_hi);

    const int32_t* table = a.b.block_table + n * a.b.table_stride;
    const int64_t head = (int64_t)h * ps * D;
    const int key0 = s.lo + u0 * UNIT + wave * KS, nb = u1 - u0;  // the wave's blocks: key0 + i UNIT
    char* vl = lds + wave * R::TILE;

    f32x4 acc[NC] = {};
    float mx = -INFINITY, sum = 0.f;
    v4u32 kr[NG * SK], vr[R::VL];
    int pg[NG], pgn[NG];  // pages of the block in registers and of the one after it; -1: none

    auto pages = [&](int i, int (&e)[NG]) {
#pragma unroll
      for (int t = 0; t < NG; ++t) {
        const int key = key0 + i * UNIT + 16 * t;
        int x = -1;
        if (i < nb && key < s.hi) x = table[key >> shift];
        x = __builtin_amdgcn_readfirstlane(x);
        e[t] = page_ok(x, a.b.num_pages) ? x : -1;
      }
    };
    auto load_k = [&](int i, const int (&e)[NG]) {
#pragma unroll
      for (int t = 0; t < NG; ++t) {
        const int key = key0 + i * UNIT + 16 * t;
        const MT* k = (const MT*)a.k_pages + max(e[t], 0) * a.k_page_stride + head + (key & (ps - 1)) * D;
#pragma unroll
        for (int j = 0; j < SK; ++j)
          kr[t * SK + j] = *reinterpret_cast<const v4u32*>(k + m * D + KS * j + R::EPL * g);
      }
    };
    auto load_v = [&](int i, const int (&e)[NG]) {
#pragma unroll
      for (int t = 0; t < NG; ++t) {
        const int key = key0 + i * UNIT + 16 * t;
        const MT* v = (const MT*)a.v_pages + max(e[t], 0) * a.v_page_stride + head + (key & (ps - 1)) * D;
#pragma unroll
        for (int j = 0; j < R::VL / NG; ++j)
          vr[t * (R::VL / NG) + j] = *reinterpret_cast<const v4u32*>(v + (j * 64 + lane) * (16 / R::ES));
      }
    };
    pages(0, pg);
    pages(1, pgn);
    if (nb > 0) {
      load_k(0, pg);
      load_v(0, pg);
    }
    for (int i = 0; i < nb; ++i) {
      const int kb = key0 + i * UNIT;
      bool whole = kb >= full_lo && kb + KS - 1 <= full_hi;
#pragma unroll
      for (int t = 0; t < NG; ++t) whole = whole && pg[t] >= 0;
      // --- scores
      f32x4 st[NG] = {};
#pragma unroll
      for (int t = 0; t < NG; ++t)
#pragma unroll
        for (int j = 0; j < SK; ++j)
          st[t] = Mma<MT>::mma(__builtin_bit_cast(frag, kr[t * SK + j]), qf[j], st[t]);
      // --- values to LDS; those that no row sees as zeros
      bool odd = false;
      if (!whole) {
#pragma unroll
        for (int j = 0; j < R::VL; ++j) {
          const int r = j * R::RPI + lane / R::RC, key = kb + r;
          if (key < any_lo || key > any_hi || pg[j * R::RPI / 16] < 0) vr[j] = v4u32{0, 0, 0, 0};
          odd |= any_nonfinite<MT>(vr[j]);
        }
        odd = __any(odd);
      }
#pragma unroll
      for (int j = 0; j < R::VL; ++j)
        *reinterpret_cast<v4u32*>(vl + v_at<MT, D>(j * R::RPI + lane / R::RC, lane % R::RC)) = vr[j];
      // --- the next block is on its way while this one is computed
      int pc[NG];
#pragma unroll
      for (int t = 0; t < NG; ++t) pc[t] = pg[t], pg[t] = pgn[t];
      if (i + 1 < nb) {
        pages(i + 2, pgn);
        load_k(i + 1, pg);
        load_v(i + 1, pg);
      }
      if (!whole) {
#pragma unroll
        for (int t = 0; t < NG; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = kb + 16 * t + 4 * g + r;
            if (key < plo || key > phi || pc[t] < 0) st[t][r] = -INFINITY;
          }
      }
      // --- running maximum and sum
      float tm = st[0][0];
#pragma unroll
      for (int t = 0; t < NG; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) tm = fmaxf(tm, st[t][r]);
      tm = across32(across16(tm, MaxOp()), MaxOp());
      if (__any(tm > mx)) {
        const float mn = fmaxf(mx, tm), al = exp2_f((mx - (mn == -INFINITY ? 0.f : mn)) * c);
        sum *= al;
#pragma unroll
        for (int j = 0; j < NC; ++j) acc[j] *= al;
        mx = mn;
      }
      const float mc = mx == -INFINITY ? 0.f : mx * c;
#pragma unroll
      for (int t = 0; t < NG; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          st[t][r] = exp2_f(fmaf(st[t][r], c, -mc));
          sum += st[t][r];
        }
      // --- O^T += V^T P^T
      const frag pf = p_frag(st, MT());
      if (!odd) {
#pragma unroll
        for (int j = 0; j < NC; ++j) acc[j] = Mma<MT>::mma(v_frag<D>(vl, j, m, g, MT()), pf, acc[j]);
      } else {
        // An infinity or NaN in a value, which a weight of 0 does not hide: it counts as 0 in the
        // product; then rows that see a key whose value is +inf or NaN gain +inf, rows that see -inf or
        // NaN gain -inf, so that NaN or both make NaN.
        f32x4 vt[NG];
#pragma unroll
        for (int t = 0; t < NG; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int key = kb + 16 * t + 4 * g + r;
            vt[t][r] = key < plo || key > phi ? 0.f : 1.f;
          }
        const frag vis = p_frag(vt, MT());
#pragma unroll
        for (int j = 0; j < NC; ++j) {
          const frag f = v_frag<D>(vl, j, m, g, MT());
          acc[j] = Mma<MT>::mma(odd_part<0>(f), pf, acc[j]);
          const f32x4 pos = Mma<MT>::mma(odd_part<1>(f), vis, f32x4{});
          const f32x4 neg = Mma<MT>::mma(odd_part<2>(f), vis, f32x4{});
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if (pos[x] > 0.f) acc[j][x] += INFINITY;
            if (neg[x] > 0.f) acc[j][x] -= INFINITY;
          }
        }
      }
    }
    sum = across32(across16(sum, SumOp()), SumOp());

    // --- the waves meet: weights of their maxima, sums of their outputs
    __syncthreads();
    if (g == 0) ml[wave][m][0] = mx, ml[wave][m][1] = sum;
    float* ot = reinterpret_cast<float*>(lds) + wave * 16 * D;
#pragma unroll
    for (int j = 0; j < NC; ++j)  // parts of 16 bytes permuted by row: lanes of a column differ in bank
      *reinterpret_cast<f32x4*>(ot + m * D + 4 * ((4 * j + g) ^ (m & 7))) = acc[j];
    __syncthreads();
    const bool done = u0 == 0 && u1 == units;
    float* part = ws.part + part_of(blockIdx.x, at, per) * part_floats(D);
    if (tid == 0 && !done && u0 == 0) ws.cut[blockIdx.x] = {at, per, n, h, tile, units};
#pragma unroll
    for (int e = 0; e < 16 * D / 4 / kThreads; ++e) {
      const int i = e * kThreads + tid, r = i / (D / 4), q4 = i % (D / 4), orow = tile * 16 + r;
      float M = ml[0][r][0];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) M = fmaxf(M, ml[w][r][0]);
      const float Mu = M == -INFINITY ? 0.f : M;
      f32x4 o = {};
      float l = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float al = exp2_f((ml[w][r][0] - Mu) * c);
        l += al * ml[w][r][1];
        o += al * *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(lds) + (w * 16 + r) * D + 4 * (q4 ^ (r & 7)));
      }
      if (orow >= s.rows) continue;
      if (done) {
        const int ti = orow / G, hh = h * G + orow - ti * G;
        const int64_t out = (s.row0 + ti) * a.num_q_heads + hh;
        o *= l == 0.f ? 0.f : 1.f / l;
        MT* dst = (MT*)a.o + out * D + 4 * q4;
#pragma unroll
        for (int x = 0; x < 4; ++x) dst[x] = from_f32<MT>(o[x]);
        if (a.lse && q4 == 0) a.lse[out] = M * a.scale + (l == 0.f ? 0.f : logf(l));
      } else {
        *reinterpret_cast<f32x4*>(part + r * D + 4 * q4) = o;
        if (q4 == 0) part[16 * D + 2 * r] = M, part[16 * D + 2 * r + 1] = l;
      }
    }
    __syncthreads();
    at += u1 - u0;
  }
}

// Joins the parts of the items that were cut: one workgroup per cut item of the row kernel (the first
// row_groups workgroups), and one per 16 rows of those of the tile kernel. 16 threads a row.
template <typename MT, int D>
__global__ __launch_bounds__(kThreads) void join_kernel(AttnArgs a, int row_groups) {
  typedef TileShape<D, sizeof(MT) == 2> S;
  constexpr int E = D / 64;  // vectors of 4 channels per thread, 16 threads apart
  const int N = a.b.num_seqs, G = a.num_q_heads / a.num_kv_heads;
  const bool tiled = (int)blockIdx.x >= row_groups;
  const int w = tiled ? ((int)blockIdx.x - row_groups) / (S::ROWS / 16) : blockIdx.x;
  const Ws ws = ws_at(a.workspace);
  const TilePlan pl = tile_plan_at(a.tile_ws, N, max_tiles(N, a.b.total_tokens, G, S::ROWS));
  const Cut cut = tiled ? pl.cut[w] : ws.cut[w];
  if (cut.n < 0) return;
  const float* parts = tiled ? pl.part : ws.part;
  const int rows = tiled ? S::ROWS : 16, r0 = tiled ? ((int)blockIdx.x - row_groups) % (S::ROWS / 16) * 16 : 0;
  const int64_t per = cut.per, size = tiled ? tile_part_floats(S::ROWS, D) : part_floats(D);
  const int64_t row0 = first_row(a.b, cut.n);
  const int64_t all = (first_row(a.b, cut.n + 1) - row0) * G, last = (cut.at + cut.units - 1) / per;
  const float c = a.scale * LOG2E;
  const int lane = threadIdx.x & 15;
  const int r = r0 + threadIdx.x / 16;
  const int64_t row = (int64_t)cut.tile * rows + r;
  if (row >= all) return;
  f32x4 o[E] = {};
  float M = -INFINITY, l = 0.f;
  for (int64_t v = w; v <= last; ++v) {
    const float* part = parts + part_of(v, cut.at, per) * size;
    const float pm = part[(int64_t)rows * D + 2 * r], pl = part[(int64_t)rows * D + 2 * r + 1];
    const float mn = fmaxf(M, pm), mu = mn == -INFINITY ? 0.f : mn;
    const float al = exp2_f((M - mu) * c), be = exp2_f((pm - mu) * c);
#pragma unroll
    for (int i = 0; i < E; ++i)
      o[i] = o[i] * al + be * *reinterpret_cast<const f32x4*>(part + (int64_t)r * D + 64 * i + 4 * lane);
    l = l * al + be * pl;
    M = mn;
  }
  const int64_t tok = row / G, out = (row0 + tok) * a.num_q_heads + cut.h * G + row - tok * G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < E; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) ((MT*)a.o)[out * D + 64 * i + 4 * lane + x] = from_f32<MT>(o[i][x] * inv);
  if (a.lse && lane == 0) a.lse[out] = M * a.scale + (l == 0.f ? 0.f : logf(l));
}

// Which kernel takes which sequence. Without cu_seqlens every sequence has the same rows; with
// it and no more tokens than sequences, the batch is one of decode steps. The row kernel reads a sequence's
// keys once for every 16 rows, the tile kernel once for 256 (fp32: 128) but pads to them. Measured with 4 query heads
// to each of 8 K/V heads of 128, bf16, row and tile kernel in us:
//   rows              16          32          48          64
//   32 x 8192 keys    195, 334    299, 331    549, 332    604, 330
//    8 x 4096         34, 58      50, 58      71, 58      86, 59
//   16 x 512          17, 36      22, 36      28, 36      30, 37
//    1 x 16384        47, 50      38, 51      48, 52      40, 52
// and fp32, whose tiles of few rows cost more (32 x 8192: 370, 651; 590, 655; 1067, 1085; 1166, 1099; 8 x
// 4096 at 64 rows 162, 166; 16 x 512 at 64 49, 74).
struct Route {
  int row_limit, tile_rows;  // tile_rows 0: no tile kernel
  bool rows;                 // whether the row kernel runs
};
constexpr int row_limit(bool bf16) { return bf16 ? 32 : 64; }
Route route(int num_seqs, int64_t total_tokens, int G, bool ragged, int tile_rows, bool bf16) {
  const int64_t rows = total_tokens / num_seqs * G;
  Route r = {INT32_MAX, 0, true};
  if (ragged ? total_tokens > num_seqs : rows > row_limit(bf16)) {
    r.row_limit = row_limit(bf16);
    r.rows = ragged;
    r.tile_rows = tile_rows;
  }
  return r;
}

template <typename MT, int D>
void launch_rows(const AttnArgs& a, bool rows) {
  const bool tiles = a.tile_rows != 0;
  if (rows) row_kernel<MT, D><<<kGroups + tiles, kThreads, 0, a.stream>>>(a);
  if (tiles) launch_attn_tile(a, !rows);
  typedef TileShape<D, sizeof(MT) == 2> S;
  const int row_groups = rows ? kGroups : 0;
  join_kernel<MT, D><<<row_groups + (tiles ? S::GROUPS * (S::ROWS / 16) : 0), kThreads, 0, a.stream>>>(a, row_groups);
}

size_t row_bytes(int head_dim) {
  return (sizeof(Cut) * kGroups + (size_t)2 * kGroups * part_floats(head_dim) * 4 + 255) / 256 * 256;
}

}  // namespace

size_t attn_workspace_bytes(int num_seqs, int64_t total_tokens, int num_q_heads, int num_kv_heads,
                            int head_dim, bool bf16) {
  const int G = num_q_heads / num_kv_heads;
  size_t tile = 0;
  for (int ragged = 0; ragged < 2; ++ragged) {
    const Route r = route(num_seqs, total_tokens, G, ragged, attn_tile_rows(head_dim, bf16), bf16);
    const size_t n = r.tile_rows ? attn_tile_bytes(num_seqs, total_tokens, G, head_dim, bf16) : 0;
    tile = n > tile ? n : tile;
  }
  return row_bytes(head_dim) + tile;
}

hipError_t launch_attn(const AttnArgs& args) {
  if (args.b.total_tokens == 0) return hipSuccess;
  AttnArgs a = args;
  const Route r = route(a.b.num_seqs, a.b.total_tokens, a.num_q_heads / a.num_kv_heads, a.b.cu_seqlens != nullptr,
                        attn_tile_rows(a.head_dim, a.dtype_bf16), a.dtype_bf16);
  a.row_limit = r.row_limit, a.tile_rows = r.tile_rows;
  a.tile_ws = a.workspace + row_bytes(a.head_dim);
  if (a.dtype_bf16) {
    if (a.head_dim == 64) launch_rows<bf16, 64>(a, r.rows);
    if (a.head_dim == 128) launch_rows<bf16, 128>(a, r.rows);
    if (a.head_dim == 256) launch_rows<bf16, 256>(a, r.rows);
  } else {
    if (a.head_dim == 64) launch_rows<float, 64>(a, r.rows);
    if (a.head_dim == 128) launch_rows<float, 128>(a, r.rows);
    if (a.head_dim == 256) launch_rows<float, 256>(a, r.rows);
  }
  return hipGetLastError();
}

}  // namespace kda
