// Bookkeeping of a paged cache's pages, and their copies.
//
// page_refs[p] counts the table entries that hold page p; the free pages are those with 0, so
// there is no list to keep in step and every choice ("the lowest free page") is a function of the
// counts: the same on every run, whatever the order in which workgroups run. Only integer
// atomics are used, whose order does not show.
//
// Alloc and fork hand out pages with one workgroup (the requests' needs are prefix-summed in
// request order, and request i's pages are the free pages of ranks rank_i ..): the counts are a few
// hundred kilobytes at most in practice, and the calls are bound by the latency of the loads that wait for each
// other, so those that do not are issued first, and claims are settled in LDS where they fit. The copies
// are bound by HBM and run over every (page, plane, 8 KB part).
// Measured: compaction of 8192 pages (516 MB moved) 96 us, of which 5 each go to the counts and the
// ranks; a fork of one sequence into four 6.4 us of plan and 4 of rows and copies.
#include "kda_device.h"
#include "kda_paged_int.h"

namespace kda {

namespace {

constexpr int kPlan = 1024;    // threads of the planning workgroup
constexpr int kCopy = 256;     // threads of the others
constexpr int kPart = 8192;    // bytes of a page that one workgroup copies at a time

__device__ __forceinline__ int pages_of(int64_t len, int ps) { return (int)((len + ps - 1) / ps); }

// Inclusive prefix sum over the workgroup's threads, in thread order; *total gets the sum.
template <typename X>
__device__ __forceinline__ X block_scan(X x, X* lds, X* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const X y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();  // lds may still be read by the previous call
  if (lane == 63) lds[wave] = x;
  __syncthreads();
  X before = 0, all = 0;
  for (int w = 0; w < waves; ++w) {
    const X s = lds[w];
    before += w < wave ? s : X(0);
    all += s;
  }
  *total = all;
  return x + before;
}

// Copies page `from` to page `to` of one pool, part `part` of plane `plane`. Neither is read again soon,
// so both pass the caches by; parts of 8 KB and a workgroup for nearly every part: a pool's 258 MB in 64 KB
// pages move in 98 us (5.3 TB/s; 114 us through the caches with 16 KB parts, 160 us with 32 KB).
__device__ __forceinline__ void copy_part(const kda_page_pool& p, int from, int to, int plane, int64_t part) {
  const int64_t at = part * kPart, n = min((int64_t)kPart, p.page_bytes - at) / 16;
  const char* base = (const char*)p.base + plane * p.outer_stride + at;
  const v4u32* s = (const v4u32*)(base + from * p.page_stride);
  v4u32* d = (v4u32*)(base + to * p.page_stride);
  v4u32 x[kPart / 16 / kCopy];
#pragma unroll
  for (int i = 0; i < kPart / 16 / kCopy; ++i)
    if (threadIdx.x + i * kCopy < n) x[i] = __builtin_nontemporal_load(s + threadIdx.x + i * kCopy);
#pragma unroll
  for (int i = 0; i < kPart / 16 / kCopy; ++i)
    if (threadIdx.x + i * kCopy < n) __builtin_nontemporal_store(x[i], d + threadIdx.x + i * kCopy);
}
__host__ __device__ __forceinline__ int64_t parts_of(const kda_page_pool& p) {
  return (p.page_bytes + kPart - 1) / kPart;
}

// ------------------------------------------------------------------ copy
// Copies pages src[i] to dst[i], i < n, as workgroup `first` of `groups`. A pair with an index outside the
// pool is passed over.
__device__ __forceinline__ void copy_pages(const Pools& pools, const int32_t* src, const int32_t* dst, int n, int first,
                                           int groups) {
  for (int k = 0; k < pools.n; ++k) {
    const kda_page_pool& p = pools.p[k];
    const int64_t parts = parts_of(p), per = parts * p.outer, total = per * n;
    for (int64_t w = first; w < total; w += groups) {
      const int i = (int)(w / per);
      const int64_t r = w - i * per;
      const int s = src[i], d = dst[i], plane = (int)(r / parts);
      if ((unsigned)s >= (unsigned)p.num_pages || (unsigned)d >= (unsigned)p.num_pages || s == d) continue;
      copy_part(p, s, d, plane, r - plane * parts);
    }
  }
}
__global__ __launch_bounds__(kCopy) void copy_kernel(Pools pools, const int32_t* src, const int32_t* dst, int n) {
  copy_pages(pools, src, dst, n, blockIdx.x, gridDim.x);
}

// ------------------------------------------------------------------ alloc and fork
// Workspace of a plan: the claims of the sequences, then per request its rank, its need and
// whether it is well formed, the pages copied (from, to), and the free pages in order.
struct Plan {
  int32_t *claim, *rank, *need, *from, *to, *len, *free_list;
};
__host__ __device__ inline Plan plan_at(char* ws, int count, int num_seqs) {
  int32_t* p = reinterpret_cast<int32_t*>(ws);
  Plan r;
  r.claim = p;
  r.rank = r.claim + num_seqs;
  r.need = r.rank + count;
  r.from = r.need + count;
  r.to = r.from + count;
  r.len = r.to + count;
  r.free_list = r.len + count;
  return r;
}

// 16 counts, from wherever they start.
struct Refs {
  int x[16];
};
__device__ __forceinline__ Refs load_refs(const int32_t* refs, int at, int n) {
  Refs r;
  if (at + 16 <= n) {
    __builtin_memcpy(&r, refs + at, sizeof r);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) r.x[j] = at + j < n ? refs[at + j] : 1;
  }
  return r;
}

constexpr int kClaims = 8192;  // sequences whose claims fit in LDS

template <bool FORK>
__global__ __launch_bounds__(kPlan) void plan_kernel(PagesArgs a) {
  __shared__ int lds[kPlan / 64], claims[kClaims];
  __shared__ int64_t sums[kPlan / 64];
  const Plan pl = plan_at(a.workspace, a.count, a.num_seqs);
  const int tid = threadIdx.x, ps = a.page_size;
  Refs refs = load_refs(a.page_refs, tid * 16, a.num_pages);  // on their way while the requests are looked at
  const bool in_lds = a.num_seqs <= kClaims;
  int32_t* claim = in_lds ? claims : pl.claim;
  // the first request that names a sequence has it
  if (a.seqs) {
    for (int i = tid; i < a.count; i += kPlan)
      if ((unsigned)a.seqs[i] < (unsigned)a.num_seqs) claim[a.seqs[i]] = 0x7fffffff;
    __syncthreads();
    for (int i = tid; i < a.count; i += kPlan)
      if ((unsigned)a.seqs[i] < (unsigned)a.num_seqs) atomicMin(&claim[a.seqs[i]], i);
    __syncthreads();
  }
  auto claimed = [&](int s) {
    // claims in memory were written by atomics, past this compute unit's own cache
    return in_lds ? claims[s] : __hip_atomic_load(&pl.claim[s], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  };
  // needs and ranks, in the order of the requests
  int64_t carry = 0;
  for (int i0 = 0; i0 < a.count; i0 += kPlan) {
    const int i = i0 + tid;
    int need = -1, len = 0;  // -1: not well formed
    if (i < a.count) {
      const int s = a.seqs ? a.seqs[i] : i;
      bool ok = (unsigned)s < (unsigned)a.num_seqs && (!a.seqs || claimed(s) == i);
      if constexpr (FORK) {
        const int f = a.parents[i];
        ok = ok && (unsigned)f < (unsigned)a.num_seqs;
        const int has = ok ? a.seq_lens[s] : 1;
        len = ok ? a.seq_lens[f] : 0;
        if (ok && has == 0 && len >= 0 && pages_of(len, ps) <= a.max_pages) need = len % ps != 0;
      } else {
        const int m = a.new_tokens[i];
        len = ok ? a.seq_lens[s] : 0;
        const int64_t to = (int64_t)len + m;
        if (ok && len >= 0 && m >= 0 && to <= 0x7fffffff && pages_of(to, ps) <= a.max_pages)
          need = pages_of(to, ps) - pages_of(len, ps);
      }
    }
    int64_t total;  // (1024 needs of long rows pass 32 bits)
    const int64_t incl = block_scan((int64_t)max(need, 0), sums, &total);
    if (i < a.count) {
      const int64_t r = carry + incl - max(need, 0);
      pl.rank[i] = (int)min(r, (int64_t)a.num_pages);  // past the last page: never granted
      pl.need[i] = need;
      pl.len[i] = len;
    }
    carry += total;
  }
  // the free pages, from the lowest, as many as are asked for
  const int want = (int)min(carry, (int64_t)a.num_pages);
  int found = 0;
  for (int p0 = 0; p0 < a.num_pages && found < want; p0 += kPlan * 16) {
    const int at = p0 + tid * 16;
    if (p0) refs = load_refs(a.page_refs, at, a.num_pages);
    int mine = 0, total;
#pragma unroll
    for (int j = 0; j < 16; ++j) mine += refs.x[j] == 0;
    int r = found + block_scan(mine, lds, &total) - mine;
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (refs.x[j] == 0) {
        if (r < want) pl.free_list[r] = at + j;
        ++r;
      }
    found += total;
  }
  __syncthreads();
  // what is granted: a fork by a thread, which takes one page at most; an alloc by 16, page by page
  constexpr int L = FORK ? 1 : 16;
  const int lane = tid % L;
  for (int i = tid / L; i < a.count; i += kPlan / L) {
    const int need = pl.need[i], rank = pl.rank[i], len = pl.len[i];
    const bool ok = need == 0 || (need > 0 && (int64_t)rank + need <= found);
    if (lane == 0) a.granted[i] = ok;
    if constexpr (FORK) {
      int from = -1, to = -1;
      if (ok && need) {
        const int s = a.seqs[i], f = a.parents[i];
        from = a.block_table[f * a.table_stride + len / ps];
        to = pl.free_list[rank];
        a.block_table[s * a.table_stride + len / ps] = to;
        a.page_refs[to] = 1;
      }
      pl.len[i] = ok ? len : -1;
      pl.from[i] = from;
      pl.to[i] = to;
    } else if (ok) {
      const int s = a.seqs ? a.seqs[i] : i, have = pages_of(len, ps);
      for (int j = lane; j < need; j += L) {
        const int p = pl.free_list[rank + j];
        a.block_table[s * a.table_stride + have + j] = p;
        a.page_refs[p] = 1;
      }
      if (lane == 0) a.seq_lens[s] = len + a.new_tokens[i];
    }
  }
  if constexpr (FORK) {
    // lengths last: a child may be named as the (empty) parent of another pair
    __syncthreads();
    for (int i = tid; i < a.count; i += kPlan)
      if (pl.len[i] >= 0) a.seq_lens[a.seqs[i]] = pl.len[i];
  }
}

// What follows the plan of a fork, in one launch (a second one costs the host 3 us). The first count * ny workgroups
// fill the rows of granted pairs: the child's full pages are the parent's, each counted once more. The others copy the
// pages that are not full.
__global__ __launch_bounds__(kCopy) void fork_kernel(PagesArgs a, int ny) {
  const Plan pl = plan_at(a.workspace, a.count, a.num_seqs);
  const int groups = a.count * ny;
  if ((int)blockIdx.x >= groups) {
    copy_pages(a.pools, pl.from, pl.to, a.count, blockIdx.x - groups, gridDim.x - groups);
    return;
  }
  const int i = blockIdx.x / ny, y = blockIdx.x % ny, full = pl.len[i] / a.page_size;
  if (pl.len[i] < 0) return;
  const int32_t* from = a.block_table + a.parents[i] * a.table_stride;
  int32_t* to = a.block_table + a.seqs[i] * a.table_stride;
  for (int j = y * kCopy + threadIdx.x; j < full; j += ny * kCopy) {
    const int p = from[j];
    to[j] = p;
    if ((unsigned)p < (unsigned)a.num_pages) atomicAdd(&a.page_refs[p], 1);
  }
}

// ------------------------------------------------------------------ free
// One workgroup per request. The length is exchanged for 0, so a sequence that is named twice is
// freed by one of its workgroups and found empty by the others.
__global__ __launch_bounds__(kCopy) void free_kernel(PagesArgs a) {
  __shared__ int len;
  const int s = a.seqs[blockIdx.x];
  if ((unsigned)s >= (unsigned)a.num_seqs) return;
  if (threadIdx.x == 0) len = atomicExch(&a.seq_lens[s], 0);
  __syncthreads();
  if (len <= 0) return;
  const int n = min(pages_of(len, a.page_size), a.max_pages);
  int32_t* row = a.block_table + s * a.table_stride;
  for (int j = threadIdx.x; j < n; j += kCopy) {
    const int p = row[j];
    row[j] = -1;
    if ((unsigned)p < (unsigned)a.num_pages) atomicSub(&a.page_refs[p], 1);
  }
}

// ------------------------------------------------------------------ compact
// With L live pages in all, the holes are the free pages below L and the movers the live pages
// at or above it, equally many; the hole of rank r (from the bottom) gets the mover of rank r
// (from the top). A page's rank follows from the number of live pages below it, b: a hole's is p - b, a
// mover's L - 1 - b. So: count the live pages of each block, then rank every page, then move.
constexpr int kPerThread = 4, kBlockPages = kPerThread * kCopy;

struct CompactAt {
  int32_t *counts, *rank_of, *hole, *mover, *moved;
};
__host__ __device__ inline CompactAt compact_at(char* ws, int num_pages) {
  const int blocks = (num_pages + kBlockPages - 1) / kBlockPages;
  CompactAt c;
  c.counts = reinterpret_cast<int32_t*>(ws);
  c.rank_of = c.counts + blocks;
  c.hole = c.rank_of + num_pages;
  c.mover = c.hole + num_pages;
  c.moved = c.mover + num_pages;
  return c;
}

__global__ __launch_bounds__(kCopy) void count_kernel(CompactArgs a) {
  __shared__ int lds[kCopy / 64];
  const int at = blockIdx.x * kBlockPages + threadIdx.x * kPerThread;
  int n = 0, total;
  for (int j = 0; j < kPerThread; ++j) n += at + j < a.num_pages && a.page_refs[at + j] > 0;
  block_scan(n, lds, &total);
  if (threadIdx.x == 0) compact_at(a.workspace, a.num_pages).counts[blockIdx.x] = total;
}

__global__ __launch_bounds__(kCopy) void rank_kernel(CompactArgs a) {
  __shared__ int lds[kCopy / 64];
  const CompactAt c = compact_at(a.workspace, a.num_pages);
  const int blocks = gridDim.x;
  int below = 0, live = 0;
  for (int i0 = 0; i0 < blocks; i0 += kCopy) {
    const int i = i0 + threadIdx.x, x = i < blocks ? c.counts[i] : 0;
    int t;
    block_scan(i < (int)blockIdx.x ? x : 0, lds, &t);
    below += t;
    block_scan(x, lds, &t);
    live += t;
  }
  const int at = blockIdx.x * kBlockPages + threadIdx.x * kPerThread;
  int n = 0, total;
  for (int j = 0; j < kPerThread; ++j) n += at + j < a.num_pages && a.page_refs[at + j] > 0;
  int b = below + block_scan(n, lds, &total) - n;
  for (int j = 0; j < kPerThread && at + j < a.num_pages; ++j) {
    const int p = at + j, r = a.page_refs[p] > 0;
    int rank = -1;
    if (!r && p < live) c.hole[p - b] = p;
    if (r && p >= live) c.mover[rank = live - 1 - b] = p;
    c.rank_of[p] = rank;
    // the pages from `live` on: all of the holes lie below them
    if (p == live) *c.moved = *a.moved = p - b;
    b += r;
  }
  if (live == a.num_pages && blockIdx.x == 0 && threadIdx.x == 0) *c.moved = *a.moved = 0;
}

// The first `groups` workgroups write the new counts and table, the others copy the pages.
__global__ __launch_bounds__(kCopy) void move_kernel(CompactArgs a, int groups) {
  const CompactAt c = compact_at(a.workspace, a.num_pages);
  const int moved = *c.moved;
  if ((int)blockIdx.x >= groups) {
    copy_pages(a.pools, c.mover, c.hole, moved, blockIdx.x - groups, gridDim.x - groups);
    return;
  }
  const int64_t first = (int64_t)blockIdx.x * kCopy + threadIdx.x, step = (int64_t)groups * kCopy;
  const int64_t entries = (int64_t)a.num_seqs * a.max_pages;
  for (int64_t e = first; e < entries; e += step) {
    const int64_t n = e / a.max_pages, j = e - n * a.max_pages;
    int p = a.block_table[n * a.table_stride + j];
    if ((unsigned)p < (unsigned)a.num_pages && c.rank_of[p] >= 0) p = c.hole[c.rank_of[p]];
    a.out_table[n * a.out_table_stride + j] = p;
  }
  // one thread writes a mover's count and its hole's, so the counts may be changed in place
  for (int64_t p = first; p < a.num_pages; p += step) {
    const int refs = a.page_refs[p], r = c.rank_of[p];
    if (r >= 0) {
      a.out_refs[c.hole[r]] = refs;
      a.out_refs[p] = 0;
    } else if (refs > 0) {
      a.out_refs[p] = refs;
    } else {
      // a free page: a hole's count is its mover's thread's to write
      int lo = 0, hi = moved;
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (c.hole[mid] < p) lo = mid + 1;
        else hi = mid;
      }
      if (lo == moved || c.hole[lo] != p) a.out_refs[p] = 0;
    }
  }
}

unsigned copy_grid(const Pools& pools, int64_t pairs) {
  int64_t most = 1;
  for (int k = 0; k < pools.n; ++k) {
    const int64_t w = parts_of(pools.p[k]) * pools.p[k].outer * pairs;
    most = w > most ? w : most;
  }
  return (unsigned)(most < 32768 ? most : 32768);
}

}  // namespace

size_t pages_plan_bytes(int count, int num_seqs, int num_pages) {
  return 4 * ((size_t)num_seqs + 5 * (size_t)count + (size_t)num_pages);
}
size_t pages_compact_bytes(int num_pages) {
  return 4 * ((size_t)(num_pages + kBlockPages - 1) / kBlockPages + 3 * (size_t)num_pages + 1);
}

hipError_t launch_pages_alloc(const PagesArgs& a) {
  plan_kernel<false><<<1, kPlan, 0, a.stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_pages_fork(const PagesArgs& a) {
  plan_kernel<true><<<1, kPlan, 0, a.stream>>>(a);
  // (count is 2^20 at most, and a grid holds 2^32 threads)
  const int per = (a.max_pages - 1) / (4 * kCopy) + 1, room = (1 << 22) / a.count, ny = per < room ? (per < 64 ? per : 64) : room;
  const unsigned copies = a.pools.n > 0 ? copy_grid(a.pools, a.count) : 0;
  fork_kernel<<<(unsigned)(a.count * ny) + copies, kCopy, 0, a.stream>>>(a, ny);
  return hipGetLastError();
}

hipError_t launch_pages_free(const PagesArgs& a) {
  free_kernel<<<a.count, kCopy, 0, a.stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_pages_compact(const CompactArgs& a) {
  const unsigned blocks = (unsigned)((a.num_pages + kBlockPages - 1) / kBlockPages);
  count_kernel<<<blocks, kCopy, 0, a.stream>>>(a);
  rank_kernel<<<blocks, kCopy, 0, a.stream>>>(a);
  const int64_t n = (int64_t)a.num_seqs * a.max_pages, m = n > a.num_pages ? n : a.num_pages;
  const int64_t want = (m + kCopy - 1) / kCopy, groups = want < 2048 ? want : 2048;
  const unsigned copies = a.pools.n > 0 ? copy_grid(a.pools, a.num_pages / 2) : 0;
  move_kernel<<<(unsigned)groups + copies, kCopy, 0, a.stream>>>(a, (int)groups);
  return hipGetLastError();
}

hipError_t launch_pages_copy(const Pools& pools, const int32_t* src, const int32_t* dst, int count,
                             hipStream_t stream) {
  copy_kernel<<<copy_grid(pools, count), kCopy, 0, stream>>>(pools, src, dst, count);
  return hipGetLastError();
}

}  // namespace kda
