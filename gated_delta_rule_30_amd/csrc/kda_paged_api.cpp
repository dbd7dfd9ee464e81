// C ABI of the full-attention layers' operators (include/kda_paged.h): argument checks and launch.
// Every check here runs on the host before anything is enqueued.
#include <hip/hip_runtime.h>
#include <math.h>

#include "kda_paged_int.h"

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int kMaxHeads = 4096;
constexpr int kMaxSeqs = 1 << 20;
constexpr int kMaxPages = 1 << 30;

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }
bool valid_dtype(kda_dtype t) { return t == KDA_DTYPE_F32 || t == KDA_DTYPE_BF16; }
int64_t esize(kda_dtype t) { return t == KDA_DTYPE_BF16 ? 2 : 4; }

// [a, a + na) and [b, b + nb) overlap
bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  if (!a || !b || na <= 0 || nb <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// Bytes from the first to the last element of rows of `width` elements, `stride` apart.
int64_t extent(int64_t rows, int64_t width, int64_t stride, int64_t es) {
  return rows > 0 ? ((rows - 1) * stride + width) * es : 0;
}

// Whether rows a and b, of na and nb bytes, overlap; with one stride they may lie between each other.
bool rows_overlap(const void* a, int64_t na, int64_t stride_a, const void* b, int64_t nb, int64_t stride_b, int64_t rows) {
  if (!overlap(a, extent(rows, na, stride_a, 1), b, extent(rows, nb, stride_b, 1))) return false;
  if (stride_a != stride_b || rows < 2) return true;
  const int64_t d = reinterpret_cast<intptr_t>(b) - reinterpret_cast<intptr_t>(a), in = (d % stride_a + stride_a) % stride_a;
  return in < na || in + nb > stride_a;
}

// Rows of heads: 16-byte pointer and stride, rows that do not overlap.
bool bad_rows(const void* p, int64_t stride, int64_t width, int64_t es) {
  return !p || !aligned(p, 16) || stride < width || stride > kMaxStride || stride * es % 16 != 0;
}
bool valid_heads(int h) { return h > 0 && h <= kMaxHeads; }

kda_status check_batch(const int32_t* block_table, int64_t table_stride, const int32_t* seq_lens,
                       const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                       int32_t num_pages, int32_t max_pages, int32_t page_size) {
  if (num_seqs <= 0 || num_seqs > kMaxSeqs || total_tokens < 0 || total_tokens > kMaxTokens ||
      num_pages <= 0 || num_pages > kMaxPages || max_pages <= 0 || table_stride < max_pages ||
      table_stride > kMaxStride)
    return KDA_ERROR_INVALID_VALUE;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256)
    return KDA_ERROR_NOT_SUPPORTED;
  if (!block_table || !seq_lens || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      (cu_seqlens && !aligned(cu_seqlens, 4)))
    return KDA_ERROR_INVALID_VALUE;
  if (!cu_seqlens && total_tokens % num_seqs != 0) return KDA_ERROR_INVALID_VALUE;
  return KDA_SUCCESS;
}

kda::PagedBatch make_batch(const int32_t* block_table, int64_t table_stride,
                           const int32_t* seq_lens, const int32_t* cu_seqlens, int32_t num_seqs,
                           int64_t total_tokens, int32_t num_pages, int32_t max_pages,
                           int32_t page_size) {
  return {block_table, table_stride, seq_lens, cu_seqlens, num_seqs, total_tokens,
          num_pages, max_pages, page_size};
}

kda_status check_rope(int32_t head_dim, int32_t rot_dim, kda_dtype dtype, uint32_t flags,
                      uint32_t known, float scale) {
  if (!valid_dtype(dtype) || (flags & ~known)) return KDA_ERROR_NOT_SUPPORTED;
  if (head_dim < 16 || head_dim > 512 || head_dim % 16 != 0) return KDA_ERROR_NOT_SUPPORTED;
  if (rot_dim < 16 || rot_dim > head_dim || rot_dim % 16 != 0) return KDA_ERROR_NOT_SUPPORTED;
  if (!isfinite(scale)) return KDA_ERROR_INVALID_VALUE;
  return KDA_SUCCESS;
}

kda_status check_pools(const kda_page_pool* pools, int32_t num_pools, int32_t num_pages,
                       kda::Pools* out) {
  if (num_pools < 0 || num_pools > KDA_MAX_POOLS || (num_pools > 0 && !pools))
    return KDA_ERROR_INVALID_VALUE;
  out->n = num_pools;
  for (int k = 0; k < num_pools; ++k) {
    const kda_page_pool& p = pools[k];
    if (!p.base || !aligned(p.base, 16) || p.outer <= 0 || p.num_pages <= 0 || p.page_bytes <= 0 ||
        p.page_bytes % 16 != 0 || p.page_stride % 16 != 0 || p.outer_stride % 16 != 0 ||
        p.page_bytes > kMaxStride || p.page_stride > kMaxStride || p.outer_stride > kMaxStride)
      return KDA_ERROR_INVALID_VALUE;
    if (num_pages > 0 && p.num_pages != num_pages) return KDA_ERROR_INVALID_VALUE;
    // planes of whole pages, or pages of whole planes: no page overlaps another
    const bool pages_in = (p.num_pages == 1 || p.page_stride >= p.page_bytes) &&
                          (p.outer == 1 || p.outer_stride >= (p.num_pages - 1) * p.page_stride + p.page_bytes);
    const bool planes_in = (p.outer == 1 || p.outer_stride >= p.page_bytes) &&
                           (p.num_pages == 1 || p.page_stride >= (p.outer - 1) * p.outer_stride + p.page_bytes);
    if (!pages_in && !planes_in) return KDA_ERROR_INVALID_VALUE;
    out->p[k] = p;
  }
  return KDA_SUCCESS;
}

kda_status check_tables(const int32_t* page_refs, const int32_t* block_table, int64_t table_stride,
                        const int32_t* seq_lens, int32_t count, int32_t num_seqs,
                        int32_t num_pages, int32_t max_pages, int32_t page_size) {
  if (count < 0 || count > kMaxSeqs || num_seqs <= 0 || num_seqs > kMaxSeqs || num_pages <= 0 ||
      num_pages > kMaxPages || max_pages <= 0 || table_stride < max_pages || table_stride > kMaxStride)
    return KDA_ERROR_INVALID_VALUE;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256)
    return KDA_ERROR_NOT_SUPPORTED;
  const void* ptrs[] = {page_refs, block_table, seq_lens};
  for (const void* p : ptrs)
    if (!p || !aligned(p, 4)) return KDA_ERROR_INVALID_VALUE;
  return KDA_SUCCESS;
}

kda_status done(hipError_t e) { return e == hipSuccess ? KDA_SUCCESS : KDA_ERROR_LAUNCH; }

}  // namespace

extern "C" kda_status kda_rope(const void* q, const void* k, const int32_t* positions,
                               const double* inv_freq, int64_t num_tokens, int32_t num_q_heads,
                               int32_t num_k_heads, int32_t head_dim, int32_t rot_dim,
                               int64_t q_stride, int64_t k_stride, kda_dtype dtype,
                               uint32_t rope_flags, float scale, void* q_out, void* k_out,
                               void* stream) {
  if (num_tokens < 0 || num_tokens > kMaxTokens) return KDA_ERROR_INVALID_VALUE;
  kda_status st = check_rope(head_dim, rot_dim, dtype, rope_flags,
                             KDA_ROPE_INTERLEAVED | KDA_ROPE_INVERSE, scale);
  if (st != KDA_SUCCESS) return st;
  if ((!q && !k) || (q == nullptr) != (q_out == nullptr) || (k == nullptr) != (k_out == nullptr))
    return KDA_ERROR_INVALID_VALUE;
  if ((q && !valid_heads(num_q_heads)) || (k && !valid_heads(num_k_heads))) return KDA_ERROR_INVALID_VALUE;
  if (!positions || !aligned(positions, 4) || !inv_freq || !aligned(inv_freq, 8))
    return KDA_ERROR_INVALID_VALUE;
  const int64_t es = esize(dtype);
  const int64_t wq = q ? (int64_t)num_q_heads * head_dim : 0, wk = k ? (int64_t)num_k_heads * head_dim : 0;
  if ((q && (bad_rows(q, q_stride, wq, es) || !aligned(q_out, 16))) ||
      (k && (bad_rows(k, k_stride, wk, es) || !aligned(k_out, 16))))
    return KDA_ERROR_INVALID_VALUE;
  const int64_t T = num_tokens, qe = extent(T, wq, q_stride, es), ke = extent(T, wk, k_stride, es);
  const bool q_in = q_out == q, k_in = k_out == k;
  // an output of its own overlaps nothing that is read or written
  if ((!q_in && (overlap(q_out, T * wq * es, q, qe) || overlap(q_out, T * wq * es, k, ke))) ||
      (!k_in && (overlap(k_out, T * wk * es, k, ke) || overlap(k_out, T * wk * es, q, qe))) ||
      (q && k && !q_in && !k_in && overlap(q_out, T * wq * es, k_out, T * wk * es)))
    return KDA_ERROR_INVALID_VALUE;
  // what is turned in place is not read as another's input
  if (q && k && (q_in || k_in) && rows_overlap(q, wq * es, q_stride * es, k, wk * es, k_stride * es, T))
    return KDA_ERROR_INVALID_VALUE;
  if (q && q == k) return KDA_ERROR_INVALID_VALUE;
  kda::RopeArgs a = {};
  a.q = q, a.k = k;
  a.q_stride = q_stride, a.k_stride = k_stride;
  a.q_out = q_out, a.k_out = k_out;
  a.q_out_stride = q_in ? q_stride : wq, a.k_out_stride = k_in ? k_stride : wk;
  a.positions = positions, a.inv_freq = inv_freq;
  a.num_q_heads = q ? num_q_heads : 0, a.num_k_heads = k ? num_k_heads : 0;
  a.head_dim = head_dim, a.rot_dim = rot_dim, a.scale = scale;
  a.interleaved = rope_flags & KDA_ROPE_INTERLEAVED, a.inverse = rope_flags & KDA_ROPE_INVERSE;
  a.dtype_bf16 = dtype == KDA_DTYPE_BF16;
  a.b.total_tokens = num_tokens;
  a.stream = static_cast<hipStream_t>(stream);
  return done(kda::launch_rope(a));
}

extern "C" kda_status kda_cache_append(
    const void* q, const void* k, const void* v, int64_t q_stride, int64_t k_stride,
    int64_t v_stride, void* k_pages, void* v_pages, int64_t k_page_stride, int64_t v_page_stride,
    const int32_t* block_table, int64_t table_stride, const int32_t* seq_lens,
    const int32_t* cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t num_q_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t num_pages, int32_t max_pages,
    int32_t page_size, kda_dtype dtype, const double* inv_freq, int32_t rot_dim,
    uint32_t rope_flags, float scale, void* q_out, void* stream) {
  kda_status st = check_batch(block_table, table_stride, seq_lens, cu_seqlens, num_seqs,
                              total_tokens, num_pages, max_pages, page_size);
  if (st != KDA_SUCCESS) return st;
  st = check_rope(head_dim, inv_freq ? rot_dim : 16, dtype, rope_flags, KDA_ROPE_INTERLEAVED,
                  inv_freq ? scale : 1.f);
  if (st != KDA_SUCCESS) return st;
  if (!valid_heads(num_kv_heads) || (q && !valid_heads(num_q_heads)) ||
      (q == nullptr) != (q_out == nullptr) || (q && !inv_freq) || (inv_freq && !aligned(inv_freq, 8)))
    return KDA_ERROR_INVALID_VALUE;
  const int64_t es = esize(dtype), T = total_tokens;
  const int64_t wq = (int64_t)num_q_heads * head_dim, wk = (int64_t)num_kv_heads * head_dim;
  const int64_t page = wk * page_size;
  if (bad_rows(k, k_stride, wk, es) || bad_rows(v, v_stride, wk, es) ||
      (q && (bad_rows(q, q_stride, wq, es) || !aligned(q_out, 16))) ||
      bad_rows(k_pages, k_page_stride, page, es) || bad_rows(v_pages, v_page_stride, page, es))
    return KDA_ERROR_INVALID_VALUE;
  // The cache is written while q, k, v are read. k's and v's pages may lie between each other
  // (a pool of [page][k, v]), so those two are held only to different first elements.
  const int64_t ke = extent(T, wk, k_stride, es), ve = extent(T, wk, v_stride, es),
                qe = q ? extent(T, wq, q_stride, es) : 0;
  const int64_t kp = extent(num_pages, page, k_page_stride, es), vp = extent(num_pages, page, v_page_stride, es);
  const void* in[] = {q, k, v};
  const int64_t in_n[] = {qe, ke, ve};
  for (int i = 0; i < 3; ++i)
    if (overlap(in[i], in_n[i], k_pages, kp) || overlap(in[i], in_n[i], v_pages, vp))
      return KDA_ERROR_INVALID_VALUE;
  if (k_pages == v_pages) return KDA_ERROR_INVALID_VALUE;
  if (q && q_out == q &&
      (rows_overlap(q, wq * es, q_stride * es, k, wk * es, k_stride * es, T) ||
       rows_overlap(q, wq * es, q_stride * es, v, wk * es, v_stride * es, T)))
    return KDA_ERROR_INVALID_VALUE;
  if (q && q_out != q) {
    const int64_t n = T * wq * es;
    if (overlap(q_out, n, q, qe) || overlap(q_out, n, k, ke) || overlap(q_out, n, v, ve) ||
        overlap(q_out, n, k_pages, kp) || overlap(q_out, n, v_pages, vp))
      return KDA_ERROR_INVALID_VALUE;
  }
  kda::RopeArgs a = {};
  a.q = q, a.k = k, a.v = v;
  a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride;
  a.q_out = q_out, a.q_out_stride = q_out == q ? q_stride : wq;
  a.k_pages = static_cast<char*>(k_pages), a.v_pages = static_cast<char*>(v_pages);
  a.k_page_stride = k_page_stride, a.v_page_stride = v_page_stride;
  a.inv_freq = inv_freq;
  a.num_q_heads = q ? num_q_heads : 0, a.num_k_heads = num_kv_heads;
  a.head_dim = head_dim, a.rot_dim = rot_dim, a.scale = scale;
  a.interleaved = rope_flags & KDA_ROPE_INTERLEAVED;
  a.dtype_bf16 = dtype == KDA_DTYPE_BF16;
  a.b = make_batch(block_table, table_stride, seq_lens, cu_seqlens, num_seqs, total_tokens,
                   num_pages, max_pages, page_size);
  a.stream = static_cast<hipStream_t>(stream);
  return done(kda::launch_append(a));
}

static kda_status check_attn_shape(int32_t num_seqs, int64_t total_tokens, int32_t num_q_heads,
                                   int32_t num_kv_heads, int32_t head_dim, kda_dtype dtype) {
  if (num_seqs <= 0 || num_seqs > kMaxSeqs || total_tokens < 0 || total_tokens > kMaxTokens ||
      !valid_heads(num_q_heads) || !valid_heads(num_kv_heads) || num_q_heads % num_kv_heads != 0 ||
      total_tokens * num_q_heads > (int64_t)1 << 30)
    return KDA_ERROR_INVALID_VALUE;
  if (!valid_dtype(dtype) || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return KDA_ERROR_NOT_SUPPORTED;
  return KDA_SUCCESS;
}

extern "C" size_t kda_attn_paged_workspace_size(int32_t num_seqs, int64_t total_tokens,
                                                int32_t num_q_heads, int32_t num_kv_heads,
                                                int32_t head_dim, kda_dtype dtype) {
  if (check_attn_shape(num_seqs, total_tokens, num_q_heads, num_kv_heads, head_dim, dtype) != KDA_SUCCESS)
    return 0;
  return kda::attn_workspace_bytes(num_seqs, total_tokens, num_q_heads, num_kv_heads, head_dim,
                                   dtype == KDA_DTYPE_BF16);
}

extern "C" kda_status kda_attn_paged(const void* q, int64_t q_stride, const void* k_pages,
                                     const void* v_pages, int64_t k_page_stride,
                                     int64_t v_page_stride, const int32_t* block_table,
                                     int64_t table_stride, const int32_t* seq_lens,
                                     const int32_t* cu_seqlens, int32_t num_seqs,
                                     int64_t total_tokens, int32_t num_q_heads,
                                     int32_t num_kv_heads, int32_t head_dim, int32_t num_pages,
                                     int32_t max_pages, int32_t page_size, kda_dtype dtype,
                                     float scale, int32_t window, void* o, float* lse,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  kda_status st = check_attn_shape(num_seqs, total_tokens, num_q_heads, num_kv_heads, head_dim, dtype);
  if (st != KDA_SUCCESS) return st;
  st = check_batch(block_table, table_stride, seq_lens, cu_seqlens, num_seqs, total_tokens,
                   num_pages, max_pages, page_size);
  if (st != KDA_SUCCESS) return st;
  if (!(scale > 0.f) || !isfinite(scale) || window < 0) return KDA_ERROR_INVALID_VALUE;
  const int64_t es = esize(dtype), T = total_tokens;
  const int64_t wq = (int64_t)num_q_heads * head_dim, page = (int64_t)num_kv_heads * head_dim * page_size;
  if (bad_rows(q, q_stride, wq, es) || !o || !aligned(o, 16) || (lse && !aligned(lse, 4)) ||
      bad_rows(k_pages, k_page_stride, page, es) || bad_rows(v_pages, v_page_stride, page, es))
    return KDA_ERROR_INVALID_VALUE;
  const int64_t qe = extent(T, wq, q_stride, es), oe = T * wq * es, le = lse ? T * num_q_heads * 4 : 0;
  const int64_t kp = extent(num_pages, page, k_page_stride, es), vp = extent(num_pages, page, v_page_stride, es);
  if (overlap(o, oe, q, qe) || overlap(o, oe, k_pages, kp) || overlap(o, oe, v_pages, vp) ||
      overlap(lse, le, q, qe) || overlap(lse, le, k_pages, kp) || overlap(lse, le, v_pages, vp) ||
      overlap(lse, le, o, oe))
    return KDA_ERROR_INVALID_VALUE;
  if (!workspace || !aligned(workspace, 256)) return KDA_ERROR_INVALID_VALUE;
  const int64_t need = (int64_t)kda::attn_workspace_bytes(num_seqs, total_tokens, num_q_heads, num_kv_heads, head_dim,
                                                          dtype == KDA_DTYPE_BF16);
  if (workspace_bytes < (size_t)need) return KDA_ERROR_WORKSPACE_TOO_SMALL;
  if (overlap(workspace, need, q, qe) || overlap(workspace, need, o, oe) || overlap(workspace, need, lse, le) ||
      overlap(workspace, need, k_pages, kp) || overlap(workspace, need, v_pages, vp))
    return KDA_ERROR_INVALID_VALUE;
  kda::AttnArgs a = {};
  a.q = q, a.q_stride = q_stride;
  a.k_pages = static_cast<const char*>(k_pages), a.v_pages = static_cast<const char*>(v_pages);
  a.k_page_stride = k_page_stride, a.v_page_stride = v_page_stride;
  a.b = make_batch(block_table, table_stride, seq_lens, cu_seqlens, num_seqs, total_tokens,
                   num_pages, max_pages, page_size);
  a.num_q_heads = num_q_heads, a.num_kv_heads = num_kv_heads, a.head_dim = head_dim;
  a.dtype_bf16 = dtype == KDA_DTYPE_BF16;
  a.scale = scale, a.window = window;
  a.o = o, a.lse = lse;
  a.workspace = static_cast<char*>(workspace);
  a.stream = static_cast<hipStream_t>(stream);
  return done(kda::launch_attn(a));
}

extern "C" size_t kda_pages_plan_workspace_size(int32_t count, int32_t num_seqs, int32_t num_pages) {
  if (count < 0 || count > kMaxSeqs || num_seqs <= 0 || num_seqs > kMaxSeqs || num_pages <= 0 || num_pages > kMaxPages)
    return 0;
  return kda::pages_plan_bytes(count, num_seqs, num_pages);
}

// granted and the workspace lie apart from each other and from the tables.
static kda_status check_plan(const kda::PagesArgs& a, const void* workspace, size_t workspace_bytes) {
  if (!a.granted || !aligned(a.granted, 4) || !workspace || !aligned(workspace, 256))
    return KDA_ERROR_INVALID_VALUE;
  const int64_t need = (int64_t)kda::pages_plan_bytes(a.count, a.num_seqs, a.num_pages), ge = (int64_t)a.count * 4;
  if (workspace_bytes < (size_t)need) return KDA_ERROR_WORKSPACE_TOO_SMALL;
  const void* tables[] = {a.page_refs, a.block_table, a.seq_lens};
  const int64_t bytes[] = {(int64_t)a.num_pages * 4, extent(a.num_seqs, a.max_pages, a.table_stride, 4),
                           (int64_t)a.num_seqs * 4};
  for (int i = 0; i < 3; ++i)
    if (overlap(workspace, need, tables[i], bytes[i]) || overlap(a.granted, ge, tables[i], bytes[i]))
      return KDA_ERROR_INVALID_VALUE;
  return overlap(workspace, need, a.granted, ge) ? KDA_ERROR_INVALID_VALUE : KDA_SUCCESS;
}

extern "C" kda_status kda_pages_alloc(int32_t* page_refs, int32_t* block_table, int64_t table_stride,
                                      int32_t* seq_lens, const int32_t* seqs,
                                      const int32_t* new_tokens, int32_t count, int32_t num_seqs,
                                      int32_t num_pages, int32_t max_pages, int32_t page_size,
                                      int32_t* granted, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  kda_status st = check_tables(page_refs, block_table, table_stride, seq_lens, count, num_seqs,
                               num_pages, max_pages, page_size);
  if (st != KDA_SUCCESS) return st;
  if (!seqs && count != num_seqs) return KDA_ERROR_INVALID_VALUE;
  if (count == 0) return KDA_SUCCESS;
  if (!new_tokens || !aligned(new_tokens, 4) || (seqs && !aligned(seqs, 4))) return KDA_ERROR_INVALID_VALUE;
  kda::PagesArgs a = {};
  a.page_refs = page_refs, a.block_table = block_table, a.seq_lens = seq_lens;
  a.table_stride = table_stride;
  a.seqs = seqs, a.new_tokens = new_tokens;
  a.count = count, a.num_seqs = num_seqs, a.num_pages = num_pages, a.max_pages = max_pages;
  a.page_size = page_size;
  a.granted = granted;
  st = check_plan(a, workspace, workspace_bytes);
  if (st != KDA_SUCCESS) return st;
  a.workspace = static_cast<char*>(workspace);
  a.stream = static_cast<hipStream_t>(stream);
  return done(kda::launch_pages_alloc(a));
}

extern "C" kda_status kda_pages_fork(const kda_page_pool* pools, int32_t num_pools,
                                     int32_t* page_refs, int32_t* block_table,
                                     int64_t table_stride, int32_t* seq_lens,
                                     const int32_t* parents, const int32_t* children,
                                     int32_t count, int32_t num_seqs, int32_t num_pages,
                                     int32_t max_pages, int32_t page_size, int32_t* granted,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  kda_status st = check_tables(page_refs, block_table, table_stride, seq_lens, count, num_seqs,
                               num_pages, max_pages, page_size);
  if (st != KDA_SUCCESS) return st;
  kda::PagesArgs a = {};
  st = check_pools(pools, num_pools, num_pages, &a.pools);
  if (st != KDA_SUCCESS) return st;
  if (count == 0) return KDA_SUCCESS;
  if (!parents || !aligned(parents, 4) || !children || !aligned(children, 4)) return KDA_ERROR_INVALID_VALUE;
  a.page_refs = page_refs, a.block_table = block_table, a.seq_lens = seq_lens;
  a.table_stride = table_stride;
  a.seqs = children, a.parents = parents;
  a.count = count, a.num_seqs = num_seqs, a.num_pages = num_pages, a.max_pages = max_pages;
  a.page_size = page_size;
  a.granted = granted;
  st = check_plan(a, workspace, workspace_bytes);
  if (st != KDA_SUCCESS) return st;
  a.workspace = static_cast<char*>(workspace);
  a.stream = static_cast<hipStream_t>(stream);
  return done(kda::launch_pages_fork(a));
}

extern "C" kda_status kda_pages_free(int32_t* page_refs, int32_t* block_table, int64_t table_stride,
                                     int32_t* seq_lens, const int32_t* seqs, int32_t count,
                                     int32_t num_seqs, int32_t num_pages, int32_t max_pages,
                                     int32_t page_size, void* stream) {
  kda_status st = check_tables(page_refs, block_table, table_stride, seq_lens, count, num_seqs,
                               num_pages, max_pages, page_size);
  if (st != KDA_SUCCESS) return st;
  if (count == 0) return KDA_SUCCESS;
  if (!seqs || !aligned(seqs, 4)) return KDA_ERROR_INVALID_VALUE;
  kda::PagesArgs a = {};
  a.page_refs = page_refs, a.block_table = block_table, a.seq_lens = seq_lens;
  a.table_stride = table_stride;
  a.seqs = seqs;
  a.count = count, a.num_seqs = num_seqs, a.num_pages = num_pages, a.max_pages = max_pages;
  a.page_size = page_size;
  a.stream = static_cast<hipStream_t>(stream);
  return done(kda::launch_pages_free(a));
}

extern "C" size_t kda_pages_compact_workspace_size(int32_t num_pages) {
  return num_pages <= 0 || num_pages > kMaxPages ? 0 : kda::pages_compact_bytes(num_pages);
}

extern "C" kda_status kda_pages_compact(const kda_page_pool* pools, int32_t num_pools,
                                        const int32_t* page_refs, const int32_t* block_table,
                                        int64_t table_stride, int32_t num_seqs, int32_t num_pages,
                                        int32_t max_pages, int32_t* out_refs, int32_t* out_table,
                                        int64_t out_table_stride, int32_t* moved, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  kda_status st = check_tables(page_refs, block_table, table_stride, page_refs, 0, num_seqs,
                               num_pages, max_pages, 16);
  if (st != KDA_SUCCESS) return st;
  kda::CompactArgs a = {};
  st = check_pools(pools, num_pools, num_pages, &a.pools);
  if (st != KDA_SUCCESS) return st;
  const void* ptrs[] = {out_refs, out_table, moved};
  for (const void* p : ptrs)
    if (!p || !aligned(p, 4)) return KDA_ERROR_INVALID_VALUE;
  if (out_table_stride < max_pages || out_table_stride > kMaxStride) return KDA_ERROR_INVALID_VALUE;
  const int64_t re = (int64_t)num_pages * 4, te = extent(num_seqs, max_pages, table_stride, 4),
                oe = extent(num_seqs, max_pages, out_table_stride, 4);
  // in place, element by element, or apart from everything that is read
  if ((out_refs != page_refs && overlap(out_refs, re, page_refs, re)) || overlap(out_refs, re, block_table, te) ||
      (out_table != block_table ? overlap(out_table, oe, block_table, te) : out_table_stride != table_stride) ||
      overlap(out_table, oe, page_refs, re) || overlap(out_table, oe, out_refs, re) ||
      overlap(moved, 4, page_refs, re) || overlap(moved, 4, block_table, te) || overlap(moved, 4, out_refs, re) ||
      overlap(moved, 4, out_table, oe))
    return KDA_ERROR_INVALID_VALUE;
  if (!workspace || !aligned(workspace, 256)) return KDA_ERROR_INVALID_VALUE;
  const int64_t need = (int64_t)kda::pages_compact_bytes(num_pages);
  if (workspace_bytes < (size_t)need) return KDA_ERROR_WORKSPACE_TOO_SMALL;
  if (overlap(workspace, need, page_refs, re) || overlap(workspace, need, block_table, te) ||
      overlap(workspace, need, out_refs, re) || overlap(workspace, need, out_table, oe) ||
      overlap(workspace, need, moved, 4))
    return KDA_ERROR_INVALID_VALUE;
  a.page_refs = page_refs, a.block_table = block_table;
  a.table_stride = table_stride, a.out_table_stride = out_table_stride;
  a.num_seqs = num_seqs, a.num_pages = num_pages, a.max_pages = max_pages;
  a.out_refs = out_refs, a.out_table = out_table, a.moved = moved;
  a.workspace = static_cast<char*>(workspace);
  a.stream = static_cast<hipStream_t>(stream);
  return done(kda::launch_pages_compact(a));
}

extern "C" kda_status kda_pages_copy(const kda_page_pool* pools, int32_t num_pools,
                                     const int32_t* src, const int32_t* dst, int32_t count,
                                     void* stream) {
  kda::Pools p = {};
  if (count < 0) return KDA_ERROR_INVALID_VALUE;
  const kda_status st = check_pools(pools, num_pools, 0, &p);
  if (st != KDA_SUCCESS) return st;
  if (count == 0 || num_pools == 0) return KDA_SUCCESS;
  if (!src || !dst || !aligned(src, 4) || !aligned(dst, 4)) return KDA_ERROR_INVALID_VALUE;
  return done(kda::launch_pages_copy(p, src, dst, count, static_cast<hipStream_t>(stream)));
}
