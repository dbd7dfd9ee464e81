// Internal host-side declarations of the full-attention layers' operators (include/kda_paged.h);
// not part of the C ABI.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/kda_paged.h"

namespace kda {

// How a batch's new tokens and its cache lie (see include/kda_paged.h).
struct PagedBatch {
  const int32_t* block_table;
  int64_t table_stride;
  const int32_t *seq_lens, *cu_seqlens;
  int num_seqs;
  int64_t total_tokens;
  int num_pages, max_pages, page_size;
};

struct RopeArgs {
  const void *q, *k, *v;       // v, k_pages, v_pages: the append alone
  int64_t q_stride, k_stride, v_stride;
  void *q_out, *k_out;
  int64_t q_out_stride, k_out_stride;
  char *k_pages, *v_pages;
  int64_t k_page_stride, v_page_stride;
  const int32_t* positions;    // kda_rope; the append takes positions from the batch
  const double* inv_freq;
  int num_q_heads, num_k_heads, head_dim, rot_dim;
  float scale;
  bool interleaved, inverse, dtype_bf16;
  PagedBatch b;
  hipStream_t stream;
};
hipError_t launch_rope(const RopeArgs& a);
hipError_t launch_append(const RopeArgs& a);

struct AttnArgs {
  const void* q;
  int64_t q_stride;
  const char *k_pages, *v_pages;
  int64_t k_page_stride, v_page_stride;  // elements
  PagedBatch b;
  int num_q_heads, num_kv_heads, head_dim;
  bool dtype_bf16;
  float scale;
  int window;
  void* o;
  float* lse;
  char* workspace;
  hipStream_t stream;
  // set by launch_attn: sequences of more rows (new tokens x query heads per K/V head) than row_limit are
  // computed in tiles of tile_rows rows, with their plan at tile_ws
  int row_limit, tile_rows;
  char* tile_ws;
};
size_t attn_workspace_bytes(int num_seqs, int64_t total_tokens, int num_q_heads, int num_kv_heads,
                            int head_dim, bool bf16);
hipError_t launch_attn(const AttnArgs& a);

struct Pools {
  kda_page_pool p[KDA_MAX_POOLS];
  int n;
};
struct PagesArgs {
  Pools pools;
  int32_t *page_refs, *block_table, *seq_lens;
  int64_t table_stride;
  const int32_t *seqs, *parents;  // seqs: the children of a fork
  const int32_t* new_tokens;
  int count, num_seqs, num_pages, max_pages, page_size;
  int32_t* granted;
  char* workspace;
  hipStream_t stream;
};
size_t pages_plan_bytes(int count, int num_seqs, int num_pages);
hipError_t launch_pages_alloc(const PagesArgs& a);
hipError_t launch_pages_fork(const PagesArgs& a);
hipError_t launch_pages_free(const PagesArgs& a);

struct CompactArgs {
  Pools pools;
  const int32_t *page_refs, *block_table;
  int64_t table_stride, out_table_stride;
  int num_seqs, num_pages, max_pages;
  int32_t *out_refs, *out_table, *moved;
  char* workspace;
  hipStream_t stream;
};
size_t pages_compact_bytes(int num_pages);
hipError_t launch_pages_compact(const CompactArgs& a);
hipError_t launch_pages_copy(const Pools& pools, const int32_t* src, const int32_t* dst, int count,
                             hipStream_t stream);

}  // namespace kda
