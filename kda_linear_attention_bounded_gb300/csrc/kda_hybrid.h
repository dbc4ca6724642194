// Internal launch interface of the calls beside the KDA layers (kda_hybrid_api.cu): arguments, launches, tensor maps.
#pragma once

#include "kda_internal.h"

namespace kda {

// Launches a kernel as a programmatic dependent of what precedes it on the stream: its launch overlaps the end of that.
// The kernel reads and writes nothing before its grid_dependency_wait, or only what the call's caller may not have
// pending in the grid directly before it.
template <typename... P, typename... A>
cudaError_t launch_dependent_clusters(void (*kernel)(P...), unsigned cluster, unsigned grid, unsigned threads, size_t smem,
                                      cudaStream_t stream, const A &...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned threads, size_t smem, cudaStream_t stream, const A &...args) {
  return launch_dependent_clusters(kernel, 1, grid, threads, smem, stream, args...);
}

// A bf16 tensor of `rank` dimensions (dims and box innermost first, strides in bytes from the second on), 128-byte swizzle.
bool make_bf16_map(CUtensorMap *map, const void *base, int rank, const uint64_t *dims, const uint64_t *strides,
                   const uint32_t *box);
// [tokens, H, 128] with the given token stride, boxes of 64 channels x 1 head x 64 tokens.
bool make_tokens_map(CUtensorMap *map, const void *base, int H, int total_tokens, int64_t token_stride);

// ---------------------------------------------------------------- gated delta rule
// Arguments of the token-by-token gated delta rule.
struct GdnRecurrentArgs {
  const uint16_t *q, *k, *v, *a, *beta;
  int64_t qk_stride, v_stride, a_stride, beta_stride, out_stride;
  const float *A_log, *dt_bias;   // [Hv]
  float scale;
  int Hv, group;             // value heads; value heads per key head
  const int32_t *cu_seqlens; // token ranges, or null: items of T tokens
  int T;
  const int32_t *slot_ids;   // non-null when a pool is read or written
  int num_slots;
  int skip_padding;          // KDA_PAD_SLOT_ID rows are skipped without a status bit
  const float *state_in;     // pool, or null = zero
  float *state_out_pool;     // pool, or null
  float *state_out_dense;    // [items, Hv, D, D], or null
  float *inter;              // [items, T, Hv, D, D], or null
  uint16_t *out;
  uint32_t *status;
};

cudaError_t launch_gdn_recurrent(const GdnRecurrentArgs &args, int num_items, cudaStream_t stream);

// Chunked prefill of the gated delta rule over the sequences of cu_host; blocks: gdn_prefill_workspace_bytes().
size_t gdn_prefill_workspace_bytes(int64_t total_tokens, int num_seqs, int Hv);
cudaError_t launch_gdn_prefill(const GdnRecurrentArgs &args, const int32_t *cu_host, int num_seqs, uint8_t *blocks,
                               cudaStream_t stream);

// ---------------------------------------------------------------- paged attention
constexpr int kPagedMaxCtas = 304;      // stretches of work at most (two CTAs on each of 152 SMs)
constexpr int kPagedPartFloats = 132;   // a part of a row: 128 sums, the maximum, the sum of weights, padding
// Where part n of a row lies whose item is cut into `parts` at the beginning of stretch `cut` (the parts of the workspace: two of every
// stretch): part 0 in the last of the stretch before the cut, part n in the first of the n-th stretch from the cut on.
constexpr int paged_part_slot(int cut, int n) { return n == 0 ? 2 * (cut - 1) + 1 : 2 * (cut + n - 1); }
// Whether a row's own words on its parts can be so.  Rows that a kernel left unwritten, after a wait that gave up, say anything.
constexpr bool paged_parts_there(int parts, int cut) {
  return parts >= 2 && cut >= 1 && parts <= kPagedMaxCtas && cut <= kPagedMaxCtas + 1 - parts;
}
struct PagedArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride;                                        // tokens of q (heads contiguous)
  int64_t k_page_stride, k_token_stride, k_head_stride;    // elements
  int64_t v_page_stride, v_token_stride, v_head_stride;
  int num_pages, page;
  const int32_t *table;
  int64_t table_stride;
  int max_len;                                             // tokens that a table row holds
  const int32_t *seq_lens;
  int B, T, Hk, G, row_blocks;                             // G: query heads per key head
  float scale;
  uint16_t *out;
  int64_t out_stride;
  float *lse;                                              // [B T, Hk G], or null
  float *parts;
  int4 *joins;                                             // one per CTA (stretches)
  int cluster;                                             // CTAs of an item's cluster (clusters)
  uint32_t *status;
  // own tokens alone (attention over shared prefixes; else null): request b's begin at own[b].x, and what its rows sum up to
  // is left for a join: rows [B T, Hk G, kPagedPartFloats], each its sums, maximum and sum of weights, or, of a cut item, behind
  // them how many parts there are and the first CTA behind the cut
  const int2 *own;
  float *rows;
  int *ticket;                                             // 0 at the beginning: stretches taken
};
// The cache's pages as [page, token, head, 128], boxes of 64 channels x `box` tokens; false: the strides or sizes are none that
// a tensor map takes.
bool make_page_map(CUtensorMap *map, const uint16_t *pages, int64_t page_stride, int64_t token_stride, int64_t head_stride,
                   const PagedArgs &a, int box);
// Rows (query heads x new tokens of a key head) that one CTA takes, for `rows` of them.
int paged_rows_per_item(int rows);
cudaError_t launch_paged_attention(const PagedArgs &args, cudaStream_t stream);
// The same over the requests' own tokens, without the join.
cudaError_t launch_paged_own(const PagedArgs &args, cudaStream_t stream);
// Checks what kda_paged_attention is given and fills its arguments (with B == 0 it leaves them without the tensors).
int check_paged(const uint16_t *q, int64_t q_token_stride, const uint16_t *k_pages, int64_t k_page_stride, int64_t k_token_stride,
                int64_t k_head_stride, const uint16_t *v_pages, int64_t v_page_stride, int64_t v_token_stride,
                int64_t v_head_stride, int num_pages, int page_size, const int32_t *block_table, int64_t table_row_stride,
                int table_width, const int32_t *seq_lens, int B, int T, int Hq, int Hk, float scale, uint16_t *out,
                int64_t out_token_stride, float *lse, void *workspace, size_t workspace_bytes, PagedArgs *args);

// ---------------------------------------------------------------- step tables
struct StepTablesArgs {
  int32_t *table;            // [B, width], row stride table_stride
  int64_t table_stride;
  int width;
  const int32_t *seq_lens, *new_lens;
  const int32_t *free_pages;
  int num_free, page, B;
  int64_t max_tokens;
  int32_t *cu_seqlens, *kv_lens, *positions, *pages_used;
  int64_t *slot_map;
  int one_cta;               // kv_lens is seq_lens: no second CTA may read it
  uint32_t *status;
};

cudaError_t launch_step_tables(const StepTablesArgs &args, cudaStream_t stream);

}  // namespace kda
