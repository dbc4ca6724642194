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
};
// Rows (query heads x new tokens of a key head) that one CTA takes, for `rows` of them.
int paged_rows_per_item(int rows);
cudaError_t launch_paged_attention(const PagedArgs &args, cudaStream_t stream);

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
