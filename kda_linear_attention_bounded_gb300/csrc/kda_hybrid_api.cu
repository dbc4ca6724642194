// C ABI of the calls beside the KDA layers (declared in include/kda.h): the gated delta rule, attention over a paged
// cache, and the step tables.  Host-side validation and launch planning only, by the rules of kda_api.cu: every check
// that can be made on the host is made before anything is launched, nothing allocates device memory or synchronises.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <iterator>

#include "kda_checks.h"
#include "kda_common.cuh"
#include "kda_hybrid.h"

namespace {

using kda::aligned16;
using kda::aligned_to;
using kda::check_workspace;
using kda::good_stride;

// The tensors of a gated-delta-rule call over `tokens` tokens; fills the token part of `a`.  Without tokens (empty
// sequences, whose final states are their initial ones) the token tensors may be NULL.
int check_gdn(int64_t tokens, const uint16_t *q, const uint16_t *k, int64_t qk_stride, const uint16_t *v, int64_t v_stride,
              const uint16_t *a_in, int64_t a_stride, const uint16_t *beta, int64_t beta_stride, const float *A_log,
              const float *dt_bias, float scale, int Hk, int Hv, uint16_t *out, int64_t out_stride,
              kda::GdnRecurrentArgs *a) {
  if (Hk <= 0 || Hv <= 0 || Hv > 4096 || Hv % Hk != 0) return KDA_ERR_INVALID_ARG;
  if (!A_log || !dt_bias) return KDA_ERR_INVALID_ARG;
  if (tokens > 0 && (!q || !k || !v || !a_in || !beta || !out)) return KDA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out)) return KDA_ERR_INVALID_ARG;
  if (!aligned_to(a_in, 2) || !aligned_to(beta, 2) || !aligned_to(A_log, 4) || !aligned_to(dt_bias, 4))
    return KDA_ERR_INVALID_ARG;
  const int64_t krow = static_cast<int64_t>(Hk) * kda::kD, vrow = static_cast<int64_t>(Hv) * kda::kD;
  if (!good_stride(qk_stride, krow) || !good_stride(v_stride, vrow) || !good_stride(out_stride, vrow))
    return KDA_ERR_INVALID_ARG;
  if (a_stride < Hv || beta_stride < Hv) return KDA_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return KDA_ERR_UNSUPPORTED;
  a->q = q; a->k = k; a->v = v; a->a = a_in; a->beta = beta;
  a->qk_stride = qk_stride; a->v_stride = v_stride; a->a_stride = a_stride;
  a->beta_stride = beta_stride; a->out_stride = out_stride;
  a->A_log = A_log; a->dt_bias = dt_bias;
  a->scale = scale;
  a->Hv = Hv; a->group = Hv / Hk;
  a->out = out;
  return KDA_OK;
}

// A piece of memory (bytes; of none, nothing meets it), or rows of it a stride apart (what lies between them is others').
struct Span {
  const void *at;
  int64_t bytes, rows = 1, stride = 0;
  bool meets(const Span &o) const {   // (o is in one piece)
    if (bytes <= 0 || rows <= 0 || o.bytes <= 0) return false;
    const int64_t from = static_cast<int64_t>(reinterpret_cast<uintptr_t>(o.at) - reinterpret_cast<uintptr_t>(at));
    const int64_t first = rows > 1 && from > 0 ? std::min(from / stride, rows - 1) : 0;   // the last row at or before it
    const auto row = [&](int64_t r) { return r < rows && r * stride < from + o.bytes && from < r * stride + bytes; };
    return row(first) || row(first + 1);
  }
};

// Batches whose sequences have so many tokens at most take the recurrence token by token.  Measured, chunks against
// tokens: 1 sequence x 2 heads of 8 tokens 11.1 and 6.7 us, of 12 11.1 and 9.0; 64 x 16 heads of 8 66 and 52 us, of 12 68 and 75.
// So a full GPU crosses between 8 and 12 and a single sequence later; 10 is right for both, at 11 and 12 a small batch loses 2 us.
constexpr int kRecurrentTokens = 10;

}  // namespace

extern "C" {

size_t kda_gdn_prefill_workspace_size(int64_t total_tokens, int num_seqs, int Hv) {
  if (total_tokens < 0 || num_seqs < 0 || Hv <= 0) return 0;
  return kda::kWorkspaceBytes + kda::gdn_prefill_workspace_bytes(total_tokens, num_seqs, Hv);
}

int kda_gdn_chunk_prefill(const uint16_t *q, const uint16_t *k, int64_t qk_token_stride, const uint16_t *v,
                          int64_t v_token_stride, const uint16_t *a, int64_t a_token_stride,
                          const uint16_t *beta_logits, int64_t beta_token_stride, const float *A_log,
                          const float *dt_bias, float scale, const int32_t *cu_seqlens_dev,
                          const int32_t *cu_seqlens_host, int num_seqs, int Hk, int Hv, float *state_pool,
                          int num_slots, const int32_t *slot_ids, int flags, uint16_t *out, int64_t out_token_stride,
                          float *final_state, void *workspace, size_t workspace_bytes, void *stream) {
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (num_seqs < 0 || !cu_seqlens_dev || !cu_seqlens_host || !aligned_to(cu_seqlens_dev, 4)) return KDA_ERR_INVALID_ARG;
  if (flags & ~(KDA_LOAD_INITIAL | KDA_FINAL_TO_POOL)) return KDA_ERR_INVALID_ARG;
  if (cu_seqlens_host[0] != 0) return KDA_ERR_INVALID_ARG;
  for (int n = 0; n < num_seqs; ++n)
    if (cu_seqlens_host[n + 1] < cu_seqlens_host[n]) return KDA_ERR_INVALID_ARG;
  if (num_seqs == 0) return KDA_OK;
  kda::GdnRecurrentArgs r{};
  if (int rc = check_gdn(cu_seqlens_host[num_seqs], q, k, qk_token_stride, v, v_token_stride, a, a_token_stride, beta_logits,
                         beta_token_stride, A_log, dt_bias, scale, Hk, Hv, out, out_token_stride, &r))
    return rc;
  const bool use_pool = flags & (KDA_LOAD_INITIAL | KDA_FINAL_TO_POOL);
  if (use_pool && (!state_pool || !slot_ids || num_slots <= 0 || !aligned16(state_pool) || !aligned_to(slot_ids, 4)))
    return KDA_ERR_INVALID_ARG;
  if (!(flags & KDA_FINAL_TO_POOL) && (!final_state || !aligned16(final_state))) return KDA_ERR_INVALID_ARG;
  if (workspace_bytes < kda_gdn_prefill_workspace_size(cu_seqlens_host[num_seqs], num_seqs, Hv)) return KDA_ERR_WORKSPACE;
  r.cu_seqlens = cu_seqlens_dev;
  r.slot_ids = use_pool ? slot_ids : nullptr;
  r.num_slots = num_slots;
  r.state_in = (flags & KDA_LOAD_INITIAL) ? state_pool : nullptr;
  r.state_out_pool = (flags & KDA_FINAL_TO_POOL) ? state_pool : nullptr;
  r.state_out_dense = (flags & KDA_FINAL_TO_POOL) ? nullptr : final_state;
  r.status = static_cast<uint32_t *>(workspace);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int longest = 0;
  for (int n = 0; n < num_seqs; ++n) longest = std::max(longest, cu_seqlens_host[n + 1] - cu_seqlens_host[n]);
  const cudaError_t e = longest <= kRecurrentTokens
                            ? kda::launch_gdn_recurrent(r, num_seqs, st)
                            : kda::launch_gdn_prefill(r, cu_seqlens_host, num_seqs,
                                                      static_cast<uint8_t *>(workspace) + kda::kWorkspaceBytes, st);
  return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_gdn_recurrent_verify(const uint16_t *q, const uint16_t *k, int64_t qk_token_stride, const uint16_t *v,
                             int64_t v_token_stride, const uint16_t *a, int64_t a_token_stride,
                             const uint16_t *beta_logits, int64_t beta_token_stride, const float *A_log,
                             const float *dt_bias, float scale, int B, int T, int Hk, int Hv,
                             const float *state_pool, int num_slots, const int32_t *slot_ids, uint16_t *out,
                             int64_t out_token_stride, float *intermediate_states, void *workspace,
                             size_t workspace_bytes, void *stream) {
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (B < 0 || T < 1 || T > 64) return KDA_ERR_INVALID_ARG;
  if (B == 0) return KDA_OK;
  kda::GdnRecurrentArgs r{};
  if (int rc = check_gdn(B, q, k, qk_token_stride, v, v_token_stride, a, a_token_stride, beta_logits,
                         beta_token_stride, A_log, dt_bias, scale, Hk, Hv, out, out_token_stride, &r))
    return rc;
  if (!state_pool || !aligned16(state_pool) || num_slots <= 0 || !slot_ids || !aligned_to(slot_ids, 4)) return KDA_ERR_INVALID_ARG;
  if (!intermediate_states || !aligned16(intermediate_states)) return KDA_ERR_INVALID_ARG;
  r.T = T;
  r.slot_ids = slot_ids;
  r.num_slots = num_slots;
  r.skip_padding = 1;
  r.state_in = state_pool;
  r.inter = intermediate_states;
  r.status = static_cast<uint32_t *>(workspace);
  return kda::launch_gdn_recurrent(r, B, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_gdn_decode(const uint16_t *q, const uint16_t *k, int64_t qk_token_stride, const uint16_t *v,
                   int64_t v_token_stride, const uint16_t *a, int64_t a_token_stride, const uint16_t *beta_logits,
                   int64_t beta_token_stride, const float *A_log, const float *dt_bias, float scale, int B, int Hk,
                   int Hv, float *state_pool, int num_slots, const int32_t *slot_ids, uint16_t *out,
                   int64_t out_token_stride, void *workspace, size_t workspace_bytes, void *stream) {
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (B < 0) return KDA_ERR_INVALID_ARG;
  if (B == 0) return KDA_OK;
  kda::GdnRecurrentArgs r{};
  if (int rc = check_gdn(B, q, k, qk_token_stride, v, v_token_stride, a, a_token_stride, beta_logits,
                         beta_token_stride, A_log, dt_bias, scale, Hk, Hv, out, out_token_stride, &r))
    return rc;
  if (!state_pool || !aligned16(state_pool) || num_slots <= 0 || !slot_ids || !aligned_to(slot_ids, 4)) return KDA_ERR_INVALID_ARG;
  r.T = 1;
  r.slot_ids = slot_ids;
  r.num_slots = num_slots;
  r.skip_padding = 1;
  r.state_in = state_pool;
  r.state_out_pool = state_pool;
  r.status = static_cast<uint32_t *>(workspace);
  return kda::launch_gdn_recurrent(r, B, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_paged_workspace_size(int Hq, int Hk, int T) {
  if (Hk <= 0 || Hq <= 0 || Hq % Hk != 0 || T < 1) return 0;
  const int64_t rows = static_cast<int64_t>(Hq / Hk) * T;
  const size_t per = kda::paged_rows_per_item(static_cast<int>(rows < 64 ? rows : 64));
  const size_t joins = kda::kPagedMaxCtas * sizeof(int4);
  return (kda::kWorkspaceBytes + joins + 2 * kda::kPagedMaxCtas * per * kda::kPagedPartFloats * sizeof(float) + 255) &
         ~size_t(255);
}

int kda_paged_attention(const uint16_t *q, int64_t q_token_stride, const uint16_t *k_pages, int64_t k_page_stride,
                        int64_t k_token_stride, int64_t k_head_stride, const uint16_t *v_pages, int64_t v_page_stride,
                        int64_t v_token_stride, int64_t v_head_stride, int num_pages, int page_size,
                        const int32_t *block_table, int64_t table_row_stride, int table_width,
                        const int32_t *seq_lens, int B, int T, int Hq, int Hk, float scale, uint16_t *out,
                        int64_t out_token_stride, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (B < 0 || T < 1 || T > 64) return KDA_ERR_INVALID_ARG;
  if (Hk <= 0 || Hq <= 0 || Hq > 4096 || Hq % Hk != 0) return KDA_ERR_INVALID_ARG;
  if (page_size < 1 || num_pages < 0 || table_width < 0 || table_row_stride < table_width) return KDA_ERR_INVALID_ARG;
  if (!std::isfinite(scale)) return KDA_ERR_UNSUPPORTED;
  if (B == 0) return KDA_OK;
  if (static_cast<int64_t>(B) * T > INT_MAX) return KDA_ERR_INVALID_ARG;
  if (!q || !seq_lens || !out || !aligned16(q) || !aligned16(out) || !aligned_to(seq_lens, 4) || !aligned_to(lse, 4))
    return KDA_ERR_INVALID_ARG;
  if (table_width > 0 && (!block_table || !aligned_to(block_table, 4))) return KDA_ERR_INVALID_ARG;
  if (num_pages > 0 && (!k_pages || !v_pages || !aligned16(k_pages) || !aligned16(v_pages))) return KDA_ERR_INVALID_ARG;
  const int64_t row = static_cast<int64_t>(Hq) * kda::kD;
  if (!good_stride(q_token_stride, row) || !good_stride(out_token_stride, row)) return KDA_ERR_INVALID_ARG;
  for (int64_t s : {k_page_stride, k_token_stride, k_head_stride, v_page_stride, v_token_stride, v_head_stride})
    if (!good_stride(s, 0)) return KDA_ERR_INVALID_ARG;
  if (workspace_bytes < kda_paged_workspace_size(Hq, Hk, T)) return KDA_ERR_WORKSPACE;
  kda::PagedArgs a{};
  a.q = q; a.k = k_pages; a.v = v_pages;
  a.q_stride = q_token_stride;
  a.k_page_stride = k_page_stride; a.k_token_stride = k_token_stride; a.k_head_stride = k_head_stride;
  a.v_page_stride = v_page_stride; a.v_token_stride = v_token_stride; a.v_head_stride = v_head_stride;
  a.num_pages = num_pages;
  a.page = page_size;
  a.table = block_table;
  a.table_stride = table_row_stride;
  const int64_t most = static_cast<int64_t>(table_width) * page_size;
  a.max_len = static_cast<int>(most < INT_MAX - 64 ? most : INT_MAX - 64);
  a.seq_lens = seq_lens;
  a.B = B; a.T = T; a.Hk = Hk; a.G = Hq / Hk;
  a.scale = scale;
  a.out = out;
  a.out_stride = out_token_stride;
  a.lse = lse;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  a.joins = reinterpret_cast<int4 *>(ws + kda::kWorkspaceBytes);
  a.parts = reinterpret_cast<float *>(ws + kda::kWorkspaceBytes + kda::kPagedMaxCtas * sizeof(int4));
  a.status = static_cast<uint32_t *>(workspace);
  return kda::launch_paged_attention(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

int kda_step_tables(int32_t *block_table, int64_t table_row_stride, int table_width, const int32_t *seq_lens,
                    const int32_t *new_lens, int B, const int32_t *free_pages, int num_free, int page_size,
                    int64_t max_tokens, int32_t *cu_seqlens, int32_t *kv_lens, int32_t *positions, int64_t *slot_map,
                    int32_t *pages_used, void *workspace, size_t workspace_bytes, void *stream) {
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (B < 0 || num_free < 0 || page_size < 1 || max_tokens < 0 || max_tokens > INT_MAX || table_width < 0)
    return KDA_ERR_INVALID_ARG;
  if (B > 0 && (!seq_lens || !new_lens || !kv_lens || (table_width > 0 && !block_table) || table_row_stride < table_width))
    return KDA_ERR_INVALID_ARG;
  if (!cu_seqlens || !pages_used || (num_free > 0 && !free_pages)) return KDA_ERR_INVALID_ARG;
  if (max_tokens > 0 && (!positions || !slot_map)) return KDA_ERR_INVALID_ARG;
  for (const void *p : {static_cast<const void *>(block_table), static_cast<const void *>(seq_lens),
                        static_cast<const void *>(new_lens), static_cast<const void *>(free_pages),
                        static_cast<const void *>(cu_seqlens), static_cast<const void *>(kv_lens),
                        static_cast<const void *>(positions), static_cast<const void *>(pages_used)})
    if (!aligned_to(p, 4)) return KDA_ERR_INVALID_ARG;
  if (!aligned_to(slot_map, 8)) return KDA_ERR_INVALID_ARG;
  // What is written lies apart from all else: every CTA reads the inputs for itself, at its own time.  The lengths may be
  // brought forward in place (kv_lens is seq_lens): one CTA then takes the call.
  const bool in_place = B > 0 && kv_lens == seq_lens;
  const auto ints = [](const int32_t *at, int64_t n) { return Span{at, n * 4}; };
  const Span inputs[] = {in_place ? Span{nullptr, 0} : ints(seq_lens, B), ints(new_lens, B), ints(free_pages, num_free)};
  const Span written[] = {Span{block_table, int64_t(4) * table_width, B, 4 * table_row_stride},
                          ints(cu_seqlens, static_cast<int64_t>(B) + 1), ints(kv_lens, B), ints(positions, max_tokens),
                          Span{slot_map, max_tokens * 8}, ints(pages_used, 1)};
  for (size_t i = 0; i < std::size(written); ++i) {
    for (const Span &x : inputs)
      if (written[i].meets(x)) return KDA_ERR_INVALID_ARG;
    for (size_t j = i + 1; j < std::size(written); ++j)
      if (written[i].meets(written[j])) return KDA_ERR_INVALID_ARG;
  }
  kda::StepTablesArgs t{};
  t.one_cta = in_place;
  t.table = block_table;
  t.table_stride = table_row_stride;
  t.width = table_width;
  t.seq_lens = seq_lens;
  t.new_lens = new_lens;
  t.free_pages = free_pages;
  t.num_free = num_free;
  t.page = page_size;
  t.B = B;
  t.max_tokens = max_tokens;
  t.cu_seqlens = cu_seqlens;
  t.kv_lens = kv_lens;
  t.positions = positions;
  t.pages_used = pages_used;
  t.slot_map = slot_map;
  t.status = static_cast<uint32_t *>(workspace);
  return kda::launch_step_tables(t, static_cast<cudaStream_t>(stream)) == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

}  // extern "C"
