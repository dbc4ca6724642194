// C ABI of the calls around the paged cache (declared in include/kda.h): rotary positions with the store into the pages,
// forking and ending requests, compacting and copying pages, attention over shared prefixes.  Host-side validation and launch
// planning only, by the rules of kda_api.cu.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>
#include <iterator>
#include <memory>
#include <new>

#include "kda_cache.h"
#include "kda_checks.h"
#include "kda_common.cuh"
#include "kda_layout.h"

namespace {

using kda::aligned16;
using kda::aligned_to;
using kda::check_workspace;
using kda::good_stride;
using kda::Pages;
using kda::Span;

Span ints(const int32_t *at, int64_t n) { return {at, 4 * n}; }
Span table_span(const int32_t *table, int64_t stride, int width, int B) { return {table, int64_t(4) * width, B, 4 * stride}; }

// From the first byte to behind the last.
struct Range {
  uintptr_t from, to;
  bool meets(const Range &o) const { return from < o.to && o.from < to; }
};
Range range_of(const Span &s) {
  const auto at = reinterpret_cast<uintptr_t>(s.at);
  return {at, s.bytes <= 0 || s.rows <= 0 ? at : at + static_cast<uintptr_t>((s.rows - 1) * s.stride + s.bytes)};
}
// Whether rows of two tensors meet: rows of one stride may lie side by side, others may not even be interleaved.
bool rows_meet(const Span &a, const Span &b) {
  if (!range_of(a).meets(range_of(b))) return false;
  if (a.rows == 1 || b.rows == 1 || a.stride != b.stride) return true;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(b.at) - reinterpret_cast<uintptr_t>(a.at)) % a.stride;
  const int64_t off = d < 0 ? d + a.stride : d;   // b's rows behind a's
  return off < a.bytes || off + b.bytes > a.stride;
}

// The part of a table that the page calls check alike.
int check_table(const int32_t *table, int64_t stride, int width, const int32_t *lens, int B, int page) {
  if (B < 0 || width < 0 || page < 1 || stride < width) return KDA_ERR_INVALID_ARG;
  if (B > 0 && (!lens || (width > 0 && !table))) return KDA_ERR_INVALID_ARG;
  if (!aligned_to(table, 4) || !aligned_to(lens, 4)) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}
kda::TableArgs table_args(const int32_t *table, int64_t stride, int width, int B, int page, void *workspace) {
  return {table, stride, width, B, page, static_cast<uint32_t *>(workspace)};
}
int status_of(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// Pages that are written: strides that keep rows of 128 channels apart, and what they reach.
bool good_pages(const Pages &p, int num_pages, int page_size, int Hk, Range *reach) {
  if (!aligned16(p.at) || (num_pages > 0 && !p.at)) return false;
  int64_t bytes = 256;
  const auto dim = [&](int64_t stride, int64_t n) {
    if (!good_stride(stride, 0) || (n > 1 && stride < kda::kD)) return false;
    int64_t far = 0;
    if (n > 1 && (__builtin_mul_overflow(stride, n - 1, &far) || far > int64_t(1) << 46)) return false;   // (behind all memory)
    bytes += 2 * far;
    return true;
  };
  if (!dim(p.page, num_pages) || !dim(p.token, page_size) || !dim(p.head, Hk)) return false;
  const auto at = reinterpret_cast<uintptr_t>(p.at);
  *reach = {at, num_pages > 0 ? at + static_cast<uintptr_t>(bytes) : at};
  return kda::rows_apart(p, num_pages, page_size, Hk);
}

// Whether two buffers of as many pages each meet, page by page.
bool buffers_meet(const Span &a, const Span &b) {
  if (a.bytes <= 0 || b.bytes <= 0 || !range_of(a).meets(range_of(b))) return false;
  if (a.rows == 1 || a.stride == b.stride) return rows_meet(a, b);
  for (int64_t r = 0; r < b.rows; ++r)
    if (a.meets({static_cast<const uint8_t *>(b.at) + r * b.stride, b.bytes})) return true;
  return false;
}
Span pages_span(const kda_page_buffer &b, int num_pages) { return {b.base, b.bytes, num_pages, b.page_stride}; }
// Whether any two do.  Buffers behind one another, in any order, are told apart by their ends; those that reach into each other with
// one stride (layers of one tensor) by the places of their first pages within it; others pair by pair.
bool any_buffers_meet(const kda_page_buffer *buffers, int n, int num_pages) {
  struct Entry {
    int64_t at;
    int buffer;
    bool operator<(const Entry &o) const { return at < o.at; }
  };
  const auto range = [&](int i) { return range_of(pages_span(buffers[i], num_pages)); };
  uintptr_t end = 0;
  int i = 0;
  for (; i < n; ++i) {   // mostly they come in order
    const Range r = range(i);
    if (r.from == r.to) continue;
    if (r.from < end) break;
    end = r.to;
  }
  if (i == n) return false;
  constexpr int kFew = 256;
  Entry few[kFew];
  const std::unique_ptr<Entry[]> many(n > kFew ? new (std::nothrow) Entry[n] : nullptr);
  Entry *const list = n > kFew ? many.get() : few;
  const auto pairs = [&](auto of, int count) {
    for (int x = 0; x < count; ++x)
      for (int y = 0; y < x; ++y)
        if (buffers_meet(pages_span(buffers[of(x)], num_pages), pages_span(buffers[of(y)], num_pages))) return true;
    return false;
  };
  if (!list) return pairs([](int x) { return x; }, n);
  int live = 0;
  for (i = 0; i < n; ++i)
    if (buffers[i].bytes > 0) list[live++] = {static_cast<int64_t>(reinterpret_cast<uintptr_t>(buffers[i].base)), i};
  std::sort(list, list + live);
  for (int from = 0, to; from < live; from = to) {
    Entry *const group = list + from;
    end = range(group[0].buffer).to;
    const int64_t stride = buffers[group[0].buffer].page_stride;
    bool same = num_pages > 1;
    for (to = from + 1; to < live && range(list[to].buffer).from < end; ++to) {
      end = std::max(end, range(list[to].buffer).to);
      same = same && buffers[list[to].buffer].page_stride == stride;
    }
    const int count = to - from;
    if (count == 1) continue;
    bool apart = same;
    if (same) {
      const int64_t first = group[0].at;
      for (i = 0; i < count; ++i) group[i].at = (group[i].at - first) % stride;
      std::sort(group, group + count);
      for (i = 0; i < count && apart; ++i)
        apart = group[i].at + buffers[group[i].buffer].bytes <= (i + 1 < count ? group[i + 1].at : group[0].at + stride);
    }
    if (!apart && pairs([&](int x) { return group[x].buffer; }, count)) return true;
  }
  return false;
}

}  // namespace

extern "C" {

int kda_rotary_to_pages(const uint16_t *q, int64_t q_token_stride, const uint16_t *k, int64_t k_token_stride, const uint16_t *v,
                        int64_t v_token_stride, int tokens, int Hq, int Hk, const int32_t *positions,
                        int64_t position_row_stride, int num_axes, const int64_t *slot_map, const float *inv_freq, int R,
                        const uint8_t *axes, int interleaved, float mscale, uint16_t *k_pages, int64_t k_page_stride,
                        int64_t k_page_token_stride, int64_t k_head_stride, uint16_t *v_pages, int64_t v_page_stride,
                        int64_t v_page_token_stride, int64_t v_head_stride, int num_pages, int page_size, uint16_t *out,
                        int64_t out_token_stride, void *workspace, size_t workspace_bytes, void *stream) {
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (tokens < 0 || Hq < 1 || Hk < 1 || Hq > 4096 || Hk > 4096 || num_pages < 0 || page_size < 1) return KDA_ERR_INVALID_ARG;
  if (num_axes < 1 || num_axes > kda::kMaxAxes) return KDA_ERR_INVALID_ARG;
  if (R < 16 || R > kda::kD || R % 16 != 0 || !std::isfinite(mscale)) return KDA_ERR_UNSUPPORTED;
  kda::RotaryArgs a{};
  for (int f = 0; axes && f < R / 2; ++f) {
    if (axes[f] >= num_axes) return KDA_ERR_INVALID_ARG;
    a.axes[f / 32] |= static_cast<uint64_t>(axes[f]) << (2 * (f % 32));
  }
  if (tokens == 0) return KDA_OK;
  if (!q || !k || !v || !out || !positions || !slot_map || !inv_freq) return KDA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned_to(positions, 4) ||
      !aligned_to(slot_map, 8) || !aligned_to(inv_freq, 4))
    return KDA_ERR_INVALID_ARG;
  const int64_t qrow = static_cast<int64_t>(Hq) * kda::kD, krow = static_cast<int64_t>(Hk) * kda::kD;
  if (!good_stride(q_token_stride, qrow) || !good_stride(k_token_stride, krow) || !good_stride(v_token_stride, krow) ||
      !good_stride(out_token_stride, qrow) || (num_axes > 1 && position_row_stride < tokens))
    return KDA_ERR_INVALID_ARG;
  const Pages kp = {k_pages, k_page_stride, k_page_token_stride, k_head_stride},
              vp = {v_pages, v_page_stride, v_page_token_stride, v_head_stride};
  Range reach[2];
  if (!good_pages(kp, num_pages, page_size, Hk, &reach[0]) || !good_pages(vp, num_pages, page_size, Hk, &reach[1]))
    return KDA_ERR_INVALID_ARG;
  // (keys and values may lie in one buffer, but not in the same places)
  if (reach[0].meets(reach[1]) && kda::pages_meet(kp, vp, num_pages, page_size, Hk)) return KDA_ERR_INVALID_ARG;
  // what is written: out (q itself, or apart from all that is read) and the pages
  const Span qs = {q, 2 * qrow, tokens, 2 * q_token_stride}, os = {out, 2 * qrow, tokens, 2 * out_token_stride},
             inputs[] = {{k, 2 * krow, tokens, 2 * k_token_stride}, {v, 2 * krow, tokens, 2 * v_token_stride},
                         {positions, 4 * ((num_axes - 1) * position_row_stride + tokens)}, {slot_map, int64_t(8) * tokens},
                         {inv_freq, 2 * R}};
  const bool in_place = out == q && (tokens == 1 || out_token_stride == q_token_stride);
  if (!in_place && rows_meet(os, qs)) return KDA_ERR_INVALID_ARG;
  for (const Span &x : inputs)
    if (rows_meet(os, x)) return KDA_ERR_INVALID_ARG;
  for (const Range &r : reach) {
    if (r.meets(range_of(qs)) || r.meets(range_of(os))) return KDA_ERR_INVALID_ARG;
    for (const Span &x : inputs)
      if (r.meets(range_of(x))) return KDA_ERR_INVALID_ARG;
  }
  a.q = q; a.k = k; a.v = v;
  a.q_stride = q_token_stride; a.k_stride = k_token_stride; a.v_stride = v_token_stride; a.out_stride = out_token_stride;
  a.tokens = tokens; a.Hq = Hq; a.Hk = Hk;
  a.positions = positions;
  a.position_stride = position_row_stride;
  a.slots = slot_map;
  a.inv_freq = inv_freq;
  a.R = R;
  a.interleaved = interleaved != 0;
  a.mscale = mscale;
  a.k_pages = k_pages; a.v_pages = v_pages; a.out = out;
  a.k_page_stride = k_page_stride; a.k_token_stride = k_page_token_stride; a.k_head_stride = k_head_stride;
  a.v_page_stride = v_page_stride; a.v_token_stride = v_page_token_stride; a.v_head_stride = v_head_stride;
  a.num_pages = num_pages;
  a.page = page_size;
  a.status = static_cast<uint32_t *>(workspace);
  return status_of(kda::launch_rotary_to_pages(a, static_cast<cudaStream_t>(stream)));
}

int kda_fork_requests(int32_t *block_table, int64_t table_row_stride, int table_width, int32_t *seq_lens, int B,
                      const int32_t *parents, const int32_t *children, int forks, const int32_t *free_pages, int num_free,
                      int page_size, int32_t *copy_src, int32_t *copy_dst, int32_t *pages_used, void *workspace,
                      size_t workspace_bytes, void *stream) {
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (int rc = check_table(block_table, table_row_stride, table_width, seq_lens, B, page_size)) return rc;
  if (forks < 0 || forks > kda::kMostEntries || num_free < 0 || !pages_used || (num_free > 0 && !free_pages)) return KDA_ERR_INVALID_ARG;
  if (forks > 0 && (!parents || !children || !copy_src || !copy_dst)) return KDA_ERR_INVALID_ARG;
  for (const int32_t *p : {parents, children, free_pages, static_cast<const int32_t *>(copy_src),
                           static_cast<const int32_t *>(copy_dst), static_cast<const int32_t *>(pages_used)})
    if (!aligned_to(p, 4)) return KDA_ERR_INVALID_ARG;
  const Span inputs[] = {ints(parents, forks), ints(children, forks), ints(free_pages, num_free)};
  const Span written[] = {table_span(block_table, table_row_stride, table_width, B), ints(seq_lens, B), ints(copy_src, forks),
                          ints(copy_dst, forks), ints(pages_used, 1)};
  for (size_t i = 0; i < std::size(written); ++i) {
    for (const Span &x : inputs)
      if (written[i].meets(x)) return KDA_ERR_INVALID_ARG;
    for (size_t j = i + 1; j < std::size(written); ++j)
      if (written[i].meets(written[j])) return KDA_ERR_INVALID_ARG;
  }
  kda::ForkArgs a{};
  a.t = table_args(block_table, table_row_stride, table_width, B, page_size, workspace);
  a.table = block_table;
  a.seq_lens = seq_lens;
  a.parents = parents; a.children = children; a.free_pages = free_pages;
  a.forks = forks;
  a.num_free = num_free;
  a.copy_src = copy_src; a.copy_dst = copy_dst; a.pages_used = pages_used;
  return status_of(kda::launch_fork_requests(a, static_cast<cudaStream_t>(stream)));
}

int kda_release_requests(const int32_t *block_table, int64_t table_row_stride, int table_width, int32_t *seq_lens, int B,
                         const int32_t *rows, int num_rows, int page_size, int32_t *free_pages, int num_pages,
                         int32_t *num_free, void *workspace, size_t workspace_bytes, void *stream) {
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (int rc = check_table(block_table, table_row_stride, table_width, seq_lens, B, page_size)) return rc;
  if (num_rows < 0 || num_rows > kda::kMostEntries || num_pages < 0 || !num_free || (num_rows > 0 && !rows) || (num_pages > 0 && !free_pages))
    return KDA_ERR_INVALID_ARG;
  if (!aligned_to(rows, 4) || !aligned_to(free_pages, 4) || !aligned_to(num_free, 4)) return KDA_ERR_INVALID_ARG;
  const Span inputs[] = {table_span(block_table, table_row_stride, table_width, B), ints(rows, num_rows)};
  const Span written[] = {ints(seq_lens, B), ints(free_pages, num_pages), ints(num_free, 1)};
  for (size_t i = 0; i < std::size(written); ++i) {
    for (const Span &x : inputs)
      if (x.meets(written[i])) return KDA_ERR_INVALID_ARG;
    for (size_t j = i + 1; j < std::size(written); ++j)
      if (written[i].meets(written[j])) return KDA_ERR_INVALID_ARG;
  }
  kda::ReleaseArgs a{};
  a.t = table_args(block_table, table_row_stride, table_width, B, page_size, workspace);
  a.seq_lens = seq_lens;
  a.rows = rows;
  a.num_rows = num_rows;
  a.free_pages = free_pages;
  a.num_free = num_free;
  a.num_pages = num_pages;
  return status_of(kda::launch_release_requests(a, static_cast<cudaStream_t>(stream)));
}

int kda_compact_pages(const int32_t *block_table, int64_t table_row_stride, int table_width, const int32_t *seq_lens, int B,
                      int page_size, int num_pages, int32_t *new_table, int64_t new_row_stride, int32_t *copy_src,
                      int32_t *copy_dst, int room, int32_t *free_pages, int32_t *num_free, void *workspace,
                      size_t workspace_bytes, void *stream) {
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (int rc = check_table(block_table, table_row_stride, table_width, seq_lens, B, page_size)) return rc;
  if (int rc = check_table(new_table, new_row_stride, table_width, seq_lens, B, page_size)) return rc;
  if (num_pages < 0 || room < num_pages / 2 || !num_free || (num_pages > 0 && !free_pages)) return KDA_ERR_INVALID_ARG;
  if (room > 0 && (!copy_src || !copy_dst)) return KDA_ERR_INVALID_ARG;
  if (!aligned_to(copy_src, 4) || !aligned_to(copy_dst, 4) || !aligned_to(free_pages, 4) || !aligned_to(num_free, 4))
    return KDA_ERR_INVALID_ARG;
  const bool in_place = new_table == block_table && (B <= 1 || new_row_stride == table_row_stride);
  const Span from = table_span(block_table, table_row_stride, table_width, B), to = table_span(new_table, new_row_stride, table_width, B);
  if (!in_place && B > 0 && table_width > 0 && rows_meet(from, to)) return KDA_ERR_INVALID_ARG;
  const Span apart[] = {ints(seq_lens, B), ints(copy_src, room), ints(copy_dst, room), ints(free_pages, num_pages), ints(num_free, 1)};
  for (size_t i = 0; i < std::size(apart); ++i) {
    if (from.meets(apart[i]) || to.meets(apart[i])) return KDA_ERR_INVALID_ARG;
    for (size_t j = i + 1; j < std::size(apart); ++j)
      if (apart[i].meets(apart[j])) return KDA_ERR_INVALID_ARG;
  }
  kda::CompactArgs a{};
  a.t = table_args(block_table, table_row_stride, table_width, B, page_size, workspace);
  a.seq_lens = seq_lens;
  a.num_pages = num_pages;
  a.room = room;
  a.new_table = new_table;
  a.new_stride = new_row_stride;
  a.copy_src = copy_src; a.copy_dst = copy_dst; a.free_pages = free_pages; a.num_free = num_free;
  return status_of(kda::launch_compact_pages(a, static_cast<cudaStream_t>(stream)));
}

int kda_copy_pages(const kda_page_buffer *buffers, int num_buffers, int num_pages, const int32_t *copy_src,
                   const int32_t *copy_dst, int count, void *workspace, size_t workspace_bytes, void *stream) {
  if (int rc = check_workspace(workspace, workspace_bytes)) return rc;
  if (num_buffers < 0 || num_pages < 0 || count < 0 || count > kda::kMostEntries || (num_buffers > 0 && !buffers)) return KDA_ERR_INVALID_ARG;
  if (count > 0 && (!copy_src || !copy_dst || !aligned_to(copy_src, 4) || !aligned_to(copy_dst, 4))) return KDA_ERR_INVALID_ARG;
  for (int i = 0; i < num_buffers; ++i) {
    const kda_page_buffer &b = buffers[i];
    if (b.bytes < 0 || b.bytes > INT_MAX || b.bytes % 16 || b.page_stride % 16 || !aligned16(b.base)) return KDA_ERR_INVALID_ARG;
    if (num_pages > 0 && b.bytes > 0 && (!b.base || (num_pages > 1 && b.page_stride < b.bytes))) return KDA_ERR_INVALID_ARG;
    // the lists are read by every CTA at its own time
    const Span pages = pages_span(b, num_pages);
    if (num_pages > 0 && (pages.meets(ints(copy_src, count)) || pages.meets(ints(copy_dst, count)))) return KDA_ERR_INVALID_ARG;
  }
  if (any_buffers_meet(buffers, num_buffers, num_pages)) return KDA_ERR_INVALID_ARG;
  if (count == 0 || num_pages == 0) return KDA_OK;
  return status_of(kda::launch_copy_pages(buffers, num_buffers, num_pages, copy_src, copy_dst, count,
                                          static_cast<uint32_t *>(workspace), static_cast<cudaStream_t>(stream)));
}

size_t kda_shared_prefix_workspace_size(int B, int T, int Hq, int Hk, int num_groups) {
  const size_t base = kda_paged_workspace_size(Hq, Hk, T);
  if (B < 0 || num_groups < 0 || base == 0) return 0;
  return base + kda::shared_prefix_bytes(B, T, Hq, Hk, num_groups, nullptr, nullptr);
}

int kda_shared_prefix_attention(const uint16_t *q, int64_t q_token_stride, const uint16_t *k_pages, int64_t k_page_stride,
                                int64_t k_token_stride, int64_t k_head_stride, const uint16_t *v_pages, int64_t v_page_stride,
                                int64_t v_token_stride, int64_t v_head_stride, int num_pages, int page_size,
                                const int32_t *block_table, int64_t table_row_stride, int table_width,
                                const int32_t *seq_lens, int B, int T, const int32_t *prefix_lens,
                                const int32_t *group_starts, int num_groups, int Hq, int Hk, float scale, uint16_t *out,
                                int64_t out_token_stride, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
  kda::PrefixArgs p{};
  if (int rc = kda::check_paged(q, q_token_stride, k_pages, k_page_stride, k_token_stride, k_head_stride, v_pages, v_page_stride,
                                v_token_stride, v_head_stride, num_pages, page_size, block_table, table_row_stride, table_width,
                                seq_lens, B, T, Hq, Hk, scale, out, out_token_stride, lse, workspace, workspace_bytes, &p.a))
    return rc;
  if (num_groups < 0 || num_groups > kda::kMostEntries || !aligned_to(prefix_lens, 4) || !aligned_to(group_starts, 4)) return KDA_ERR_INVALID_ARG;
  if (num_groups > 0 && (!prefix_lens || !group_starts)) return KDA_ERR_INVALID_ARG;
  if (B == 0) return KDA_OK;
  if (workspace_bytes < kda_shared_prefix_workspace_size(B, T, Hq, Hk, num_groups)) return KDA_ERR_WORKSPACE;
  p.prefix_lens = prefix_lens;
  p.group_starts = group_starts;
  p.groups = num_groups;
  kda::shared_prefix_bytes(B, T, Hq, Hk, num_groups, static_cast<uint8_t *>(workspace) + kda_paged_workspace_size(Hq, Hk, T), &p);
  return status_of(kda::launch_shared_prefix(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
