// Host-side argument checks shared by the entry points (kda_api.cu, kda_hybrid_api.cu, kda_cache_api.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "kda.h"
#include "kda_internal.h"

namespace kda {

// Bytes every workspace starts with: the status word and the counters that kda_workspace_reset clears.
constexpr size_t kWorkspaceBytes = 1024;
static_assert(kDoneCounterOffset + sizeof(uint32_t) <= kWorkspaceBytes,
              "the spec step's CTA counter must sit in the cleared header");
static_assert(kSplitCounterOffset >= kDoneCounterOffset + sizeof(uint32_t) &&
                  kSplitCounterOffset + kMaxSplitCounters * sizeof(uint32_t) <= kWorkspaceBytes,
              "the split schedule's counters lie in the part kda_workspace_reset clears");

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned_to(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool good_stride(int64_t stride, int64_t min_elems) { return stride >= min_elems && stride % 8 == 0; }

// Entries at most of a list that a kernel goes through in steps of up to 65536, with 32-bit places.
constexpr int kMostEntries = 0x7FFFFFFF - 65536;

inline int check_workspace(const void *ws, size_t bytes) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || bytes < kWorkspaceBytes) return KDA_ERR_WORKSPACE;
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

}  // namespace kda
