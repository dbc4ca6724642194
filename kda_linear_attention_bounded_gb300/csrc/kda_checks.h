// Host-side argument checks shared by the entry points (kda_api.cu, kda_hybrid_api.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

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

inline int check_workspace(const void *ws, size_t bytes) {
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u) != 0 || bytes < kWorkspaceBytes) return KDA_ERR_WORKSPACE;
  return KDA_OK;
}

}  // namespace kda
