// Whether rows of a cache's pages, one tensor's or two, meet: arithmetic on strides, on the host.
#pragma once

#include <stdint.h>

#include <algorithm>
#include <utility>

namespace kda {

constexpr int64_t kRow = 128;   // channels of a row

// Whether rows of 128 channels meet whose places differ by sums of stride * x, one x in lo .. hi for each term: some sum comes
// nearer than a row to `apart` (elements).  The largest strides first, a term's x are only those that the terms behind it can make up
// for: one to three where strides nest, so the search is short; one that is not (no layout of a cache) counts as meeting.
struct Steps {
  int64_t stride, lo, hi;
};
struct RowSearch {
  Steps term[6];
  int64_t least[7], most[7];   // sums of the terms from one on
  int terms = 0, left = 1 << 16;
  bool others;                 // not counting the sum of zeros alone (rows of one tensor)
  void add(int64_t stride, int64_t lo, int64_t hi, bool join) {
    for (int i = 0; join && i < terms; ++i)
      if (term[i].stride == stride) {
        term[i].lo += lo;
        term[i].hi += hi;
        return;
      }
    term[terms++] = {stride, lo, hi};
  }
  void sort() {   // (at most six)
    for (int i = 1; i < terms; ++i)
      for (int j = i; j > 0 && term[j - 1].stride < term[j].stride; --j) std::swap(term[j - 1], term[j]);
  }
  // Whether every stride passes all that the smaller ones reach: rows of one tensor are apart then, and mostly so.
  bool nest() {
    sort();
    int64_t reach = kRow;
    for (int i = terms - 1; i >= 0; --i) {
      if (term[i].stride < reach) return false;
      reach += term[i].stride * term[i].hi;
    }
    return true;
  }
  bool meet(int64_t apart) {
    sort();
    least[terms] = most[terms] = 0;
    for (int i = terms - 1; i >= 0; --i) {
      least[i] = least[i + 1] + term[i].stride * term[i].lo;
      most[i] = most[i + 1] + term[i].stride * term[i].hi;
    }
    return look(0, apart, true);
  }
  bool look(int i, int64_t apart, bool zeros) {
    if (--left < 0) return true;
    if (i == terms) return apart > -kRow && apart < kRow && !(others && zeros);
    const Steps &t = term[i];
    const auto floor_div = [](int64_t a, int64_t b) { return a / b - (a % b < 0); };
    const int64_t lo = std::max(t.lo, -floor_div(most[i + 1] + kRow - 1 - apart, t.stride)),
                  hi = std::min(t.hi, floor_div(apart + kRow - 1 - least[i + 1], t.stride));
    for (int64_t x = lo; x <= hi; ++x)
      if (look(i + 1, apart - t.stride * x, zeros && x == 0)) return true;
    return false;
  }
};

// A tensor [pages, page_size, Hk, 128] of 16-bit channels, strides in channels.
struct Pages {
  const uint16_t *at;
  int64_t page, token, head;
};

// Whether no two rows of a tensor meet (strides of dimensions larger than one: at least a row, no product with their sizes beyond
// 2^46).
inline bool rows_apart(const Pages &p, int num_pages, int page_size, int Hk) {
  if (num_pages < 1) return true;
  RowSearch own;
  own.others = true;
  const int64_t strides[3] = {p.page, p.token, p.head}, n[3] = {num_pages, page_size, Hk};
  for (int d = 0; d < 3; ++d)
    if (n[d] > 1) own.add(strides[d], 1 - n[d], n[d] - 1, false);
  return own.nest() || !own.meet(0);
}

// Whether a row of one tensor meets one of the other (of both, the rows are apart).
inline bool pages_meet(const Pages &a, const Pages &b, int num_pages, int page_size, int Hk) {
  if (num_pages < 1) return false;
  RowSearch both;
  both.others = false;
  const int64_t strides[2][3] = {{a.page, a.token, a.head}, {b.page, b.token, b.head}}, n[3] = {num_pages, page_size, Hk};
  for (int d = 0; d < 3; ++d)
    if (n[d] > 1) {
      both.add(strides[0][d], 0, n[d] - 1, true);
      both.add(strides[1][d], 1 - n[d], 0, true);
    }
  return both.meet((reinterpret_cast<intptr_t>(b.at) - reinterpret_cast<intptr_t>(a.at)) / 2);
}

}  // namespace kda
