// The tree that a sequence's drafts form: plain functions, which the host's tests run as well.
#pragma once

#include <stdint.h>

namespace tkp {

// A draft's token and the row that it follows: row 0 follows the last token, row
// j + 1 draft j. Token -1: the draft counts as not there and follows no row, whatever
// its parent was.
struct DraftPlace {
  int32_t token, node;
};
constexpr DraftPlace draft_place(int j, int32_t token, int32_t parent, int V) {
  const bool there = token >= 0 && token < V && parent >= -1 && parent < j;
  return there ? DraftPlace{token, parent + 1} : DraftPlace{-1, -1};
}

// Whether row r lies at or behind row `node`, and so do all drafts on the way: token
// and above are the drafts' places. Every step goes to a smaller row, or there is none.
constexpr bool row_behind(int r, int node, const int32_t* token, const int32_t* above) {
  while (r > node) {
    const int up = above[r - 1];
    if (token[r - 1] < 0 || up < 0 || up >= r) return false;
    r = up;
  }
  return r == node;
}

}  // namespace tkp
