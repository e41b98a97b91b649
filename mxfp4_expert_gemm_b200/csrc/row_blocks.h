// How a weight gradient copies an expert's token rows.
//
// Its contraction runs over the rows in blocks of 64, and no row of a neighbour (its values may be
// infinite) may enter the sum: a block of fewer rows is copied as 64 whose others read zeros, in both
// operands alike.  The tensor maps are views [rows - w + 1][w][values] whose two row axes share one
// stride (row d1 + d2): a window of w rows ends where one likes, and d1 past it reads zeros.  The views
// cover the buffer's rows and nothing behind it, and no copy starts at a negative coordinate.  (A view
// that covered the 63 rows behind the buffer as well, with the zero rows in front of a short block,
// d1 < 0, made the copy touch memory behind the buffer: a fault where nothing is mapped there.)
//   Map 0: w = min(64, rows), for ranges of rows that end at or behind row w.
//   Maps 1 and 2: w = 8 and w = 1.  A range that ends before row w is copied eight rows at a time, then
//   one at a time: an expert within the first 63 rows of the buffer, at most 14 blocks.
#pragma once

#include <cstdint>

namespace moe {

constexpr int kBlockRows = 64;

struct RowBlock {
  int32_t map, d1, d2;
};

constexpr int32_t window_rows(int map, int32_t rows) {
  const int32_t w = map == 0 ? kBlockRows : map == 1 ? 8 : 1;
  return w < rows ? w : rows;
}

// Blocks of the rows c0 .. c0 + clen - 1 (win: map 0's window).
constexpr int weight_blocks(int win, int c0, int clen) {
  return c0 + clen >= win ? (clen + kBlockRows - 1) / kBlockRows : clen / 8 + clen % 8;
}

// Block kb of them: the map, and the coordinates of its copy along the view's row axes.
constexpr RowBlock weight_block(int win, int c0, int clen, int kb) {
  if (c0 + clen >= win) {
    const int left = clen - kBlockRows * kb, n = left < kBlockRows ? left : kBlockRows;
    return RowBlock{0, win - n, c0 + kBlockRows * kb + n - win};
  }
  const int eights = clen / 8;   // (clen < win <= 64)
  return kb < eights ? RowBlock{1, 0, c0 + 8 * kb} : RowBlock{2, 0, c0 + 7 * eights + kb};
}

}  // namespace moe
