// Whether two strided tensors of a call share a byte (host).
#pragma once

#include <cstdint>

namespace oscar {

// n x heads pieces of `bytes` bytes each, `row` and `head` bytes apart.
struct Pieces {
  uintptr_t at;
  long long n, heads, row, head, bytes;
};

// The same bytes in fewer pieces.
inline Pieces joined(Pieces p) {
  if (p.heads == 1 || p.head == 0) p.heads = 1, p.head = 0;
  if (p.n == 1 || p.row == 0) p.n = 1, p.row = 0;
  if (p.heads > 1 && p.head == p.bytes) p.bytes *= p.heads, p.heads = 1, p.head = 0;
  if (p.heads == 1 && p.n > 1 && p.row == p.bytes) p.bytes *= p.n, p.n = 1, p.row = 0;
  return p;
}

// a's pieces do not overlap: its heads lie inside their row, or its rows inside their head.  For disjoint ranges
// and for slices of the same rows (a fused projection's) no more than a few steps for each of b's heads, else
// for each of its pieces.
inline bool share_bytes(Pieces a, Pieces b) {
  a = joined(a);
  b = joined(b);
  auto reach = [](const Pieces& p) { return (p.n - 1) * p.row + (p.heads - 1) * p.head + p.bytes; };
  if (a.at + uintptr_t(reach(a)) <= b.at || b.at + uintptr_t(reach(b)) <= a.at) return false;
  const long long d = (long long)(b.at - a.at);
  auto below = [](long long x, long long y) { return x / y - (x % y != 0 && x < 0); };  // floor(x / y), y > 0
  // the members i of [0, count), `size` bytes each every `stride`, that [x, x + b.bytes) meets: first .. last
  auto range = [&](long long x, long long size, long long stride, long long count, long long* first, long long* last) {
    *first = stride ? below(x - size, stride) + 1 : x >= size;  // (i stride + size > x)
    *last = stride ? below(x + b.bytes - 1, stride) : (x + b.bytes > 0) - 1;
    if (*first < 0) *first = 0;
    if (*last > count - 1) *last = count - 1;
  };
  long long i0, i1;
  if (a.n == 1 || b.n == 1 || a.row == b.row) {
    // Rows of one stride: row j of b begins d + (j - i) stride bytes behind row i of a.  The differences for
    // which the rows' ranges meet:
    const long long stride = a.n > 1 ? a.row : b.row;
    const long long span_a = (a.heads - 1) * a.head + a.bytes, span_b = (b.heads - 1) * b.head + b.bytes;
    long long k0 = stride ? below(-span_b - d, stride) + 1 : 0, k1 = stride ? below(span_a - 1 - d, stride) : 0;
    if (k0 < -(a.n - 1)) k0 = -(a.n - 1);
    if (k1 > b.n - 1) k1 = b.n - 1;
    if (k1 - k0 < 8) {  // (rows whose heads lie far apart meet more of the others: below)
      for (long long k = k0; k <= k1; ++k)
        for (long long h = 0; h < b.heads; ++h) {
          range(d + k * stride + h * b.head, a.bytes, a.head, a.heads, &i0, &i1);
          if (i0 <= i1) return true;
        }
      return false;
    }
  }
  // a as groups of pieces, the wider stride outside
  const bool rows_out = a.heads == 1 || a.row >= a.head * (a.heads - 1) + a.bytes;
  const long long outer = rows_out ? a.row : a.head, inner = rows_out ? a.head : a.row;
  const long long n_outer = rows_out ? a.n : a.heads, n_inner = rows_out ? a.heads : a.n;
  const long long group = (n_inner - 1) * inner + a.bytes;
  for (long long r = 0; r < b.n; ++r)
    for (long long h = 0; h < b.heads; ++h) {
      const long long x = d + r * b.row + h * b.head;
      long long o0, o1;
      range(x, group, outer, n_outer, &o0, &o1);
      for (long long o = o0; o <= o1; ++o) {
        range(x - o * outer, a.bytes, inner, n_inner, &i0, &i1);
        if (i0 <= i1) return true;
      }
    }
  return false;
}

}  // namespace oscar
