/* seq_index.h -- where the rows of a sequence are: the one place that reads boundaries, lengths
 * and page tables, for every sequence kernel. Compiles as plain C++ too, so that its answers to
 * broken tables can be checked without a GPU.
 *
 * Boundaries, lengths and tables live in device memory, so no host check sees them. Whatever they
 * hold, the rows that come out lie inside the tensors: a span that is wrong is cut (or empty) and
 * says so, and the kernels then set the status word. */
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define WK_SEQ_FN __host__ __device__ __forceinline__
#else
#define WK_SEQ_FN static inline
#endif

namespace wk {

struct SeqSpan {
  int64_t begin; /* first row of the sequence */
  int32_t len;   /* rows of it that take part, 0 .. most */
  int32_t room;  /* rows up to the next sequence (>= len; padding behind len) */
  int32_t bad;   /* the boundaries or the length were out of range */
};

/* Sequence b of boundaries off [batch + 1] over `total` rows: rows off[b] .. off[b + 1], of which
 * the first lens[b] take part (all of them when lens is NULL), and at most `most`. */
WK_SEQ_FN SeqSpan seq_span(const int32_t* off, const int32_t* lens, int64_t b, int64_t total, int32_t most) {
  SeqSpan s;
  const int64_t lo = off[b], hi = off[b + 1];
  s.bad = lo < 0 || hi < lo || hi > total;
  const int64_t l = lo < 0 ? 0 : (lo > total ? total : lo);
  const int64_t h = hi < l ? l : (hi > total ? total : hi);
  int64_t len = h - l;
  s.begin = l;
  s.room = static_cast<int32_t>(len);
  if (lens) {
    const int64_t want = lens[b];
    if (want < 0 || want > len) s.bad = 1;
    len = want < 0 ? 0 : (want > len ? len : want);
  }
  if (len > most) {
    s.bad = 1;
    len = most;
  }
  s.len = static_cast<int32_t>(len);
  return s;
}

/* Length of cached sequence b: lens[b], cut to what its row of the table can hold and to `most`. */
WK_SEQ_FN SeqSpan seq_cached(const int32_t* lens, int64_t b, int64_t capacity, int32_t most) {
  SeqSpan s;
  const int64_t want = lens[b];
  const int64_t cap = capacity < most ? capacity : most;
  const int64_t len = want < 0 ? 0 : (want > cap ? cap : want);
  s.begin = 0;
  s.bad = want != len;
  s.len = static_cast<int32_t>(len);
  s.room = s.len;
  return s;
}

/* Page of table row `row` that holds position pos, or -1 if the entry names no page. */
WK_SEQ_FN int32_t seq_page(const int32_t* row, int64_t pos, int32_t page_shift, int32_t num_pages) {
  const int32_t p = row[pos >> page_shift];
  return (p < 0 || p >= num_pages) ? -1 : p;
}

/* Keys that query row i of `new_rows` new tokens sees in a sequence of `len`: all of them, or with
 * `causal` those up to its own position len - new_rows + i (none when that is negative). */
WK_SEQ_FN int32_t seq_seen(int32_t len, int32_t new_rows, int32_t i, int32_t causal) {
  if (!causal) return len;
  const int64_t s = static_cast<int64_t>(len) - new_rows + i + 1;
  return s < 0 ? 0 : (s > len ? len : static_cast<int32_t>(s));
}

}  // namespace wk
