/* Reads "off[2] lens have most total" style questions from stdin and prints what csrc/seq_index.h
 * answers, one line each. Built and run by tests/test_seq_cpu.py. */
#include <cstdio>
#include <cstring>

#include "seq_index.h"

int main() {
  char what[16];
  long long a, b, c, d, e;
  while (std::scanf("%15s %lld %lld %lld %lld %lld", what, &a, &b, &c, &d, &e) == 6) {
    if (!std::strcmp(what, "span")) { /* lo hi len(or -99: none) total most */
      const int32_t off[2] = {static_cast<int32_t>(a), static_cast<int32_t>(b)};
      const int32_t len = static_cast<int32_t>(c);
      const wk::SeqSpan s = wk::seq_span(off, c == -99 ? nullptr : &len, 0, d, static_cast<int32_t>(e));
      std::printf("%lld %d %d %d\n", static_cast<long long>(s.begin), s.len, s.room, s.bad ? 1 : 0);
    } else if (!std::strcmp(what, "cached")) { /* len capacity most */
      const int32_t len = static_cast<int32_t>(a);
      const wk::SeqSpan s = wk::seq_cached(&len, 0, b, static_cast<int32_t>(c));
      std::printf("%lld %d %d %d\n", static_cast<long long>(s.begin), s.len, s.room, s.bad ? 1 : 0);
    } else if (!std::strcmp(what, "page")) { /* entry pos shift pages */
      int32_t row[64];
      for (int i = 0; i < 64; ++i) row[i] = 1000000;
      row[b >> c] = static_cast<int32_t>(a);
      std::printf("%d\n", wk::seq_page(row, b, static_cast<int32_t>(c), static_cast<int32_t>(d)));
    } else { /* seen: len new i causal */
      std::printf("%d\n", wk::seq_seen(static_cast<int32_t>(a), static_cast<int32_t>(b), static_cast<int32_t>(c),
                                       static_cast<int32_t>(d)));
    }
  }
  return 0;
}
