// rule_schedule.hpp -- which rows of a sequence the rule's scans request ahead, apart from what is
// done with them.  Plain C++: the kernels walk it, tests/rule_schedule_model.cpp writes down the rows.
//
// A lane keeps its rows as offsets from a chunk's first row, the same ones for chunk after chunk.
// Every chunk but a sequence's last has kC rows; in the last one, rows past its end are requested as its
// last row.  Requests are made for a chunk ahead and never skipped (the compiler counts them), so at
// the end of a walk the chunk at hand is requested once more.
//
// places(rows) sets the offsets for a chunk of that many rows, load(c) requests chunk c's rows at them.
#pragma once

namespace gdn {

constexpr int kC = 64;                       // rows of a chunk

#define GDN_WALK __attribute__((always_inline)) constexpr

GDN_WALK int chunks_of(int n) { return (n + kC - 1) / kC; }
GDN_WALK int last_rows(int n) { return n - (chunks_of(n) - 1) * kC; }
// What is requested for row `row` of a chunk of `rows` rows.
GDN_WALK int row_in(int row, int rows) { return row < rows ? row : rows - 1; }

// From the first chunk to the last, the offsets being those of a whole chunk at first.
template <class Places, class Load>
GDN_WALK void request_forward(int n, int c, Places places, Load load) {
    if (c == chunks_of(n) - 1 && last_rows(n) < kC) places(last_rows(n));
    load(c);
}
GDN_WALK int after(int n, int c) { return c + 1 < chunks_of(n) ? c + 1 : c; }

// From the last chunk to the first: before the loop, and what is requested while chunk c is worked on.
// The offsets are those of a whole chunk from the second request on, where that is another chunk's.
template <class Places, class Load>
GDN_WALK void request_back_first(int n, Places places, Load load) {
    places(last_rows(n));
    load(chunks_of(n) - 1);
    if (chunks_of(n) > 1) places(kC);
}
GDN_WALK int before(int c) { return c > 0 ? c - 1 : 0; }

}  // namespace gdn
