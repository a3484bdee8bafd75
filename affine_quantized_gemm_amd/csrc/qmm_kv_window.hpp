// Which steps of a sequence attention with a window takes, in which order
// (plain C++: the host's tests include it as it is).
#pragma once

#include <stdint.h>

// (constexpr functions are for the device as well)
#define QMM_WINDOW_FN __attribute__((always_inline)) constexpr

namespace qmm {
namespace kv {

// With a window a sequence's steps are taken in another order, and those that
// no row sees not at all: first the steps that all rows see whole (among the
// sinks, then from where the last row's window surely begins to the new
// tokens), then the others (the sinks' last, the window's begin, the new
// ones).  So there is one loop for each form of a step, as without a window;
// a branch in one loop, a third loop or a loop around two had up to 370
// registers spilled.  Positions are counted in this order; each of the five
// pieces lies `by` further on in the sequence.
//
// `by` is chosen by position, which the compiler makes a choice of addresses:
// the struct lies in 48 bytes of scratch memory a lane, and each step's loads
// follow a read of it that waits for the loads before, so that one step is on
// its way and not two (one token over 4100 tokens 15.4 us, without a window
// 13.2; 16 sequences of 5 rows over 1030 23.8 and 20.3; 64 rows of 4 sequences
// over 4200 43 and 38).
struct Window {
    int len;         // tokens of all pieces
    int all;         // of those that all rows see
    int end[4], by[5];
    QMM_WINDOW_FN int real(int t) const {
        return t + (t < end[0] ? by[0] : t < end[1] ? by[1] : t < end[2] ? by[2] : t < end[3] ? by[3] : by[4]);
    }
};
// n new tokens from position pos0 on, in a table of `cap`.  masked: a row may
// see none of the new tokens (without a mask its own at least, so that the
// first row's window begins one token later).
QMM_WINDOW_FN Window window_of(int pos0, int n, int64_t cap, int window, int sinks, bool masked) {
    auto down = [](int t) { return t & ~31; };
    auto up = [](int t) { return (t + 31) & ~31; };
    auto least = [](int x, int y) { return x < y ? x : y; };
    auto most = [](int x, int y) { return x > y ? x : y; };
    const int len = most(0, static_cast<int>(pos0 + n < cap ? pos0 + n : cap));
    const int before = most(0, least(pos0, len));
    const int sinks_whole = down(least(sinks, before)), sinks_end = least(up(least(sinks, len)), len);
    const int low = down(most(0, pos0 + (masked ? 0 : 1) - window));  // no row sees what is before it, and no sink
    const int whole = most(up(most(0, pos0 + n - window)), sinks_whole);  // (a row sees at most n new ones)
    const int fresh = most(down(before), 0);
    // pieces: begin and tokens
    const bool some = whole < fresh;
    const int n1 = some ? fresh - whole : 0;
    const int n2 = some ? most(0, least(sinks_end, whole) - sinks_whole) : sinks_end - sinks_whole;
    const int b3 = most(low, sinks_end), n3 = most(0, (some ? whole : len) - b3);
    const int n4 = some ? len - fresh : 0;
    Window w{};
    w.all = sinks_whole + n1;
    w.end[0] = sinks_whole;
    w.end[1] = w.all;
    w.end[2] = w.all + n2;
    w.end[3] = w.end[2] + n3;
    w.len = w.end[3] + n4;
    w.by[0] = 0;
    w.by[1] = whole - w.end[0];
    w.by[2] = sinks_whole - w.end[1];
    w.by[3] = b3 - w.end[2];
    w.by[4] = fresh - w.end[3];
    return w;
}

}  // namespace kv
}  // namespace qmm
