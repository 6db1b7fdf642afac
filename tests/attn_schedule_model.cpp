// Runs the tree attention's tile loops (tree_masked_gated_amd/csrc/attn_schedule.hpp) against a model of
// LDS that promises no more than the hardware does, and prints what a read could find that it must not.
//
// Each group of waves runs alone and writes down its sends, its waits and its reads with the number
// of barriers that it has passed.  Between two barriers the groups (and the waves of one group)
// are not ordered, so that
//   - a read in interval x needs the tile's pieces of every group, waited for by their sender in an
//     interval before x,
//   - a send in interval x may only go over a tile that every group has read in an interval before x,
//     and whose pieces have arrived.
// A wait for all but n sends takes the n newest to be under way; page ids take part in the count on
// the device, which only makes a wait longer.  With `uneven` (waves that send less) a wait that leaves
// any sends under way promises nothing.
//
//   model turns|step SLOTS UNEVEN DROP     DROP: none, wait_k, wait_sent
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <vector>

#include "attn_schedule.hpp"

namespace {

struct Send {
    int kind, tile, slot, x, order, arrived;     // arrived: interval of the wait that covers it, or -1
};
struct Read {
    int kind, tile, slot, x, order;
};

struct Group {
    int last = 0, x = 0, order = 0;
    bool uneven = false;
    const char* drop = "";
    std::vector<Send> sends;
    std::vector<Read> reads;
    std::vector<const char*> faults;
    int pid = -1, ids = -1, at = -1, old = -1;   // tiles that the page ids and addresses belong to
    int scores_of = -1, values_of = -1, early_of = -1;
    int first = 0;

    void fetch(int t) { pid = t; }
    void keep() { ids = pid; }
    void locate(int t) { place(t, pid); }
    void locate_kept(int t) { place(t, ids); }
    void place(int t, int from) {
        if (t != from) faults.push_back("addresses from another tile's page ids");
        if (t < first || t > last) faults.push_back("a tile outside the run");
        old = at;
        at = t;
    }
    void send_k(int slot) { sends.push_back({0, at, slot, x, order++, -1}); }
    void send_v(int slot) { sends.push_back({1, old, slot, x, order++, -1}); }
    void wait(size_t leave) {
        if (uneven && leave > 0) return;
        for (size_t i = 0; i + leave < sends.size(); ++i)
            if (sends[i].arrived < 0) sends[i].arrived = x;
    }
    void wait_k() {
        if (strcmp(drop, "wait_k") != 0) wait(uneven ? 0 : 1);
    }
    void wait_sent(bool all) {
        if (strcmp(drop, "wait_sent") != 0 || all) wait(all || uneven ? 0 : 2);
    }
    void barrier() { ++x; }
    void turn() { ++x; }
    void read(int kind, int tile, int slot) { reads.push_back({kind, tile, slot, x, order++}); }
    void scores(int slot) {
        scores_of = scores_of < 0 ? first : scores_of + 1;
        read(0, scores_of, slot);
    }
    void values(int slot) {
        values_of = values_of < 0 ? first : values_of + 1;
        if (values_of != scores_of) faults.push_back("values of a tile whose weights are not formed");
        read(1, values_of, slot);
    }
    void early(int here, int) { read(1, early_of = values_of < 0 ? first : values_of + 1, here); }
    void weights() {}
    void products(int here, int next) {
        values(here);
        scores(next);
    }
    void tile(int here, int next) {
        values(here);
        scores(next);
    }
    void finish(int here) {
        values(here);
        if (values_of != last) faults.push_back("not all tiles");
    }
};

int check(std::vector<Group>& groups, bool say, int t0, int full) {
    int bad = 0;
    auto fault = [&](const char* what, int tile, int kind) {
        if (say) printf("tiles [%d, %d): %c of tile %d: %s\n", t0, full, kind ? 'V' : 'K', tile, what);
        ++bad;
    };
    for (Group& g : groups) {
        for (const char* f : g.faults) fault(f, -1, 0);
        if (g.x != groups[0].x) fault("barriers of the groups differ", -1, 0);
        for (const Read& r : g.reads)
            for (Group& h : groups) {
                bool found = false;
                for (const Send& s : h.sends) {
                    if (s.kind != r.kind || s.slot != r.slot) continue;
                    if (s.tile == r.tile) {
                        found |= s.arrived >= 0 && s.arrived < r.x;
                    } else if (s.tile > r.tile && s.x <= r.x) {
                        fault("overwritten before it is read", r.tile, r.kind);
                    }
                }
                if (!found) fault("read before it has arrived", r.tile, r.kind);
            }
        // a thread's own pieces land in one place of the slot: not before the last one's have arrived.
        // (Beyond the last tile its addresses repeat: the same bytes again.)
        for (const Send& s : g.sends)
            for (const Send& u : g.sends)
                if (s.kind == u.kind && s.slot == u.slot && s.order < u.order && s.tile != u.tile &&
                    (s.arrived < 0 || s.arrived > u.x))
                    fault("sent over pieces under way", u.tile, u.kind);
    }
    return bad;
}

template <int S>
int run(bool turns, bool uneven, const char* drop, int t0, int full, bool say) {
    std::vector<Group> groups(turns ? 2 : 1);
    for (size_t i = 0; i < groups.size(); ++i) {
        Group& g = groups[i];
        g.first = t0;
        g.last = full - 1;
        g.uneven = uneven;
        g.drop = drop;
        if constexpr (S == 3) {
            if (turns) gdn::attn::walk_in_turns<S>(t0, full, i == 0, g);
        }
        if (!turns) gdn::attn::walk_in_step<S>(t0, full, g);
    }
    return check(groups, say, t0, full);
}

}  // namespace

int main(int argc, char** argv) {
    if (argc != 5) return 2;
    const bool turns = strcmp(argv[1], "turns") == 0;
    const int slots = atoi(argv[2]);
    int bad = 0, runs = 0;
    for (int t0 : {0, 1, 5})
        for (int n = 1; n <= 24; ++n, ++runs)
            bad += slots == 3 ? run<3>(turns, atoi(argv[3]) != 0, argv[4], t0, t0 + n, bad < 5)
                              : run<2>(turns, atoi(argv[3]) != 0, argv[4], t0, t0 + n, bad < 5);
    printf("%d runs, %d faults\n", runs, bad);
    return bad != 0;
}
