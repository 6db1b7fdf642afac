// attn_schedule.hpp -- the order in which the tree attention's loops over shared tiles send tiles
// to LDS, wait for them, meet at barriers and read them, apart from what is computed.  Plain C++: the
// kernel walks it with its own operations, tests/attn_schedule_model.cpp with ones that
// record what each read may rely on.
//
// K and V of tile t lie in slot (t - t0) % S.  K of t is read by the scores of t, which are formed
// while the values of t - 1 are added, V of t by the values of t.  Tiles are sent through page ids
// (fetched a tile earlier) and addresses (located from them): send_k takes the newest
// addresses, send_v those before.
//
// A piece that a thread has sent is in LDS once that thread has waited for it, and other
// waves may read it from the next barrier on.  A wait leaves the newest sends under way: wait_k()
// all of them but one tile's K, wait_sent(false) all but one tile's K and V, wait_sent(true) none.  Where
// some waves send less (a head that leaves columns of the tile unused) the kernel makes each
// of them a wait for everything.
#pragma once

namespace gdn {
namespace attn {

#define GDN_INLINE __attribute__((always_inline)) constexpr

GDN_INLINE int min_tile(int a, int b) { return a < b ? a : b; }

// K of the first S tiles and V of the first S - 1; on return page ids of tile t0 + S are on their way.
template <int S, class O>
GDN_INLINE void fill_slots(int t0, int last, O& o) {
    o.fetch(t0);
    o.locate(t0);
    o.send_k(0);
#pragma unroll
    for (int i = 1; i < S; ++i) {
        o.fetch(min_tile(t0 + i, last));
        o.locate(min_tile(t0 + i, last));
        o.send_v(i - 1);
        o.send_k(i);
    }
    o.fetch(min_tile(t0 + S, last));
    o.wait_sent(true);
    o.barrier();
    o.scores(0);
}

// Two groups of waves, the second half a tile behind the first, a barrier after each half.  With
// i = t - t0, and x barriers passed:
//
//   x = 2 i        leading: weights(t), first reads of V(t)
//   x = 2 i + 1    leading: send V(t + 2), K(t + 3); values(t), scores(t + 1)
//                  trailing: weights(t), first reads of V(t)
//   x = 2 i + 2    trailing: send V(t + 2), K(t + 3); values(t), scores(t + 1)
//
// What may be relied on:
//   - The leading group reads V(t) from x = 2 i on.  The trailing one has sent its share at 2 i - 2, so
//     that the wait at the end of its half 2 i - 1, weights(t - 1), must cover V(t): wait_k(), as only
//     K(t + 1) was sent later.
//   - The leading group reads K(t + 1) at 2 i + 1.  The trailing one has sent its share at 2 i - 2 and
//     its half 2 i ends with wait_sent(false), which leaves what that half itself has sent.
//   - V(t + 2) goes over V(t - 1), which the trailing group has read at 2 i, and K(t + 3) over K(t), which it
//     has read at 2 i, both before the leading group sends at 2 i + 1.
template <int S, class O>
GDN_INLINE void walk_in_turns(int t0, int full, bool leading, O& o) {
    static_assert(S == 3, "slots of tiles t - 1, t and t + 1");
    const int last = full - 1;
    fill_slots<S>(t0, last, o);
    int here = 0, next = 1, prev = S - 1;    // slots of t, t + 1 and t - 1
    o.locate(min_tile(t0 + S, last));
    o.fetch(min_tile(t0 + S + 1, last));
    if (!leading) o.turn();
    for (int t = t0; t < last; ++t) {
        o.early(here, next);
        o.weights();
        o.wait_k();
        o.turn();
        o.keep();
        o.fetch(min_tile(t + S + 2, last));
        if (t + S - 1 < full) o.send_v(prev);
        if (t + S < full) o.send_k(here);
        o.locate_kept(min_tile(t + S + 1, last));
        o.products(here, next);
        o.wait_sent(t + S >= full);
        o.turn();
        prev = here;
        here = next;
        next = next + 1 == S ? 0 : next + 1;
    }
    if (leading) o.turn();
    o.finish(here);
}

// All waves together, one barrier per tile.  At the barrier of t, K(t + 1) and V(t) are needed, sent
// S - 1 tiles ago, and every wave is done with V(t - 1) and K(t), over which the next ones go.
template <int S, class O>
GDN_INLINE void walk_in_step(int t0, int full, O& o) {
    const int last = full - 1;
    fill_slots<S>(t0, last, o);
    int here = 0, next = 1, prev = S - 1;
    for (int t = t0; t < last; ++t) {
        // fewer pieces are under way near the end
        o.wait_sent(S == 2 || t + S > last || t == t0);
        o.barrier();
        o.locate(min_tile(t + S, last));
        o.fetch(min_tile(t + S + 1, last));
        if (t + S - 1 < full) o.send_v(prev);
        if (t + S < full) o.send_k(here);
        o.tile(here, next);
        prev = here;
        here = next;
        next = next + 1 == S ? 0 : next + 1;
    }
    o.wait_sent(true);
    o.barrier();
    o.finish(here);
}

}  // namespace attn
}  // namespace gdn
