// Host-only check of csrc/notice_ring.h: every interleaving of the warps around a ring of key and
// value tiles (the loads, the warp that looks through some value tiles and gives notice, the warps
// that use them) reaches its end, and no tile that is looked through is used before. Compiled and
// run by tests/test_notice_ring.py. Prints "ok" and exits 0 when every check holds.
#include <cstdio>
#include <set>
#include <vector>

#include "notice_ring.h"

namespace {

constexpr int kTiles = 8;

// Whether an mbarrier with `phases` completed phases lets a wait for `parity` through.
bool passes(int phases, unsigned parity) { return (static_cast<unsigned>(phases) & 1u) != parity; }

struct State {
    int units = 0;               // units loaded: K of tile 0, V of tile 0, K of tile 1, ...
    int seen = 0, notices = 0;   // tiles the looking warp is past, notices it gave
    int used[2] = {0, 0}, waited[2] = {0, 0};  // per using warp: tiles used, notices waited for
    std::vector<int> key() const { return {units, seen, notices, used[0], used[1], waited[0], waited[1]}; }
};

// Completed phases of notice barrier `bar` after `given` notices.
int phases(int given, int bar, int rings) {
    int n = 0;
    for (int i = 0; i < given; ++i) n += fa::notice_bar(i, rings) == bar;
    return n;
}

// 0: sound; 1: some order of steps stops for good; 2: a tile is used before it was looked through.
// Keys are used at once (which lets the loads run as far ahead as they ever can).
int explore(int units, int users, unsigned looked, int rings) {
    std::set<std::vector<int>> done;
    std::vector<State> todo{State{}};
    while (!todo.empty()) {
        const State s = todo.back();
        todo.pop_back();
        if (!done.insert(s.key()).second) continue;
        bool moved = false;
        auto go = [&](const State& n) {
            moved = true;
            todo.push_back(n);
        };
        int freed = s.used[0];  // value tiles every user is past
        for (int i = 1; i < users; ++i) freed = s.used[i] < freed ? s.used[i] : freed;
        if (s.units < 2 * kTiles) {
            const int before = s.units - units;  // the unit whose slot this load takes
            if (before < 0 || before % 2 == 0 || before / 2 < freed) {
                State n = s;
                ++n.units;
                go(n);
            }
        }
        auto here = [&](int tile) { return s.units > 2 * tile + 1; };
        if (s.seen < kTiles) {
            if (!(looked >> s.seen & 1u)) {
                State n = s;
                ++n.seen;
                go(n);
            } else if (here(s.seen)) {
                State n = s;
                ++n.seen;
                ++n.notices;
                go(n);
            }
        }
        bool end = s.units == 2 * kTiles && s.seen == kTiles;
        for (int i = 0; i < users; ++i) {
            const int tile = s.used[i];
            if (tile == kTiles) continue;
            end = false;
            if (!here(tile)) continue;
            State n = s;
            ++n.used[i];
            if (looked >> tile & 1u) {
                const int w = s.waited[i], bar = fa::notice_bar(w, rings);
                if (!passes(phases(s.notices, bar, rings), fa::notice_parity(w, rings))) continue;
                if (s.seen <= tile) return 2;
                ++n.waited[i];
            }
            go(n);
        }
        if (!moved && !end) return 1;
    }
    return 0;
}

}  // namespace

int main() {
    int failures = 0;
    for (int units : {5, 6})  // the rings of the two forms
        for (int users : {1, 2})
            for (unsigned looked = 0; looked < 1u << kTiles; ++looked) {
                const int r = explore(units, users, looked, fa::kNotices);
                if (r != 0 && ++failures < 10)
                    std::printf("FAILED units %d users %d tiles %02x: %s\n", units, users, looked, r == 1 ? "stops" : "used too early");
            }
    // The model tells the difference: one or two barriers are not enough for three tiles.
    for (int units : {5, 6})
        for (int rings : {1, 2})
            if (explore(units, 1, (1u << kTiles) - 1, rings) == 0 && ++failures)
                std::printf("FAILED: %d barriers pass with %d units\n", rings, units);
    if (explore(5, 1, 0x06, 1) != 1 && ++failures) std::printf("FAILED: two tiles in a row pass one barrier\n");
    if (fa::ring_values(5) != 3 || fa::ring_values(6) != 3) {
        ++failures;
        std::printf("FAILED: ring_values\n");
    }
    if (failures) return 1;
    std::printf("ok\n");
    return 0;
}
