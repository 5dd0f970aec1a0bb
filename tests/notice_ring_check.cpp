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
    int units = 0, landed = 0;  // loads begun, and which of the ring's last ones are over (bit: slot)
    int over[6] = {};           // per slot: loads that are over
    int due = 0;                // notices the loads gave
    int seen = 0, notices = 0;  // tiles the looking warp is past, notices it gave
    bool told = false;          // it knows that its next tile's load has begun
    int used[2] = {0, 0}, waited[2] = {0, 0};  // per using warp: tiles used, notices waited for
    std::vector<int> key() const {
        return {units, landed, due, seen, notices, told, used[0], used[1], waited[0], waited[1]};
    }
};

// Completed phases of notice barrier `bar` after `given` notices.
int phases(int given, int bar, int rings) {
    int n = 0;
    for (int i = 0; i < given; ++i) n += fa::notice_bar(i, rings) == bar;
    return n;
}

enum Result { kSound, kStops, kUsedEarly, kLookedEarly };
const char* const kNames[] = {"sound", "some order of steps stops for good", "a tile is used before it was looked through",
                              "a tile is looked through before it is there"};

// Units 0, 1, 2, ... are K of tile 0, V of tile 0, K of tile 1, ...; loads land in any order. Keys
// are used as they land (which lets the loads run as far ahead as they ever can). `looked`: the
// tiles (bits) that are looked through; `told`: the loads give notice of them.
Result explore(int units, int users, unsigned looked, int rings, bool told = true) {
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
            const int before = s.units - units, slot = s.units % units;  // the unit whose slot this load takes
            if (before < 0 || ((s.landed >> slot & 1) && (before % 2 == 0 || before / 2 < freed))) {
                State n = s;
                n.landed &= ~(1 << slot);
                if (s.units % 2 == 1 && (looked >> s.units / 2 & 1u)) ++n.due;
                ++n.units;
                go(n);
            }
        }
        for (int u = s.units > units ? s.units - units : 0; u < s.units; ++u)
            if (!(s.landed >> u % units & 1)) {
                State n = s;
                n.landed |= 1 << u % units;
                ++n.over[u % units];
                go(n);
            }
        // Whether tile's values are there, and what a wait for their slot by parity says.
        auto there = [&](int tile) { return s.over[(2 * tile + 1) % units] > (2 * tile + 1) / units; };
        auto full = [&](int tile) {
            return passes(s.over[(2 * tile + 1) % units], static_cast<unsigned>((2 * tile + 1) / units) & 1u);
        };
        if (s.seen < kTiles) {
            State n = s;
            if (!(looked >> s.seen & 1u)) {
                ++n.seen;
                go(n);
            } else if (told && !s.told) {
                n.told = true;
                if (passes(phases(s.due, fa::notice_bar(s.notices, rings), rings), fa::notice_parity(s.notices, rings))) go(n);
            } else if (full(s.seen)) {
                if (!there(s.seen)) return kLookedEarly;
                ++n.seen;
                ++n.notices;
                n.told = false;
                go(n);
            }
        }
        bool end = s.units == 2 * kTiles && s.seen == kTiles;
        for (int i = 0; i < users; ++i) {
            const int tile = s.used[i];
            if (tile == kTiles) continue;
            end = false;
            if (!there(tile)) continue;
            State n = s;
            ++n.used[i];
            if (looked >> tile & 1u) {
                const int w = s.waited[i], bar = fa::notice_bar(w, rings);
                if (!passes(phases(s.notices, bar, rings), fa::notice_parity(w, rings))) continue;
                if (s.seen <= tile) return kUsedEarly;
                ++n.waited[i];
            }
            go(n);
        }
        if (!moved && !end) return kStops;
    }
    return kSound;
}

}  // namespace

int main() {
    int failures = 0;
    for (int units : {5, 6})  // the rings of the two forms
        for (int users : {1, 2})
            for (unsigned looked = 0; looked < 1u << kTiles; ++looked) {
                const Result r = explore(units, users, looked, fa::kNotices);
                if (r != kSound && ++failures < 10)
                    std::printf("FAILED units %d users %d tiles %02x: %s\n", units, users, looked, kNames[r]);
            }
    // The model tells the difference: one or two barriers are not enough for three tiles.
    for (int units : {5, 6})
        for (int rings : {1, 2})
            if (explore(units, 1, (1u << kTiles) - 1, rings) == kSound && ++failures)
                std::printf("FAILED: %d barriers pass with %d units\n", rings, units);
    if (explore(5, 1, 0x06, 1) != kStops && ++failures) std::printf("FAILED: two tiles in a row pass one barrier\n");
    // Without the loads' notices a segment's last tile is taken for an earlier one of its slot.
    for (int units : {5, 6})
        if (explore(units, 1, 0x80, fa::kNotices, false) != kLookedEarly && ++failures)
            std::printf("FAILED: %d units pass without the loads' notices\n", units);
    if (fa::ring_values(5) != 3 || fa::ring_values(6) != 3) {
        ++failures;
        std::printf("FAILED: ring_values\n");
    }
    if (failures) return 1;
    std::printf("ok\n");
    return 0;
}
