// notice_ring.h: the barriers around a warp that looks through some of the value tiles in shared
// memory (fa_decode_fp8.cuh, dec8_hide_nan): the loads tell it of every such tile, and it tells the
// warps that use the tiles. No CUDA types, so the protocol can be checked on any machine.
#pragma once

namespace fa {

// Key and value tiles alternate in a ring of `units` slots, loaded in order, a slot again only when
// its tile was used. So many value tiles can be there at once, none of them used yet.
constexpr int ring_values(int units) { return (units + 1) / 2; }

// The warp that looks through the tiles runs ahead of the one that uses them by what the ring holds.
// An mbarrier waited on by parity tells one completed phase from none, not from two: with a single
// barrier, a second notice before the first was waited for makes that wait go on for ever. Notice n
// completes phase n / notices of barrier n % notices: its next phase needs the notice of a tile
// `notices` further on, which is not loaded before the tile of notice n was used.
//
// For the same reason the looking warp may not wait for a slot's load alone: it skips the tiles it
// does not look through, so the slot may be an odd number of loads behind the tile it wants, and the
// wait lets it through at once, to another tile's bytes. The loads therefore give a notice of their
// own (same numbering) once they have begun such a tile; every earlier load into its slot is then over.
constexpr int kNotices = 3;
constexpr int notice_bar(int n, int notices = kNotices) { return n % notices; }
constexpr unsigned notice_parity(int n, int notices = kNotices) { return static_cast<unsigned>(n / notices) & 1u; }

}  // namespace fa
