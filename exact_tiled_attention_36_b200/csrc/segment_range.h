// segment_range.h: which partial results of an item the merge of the E4M3 decode reads. No CUDA
// types, so the rule can be checked on any machine.
#pragma once

namespace fa {

struct SegmentRange {
    int first, last;  // teams (last < first: none)
};

// `first` and `last` as the split kernel noted them: the teams that hold the item's first and last
// tile. Nothing was noted for an item without keys, nor where the split gave up (a wait that ran out
// of its limit): what stands there may be anything, and must not lead past the workspace's slots.
// (Both stay near the teams' range, so that steps from them cannot overflow.)
constexpr int clamp_team(int x, int least, int most) { return x < least ? least : (x < most ? x : most); }
constexpr SegmentRange segment_range(int first, int last, int keys, int teams) {
    return keys <= 0 ? SegmentRange{0, -1}
                     : SegmentRange{clamp_team(first, 0, teams), clamp_team(last, -1, teams - 1)};
}

}  // namespace fa
