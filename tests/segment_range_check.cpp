// Host-only check of fa::segment_range (csrc/segment_range.h), compiled and run by
// tests/test_segment_range.py. Prints "ok" and exits 0 when every check holds.
#include <climits>
#include <cstdio>
#include <initializer_list>

#include "segment_range.h"

int main() {
    const int any[] = {INT_MIN, -7, -1, 0, 1, 5, 36, 37, 295, 296, 1 << 20, INT_MAX};
    int failures = 0;
    for (int teams : {1, 2, 37, 148, 296})
        for (int first : any)
            for (int last : any)
                for (int keys : {INT_MIN, -1, 0, 1, 8192, INT_MAX}) {
                    const fa::SegmentRange r = fa::segment_range(first, last, keys, teams);
                    bool ok = true;
                    for (long long c = r.first; c <= r.last && ok; ++c) ok = c >= 0 && c < teams;  // slots of teams only
                    ok = ok && r.first >= 0 && r.first <= teams && r.last >= -1 && r.last < teams;
                    if (keys <= 0) ok = ok && r.last < r.first;
                    // what the split notes is taken as it is
                    if (keys > 0 && 0 <= first && first <= last && last < teams) ok = ok && r.first == first && r.last == last;
                    if (!ok && ++failures < 10) std::printf("FAILED %d..%d keys %d teams %d\n", first, last, keys, teams);
                }
    if (failures) return 1;
    std::printf("ok\n");
    return 0;
}
