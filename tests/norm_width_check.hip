// Host-side check of the group norm's thread map (built with --cuda-host-only and run on the CPU by
// test_norm_widths.py): whether every variant that norm_variant() chooses has a place for every channel
// of a group, wherever the group begins in its row.  Prints one line per width that is not covered,
// then "widths checked N".
#include <stdio.h>

#include "gdr_norm.hpp"

using namespace gdr;

int main() {
    int checked = 0;
    for (const bool aligned : {false, true}) {
        for (int D = 1; D <= NORM_WIDTH_MAX; ++D) {
            const NormVariant v = norm_variant(D, aligned);
            // the group that begins furthest past a multiple of 8 channels, among eight of them
            int shift = 0;
            if (v.vec == 8)
                for (int g = 0; g < 8; ++g) shift = (g * D & 7) > shift ? (g * D & 7) : shift;
            const bool lanes = v.lanes == NORM_THREADS || (v.lanes <= 64 && (v.lanes & (v.lanes - 1)) == 0);
            const bool known = v.vec == 8 ? v.values == 8 || v.values == 16 || v.values == 32 : v.vec == 1 && (v.values == 8 || v.values == 32);
            const bool masked = shift == 0 || v.ragged;
            if (v.lanes * v.values < shift + D || !lanes || !known || !masked)
                printf("%d %s: %d lanes of %d values, %d channels from %d on\n", D, aligned ? "aligned" : "any", v.lanes, v.values, D, shift);
            ++checked;
        }
    }
    printf("widths checked %d\n", checked);
    return 0;
}
