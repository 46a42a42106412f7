// CPU check of the rows that the tree pass and merge over the 8-bit cache reads
// and writes (csrc/layout.h): over every row count of a unit, both tile sizes and
// the whole launch grid, each row that a lane reads queries of is one of the
// unit's, and every row of the unit belongs to exactly one CTA.
// Prints "OK" and exits 0, or prints the first failure and exits 1.
#include <cstdio>
#include <vector>

#include "layout.h"

using namespace treeattn;

int main() {
    for (int M = 1; M <= 64 * 16; ++M) {
        const int RB = (M + kRows - 1) / kRows;
        for (int rows : {4, 16}) {
            std::vector<int> owners(M, 0);
            for (int rb = 0; rb < RB; ++rb)
                for (int y = 0; y < merge_groups(M, rows); ++y)
                    for (int r = 0; r < 16; ++r) {  // rows of the score tile
                        const int r0 = y * rows;
                        const int at = merge_reads_row(rb, r0, r, rows, M);
                        if (at < 0 || at >= M) {
                            std::printf("M %d tile %d block %d: row %d + %d reads row %d\n", M,
                                        rows, rb, r0, r, at);
                            return 1;
                        }
                        if (!merge_has_row(rb, r0, r, rows, M)) continue;
                        if (at != rb * kRows + r0 + r) {
                            std::printf("M %d tile %d block %d: row %d + %d reads row %d\n", M,
                                        rows, rb, r0, r, at);
                            return 1;
                        }
                        ++owners[at];
                    }
            for (int i = 0; i < M; ++i)
                if (owners[i] != 1) {
                    std::printf("M %d tile %d: row %d has %d owners\n", M, rows, i, owners[i]);
                    return 1;
                }
        }
    }
    std::printf("OK\n");
    return 0;
}
