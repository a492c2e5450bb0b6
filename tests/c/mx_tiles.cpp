// Prints the tile that the MXFP4 projection takes (csrc/nhm_internal.h) for each "m n f32" of the command line: its features,
// its rows, and the workgroups of it that a CU holds.
#include <stdio.h>
#include <stdlib.h>

#include "../../fp8_w8a8_linear_amd/csrc/nhm_internal.h"

int main(int argc, char** argv) {
    for (int i = 1; i + 2 < argc; i += 3) {
        const nhm::MxTile t = nhm::mx_tile(atoll(argv[i]), atoll(argv[i + 1]), atoi(argv[i + 2]) != 0);
        printf("%d %d %d\n", t.tn, t.tm, t.per_cu);
    }
    return 0;
}
