// Host functions of lm_common.hpp.  Grids (long_grid): within HIP's limits, and
// no workgroup missing, for up to 2^31 - 1 workgroups.  Partial outputs
// (part_outputs): past the maxima and sums, and aligned to 16-byte stores.
#include <stdio.h>
#include <stdlib.h>

#include "../../newton_schulz_09_amd/csrc/lm_common.hpp"

int main() {
    long checked = 0;
    for (const int threads : {64, 128, 192, 256, 512, 1024})
        for (int64_t at = 1; at < int64_t{1} << 31; at = at < 4096 ? at + 1 : at + at / 97)
            for (const int64_t blocks : {at, ((int64_t{1} << 32) - 1) / threads, ((int64_t{1} << 32) - 1) / threads + 1,
                                         (int64_t{1} << 31) - 1}) {
                if (blocks > (int64_t{1} << 31) - 1) continue;
                const dim3 g = muon::long_grid(blocks, threads, 4096);
                const uint64_t x = g.x, z = g.z;
                if (x * threads >= uint64_t{1} << 32 || z > 65535 || g.y != 4096 || x * z < static_cast<uint64_t>(blocks) ||
                    x * z > 0xffffffffull || (blocks * threads < int64_t{1} << 32) != (z == 1)) {
                    fprintf(stderr, "%lld workgroups of %d: %u x %u x %u\n", (long long)blocks, threads, g.x, g.y, g.z);
                    return 1;
                }
                ++checked;
            }
    for (int64_t n = 1; n < 100000; ++n)
        if (muon::part_outputs(n) < 2 * n || muon::part_outputs(n) > 2 * n + 3 || muon::part_outputs(n) % 4 != 0) {
            fprintf(stderr, "outputs of %lld pairs at %lld\n", (long long)n, (long long)muon::part_outputs(n));
            return 1;
        }
    printf("grids ok: %ld\n", checked);
    return 0;
}
