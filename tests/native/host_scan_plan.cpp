// The cut of recurrence calls whose rows are far apart (no GPU): as many channel
// blocks as the channels take, no more, and none missing.
#include <cstdio>
#include <cstdlib>

#include "fields.hpp"

using namespace nerf;

static int g_checks = 0;
static void check(const ScanPlan& p, int d, int gates, const char* what) {
    const int V = p.vec ? 4 : 1, m = d / gates;
    // channels (or, grouped, gates) that one block holds, and how many there are
    const int64_t each = p.grouped ? (p.parts > 1 ? 1 : p.cl / p.lg) : (int64_t)p.cl * V, all = p.grouped ? gates : d;
    const int64_t blocks = p.blocks / p.parts;
    const bool fits = p.blocks % p.parts == 0 && blocks * each >= all && (blocks - 1) * each < all &&
                      (!p.grouped || (int64_t)p.lg * p.parts * V >= m);
    ++g_checks;
    if (!fits) {
        std::fprintf(stderr, "FAILED %s: d %d gates %d cl %d lg %d parts %d blocks %d\n", what, d, gates, p.cl, p.lg,
                     p.parts, p.blocks);
        std::exit(1);
    }
}

int main() {
    const int widths[] = {1, 2, 3, 4, 5, 16, 24, 33, 63, 64, 70, 96, 130, 256, 257, 600, 1024, 1030, 4096, 65536};
    const int64_t shapes[][2] = {{0, 1}, {1, 1}, {40, 8}, {9000, 1}, {40000, 2}, {300000, 3}, {131072, 65536}, {32768, 16}};
    for (int d : widths)
        for (int gates : {1, 2, 3, 8, 16, d})
            for (const auto& s : shapes)
                for (int elt : {2, 4})
                    for (bool backward : {false, true}) {
                        if (gates > d || d % gates) continue;
                        ScanPlan p = scan_plan(elt, s[0], s[1], d, gates, backward);
                        check(p, d, gates, "rows together");
                        const size_t parts = scan_workspace(p, s[0], gates, backward);
                        scan_plan_strides(p, d, gates, d);
                        check(p, d, gates, "rows side by side");
                        scan_plan_strides(p, d, gates, kScanMaxLd);
                        check(p, d, gates, "rows far apart");
                        // (steps of a tile within 32-bit offsets, and no more workspace than the sizes alone ask for)
                        if ((64 / p.cl) * 8 * kScanMaxLd + 65536 > (int64_t)1 << 30 ||
                            scan_workspace(p, s[0], gates, backward) > parts) {
                            std::fprintf(stderr, "FAILED far apart: d %d gates %d cl %d\n", d, gates, p.cl);
                            return 1;
                        }
                    }
    std::printf("all %d checks passed\n", g_checks);
    return 0;
}
