// How a call of the gated linear recurrence is cut up: host code, shared by the
// launchers and the workspace sizes.
#include "fields.hpp"

namespace nerf {

namespace {

int pow2_at_least(int64_t v) {
    int p = 1;
    while (p < v) p <<= 1;
    return p;
}

}  // namespace

ScanPlan scan_plan(int elt, int64_t rows, int64_t n_seq, int d, int gates) {
    ScanPlan p{};
    const int m = d / gates, wide = 4;
    p.grouped = gates < d;
    p.vec = (p.grouped ? m : d) >= wide;
    const int V = p.vec ? wide : 1;
    p.lg = p.parts = 1;
    if (!p.grouped) {
        const int lanes = (d + V - 1) / V;
        p.cl = pow2_at_least(lanes < 64 ? lanes : 64);
        p.blocks = (int)(((int64_t)d + p.cl * V - 1) / (p.cl * V));
    } else {
        const int lanes = (m + V - 1) / V;
        if (lanes <= 64) {
            p.lg = pow2_at_least(lanes);
            const int64_t all = (int64_t)p.lg * gates;
            p.cl = pow2_at_least(all < 64 ? all : 64);
            const int per = p.cl / p.lg;
            p.blocks = (gates + per - 1) / per;
        } else {
            p.lg = p.cl = 64;
            p.parts = (lanes + 63) / 64;
            p.blocks = gates * p.parts;
        }
    }
    const int64_t run = (int64_t)(64 / p.cl) * 8;  // steps of one wave's tile
    const int64_t average = n_seq > 0 ? (rows + n_seq - 1) / n_seq : 0, units = n_seq * p.blocks;
    p.waves = units >= 16384 || average <= run ? 1 : units >= 1024 || average <= 4 * run ? 4 : 8;
    if (units < 256 && average > 32 * run) {
        p.waves = 4;
        const int64_t each = (2048 + units - 1) / units, tile = 4 * run;  // chunks of a sequence
        p.chunk = ((average + each - 1) / each + tile - 1) / tile * tile;
        p.slots = rows / p.chunk + n_seq;
    }
    return p;
}

// The steps of a wave's tile are within 32-bit byte offsets of each other: rows
// far apart get all lanes for their channels, and so eight steps a tile.
void scan_plan_strides(ScanPlan& p, int64_t ld) {
    if ((64 / p.cl) * 8 * ld + 65536 > (int64_t)1 << 30) p.cl = 64;
}

size_t scan_workspace(const ScanPlan& p, int64_t rows, int d, int gates, bool backward) {
    size_t floats = p.chunk ? 2 * (size_t)p.slots * (size_t)d : 0;
    if (backward && p.parts > 1) floats += (size_t)p.parts * (size_t)rows * (size_t)gates;
    return floats * sizeof(float);
}

}  // namespace nerf
