// How a call of the gated linear recurrence is cut up: host code, shared by the
// launchers and the workspace sizes.  It knows the sequences' average length only:
// offsets are on the device.  Where one sequence is far longer than the average, a
// lane or a workgroup walks it while the card idles (one of 30000 steps beside 10000
// of up to one step, 4 channels: 4.9 ms, by itself 17 us; one of 32768 beside 300 of one
// step, 64 channels: 644 us, by itself 16).
#include "fields.hpp"

namespace nerf {

namespace {

int pow2_at_least(int64_t v) {
    int p = 1;
    while (p < v) p <<= 1;
    return p;
}

// A block of `cl` channel lanes, and as many as the channels take (no gate over
// several blocks).
void lanes_of_channels(ScanPlan& p, int d, int gates, int cl) {
    const int V = p.vec ? 4 : 1;
    p.cl = cl;
    p.blocks = p.grouped ? (gates + cl / p.lg - 1) / (cl / p.lg) : (int)(((int64_t)d + cl * V - 1) / (cl * V));
}

}  // namespace

ScanPlan scan_plan(int elt, int64_t rows, int64_t n_seq, int d, int gates, bool backward) {
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
    const int64_t average = n_seq > 0 ? (rows + n_seq - 1) / n_seq : 0;
    auto run = [&] { return (int64_t)(64 / p.cl) * 8; };  // steps of one wave's tile
    // Too few workgroups for long sequences: fewer channels each (64, whole lines of bfloat16) if that gives
    // every CU one (16 sequences of 2048 steps of 1024 bfloat16 channels: 50 us, 91 else).
    const int narrow = p.lg > 16 ? p.lg : 16;
    if (p.parts == 1 && p.cl > narrow && n_seq * p.blocks < 256 && average > 16 * run() &&
        n_seq * p.blocks * (p.cl / narrow) >= 256)
        lanes_of_channels(p, d, gates, narrow);
    const int64_t units = n_seq * p.blocks;
    // Waves of a workgroup, which share a tile: no more than a sequence has tiles, and fewer the more
    // workgroups there are (65536 rays of 64 steps: 109 us with single waves, 139 with four).
    p.waves = units >= 16384 || average <= run() ? 1 : units >= 1024 || average <= 4 * run() ? 4 : 8;
    // Outputs past the caches where a step's are whole 64-byte sectors: the inputs stay in them (the gradient
    // of 16 sequences of 2048 steps of 1024 channels 67 us, 83 else; but 16-byte rows 5 us against 33).  Before
    // chunks of fewer channels, whose neighbours write the rest (3 of 300000 steps of 64: 101 us, 128 else).
    p.stream = p.cl * V * elt >= 64;
    // A sequence to a lane's channels, walked alone, saves the exchanges between lanes that a tile needs: for
    // the shortest always (35393 sequences of 2 steps of 32 channels: 10 us, 45 in tiles), else if there are
    // lanes enough (16183 of 14: 9.7 us against 25; 256 rays of 64 by 16 channels: 18 against 7) and rows so
    // short that a line serves the steps behind it (65536 rays of 64 steps of 4 channels: 80 us against 84;
    // of 16 channels 169 against 122).
    p.alone = average <= 4 || (units * p.cl >= 32768 && average <= (p.cl * V * elt <= 32 ? 128 : 16));
    // In chunks of one tile, worked on at once: few sequences for the CUs (2 of 32768 steps of 1024 channels
    // 123 us, by whole sequences 1.6 ms; the gradient of 46 of 392 steps of 33 15 us against 26), if they are
    // longer than two tiles of eight waves (30 of 200 steps of 256 channels 11.3 us against 15.7, of 100 10.2
    // against 9.5: a chunk's words have to be made ready first).
    // Chunks of one wide gate's channels are short, and of given offsets come sequence after sequence: fewer
    // sequences then (of 1551 steps of 160 channels 64 take 81 us against 113, 128 take 144 against 115).
    const int64_t most = p.parts > 1 || narrow > 16 ? 96 : kScanMaxSplit;
    if (units < most && average > 16 * (64 / p.cl) * scan_steps(backward)) {
        // A chunk waits for the one in front, so fewer channels and longer chunks shorten the chain; whole lines
        // where there are chains enough (3 sequences of 300000 steps of 64 channels: 100 us with 16 channels a
        // workgroup, 183 with 64; 2 of 32768 of 1024 channels: 125 us with 64, 141 with 32).
        if (p.parts == 1) {
            const int least = p.lg > 4 ? p.lg : 4;
            if (p.cl > narrow) lanes_of_channels(p, d, gates, narrow);
            while (p.cl > least && n_seq * p.blocks < 8) lanes_of_channels(p, d, gates, p.cl / 2);
        }
        p.waves = kScanChainWaves;
        p.chunk = (int64_t)p.waves * (64 / p.cl) * scan_steps(backward);
        p.slots = rows / p.chunk + n_seq;
    }
    return p;
}

// The steps of a wave's tile are within 32-bit byte offsets of each other: rows
// far apart get all lanes for their channels, and so eight steps a tile, and
// whole sequences, as chunks would be more than the workspace has room for.
void scan_plan_strides(ScanPlan& p, int d, int gates, int64_t ld) {
    if ((64 / p.cl) * 8 * ld + 65536 > (int64_t)1 << 30) {
        lanes_of_channels(p, d, gates, 64);  // (a gate over several blocks has them already)
        p.chunk = 0;
    }
}

size_t scan_chain_words(const ScanPlan& p) {
    const size_t each = (size_t)p.slots * p.blocks * p.cl * (p.vec ? 4 : 1);
    return 4 + 3 * ((each + 3) & ~(size_t)3);
}

size_t scan_workspace(const ScanPlan& p, int64_t rows, int gates, bool backward) {
    size_t words = p.chunk ? scan_chain_words(p) : 0;
    if (backward && p.parts > 1) words += (size_t)p.parts * (size_t)rows * (size_t)gates;
    return words * sizeof(float);
}

}  // namespace nerf
