// The gated linear recurrence's forward pass, how calls are cut up, and the
// states between the chunks of split sequences (both passes).
#include "scan_kernels.hpp"

namespace nerf {

namespace {

int pow2_at_least(int64_t v) {
    int p = 1;
    while (p < v) p <<= 1;
    return p;
}

// ---------------------------------------------------------------------------
// The state before every chunk of a sequence, from the chunks' sums: a
// workgroup takes a sequence and 64 channels, its waves runs of consecutive
// chunks.  sum_a is read for the last time here and becomes those states.
// ---------------------------------------------------------------------------
constexpr int kCarryWaves = 16;

__global__ void __launch_bounds__(64 * kCarryWaves) k_scan_carry(ScanArgs a, const float* first, float* last,
                                                                 int blocks) {
    __shared__ float pa[kCarryWaves][64], pb[kCarryWaves][64];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    for (int64_t u = blockIdx.x; u < a.n_seq * blocks; u += gridDim.x) {
        const int64_t seq = u / blocks, c = u % blocks * 64 + lane;
        const bool live = c < a.d;
        int64_t lo, len;
        sequence_rows(a, seq, lo, len);
        const int64_t chunks = (len + a.p.chunk - 1) / a.p.chunk, slot = first_slot(a, seq);
        const int64_t per = (chunks + kCarryWaves - 1) / kCarryWaves;
        const int64_t i0 = wave * per < chunks ? wave * per : chunks, i1 = i0 + per < chunks ? i0 + per : chunks;
        float A = 1.0f, B = 0.0f;
        float s = first && live ? first[seq * a.d + c] : 0.0f;
        if (live)
#pragma unroll 8
            for (int64_t i = i0; i < i1; ++i) {
                const int64_t at = (slot + i) * a.d + c;
                const float ai = a.sum_a[at];
                B = fmaf(ai, B, a.sum_b[at]);
                A *= ai;
            }
        pa[wave][lane] = A;
        pb[wave][lane] = B;
        __syncthreads();
        for (int w = 0; w < wave; ++w) s = fmaf(pa[w][lane], s, pb[w][lane]);
        if (live) {
#pragma unroll 8
            for (int64_t i = i0; i < i1; ++i) {
                const int64_t at = (slot + i) * a.d + c;
                const float ai = a.sum_a[at], bi = a.sum_b[at];
                a.sum_a[at] = s;
                s = fmaf(ai, s, bi);
            }
            if (last && wave == kCarryWaves - 1) last[seq * a.d + c] = s;
        }
        __syncthreads();
    }
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

void launch_scan_carry(const ScanArgs& a, const float* first, float* last, hipStream_t s) {
    const int blocks = (a.d + 63) / 64;
    const int64_t units = a.n_seq * blocks;
    k_scan_carry<<<(unsigned)(units < kScanGrid ? units : kScanGrid), 64 * kCarryWaves, 0, s>>>(a, first, last, blocks);
}

void launch_scan(bool bf16, bool gate_bf16, const ScanArgs& a, hipStream_t s) {
    if (!bf16)
        pick_scan<float, float, false>(a, s);
    else if (gate_bf16)
        pick_scan<__bf16, __bf16, false>(a, s);
    else
        pick_scan<float, __bf16, false>(a, s);
}

}  // namespace nerf
