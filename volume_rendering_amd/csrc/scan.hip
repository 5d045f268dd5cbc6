// The gated linear recurrence's forward pass, and the states between the chunks
// of split sequences (both passes).
#include "scan_kernels.hpp"

namespace nerf {

namespace {

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
        const int64_t chunks = chunks_of(a, len), slot = first_slot(a, seq);
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
