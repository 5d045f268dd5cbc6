// The gradient of the gated linear recurrence.
#include "scan_kernels.hpp"

namespace nerf {

namespace {

// Gates whose channels take several blocks: their partial sums, in order, for
// the rows of sequences (the others keep what they hold).
template <class TA>
__global__ void __launch_bounds__(256) k_scan_gate_sums(ScanArgs a) {
    const int64_t lo = a.offsets ? clamp_row(a.offsets[0], a.rows) : 0;
    const int64_t hi = a.offsets ? clamp_row(a.offsets[a.n_seq], a.rows) : a.rows;
    const int64_t all = a.rows * a.gates;
    for (int64_t i = lo * a.gates + (int64_t)blockIdx.x * 256 + threadIdx.x; i < hi * a.gates;
         i += (int64_t)gridDim.x * 256) {
        float s = a.part_da[i];
        for (int p = 1; p < a.p.parts; ++p) s += a.part_da[p * all + i];
        ((TA*)a.da)[i] = (TA)s;
    }
}

template <class TA, class T>
void launch(const ScanArgs& a, hipStream_t s) {
    pick_scan<TA, T, true>(a, s);
    if (a.p.parts > 1 && a.rows > 0) {
        const int64_t blocks = (a.rows * a.gates + 255) / 256;
        k_scan_gate_sums<TA><<<(unsigned)(blocks < kScanGrid ? blocks : kScanGrid), 256, 0, s>>>(a);
    }
}

}  // namespace

void launch_scan_grad(bool bf16, bool gate_bf16, const ScanArgs& a, hipStream_t s) {
    if (!bf16)
        launch<float, float>(a, s);
    else if (gate_bf16)
        launch<__bf16, __bf16>(a, s);
    else
        launch<float, __bf16>(a, s);
}

}  // namespace nerf
