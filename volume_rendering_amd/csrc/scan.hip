// The gated linear recurrence's forward pass, and the words between chunks made
// ready (both passes).
#include "scan_kernels.hpp"

namespace nerf {

namespace {

__global__ void __launch_bounds__(256) k_scan_reset(ScanArgs a, int64_t fours) {
    const uint4 none = {kNotYet, kNotYet, kNotYet, kNotYet};
    // (from the counter on, which lies in front of the words)
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < fours; i += (int64_t)gridDim.x * 256)
        ((uint4*)a.ticket)[i] = i == 0 ? uint4{} : none;
}

}  // namespace

void launch_scan_reset(const ScanArgs& a, hipStream_t s) {
    const int64_t fours = (int64_t)(scan_chain_words(a.p) / 4), blocks = (fours + 255) / 256;
    k_scan_reset<<<(unsigned)(blocks < 2048 ? blocks : 2048), 256, 0, s>>>(a, fours);
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
