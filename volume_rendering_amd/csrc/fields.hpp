// Argument structs and launchers of the streaming-field operators: the gate
// (gate.hip), the routed layer for a few samples (routed_mlp.hip), the gated
// linear recurrence (scan.hip, scan_grad.hip) and the norm of a list of
// gradients (clip.hip).  Shapes and pointers are validated by fields_abi.cpp
// before any launcher is called; the contents of device index arrays are not,
// so every kernel keeps them in range itself.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "nerf_mi355x.h"

namespace nerf {

// Bits of the checked build (continuing ExpertCheckBit in experts.hpp).
enum FieldCheckBit : unsigned {
    kCheckScanOffset = 11,  // sequence offsets decreasing or past the rows
};

// ---- gate (gate.hip) ----
struct GateArgs {
    const void* logits;  // [n, n_experts]
    int64_t ld;
    int64_t n;
    int n_experts, k;
    int renorm;          // weights are a softmax over the chosen experts, not over all
    int32_t* ids;        // [n, k]: out (forward) or in
    float* weights;      // [n, k]: out (forward) or in
    const float* dweights;
    void* dlogits;       // [n, n_experts]
    int64_t ld_d;
};
void launch_gate(bool bf16, const GateArgs& a, hipStream_t s);
void launch_gate_grad(bool bf16, const GateArgs& a, hipStream_t s);

// ---- routed layer for a few samples (routed_mlp.hip) ----
struct MlpArgs {
    int n, k, n_experts;
    int d_in, hidden, d_out;
    int act;               // NERF_ACT_*
    const void* x;         // [n, d_in]
    int64_t ld_x;
    const int32_t* ids;    // [n, k]
    const float* weights;  // [n, k] or NULL (1)
    const void* w1;        // [n_experts][hidden, or 2 hidden][d_in]
    const float* b1;
    const void* w2;        // [n_experts][d_out][hidden]
    const float* b2;
    float* h;              // workspace [n k][ld_h], or three bfloat16 planes of that
    int64_t ld_h;
    int64_t plane;         // elements of a plane
    float* y;              // workspace [n k][d_out]
    void* plan;            // workspace: the sorted pairs, above kMlpSelfSorted
    void* out;             // [n, d_out]
    int64_t ld_out;
};
constexpr int kMlpSelfSorted = 64;       // pairs that need no plan
constexpr size_t kMlpPlanBytes = 16640;  // whole 256 bytes
void launch_routed_mlp(bool bf16, const MlpArgs& a, hipStream_t s);

// ---- gated linear recurrence (scan_kernels.hpp, scan.hip, scan_grad.hip) ----
// How a call is cut up.  Lanes of a wave are CL channel lanes (V channels each)
// times 64 / CL runs of consecutive steps; a gate's channels take LG of them.
struct ScanPlan {
    bool vec;        // V is 4 (8 bytes of bfloat16, 16 of float32), or 1
    bool grouped;    // fewer gates than channels
    int cl, lg;      // channel lanes, lanes of a gate's channels (powers of two)
    int blocks;      // channel blocks: workgroups side by side
    int parts;       // channel blocks of one gate (partial sums of its gradient)
    int waves;       // waves that share a sequence (or chunk)
    bool alone;      // a lane walks a sequence alone
    bool stream;     // outputs are stored past the caches
    int64_t chunk;   // steps of a chunk (one tile), 0: sequences are not split
    int64_t slots;   // chunks at most
};
struct ScanArgs {
    int64_t rows, n_seq, len;  // len: of every sequence where offsets is NULL
    const int32_t* offsets;    // [n_seq + 1] or NULL
    int d, gates;
    int reverse, mix;
    const void* a;             // [rows, gates]
    int64_t ld_a;
    const void* x;             // [rows, d]
    int64_t ld_x;
    const float* h0;           // [n_seq, d] or NULL (0)
    void* h;                   // [rows, d]: out (forward) or in
    int64_t ld_h;
    float* h_last;             // [n_seq, d] or NULL
    const void* dh;            // gradient: [rows, d]
    int64_t ld_dh;
    const float* dh_last;      // [n_seq, d] or NULL (0)
    void* da;                  // [rows, gates]
    void* dx;                  // [rows, d]
    float* dh0;                // [n_seq, d] or NULL
    uint32_t* ticket;          // split: the next chunk to take (64 bits)
    uint32_t* sum_a;           // split: per chunk, block and channel lane: the gates' products,
    uint32_t* sum_b;           //   the states of a chunk that began with 0,
    uint32_t* state;           //   and the states after the chunk
    float* part_da;            // [parts, rows, gates]
    ScanPlan p;
};
// The strides may take a plan's workspace away, but not change its size.
ScanPlan scan_plan(int elt, int64_t rows, int64_t n_seq, int d, int gates, bool backward);
void scan_plan_strides(ScanPlan& p, int d, int gates, int64_t ld);
// Steps of a lane, and waves of a chunk's workgroup.
constexpr int scan_steps(bool backward) { return backward ? 4 : 8; }
constexpr int kScanChainWaves = 8;
// 32-bit words of a split call's workspace: the counter's four, and the chunks'.
size_t scan_chain_words(const ScanPlan& p);
constexpr int kScanMaxSplit = 256;  // sequences of a call that is split
constexpr int64_t kScanMaxLd = (int64_t)1 << 26;  // elements
size_t scan_workspace(const ScanPlan& p, int64_t rows, int gates, bool backward);
// gate_bf16 implies bf16.
void launch_scan(bool bf16, bool gate_bf16, const ScanArgs& a, hipStream_t s);
void launch_scan_grad(bool bf16, bool gate_bf16, const ScanArgs& a, hipStream_t s);
// The words of a split call's workspace before its chunks.
void launch_scan_reset(const ScanArgs& a, hipStream_t s);

// ---- gradient norm (clip.hip) ----
size_t grad_norm_partials(const nerf_tensor* list, int n);
void launch_grad_norm(const nerf_tensor* list, int n, double* partials, float* norm, hipStream_t s);
void launch_grad_clip(const nerf_tensor* list, int n, float max_norm, double* partials, float* norm, hipStream_t s);

}  // namespace nerf
