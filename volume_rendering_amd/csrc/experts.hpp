// Argument structs and launchers of the routed-field operators: routing
// plans and row movement (route.hip), the experts' products (experts.hip)
// and the distillation loss (distill.hip).  Shapes and pointers are validated
// by experts_abi.cpp before any launcher is called; the contents of device
// index arrays are not, so every kernel keeps them in range itself.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace nerf {

// HIP launches hold fewer than 2^32 work items.
constexpr int64_t kMaxWorkItems = ((int64_t)1 << 32) - 1;

// Bits of the checked build (continuing CheckBit in common.hpp).
enum ExpertCheckBit : unsigned {
    kCheckRouteSlot = 9,    // slot of a pair outside the slots, or a sorted pair outside the pairs
    kCheckRouteOffset = 10, // expert offsets decreasing or past the slots
};

// ---- routing (route.hip) ----
// Pairs one workgroup sorts; the plan's workspace holds a row of E + 1 counts
// per workgroup and one of totals.
constexpr int kRouteWaves = 8;
constexpr int kRouteBatch = 8;  // pairs a lane holds in registers
inline int64_t route_chunk(int64_t pairs) {
    // one batch a lane; beyond 2^22 pairs more, so that the counts of 1024
    // workgroups stay a small part of what is read
    int64_t c = 64 * kRouteWaves * kRouteBatch;
    const int64_t per = (pairs + 1023) / 1024;
    if (c < per) c = (per + c - 1) / c * c;
    return c;
}
inline int64_t route_blocks(int64_t pairs) { return (pairs + route_chunk(pairs) - 1) / route_chunk(pairs); }

struct RouteRows {
    int64_t n;  // samples
    int k, d;
    int n_experts;
    const int32_t* offsets;  // [n_experts + 1]; offsets[n_experts] = slots in use
    const int32_t* place;    // [n, k] slot of each pair
    const float* weights;    // [n, k] or NULL (1)
    const void* a;           // gather: x; combine: y; combine gradient: dout
    int64_t lda;             // elements per row of x or dout
    const void* y;           // combine gradient: y
    void* out;               // gather: rows; combine: out; combine gradient: dy
    int64_t ldo;             // elements per row of the combined rows
    float* dweights;         // combine gradient, or NULL
};
void launch_route_plan(const int32_t* ids, int64_t pairs, int n_experts, int32_t* offsets, int32_t* order,
                       int32_t* place, int32_t* counts, hipStream_t s);
void launch_route_gather(bool bf16, const RouteRows& r, hipStream_t s);
void launch_route_combine(bool bf16, const RouteRows& r, hipStream_t s);
void launch_route_combine_grad(bool bf16, const RouteRows& r, hipStream_t s);

// ---- experts' products (experts.hip) ----
struct ExpertArgs {
    int n_experts, d_in, d_out;
    int64_t slots;           // rows of y, dz and dx
    const int32_t* offsets;  // [n_experts + 1]
    const int32_t* order;    // [slots] pair of each slot (x row = pair / k), or NULL (x row = slot)
    uint32_t k_mul;          // pair / k = (pair k_mul) >> k_shift for pairs below 2^31
    int k_shift;
    int64_t x_rows;          // rows of x
    const void* x;
    int64_t ld_x;
    const void* w;           // [n_experts][d_out][d_in]
    const float* bias;       // [n_experts][d_out] or NULL
    int relu;                // forward: of the output; gradient: x is a ReLU's output
    void* y;                 // forward: y; gradient: dx
    int64_t ld_y;
    const void* dz;          // gradient
    int64_t ld_dz;
    float* dw;               // [n_experts][d_out][d_in]
    float* db;               // [n_experts][d_out] or NULL
    float* part;             // partial weight gradients (row ranges), or NULL
    float* bpart;
    int64_t chunk;           // rows per partial sum (0: one range per expert)
};
// Rows per partial weight gradient, 0 if each expert's rows are one range.
int64_t expert_grad_chunk(int64_t slots, int n_experts, int d_in, int d_out);
void launch_expert_linear(bool bf16, const ExpertArgs& a, hipStream_t s);
void launch_expert_grad_x(bool bf16, const ExpertArgs& a, hipStream_t s);
void launch_expert_grad_w(bool bf16, const ExpertArgs& a, hipStream_t s);

// ---- distillation (distill.hip) ----
struct DistillArgs {
    const void* logits;
    int64_t ld, n, classes;
    const float* t_logits;    // [n, top]
    const int32_t* t_ids;     // [n, top]
    int top;
    float temperature;
    const float* row_scale;   // [n] or NULL (1)
    float* loss;              // [n] (forward)
    float* lse;               // [n]: out (forward, optional) or in (gradient)
    void* grad;               // [n, classes] or NULL
    int64_t ld_grad;
    float* part;              // split forward: [n][splits][2] running maxima and sums
};
constexpr int kDistillMaxTop = 256;
// Workgroups that share one row of the forward pass (1: a row each).
int distill_splits(int64_t n, int64_t classes);
void launch_distill(bool bf16, const DistillArgs& a, hipStream_t s);
void launch_distill_grad(bool bf16, const DistillArgs& a, hipStream_t s);

}  // namespace nerf
