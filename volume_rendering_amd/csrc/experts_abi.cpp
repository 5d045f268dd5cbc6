// C ABI of the routed-field operators (routing, experts' products,
// distillation): argument validation, workspaces and dispatch.  Nothing is
// enqueued unless every argument checks out.
#include <hip/hip_runtime.h>

#include <cmath>

#include "abi_util.hpp"
#include "experts.hpp"
#include "nerf_mi355x.h"

using namespace nerf;

namespace {

constexpr int kMaxWidth = 65536;
constexpr int64_t kMaxPairs = ((int64_t)1 << 31) - 1;
constexpr int64_t kMaxLogits = (int64_t)1 << 40;  // more than a card holds

hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(bytes - 1)) == 0; }
int elt_bytes(int dtype) { return dtype == NERF_BF16 ? 2 : 4; }

#define NERF_REQUIRE(cond, ...)                                                \
    do {                                                                       \
        if (!(cond)) return nerf_fail(NERF_ERR_INVALID_ARGUMENT, __VA_ARGS__); \
    } while (0)

nerf_status check_launch(const char* who) {
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return nerf_fail(NERF_ERR_HIP, "%s: %s", who, hipGetErrorString(e));
    return NERF_OK;
}

// The caller's workspace, or one allocated in stream order for the call.
struct Workspace {
    void* p = nullptr;
    bool own = false;

    nerf_status take(const char* who, void* given, size_t bytes, size_t need, void* stream) {
        if (need == 0) return NERF_OK;
        if (given) {
            if (bytes < need)
                return nerf_fail(NERF_ERR_WORKSPACE, "%s: workspace has %zu bytes, needs %zu", who, bytes, need);
            NERF_REQUIRE(aligned(given, 16), "%s: workspace must be 16-byte aligned", who);
            p = given;
            return NERF_OK;
        }
        (void)hipGetLastError();
        const hipError_t e = hipMallocAsync(&p, need, as_stream(stream));
        if (e != hipSuccess)
            return nerf_fail(NERF_ERR_WORKSPACE, "%s: cannot allocate %zu workspace bytes: %s", who, need,
                             hipGetErrorString(e));
        own = true;
        return NERF_OK;
    }
    nerf_status release(const char* who, nerf_status st, void* stream) {
        if (!own) return st;
        const hipError_t e = hipFreeAsync(p, as_stream(stream));
        if (st == NERF_OK && e != hipSuccess)
            return nerf_fail(NERF_ERR_HIP, "%s: workspace free: %s", who, hipGetErrorString(e));
        return st;
    }
};

nerf_status check_route(const char* who, int64_t n, int k, int n_experts) {
    NERF_REQUIRE(n >= 0, "%s: n %lld < 0", who, (long long)n);
    NERF_REQUIRE(k >= 1 && k <= NERF_MAX_CHOICES, "%s: k %d outside 1..%d", who, k, NERF_MAX_CHOICES);
    NERF_REQUIRE(n_experts >= 1, "%s: n_experts %d < 1", who, n_experts);
    NERF_REQUIRE(n <= kMaxPairs / k, "%s: %lld x %d pairs (fewer than 2^31)", who, (long long)n, k);
    if (n_experts > NERF_MAX_EXPERTS)
        return nerf_fail(NERF_ERR_UNSUPPORTED, "%s: n_experts %d above %d", who, n_experts, NERF_MAX_EXPERTS);
    return NERF_OK;
}

nerf_status check_rows(const char* who, const RouteRows& r, int dtype, int64_t ld) {
    NERF_REQUIRE(dtype == NERF_F32 || dtype == NERF_BF16, "%s: dtype %d", who, dtype);
    NERF_REQUIRE(r.d >= 1 && r.d <= kMaxWidth, "%s: d %d outside 1..%d", who, r.d, kMaxWidth);
    NERF_REQUIRE(ld == 0 || ld >= r.d, "%s: row stride %lld below d %d", who, (long long)ld, r.d);
    return check_route(who, r.n, r.k, r.n_experts);
}

nerf_status check_row_pointers(const char* who, const RouteRows& r, int dtype) {
    const int b = elt_bytes(dtype);
    NERF_REQUIRE(r.offsets && r.place && r.out, "%s: NULL offsets, place or output", who);
    NERF_REQUIRE(aligned(r.offsets, 4) && aligned(r.place, 4) && aligned(r.weights, 4) && aligned(r.dweights, 4) &&
                     aligned(r.a, b) && aligned(r.y, b) && aligned(r.out, b),
                 "%s: misaligned pointer", who);
    return NERF_OK;
}

nerf_status check_layer(const char* who, const nerf_expert_layer* L, const int32_t* order, int64_t slots) {
    NERF_REQUIRE(L, "%s: layer is NULL", who);
    NERF_REQUIRE(L->dtype == NERF_F32 || L->dtype == NERF_BF16, "%s: dtype %d", who, L->dtype);
    NERF_REQUIRE(L->n_experts >= 1, "%s: n_experts %d < 1", who, L->n_experts);
    NERF_REQUIRE(L->d_in >= 1 && L->d_in <= kMaxWidth && L->d_out >= 1 && L->d_out <= kMaxWidth,
                 "%s: widths %d -> %d outside 1..%d", who, L->d_in, L->d_out, kMaxWidth);
    NERF_REQUIRE(L->ld_x == 0 || L->ld_x >= L->d_in, "%s: ld_x %lld below d_in", who, (long long)L->ld_x);
    NERF_REQUIRE(L->ld_y == 0 || L->ld_y >= L->d_out, "%s: ld_y %lld below d_out", who, (long long)L->ld_y);
    NERF_REQUIRE(slots >= 0 && slots <= kMaxPairs, "%s: slots %lld", who, (long long)slots);
    NERF_REQUIRE(L->x_rows >= 0 && (L->x_rows > 0 || !order || slots == 0), "%s: x_rows %lld", who,
                 (long long)L->x_rows);
    NERF_REQUIRE(!order || (L->k >= 1 && L->k <= NERF_MAX_CHOICES), "%s: k %d outside 1..%d", who, L->k,
                 NERF_MAX_CHOICES);
    if (L->n_experts > NERF_MAX_EXPERTS)
        return nerf_fail(NERF_ERR_UNSUPPORTED, "%s: n_experts %d above %d", who, L->n_experts, NERF_MAX_EXPERTS);
    // The largest grids: four waves for each 128 slots x 128 columns, or, with up to
    // 64 columns, a wave for each 32 slots.  (Tiles of 32 slots x 64 of more columns
    // are for fewer than 2^20 slots, and few enough for any width.  Steps of 64 slots
    // are counted in 32 bits, two past the end.)
    const int64_t width = L->d_in > L->d_out ? L->d_in : L->d_out;
    if (slots > kMaxPairs - 255 || (slots / 128 + L->n_experts + 1) * ((width + 127) / 128) * 256 > kMaxWorkItems)
        return nerf_fail(NERF_ERR_UNSUPPORTED, "%s: %lld slots x %lld columns exceed one launch", who,
                         (long long)slots, (long long)width);
    return NERF_OK;
}

ExpertArgs expert_args(const nerf_expert_layer* L, const void* x, const void* w, const int32_t* offsets,
                       const int32_t* order, int64_t slots) {
    ExpertArgs a{};
    a.n_experts = L->n_experts;
    a.d_in = L->d_in;
    a.d_out = L->d_out;
    a.slots = slots;
    a.offsets = offsets;
    a.order = order;
    // ceil(2^(31 + b) / k) with k <= 2^b: an exact quotient of 31-bit numbers
    const uint32_t k = order ? (uint32_t)L->k : 1u;
    int b = 0;
    while ((1u << b) < k) ++b;
    a.k_mul = (uint32_t)((((uint64_t)1 << (31 + b)) + k - 1) / k);
    a.k_shift = 31 + b;
    a.x_rows = L->x_rows;
    a.x = x;
    a.ld_x = L->ld_x ? L->ld_x : L->d_in;
    a.w = w;
    a.relu = L->relu != 0;
    return a;
}

nerf_status check_distill(const char* who, int dtype, int64_t ld, int64_t n, int64_t classes, int top,
                          float temperature) {
    NERF_REQUIRE(dtype == NERF_F32 || dtype == NERF_BF16, "%s: dtype %d", who, dtype);
    NERF_REQUIRE(n >= 0, "%s: n %lld < 0", who, (long long)n);
    NERF_REQUIRE(classes >= 1 && classes <= kMaxPairs, "%s: classes %lld", who, (long long)classes);
    NERF_REQUIRE(ld == 0 || ld >= classes, "%s: row stride %lld below the classes", who, (long long)ld);
    NERF_REQUIRE(top >= 1 && top <= kDistillMaxTop, "%s: top %d outside 1..%d", who, top, kDistillMaxTop);
    NERF_REQUIRE(temperature > 0.0f && std::isfinite(temperature), "%s: temperature %g", who, (double)temperature);
    if (n > kMaxLogits / classes)
        return nerf_fail(NERF_ERR_UNSUPPORTED, "%s: %lld rows x %lld classes (at most 2^40)", who, (long long)n,
                         (long long)classes);
    return NERF_OK;
}

}  // namespace

extern "C" {

size_t nerf_route_workspace_size(int64_t n, int k, int n_experts) {
    if (n < 0 || k < 1 || k > NERF_MAX_CHOICES || n_experts < 1 || n_experts > NERF_MAX_EXPERTS || n > kMaxPairs / k)
        return 0;
    const int64_t nb = route_blocks(n * k);
    return nb > 1 ? (size_t)(nb + 1) * (size_t)(n_experts + 1) * sizeof(int32_t) : 0;
}

nerf_status nerf_route_plan(const int32_t* ids, int64_t n, int k, int n_experts, int32_t* offsets, int32_t* order,
                            int32_t* place, void* workspace, size_t workspace_bytes, void* stream) {
    const char* who = "nerf_route_plan";
    nerf_status st = check_route(who, n, k, n_experts);
    if (st != NERF_OK) return st;
    NERF_REQUIRE(offsets && (n == 0 || (ids && order && place)), "%s: NULL input or output", who);
    NERF_REQUIRE(aligned(ids, 4) && aligned(offsets, 4) && aligned(order, 4) && aligned(place, 4),
                 "%s: misaligned pointer", who);
    Workspace ws;
    st = ws.take(who, workspace, workspace_bytes, nerf_route_workspace_size(n, k, n_experts), stream);
    if (st != NERF_OK) return st;
    (void)hipGetLastError();
    launch_route_plan(ids, n * k, n_experts, offsets, order, place, static_cast<int32_t*>(ws.p), as_stream(stream));
    return ws.release(who, check_launch(who), stream);
}

nerf_status nerf_route_gather(const void* x, int dtype, int64_t ld_x, int64_t n, int k, int d, int n_experts,
                              const int32_t* offsets, const int32_t* place, void* rows, void* stream) {
    const char* who = "nerf_route_gather";
    RouteRows r{};
    r.n = n, r.k = k, r.d = d, r.n_experts = n_experts, r.offsets = offsets, r.place = place;
    r.a = x, r.lda = ld_x ? ld_x : d, r.out = rows;
    nerf_status st = check_rows(who, r, dtype, ld_x);
    if (st != NERF_OK || n == 0) return st;
    NERF_REQUIRE(x, "%s: x is NULL", who);
    if ((st = check_row_pointers(who, r, dtype)) != NERF_OK) return st;
    (void)hipGetLastError();
    launch_route_gather(dtype == NERF_BF16, r, as_stream(stream));
    return check_launch(who);
}

nerf_status nerf_route_combine(const void* y, int dtype, int64_t n, int k, int d, int n_experts,
                               const int32_t* offsets, const int32_t* place, const float* weights, void* out,
                               int64_t ld_out, void* stream) {
    const char* who = "nerf_route_combine";
    RouteRows r{};
    r.n = n, r.k = k, r.d = d, r.n_experts = n_experts, r.offsets = offsets, r.place = place;
    r.weights = weights, r.y = y, r.out = out, r.ldo = ld_out ? ld_out : d;
    nerf_status st = check_rows(who, r, dtype, ld_out);
    if (st != NERF_OK || n == 0) return st;
    NERF_REQUIRE(y, "%s: y is NULL", who);
    if ((st = check_row_pointers(who, r, dtype)) != NERF_OK) return st;
    (void)hipGetLastError();
    launch_route_combine(dtype == NERF_BF16, r, as_stream(stream));
    return check_launch(who);
}

nerf_status nerf_route_combine_grad(const void* dout, int64_t ld_dout, const void* y, int dtype, int64_t n, int k,
                                    int d, int n_experts, const int32_t* offsets, const int32_t* place,
                                    const float* weights, void* dy, float* dweights, void* stream) {
    const char* who = "nerf_route_combine_grad";
    RouteRows r{};
    r.n = n, r.k = k, r.d = d, r.n_experts = n_experts, r.offsets = offsets, r.place = place;
    r.weights = weights, r.a = dout, r.lda = ld_dout ? ld_dout : d, r.y = y, r.out = dy, r.dweights = dweights;
    nerf_status st = check_rows(who, r, dtype, ld_dout);
    if (st != NERF_OK || n == 0) return st;
    NERF_REQUIRE(dout && y, "%s: dout or y is NULL", who);
    if ((st = check_row_pointers(who, r, dtype)) != NERF_OK) return st;
    (void)hipGetLastError();
    launch_route_combine_grad(dtype == NERF_BF16, r, as_stream(stream));
    return check_launch(who);
}

nerf_status nerf_expert_linear(const nerf_expert_layer* layer, const void* x, const void* weights, const float* bias,
                               const int32_t* offsets, const int32_t* order, int64_t slots, void* y, void* stream) {
    const char* who = "nerf_expert_linear";
    const nerf_status st = check_layer(who, layer, order, slots);
    if (st != NERF_OK || slots == 0) return st;
    const int b = elt_bytes(layer->dtype);
    NERF_REQUIRE(x && weights && offsets && y, "%s: NULL input or output", who);
    NERF_REQUIRE(order || layer->x_rows >= slots, "%s: x has %lld rows for %lld slots", who,
                 (long long)layer->x_rows, (long long)slots);
    NERF_REQUIRE(aligned(x, b) && aligned(weights, b) && aligned(y, b) && aligned(bias, 4) && aligned(offsets, 4) &&
                     aligned(order, 4),
                 "%s: misaligned pointer", who);
    ExpertArgs a = expert_args(layer, x, weights, offsets, order, slots);
    a.bias = bias;
    a.y = y;
    a.ld_y = layer->ld_y ? layer->ld_y : layer->d_out;
    (void)hipGetLastError();
    launch_expert_linear(layer->dtype == NERF_BF16, a, as_stream(stream));
    return check_launch(who);
}

size_t nerf_expert_linear_grad_workspace_size(int64_t slots, int n_experts, int d_in, int d_out) {
    if (slots < 0 || slots > kMaxPairs - 255 || n_experts < 1 || n_experts > NERF_MAX_EXPERTS || d_in < 1 ||
        d_in > kMaxWidth || d_out < 1 || d_out > kMaxWidth)
        return 0;
    const int64_t chunk = expert_grad_chunk(slots, n_experts, d_in, d_out);
    if (chunk == 0) return 0;
    return (size_t)(slots / chunk + n_experts) * ((size_t)d_in + 1) * (size_t)d_out * sizeof(float);
}

nerf_status nerf_expert_linear_grad(const nerf_expert_layer* layer, const void* dz, const void* x, const void* weights,
                                    const int32_t* offsets, const int32_t* order, int64_t slots, void* dx,
                                    float* dweights, float* dbias, void* workspace, size_t workspace_bytes,
                                    void* stream) {
    const char* who = "nerf_expert_linear_grad";
    nerf_status st = check_layer(who, layer, order, slots);
    if (st != NERF_OK) return st;
    const int b = elt_bytes(layer->dtype);
    NERF_REQUIRE(dx || dweights, "%s: neither dx nor dweights asked for", who);
    NERF_REQUIRE(!dbias || dweights, "%s: dbias needs dweights", who);
    NERF_REQUIRE(offsets && (slots == 0 || dz), "%s: NULL offsets or dz", who);
    NERF_REQUIRE(slots == 0 || x || (!dweights && !layer->relu), "%s: x is NULL", who);
    NERF_REQUIRE(slots == 0 || weights || !dx, "%s: weights are NULL", who);
    NERF_REQUIRE(!x || order || layer->x_rows >= slots, "%s: x has %lld rows for %lld slots", who,
                 (long long)layer->x_rows, (long long)slots);
    NERF_REQUIRE(aligned(dz, b) && aligned(x, b) && aligned(weights, b) && aligned(dx, b) && aligned(dweights, 4) &&
                     aligned(dbias, 4) && aligned(offsets, 4) && aligned(order, 4),
                 "%s: misaligned pointer", who);
    ExpertArgs a = expert_args(layer, x, weights, offsets, order, slots);
    a.dz = dz;
    a.ld_dz = layer->ld_y ? layer->ld_y : layer->d_out;
    a.y = dx;
    a.ld_y = layer->d_in;
    a.dw = dweights;
    a.db = dbias;
    Workspace ws;
    if (dweights) {
        st = ws.take(who, workspace, workspace_bytes,
                     nerf_expert_linear_grad_workspace_size(slots, layer->n_experts, layer->d_in, layer->d_out),
                     stream);
        if (st != NERF_OK) return st;
        a.chunk = expert_grad_chunk(slots, layer->n_experts, layer->d_in, layer->d_out);
        if (a.chunk) {
            a.part = static_cast<float*>(ws.p);
            a.bpart = a.part + (slots / a.chunk + layer->n_experts) * (int64_t)layer->d_in * layer->d_out;
        }
    }
    (void)hipGetLastError();
    if (dx && slots > 0) launch_expert_grad_x(layer->dtype == NERF_BF16, a, as_stream(stream));
    if (dweights) launch_expert_grad_w(layer->dtype == NERF_BF16, a, as_stream(stream));
    return ws.release(who, check_launch(who), stream);
}

size_t nerf_distill_workspace_size(int64_t n, int64_t classes) {
    if (n < 1 || classes < 1) return 0;
    const int splits = distill_splits(n, classes);
    return splits > 1 ? (size_t)n * (size_t)splits * 2 * sizeof(float) : 0;
}

nerf_status nerf_distill_topk(const void* logits, int dtype, int64_t ld_logits, int64_t n, int64_t classes,
                              const float* t_logits, const int32_t* t_ids, int top, float temperature,
                              const float* row_scale, float* loss, float* lse, void* grad, int64_t ld_grad,
                              void* workspace, size_t workspace_bytes, void* stream) {
    const char* who = "nerf_distill_topk";
    nerf_status st = check_distill(who, dtype, ld_logits, n, classes, top, temperature);
    if (st != NERF_OK) return st;
    NERF_REQUIRE(ld_grad == 0 || ld_grad >= classes, "%s: ld_grad %lld below the classes", who, (long long)ld_grad);
    if (n == 0) return NERF_OK;
    const int b = elt_bytes(dtype);
    NERF_REQUIRE(logits && t_logits && t_ids && loss, "%s: NULL input or output", who);
    NERF_REQUIRE(grad != logits, "%s: grad must not overlap logits", who);
    NERF_REQUIRE(aligned(logits, b) && aligned(grad, b) && aligned(t_logits, 4) && aligned(t_ids, 4) &&
                     aligned(row_scale, 4) && aligned(loss, 4) && aligned(lse, 4),
                 "%s: misaligned pointer", who);
    DistillArgs a{logits, ld_logits ? ld_logits : classes, n, classes, t_logits, t_ids, top, temperature, row_scale,
                  loss, lse, grad, ld_grad ? ld_grad : classes, nullptr};
    Workspace ws;
    st = ws.take(who, workspace, workspace_bytes, nerf_distill_workspace_size(n, classes), stream);
    if (st != NERF_OK) return st;
    a.part = static_cast<float*>(ws.p);
    (void)hipGetLastError();
    launch_distill(dtype == NERF_BF16, a, as_stream(stream));
    return ws.release(who, check_launch(who), stream);
}

nerf_status nerf_distill_topk_grad(const void* logits, int dtype, int64_t ld_logits, int64_t n, int64_t classes,
                                   const float* t_logits, const int32_t* t_ids, int top, float temperature,
                                   const float* row_scale, const float* lse, void* grad, int64_t ld_grad,
                                   void* stream) {
    const char* who = "nerf_distill_topk_grad";
    const nerf_status st = check_distill(who, dtype, ld_logits, n, classes, top, temperature);
    if (st != NERF_OK) return st;
    NERF_REQUIRE(ld_grad == 0 || ld_grad >= classes, "%s: ld_grad %lld below the classes", who, (long long)ld_grad);
    if (n == 0) return NERF_OK;
    const int b = elt_bytes(dtype);
    NERF_REQUIRE(logits && t_logits && t_ids && lse && grad, "%s: NULL input or output", who);
    NERF_REQUIRE(grad != logits, "%s: grad must not overlap logits", who);
    NERF_REQUIRE(aligned(logits, b) && aligned(grad, b) && aligned(t_logits, 4) && aligned(t_ids, 4) &&
                     aligned(row_scale, 4) && aligned(lse, 4),
                 "%s: misaligned pointer", who);
    DistillArgs a{logits, ld_logits ? ld_logits : classes, n, classes, t_logits, t_ids, top, temperature, row_scale,
                  nullptr, const_cast<float*>(lse), grad, ld_grad ? ld_grad : classes, nullptr};
    (void)hipGetLastError();
    launch_distill_grad(dtype == NERF_BF16, a, as_stream(stream));
    return check_launch(who);
}

}  // extern "C"
