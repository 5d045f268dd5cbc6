// C ABI of the streaming-field operators (gate, routed layer for a few
// samples, gated linear recurrence, gradient norm): argument validation,
// workspaces and dispatch.  Nothing is enqueued unless every argument checks
// out.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdlib>

#include "abi_args.hpp"
#include "fields.hpp"
#include "nerf_mi355x.h"

using namespace nerf;

namespace {

constexpr int kMaxWidth = 65536;
constexpr int64_t kMaxRows = ((int64_t)1 << 31) - 1;
constexpr int kMaxTensors = 1 << 20;

nerf_status check_gate(const char* who, int dtype, int64_t ld, int64_t n, int n_experts, int k) {
    NERF_REQUIRE(dtype == NERF_F32 || dtype == NERF_BF16, "%s: dtype %d", who, dtype);
    NERF_REQUIRE(n >= 0, "%s: n %lld < 0", who, (long long)n);
    NERF_REQUIRE(n_experts >= 1, "%s: n_experts %d < 1", who, n_experts);
    NERF_REQUIRE(k >= 1 && k <= NERF_MAX_CHOICES && k <= n_experts, "%s: k %d outside 1..%d", who, k,
                 n_experts < NERF_MAX_CHOICES ? n_experts : NERF_MAX_CHOICES);
    NERF_REQUIRE(ld == 0 || ld >= n_experts, "%s: row stride %lld below the experts", who, (long long)ld);
    NERF_REQUIRE(n <= kMaxRows / k, "%s: %lld x %d pairs (fewer than 2^31)", who, (long long)n, k);
    if (n_experts > NERF_MAX_EXPERTS)
        return nerf_fail(NERF_ERR_UNSUPPORTED, "%s: n_experts %d above %d", who, n_experts, NERF_MAX_EXPERTS);
    return NERF_OK;
}

nerf_status check_scan(const char* who, const nerf_scan_cfg* c, bool offsets, bool backward) {
    NERF_REQUIRE(c, "%s: cfg is NULL", who);
    NERF_REQUIRE(c->dtype == NERF_F32 || c->dtype == NERF_BF16, "%s: dtype %d", who, c->dtype);
    NERF_REQUIRE(c->gate_dtype == NERF_F32 || c->gate_dtype == NERF_BF16, "%s: gate_dtype %d", who, c->gate_dtype);
    NERF_REQUIRE(c->d >= 1 && c->d <= kMaxWidth, "%s: d %d outside 1..%d", who, c->d, kMaxWidth);
    NERF_REQUIRE(c->gates >= 1 && c->gates <= c->d && c->d % c->gates == 0, "%s: %d gates for %d channels", who,
                 c->gates, c->d);
    NERF_REQUIRE(c->rows >= 0 && c->rows <= kMaxRows, "%s: rows %lld", who, (long long)c->rows);
    NERF_REQUIRE(c->n_seq >= 0 && c->n_seq < kMaxRows, "%s: n_seq %lld", who, (long long)c->n_seq);
    NERF_REQUIRE(offsets || c->n_seq == 0 || c->rows % c->n_seq == 0, "%s: %lld rows are not %lld equal sequences", who,
                 (long long)c->rows, (long long)c->n_seq);
    NERF_REQUIRE(c->ld_a == 0 || c->ld_a >= c->gates, "%s: ld_a %lld below the gates", who, (long long)c->ld_a);
    NERF_REQUIRE(c->ld_x == 0 || c->ld_x >= c->d, "%s: ld_x %lld below d", who, (long long)c->ld_x);
    NERF_REQUIRE(c->ld_h == 0 || c->ld_h >= c->d, "%s: ld_h %lld below d", who, (long long)c->ld_h);
    NERF_REQUIRE(!backward || c->ld_dh == 0 || c->ld_dh >= c->d, "%s: ld_dh %lld below d", who, (long long)c->ld_dh);
    if (c->gate_dtype == NERF_BF16 && c->dtype != NERF_BF16)
        return nerf_fail(NERF_ERR_UNSUPPORTED, "%s: bfloat16 gates of float32 rows", who);
    if (std::max(std::max(c->ld_a, c->ld_x), std::max(c->ld_h, c->ld_dh)) > kScanMaxLd)
        return nerf_fail(NERF_ERR_UNSUPPORTED, "%s: row strides above 2^26 elements", who);
    return NERF_OK;
}

// Rows of the hidden values start at whole 16 bytes of either form.
size_t hidden_bytes(size_t pairs, int hidden) { return pairs * (((size_t)hidden + 7) & ~(size_t)7) * 6; }

ScanArgs scan_args(const nerf_scan_cfg* c, const void* a, const void* x, const float* h0, const int32_t* offsets,
                   bool backward) {
    ScanArgs s{};
    s.rows = c->rows;
    s.n_seq = c->n_seq;
    s.len = offsets ? 0 : c->rows / c->n_seq;
    s.offsets = offsets;
    s.d = c->d;
    s.gates = c->gates;
    s.reverse = c->reverse != 0;
    s.mix = c->mix != 0;
    s.a = a;
    s.ld_a = c->ld_a ? c->ld_a : c->gates;
    s.x = x;
    s.ld_x = c->ld_x ? c->ld_x : c->d;
    s.h0 = h0;
    s.ld_h = c->ld_h ? c->ld_h : c->d;
    s.ld_dh = c->ld_dh ? c->ld_dh : c->d;
    s.p = scan_plan(elt_bytes(c->dtype), c->rows, c->n_seq, c->d, c->gates, backward);
    scan_plan_strides(s.p, c->d, c->gates, std::max(std::max(s.ld_a, s.ld_x), std::max(s.ld_h, s.ld_dh)));
    return s;
}

void scan_parts(ScanArgs& s, void* ws) {
    uint32_t* w = static_cast<uint32_t*>(ws);
    if (s.p.chunk) {
        const size_t each = (scan_chain_words(s.p) - 4) / 3;
        s.ticket = w;
        s.sum_a = w + 4;
        s.sum_b = s.sum_a + each;
        s.state = s.sum_b + each;
        w = s.state + each;
    }
    s.part_da = reinterpret_cast<float*>(w);
}

nerf_status check_list(const char* who, const nerf_tensor* list, int n) {
    NERF_REQUIRE(n >= 0 && n <= kMaxTensors, "%s: %d tensors", who, n);
    NERF_REQUIRE(n == 0 || list, "%s: list is NULL", who);
    int64_t left = kMaxRows << 10;  // elements of all tensors
    for (int i = 0; i < n; ++i) {
        const nerf_tensor& t = list[i];
        NERF_REQUIRE(t.dtype == NERF_F32 || t.dtype == NERF_BF16, "%s: tensor %d: dtype %d", who, i, t.dtype);
        NERF_REQUIRE(t.count >= 0 && t.count <= left, "%s: tensor %d: %lld elements", who, i, (long long)t.count);
        NERF_REQUIRE(t.count == 0 || t.src, "%s: tensor %d is NULL", who, i);
        NERF_REQUIRE(aligned(t.src, elt_bytes(t.dtype)), "%s: tensor %d is misaligned", who, i);
        left -= t.count;
    }
    return NERF_OK;
}

// Bytes that a list reads or writes.
struct Range {
    uintptr_t lo, hi;
    bool written;
};

// Whether a written range overlaps any other (tensors scaled in place have one
// range); -1 without memory for the look.
int overlaps(const nerf_tensor* list, int n) {
    constexpr int kLocal = 128;
    Range local[kLocal];
    Range* r = 2 * (int64_t)n <= kLocal ? local : static_cast<Range*>(std::malloc(2 * (size_t)n * sizeof(Range)));
    if (!r) return -1;
    int m = 0;
    for (int i = 0; i < n; ++i) {
        if (list[i].count == 0) continue;
        const size_t bytes = (size_t)list[i].count * elt_bytes(list[i].dtype);
        const uintptr_t s = reinterpret_cast<uintptr_t>(list[i].src), d = reinterpret_cast<uintptr_t>(list[i].dst);
        r[m++] = {d, d + bytes, true};
        if (s != d) r[m++] = {s, s + bytes, false};
    }
    std::sort(r, r + m, [](const Range& a, const Range& b) { return a.lo < b.lo; });
    uintptr_t any = 0, written = 0;  // ends of the ranges so far
    int found = 0;
    for (int i = 0; i < m && !found; ++i) {
        found = r[i].lo < (r[i].written ? any : written);
        any = std::max(any, r[i].hi);
        if (r[i].written) written = std::max(written, r[i].hi);
    }
    if (r != local) std::free(r);
    return found;
}

}  // namespace

extern "C" {

nerf_status nerf_route_gate(const void* logits, int dtype, int64_t ld_logits, int64_t n, int n_experts, int k,
                            int renorm, int32_t* ids, float* weights, void* stream) {
    const char* who = "nerf_route_gate";
    const nerf_status st = check_gate(who, dtype, ld_logits, n, n_experts, k);
    if (st != NERF_OK || n == 0) return st;
    NERF_REQUIRE(logits && ids && weights, "%s: NULL input or output", who);
    NERF_REQUIRE(aligned(logits, elt_bytes(dtype)) && aligned(ids, 4) && aligned(weights, 4), "%s: misaligned pointer",
                 who);
    GateArgs a{};
    a.logits = logits;
    a.ld = ld_logits ? ld_logits : n_experts;
    a.n = n;
    a.n_experts = n_experts;
    a.k = k;
    a.renorm = renorm != 0;
    a.ids = ids;
    a.weights = weights;
    (void)hipGetLastError();
    launch_gate(dtype == NERF_BF16, a, as_stream(stream));
    return check_launch(who);
}

nerf_status nerf_route_gate_grad(const float* dweights, const void* logits, int dtype, int64_t ld_logits, int64_t n,
                                 int n_experts, int k, int renorm, const int32_t* ids, const float* weights,
                                 void* dlogits, int64_t ld_dlogits, void* stream) {
    const char* who = "nerf_route_gate_grad";
    const nerf_status st = check_gate(who, dtype, ld_logits, n, n_experts, k);
    if (st != NERF_OK) return st;
    NERF_REQUIRE(ld_dlogits == 0 || ld_dlogits >= n_experts, "%s: row stride %lld below the experts", who,
                 (long long)ld_dlogits);
    if (n == 0) return NERF_OK;
    NERF_REQUIRE(dweights && ids && weights && dlogits, "%s: NULL input or output", who);
    NERF_REQUIRE(logits || renorm, "%s: logits are NULL", who);
    NERF_REQUIRE(dlogits != logits, "%s: dlogits must not overlap logits", who);
    const int b = elt_bytes(dtype);
    NERF_REQUIRE(aligned(logits, b) && aligned(dlogits, b) && aligned(dweights, 4) && aligned(ids, 4) &&
                     aligned(weights, 4),
                 "%s: misaligned pointer", who);
    GateArgs a{};
    a.logits = logits;
    a.ld = ld_logits ? ld_logits : n_experts;
    a.n = n;
    a.n_experts = n_experts;
    a.k = k;
    a.renorm = renorm != 0;
    a.ids = const_cast<int32_t*>(ids);
    a.weights = const_cast<float*>(weights);
    a.dweights = dweights;
    a.dlogits = dlogits;
    a.ld_d = ld_dlogits ? ld_dlogits : n_experts;
    (void)hipGetLastError();
    launch_gate_grad(dtype == NERF_BF16, a, as_stream(stream));
    return check_launch(who);
}

// The sorted pairs, the hidden values (float32, or three bfloat16 parts) and the
// outputs per pair.
size_t nerf_routed_mlp_workspace_size(int64_t n, int k, int hidden, int d_out) {
    if (n < 1 || k < 1 || n > NERF_FEW_PAIRS / k || hidden < 1 || hidden > kMaxWidth || d_out < 1 || d_out > kMaxWidth)
        return 0;
    const size_t pairs = (size_t)n * (size_t)k;
    return kMlpPlanBytes + hidden_bytes(pairs, hidden) + pairs * (size_t)d_out * sizeof(float);
}

nerf_status nerf_routed_mlp(const nerf_routed_layer* L, const void* x, const int32_t* ids, const float* weights,
                            int64_t n, const void* w1, const float* b1, const void* w2, const float* b2, void* out,
                            void* workspace, size_t workspace_bytes, void* stream) {
    const char* who = "nerf_routed_mlp";
    NERF_REQUIRE(L, "%s: layer is NULL", who);
    NERF_REQUIRE(L->dtype == NERF_F32 || L->dtype == NERF_BF16, "%s: dtype %d", who, L->dtype);
    NERF_REQUIRE(L->act == NERF_ACT_NONE || L->act == NERF_ACT_RELU || L->act == NERF_ACT_GATED, "%s: act %d", who,
                 L->act);
    NERF_REQUIRE(L->d_in >= 1 && L->d_in <= kMaxWidth && L->hidden >= 1 && L->hidden <= kMaxWidth && L->d_out >= 1 &&
                     L->d_out <= kMaxWidth,
                 "%s: widths %d -> %d -> %d outside 1..%d", who, L->d_in, L->hidden, L->d_out, kMaxWidth);
    NERF_REQUIRE(L->n_experts >= 1, "%s: n_experts %d < 1", who, L->n_experts);
    NERF_REQUIRE(L->k >= 1 && L->k <= NERF_MAX_CHOICES, "%s: k %d outside 1..%d", who, L->k, NERF_MAX_CHOICES);
    NERF_REQUIRE(L->ld_x == 0 || L->ld_x >= L->d_in, "%s: ld_x %lld below d_in", who, (long long)L->ld_x);
    NERF_REQUIRE(L->ld_out == 0 || L->ld_out >= L->d_out, "%s: ld_out %lld below d_out", who, (long long)L->ld_out);
    NERF_REQUIRE(n >= 0, "%s: n %lld < 0", who, (long long)n);
    if (L->n_experts > NERF_MAX_EXPERTS)
        return nerf_fail(NERF_ERR_UNSUPPORTED, "%s: n_experts %d above %d", who, L->n_experts, NERF_MAX_EXPERTS);
    if (n > NERF_FEW_PAIRS / L->k)
        return nerf_fail(NERF_ERR_UNSUPPORTED, "%s: %lld x %d pairs (at most %d: nerf_expert_linear takes more%s)", who,
                         (long long)n, L->k, NERF_FEW_PAIRS,
                         L->act == NERF_ACT_GATED ? ", but has no gated hidden layer: its caller gates in between" : "");
    if (n == 0) return NERF_OK;
    const int b = elt_bytes(L->dtype);
    NERF_REQUIRE(x && ids && w1 && w2 && out, "%s: NULL input or output", who);
    NERF_REQUIRE(aligned(x, b) && aligned(w1, b) && aligned(w2, b) && aligned(out, b) && aligned(ids, 4) &&
                     aligned(weights, 4) && aligned(b1, 4) && aligned(b2, 4),
                 "%s: misaligned pointer", who);
    MlpArgs a{};
    a.n = (int)n;
    a.k = L->k;
    a.n_experts = L->n_experts;
    a.d_in = L->d_in;
    a.hidden = L->hidden;
    a.d_out = L->d_out;
    a.act = L->act;
    a.x = x;
    a.ld_x = L->ld_x ? L->ld_x : L->d_in;
    a.ids = ids;
    a.weights = weights;
    a.w1 = w1;
    a.b1 = b1;
    a.w2 = w2;
    a.b2 = b2;
    a.ld_h = (L->hidden + 7) & ~7;
    a.out = out;
    a.ld_out = L->ld_out ? L->ld_out : L->d_out;
    Workspace ws;
    const nerf_status st = ws.take(who, workspace, workspace_bytes,
                                   nerf_routed_mlp_workspace_size(n, L->k, L->hidden, L->d_out), stream);
    if (st != NERF_OK) return st;
    char* const p = static_cast<char*>(ws.p);
    a.plan = p;
    a.h = reinterpret_cast<float*>(p + kMlpPlanBytes);
    a.y = reinterpret_cast<float*>(p + kMlpPlanBytes + hidden_bytes((size_t)n * L->k, L->hidden));
    (void)hipGetLastError();
    launch_routed_mlp(L->dtype == NERF_BF16, a, as_stream(stream));
    return ws.release(who, check_launch(who), stream);
}

size_t nerf_scan_workspace_size(int64_t rows, int64_t n_seq, int d, int gates, int backward) {
    if (rows < 0 || rows > kMaxRows || n_seq < 1 || n_seq >= kMaxRows || d < 1 || d > kMaxWidth || gates < 1 ||
        gates > d || d % gates)
        return 0;
    // (of either type of rows)
    const bool b = backward != 0;
    return std::max(scan_workspace(scan_plan(2, rows, n_seq, d, gates, b), rows, gates, b),
                    scan_workspace(scan_plan(4, rows, n_seq, d, gates, b), rows, gates, b));
}

nerf_status nerf_scan(const nerf_scan_cfg* cfg, const void* a, const void* x, const int32_t* offsets, const float* h0,
                      void* h, float* h_last, void* workspace, size_t workspace_bytes, void* stream) {
    const char* who = "nerf_scan";
    nerf_status st = check_scan(who, cfg, offsets != nullptr, false);
    if (st != NERF_OK || cfg->n_seq == 0) return st;
    const int b = elt_bytes(cfg->dtype);
    NERF_REQUIRE(cfg->rows == 0 || (a && x && h), "%s: NULL input or output", who);
    NERF_REQUIRE(cfg->rows == 0 || (h != x && h != a), "%s: h must not overlap a or x", who);
    NERF_REQUIRE(aligned(a, elt_bytes(cfg->gate_dtype)) && aligned(x, b) && aligned(h, b) && aligned(offsets, 4) &&
                     aligned(h0, 4) && aligned(h_last, 4),
                 "%s: misaligned pointer", who);
    ScanArgs s = scan_args(cfg, a, x, h0, offsets, false);
    s.h = h;
    s.h_last = h_last;
    Workspace ws;
    st = ws.take(who, workspace, workspace_bytes, scan_workspace(s.p, s.rows, s.gates, false), stream);
    if (st != NERF_OK) return st;
    scan_parts(s, ws.p);
    (void)hipGetLastError();
    launch_scan(cfg->dtype == NERF_BF16, cfg->gate_dtype == NERF_BF16, s, as_stream(stream));
    return ws.release(who, check_launch(who), stream);
}

nerf_status nerf_scan_grad(const nerf_scan_cfg* cfg, const void* dh, const float* dh_last, const void* a,
                           const void* x, const void* h, const float* h0, const int32_t* offsets, void* da, void* dx,
                           float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
    const char* who = "nerf_scan_grad";
    nerf_status st = check_scan(who, cfg, offsets != nullptr, true);
    if (st != NERF_OK || cfg->n_seq == 0) return st;
    const int b = elt_bytes(cfg->dtype), ba = elt_bytes(cfg->gate_dtype);
    NERF_REQUIRE(cfg->rows == 0 || (dh && a && h && da && dx), "%s: NULL input or output", who);
    NERF_REQUIRE(cfg->rows == 0 || x || !cfg->mix, "%s: x is NULL", who);
    NERF_REQUIRE(cfg->rows == 0 || (da != a && da != dh && da != h && da != x && dx != a && dx != dh && dx != h &&
                                    dx != x && da != dx),
                 "%s: da and dx must not overlap each other or an input", who);
    NERF_REQUIRE(aligned(dh, b) && aligned(a, ba) && aligned(x, b) && aligned(h, b) && aligned(da, ba) &&
                     aligned(dx, b) && aligned(offsets, 4) && aligned(h0, 4) && aligned(dh_last, 4) && aligned(dh0, 4),
                 "%s: misaligned pointer", who);
    ScanArgs s = scan_args(cfg, a, x, h0, offsets, true);
    s.h = const_cast<void*>(h);
    s.dh = dh;
    s.dh_last = dh_last;
    s.da = da;
    s.dx = dx;
    s.dh0 = dh0;
    Workspace ws;
    st = ws.take(who, workspace, workspace_bytes, scan_workspace(s.p, s.rows, s.gates, true), stream);
    if (st != NERF_OK) return st;
    scan_parts(s, ws.p);
    (void)hipGetLastError();
    launch_scan_grad(cfg->dtype == NERF_BF16, cfg->gate_dtype == NERF_BF16, s, as_stream(stream));
    return ws.release(who, check_launch(who), stream);
}

size_t nerf_grad_norm_workspace_size(const nerf_tensor* list, int n) {
    if (check_list("nerf_grad_norm_workspace_size", list, n) != NERF_OK) return 0;
    return grad_norm_partials(list, n) * sizeof(double);
}

nerf_status nerf_grad_norm(const nerf_tensor* list, int n, float* norm, void* workspace, size_t workspace_bytes,
                           void* stream) {
    const char* who = "nerf_grad_norm";
    nerf_status st = check_list(who, list, n);
    if (st != NERF_OK) return st;
    NERF_REQUIRE(norm && aligned(norm, 4), "%s: NULL or misaligned norm", who);
    Workspace ws;
    st = ws.take(who, workspace, workspace_bytes, grad_norm_partials(list, n) * sizeof(double), stream);
    if (st != NERF_OK) return st;
    (void)hipGetLastError();
    launch_grad_norm(list, n, static_cast<double*>(ws.p), norm, as_stream(stream));
    return ws.release(who, check_launch(who), stream);
}

nerf_status nerf_grad_clip(const nerf_tensor* list, int n, float max_norm, float* norm, void* workspace,
                           size_t workspace_bytes, void* stream) {
    const char* who = "nerf_grad_clip";
    nerf_status st = check_list(who, list, n);
    if (st != NERF_OK) return st;
    NERF_REQUIRE(norm && aligned(norm, 4), "%s: NULL or misaligned norm", who);
    NERF_REQUIRE(max_norm >= 0.0f, "%s: max_norm %g", who, (double)max_norm);
    for (int i = 0; i < n; ++i) {
        NERF_REQUIRE(list[i].count == 0 || list[i].dst, "%s: tensor %d has no destination", who, i);
        NERF_REQUIRE(aligned(list[i].dst, elt_bytes(list[i].dtype)), "%s: tensor %d is misaligned", who, i);
    }
    const int bad = overlaps(list, n);
    NERF_REQUIRE(bad != 1, "%s: a destination overlaps another tensor", who);
    if (bad < 0) return nerf_fail(NERF_ERR_WORKSPACE, "%s: no host memory to check %d tensors", who, n);
    Workspace ws;
    st = ws.take(who, workspace, workspace_bytes, grad_norm_partials(list, n) * sizeof(double), stream);
    if (st != NERF_OK) return st;
    (void)hipGetLastError();
    launch_grad_clip(list, n, max_norm, static_cast<double*>(ws.p), norm, as_stream(stream));
    return ws.release(who, check_launch(who), stream);
}

}  // extern "C"
