// Host-side checks of the streaming-field entry points under AddressSanitizer and
// UndefinedBehaviorSanitizer, without a GPU: the real argument checks, workspace
// code and plans of the recurrence (fields_abi.cpp, scan_plan.cpp) with stand-ins
// for the launchers, which touch every byte of a workspace that the kernels would,
// and for the HIP calls, whose failures can be forced.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "abi_util.hpp"
#include "fields.hpp"
#include "nerf_mi355x.h"

static int g_launches = 0, g_live_allocs = 0, g_checks = 0;
static bool g_fail_malloc = false, g_pending = false, g_fail_launch = false;
static size_t g_last_alloc = 0;
static char g_error[512];

extern "C" {
hipError_t hipMallocAsync(void** p, size_t bytes, hipStream_t) {
    if (g_fail_malloc) return hipErrorOutOfMemory;
    *p = std::malloc(bytes);  // (not rounded up: the sanitizer sees a byte too many)
    g_last_alloc = bytes;
    ++g_live_allocs;
    return hipSuccess;
}
hipError_t hipFreeAsync(void* p, hipStream_t) {
    std::free(p);
    --g_live_allocs;
    return hipSuccess;
}
hipError_t hipGetLastError(void) {
    const hipError_t e = g_pending ? hipErrorLaunchFailure : hipSuccess;
    g_pending = false;
    return e;
}
const char* hipGetErrorString(hipError_t e) { return e == hipSuccess ? "no error" : "forced error"; }
}

nerf_status nerf_fail(nerf_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(g_error, sizeof(g_error), fmt, ap);
    va_end(ap);
    return s;
}

#define CHECK(cond)                                                                                  \
    do {                                                                                             \
        ++g_checks;                                                                                  \
        if (!(cond)) {                                                                               \
            std::fprintf(stderr, "FAILED %s:%d: %s (%s)\n", __FILE__, __LINE__, #cond, g_error);     \
            std::exit(1);                                                                            \
        }                                                                                            \
    } while (0)

static void launched() {
    ++g_launches;
    if (g_fail_launch) {
        g_pending = true;
        g_fail_launch = false;
    }
}

static bool power_of_two(int v) { return v > 0 && (v & (v - 1)) == 0; }

static void check_plan(const nerf::ScanArgs& a, bool backward) {
    const nerf::ScanPlan& p = a.p;
    CHECK(power_of_two(p.cl) && p.cl <= 64 && power_of_two(p.lg) && p.lg <= p.cl && p.parts >= 1);
    CHECK(p.waves == 1 || p.waves == 4 || p.waves == 8);
    const int m = a.d / a.gates, V = p.vec ? 4 : 1;
    if (p.grouped) {  // every gate has lanes for all its channels, every block whole gates
        CHECK(!p.vec || m >= V);
        CHECK((int64_t)p.parts * p.lg * V >= m && (p.parts == 1 || p.lg == 64));
        CHECK((int64_t)p.blocks / p.parts * (p.cl / p.lg) >= a.gates);
    } else {
        CHECK(!p.vec || a.d >= V);
        CHECK((int64_t)p.blocks * p.cl * V >= a.d);
    }
    // a wave's tile lies within 32-bit byte offsets
    int64_t ld = a.ld_a > a.ld_x ? a.ld_a : a.ld_x;
    ld = a.ld_h > ld ? a.ld_h : ld;
    if (backward && a.ld_dh > ld) ld = a.ld_dh;
    CHECK((64 / p.cl * 8 * ld + a.d) * 4 < (int64_t)1 << 32);
    CHECK(!p.chunk || (!p.alone && a.n_seq < nerf::kScanMaxSplit));
    if (p.chunk) {
        CHECK(p.slots >= a.rows / p.chunk + a.n_seq && p.chunk == p.waves * (64 / p.cl) * (backward ? 4 : 8));
        const size_t words = (size_t)p.slots * p.blocks * p.cl * V;
        CHECK(reinterpret_cast<uintptr_t>(a.ticket) % 16 == 0 && reinterpret_cast<uintptr_t>(a.sum_a) % 16 == 0);
        CHECK(reinterpret_cast<uintptr_t>(a.sum_b) % 16 == 0 && reinterpret_cast<uintptr_t>(a.state) % 16 == 0);
        std::memset(a.ticket, 0, nerf::scan_chain_words(p) * 4);
        std::memset(a.sum_a, 0, words * 4);
        std::memset(a.sum_b, 0, words * 4);
        std::memset(a.state, 0, words * 4);
    }
    if (backward && p.parts > 1 && a.rows > 0) std::memset(a.part_da, 0, (size_t)p.parts * a.rows * a.gates * 4);
    launched();
}

namespace nerf {
void launch_gate(bool, const GateArgs& a, hipStream_t) {
    CHECK(a.ld >= a.n_experts && a.k <= a.n_experts);
    launched();
}
void launch_gate_grad(bool, const GateArgs& a, hipStream_t) {
    CHECK(a.ld >= a.n_experts && a.ld_d >= a.n_experts && (a.logits || a.renorm));
    launched();
}
void launch_routed_mlp(bool, const MlpArgs& a, hipStream_t) {
    CHECK(a.n * a.k <= NERF_FEW_PAIRS && a.ld_h % 8 == 0 && a.ld_h >= a.hidden);
    CHECK(reinterpret_cast<uintptr_t>(a.h) % 16 == 0 && reinterpret_cast<uintptr_t>(a.plan) % 16 == 0);
    std::memset(a.plan, 0, kMlpPlanBytes);
    std::memset(a.h, 0, (size_t)a.n * a.k * a.ld_h * 6);
    std::memset(a.y, 0, (size_t)a.n * a.k * a.d_out * 4);
    launched();
}
void launch_scan(bool bf16, bool gate_bf16, const ScanArgs& a, hipStream_t) {
    CHECK(bf16 || !gate_bf16);
    check_plan(a, false);
}
void launch_scan_grad(bool bf16, bool gate_bf16, const ScanArgs& a, hipStream_t) {
    CHECK(bf16 || !gate_bf16);
    check_plan(a, true);
}
size_t grad_norm_partials(const nerf_tensor* list, int n) {
    size_t used = 1;
    for (int i = 0; i < n; ++i) used += (size_t)(list[i].count > 0);
    return used;
}
void launch_grad_norm(const nerf_tensor* list, int n, double* partials, float*, hipStream_t) {
    std::memset(partials, 0, grad_norm_partials(list, n) * sizeof(double));
    launched();
}
void launch_grad_clip(const nerf_tensor* list, int n, float, double* partials, float*, hipStream_t) {
    std::memset(partials, 0, grad_norm_partials(list, n) * sizeof(double));
    launched();
}
}  // namespace nerf

static float g_buf[64] __attribute__((aligned(256)));
static int32_t g_int[64] __attribute__((aligned(256)));

int main() {
    float* f = g_buf;
    int32_t* i = g_int;
    // gate
    for (int dt = 0; dt < 2; ++dt)
        for (int64_t ld : {(int64_t)0, (int64_t)70}) {
            CHECK(nerf_route_gate(f, dt, ld, 5, 64, 64, 1, i, f, nullptr) == NERF_OK);
            CHECK(nerf_route_gate_grad(f, nullptr, dt, ld, 5, 64, 3, 1, i, f, f, ld, nullptr) == NERF_OK);
            CHECK(nerf_route_gate_grad(f, f + 8, dt, ld, 5, 64, 3, 0, i, f, f, ld, nullptr) == NERF_OK);
        }
    // layer: every workspace byte, with and without one of the caller's
    for (int n : {1, 8, 64, 65, 512})
        for (int hidden : {1, 7, 8, 513}) {
            const nerf_routed_layer L{NERF_BF16, 9, 16, hidden, 24, NERF_ACT_GATED, 1, 0, 0};
            CHECK(nerf_routed_mlp(&L, f, i, nullptr, n, f, f, f, f, f, nullptr, 0, nullptr) == NERF_OK);
            const size_t need = nerf_routed_mlp_workspace_size(n, 1, hidden, 24);
            CHECK(g_last_alloc == need && g_live_allocs == 0);
            void* own = std::aligned_alloc(16, (need + 15) / 16 * 16);
            CHECK(nerf_routed_mlp(&L, f, i, nullptr, n, f, f, f, f, f, own, need, nullptr) == NERF_OK);
            CHECK(nerf_routed_mlp(&L, f, i, nullptr, n, f, f, f, f, f, own, need - 1, nullptr) == NERF_ERR_WORKSPACE);
            std::free(own);
        }
    // recurrence: plans over its range
    for (int dt = 0; dt < 2; ++dt)
        for (int64_t rows : {0, 1, 7, 64, 1000, 5000, 200000})
            for (int64_t n : {1, 2, 7, 16, 255, 300, 5000})
                for (int d : {1, 2, 3, 4, 5, 16, 33, 63, 256, 257, 600, 1024, 1030})
                    for (int m : {1, 2, 3, 4, 5, 11, 33, 257, 515, 1030}) {
                        if (d % m) continue;
                        for (int64_t ld : {(int64_t)0, (int64_t)1 << 20, (int64_t)1 << 26}) {
                            nerf_scan_cfg c{dt, NERF_F32, d, d / m, 0, 1, rows, n, ld, ld, ld, ld};
                            const int before = g_launches;
                            CHECK(nerf_scan(&c, f, f + 8, i, nullptr, f + 16, nullptr, nullptr, 0, nullptr) == NERF_OK);
                            const size_t forward = g_last_alloc;
                            CHECK(nerf_scan_grad(&c, f, f, f + 8, f + 16, f + 24, f, i, f + 32, f + 40, f, nullptr, 0,
                                                 nullptr) == NERF_OK);
                            CHECK(g_launches == before + 2 && g_live_allocs == 0);
                            CHECK(nerf_scan_workspace_size(rows, n, d, d / m, 0) <= nerf_scan_workspace_size(rows, n, d, d / m, 1));
                            (void)forward;
                        }
                    }
    {
        // a workspace of exactly the size asked for, either type of rows
        for (int dt = 0; dt < 2; ++dt) {
            nerf_scan_cfg c{dt, NERF_F32, 600, 1, 0, 0, 90000, 1, 0, 0, 0, 0};
            const size_t need = nerf_scan_workspace_size(90000, 1, 600, 1, 1);
            CHECK(need > 0);
            void* own = std::aligned_alloc(16, (need + 15) / 16 * 16);
            CHECK(nerf_scan_grad(&c, f, f, f + 8, nullptr, f + 24, f, nullptr, f + 32, f + 40, f, own, need, nullptr) == NERF_OK);
            std::free(own);
        }
        nerf_scan_cfg c{NERF_F32, NERF_F32, 8, 8, 0, 0, 90000, 1, ((int64_t)1 << 26) + 1, 0, 0, 0};
        CHECK(nerf_scan(&c, f, f + 8, nullptr, nullptr, f + 16, nullptr, nullptr, 0, nullptr) == NERF_ERR_UNSUPPORTED);
        c.ld_a = 0;
        g_fail_malloc = true;
        int before = g_launches;
        CHECK(nerf_scan(&c, f, f + 8, nullptr, nullptr, f + 16, nullptr, nullptr, 0, nullptr) == NERF_ERR_WORKSPACE);
        CHECK(g_launches == before);
        g_fail_malloc = false;
        g_fail_launch = true;  // a failed launch is reported, and the workspace freed all the same
        CHECK(nerf_scan(&c, f, f + 8, nullptr, nullptr, f + 16, nullptr, nullptr, 0, nullptr) == NERF_ERR_HIP);
        CHECK(g_live_allocs == 0);
        g_pending = true;  // another call's error is not this one's
        CHECK(nerf_scan(&c, f, f + 8, nullptr, nullptr, f + 16, nullptr, nullptr, 0, nullptr) == NERF_OK);
    }
    // lists: short ones on the stack, long ones in host memory
    for (int n : {0, 1, 63, 64, 65, 200, 5000}) {
        nerf_tensor* list = new nerf_tensor[n + 1];
        for (int t = 0; t < n; ++t) {
            char* at = reinterpret_cast<char*>((uintptr_t)1 << 30) + 64 * ((t * 7919LL) % 10007);
            list[t] = nerf_tensor{at, t % 2 ? at : at + ((uintptr_t)1 << 32), t % 5 ? 16 : 0, t % 3 == 0, 0};
        }
        CHECK(nerf_grad_norm(list, n, f, nullptr, 0, nullptr) == NERF_OK);
        CHECK(nerf_grad_clip(list, n, 1.0f, f, nullptr, 0, nullptr) == NERF_OK);
        CHECK(g_live_allocs == 0);
        if (n > 63) {  // one element shared with the next tensor in memory
            list[1].count = 17;
            list[2] = list[1];
            list[2].src = list[2].dst = static_cast<char*>(list[1].dst) + 64;
            list[2].count = 1;
            CHECK(nerf_grad_clip(list, n, 1.0f, f, nullptr, 0, nullptr) == NERF_ERR_INVALID_ARGUMENT);
        }
        delete[] list;
    }
    std::printf("all %d checks passed\n", g_checks);
    return 0;
}
