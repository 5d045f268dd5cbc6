// Host-side checks of the routed-field and distillation entry points under
// AddressSanitizer and UndefinedBehaviorSanitizer, without a GPU: the real
// argument checks and workspace code (experts_abi.cpp) with stand-ins for the
// launchers, which only look at what they are given, and for the HIP calls,
// whose failures can be forced.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "abi_util.hpp"
#include "experts.hpp"
#include "nerf_mi355x.h"

static int g_launches = 0, g_live_allocs = 0, g_checks = 0;
static bool g_fail_malloc = false, g_pending = false, g_fail_launch = false;
static size_t g_last_alloc = 0;
static char g_error[512];

extern "C" {
hipError_t hipMallocAsync(void** p, size_t bytes, hipStream_t) {
    if (g_fail_malloc) return hipErrorOutOfMemory;
    *p = std::aligned_alloc(256, (bytes + 255) / 256 * 256);
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

namespace nerf {
void launch_route_plan(const int32_t*, int64_t pairs, int n_experts, int32_t*, int32_t*, int32_t*, int32_t* counts,
                       hipStream_t) {
    const int64_t nb = route_blocks(pairs);
    if (nb > 1) {  // the counts and totals the kernels write lie in the workspace
        CHECK(counts);
        std::memset(counts, 0, (size_t)(nb + 1) * (n_experts + 1) * sizeof(int32_t));
    }
    launched();
}
void launch_route_gather(bool, const RouteRows& r, hipStream_t) {
    CHECK(r.lda >= r.d);
    launched();
}
void launch_route_combine(bool, const RouteRows& r, hipStream_t) {
    CHECK(r.ldo >= r.d);
    launched();
}
void launch_route_combine_grad(bool, const RouteRows& r, hipStream_t) {
    CHECK(r.lda >= r.d);
    launched();
}
int64_t expert_grad_chunk(int64_t slots, int, int, int) { return slots > 1000 ? 512 : 0; }
static void check_args(const ExpertArgs& a) {
    CHECK(a.ld_x >= a.d_in);
    for (int64_t p : {(int64_t)0, (int64_t)1, (int64_t)12345, ((int64_t)1 << 31) - 1}) {
        // the quotient by multiplication is exact
        const int64_t k = ((int64_t)1 << a.k_shift) / a.k_mul;
        bool some = false;
        for (int64_t c = k > 1 ? k - 1 : 1; c <= k + 1; ++c) some = some || (int64_t)(((uint64_t)p * a.k_mul) >> a.k_shift) == p / c;
        CHECK(some);
    }
    launched();
}
void launch_expert_linear(bool, const ExpertArgs& a, hipStream_t) { check_args(a); }
void launch_expert_grad_x(bool, const ExpertArgs& a, hipStream_t) { check_args(a); }
void launch_expert_grad_w(bool, const ExpertArgs& a, hipStream_t) {
    if (a.chunk) {  // partial sums of every range lie in the workspace
        const int64_t items = a.slots / a.chunk + a.n_experts;
        CHECK(a.part && a.bpart);
        std::memset(a.part, 0, (size_t)items * a.d_in * a.d_out * 4);
        std::memset(a.bpart, 0, (size_t)items * a.d_out * 4);
    }
    check_args(a);
}
int distill_splits(int64_t n, int64_t classes) { return n < 8 && classes > 1000 ? 16 : 1; }
void launch_distill(bool, const DistillArgs& a, hipStream_t) {
    const int s = distill_splits(a.n, a.classes);
    if (s > 1) std::memset(a.part, 0, (size_t)a.n * s * 8);
    launched();
}
void launch_distill_grad(bool, const DistillArgs& a, hipStream_t) {
    CHECK(a.lse && a.grad);
    launched();
}
}  // namespace nerf

static float g_buf[64] __attribute__((aligned(256)));
static int32_t g_int[64] __attribute__((aligned(256)));

int main() {
    float* f = g_buf;
    int32_t* i = g_int;
    void* own = nullptr;
    // plans: with and without a workspace of the caller's
    CHECK(nerf_route_plan(i, 100, 2, 8, i, i, i, nullptr, 0, nullptr) == NERF_OK && g_launches == 1);
    CHECK(g_live_allocs == 0);  // small plans need none
    CHECK(nerf_route_plan(i, 200000, 2, 4096, i, i, i, nullptr, 0, nullptr) == NERF_OK && g_live_allocs == 0);
    const size_t need = nerf_route_workspace_size(200000, 2, 4096);
    CHECK(need == g_last_alloc);
    own = std::aligned_alloc(256, (need + 255) / 256 * 256);
    CHECK(nerf_route_plan(i, 200000, 2, 4096, i, i, i, own, need, nullptr) == NERF_OK);
    CHECK(nerf_route_plan(i, 200000, 2, 4096, i, i, i, own, need - 1, nullptr) == NERF_ERR_WORKSPACE);
    std::free(own);
    int before = g_launches;
    g_fail_malloc = true;
    CHECK(nerf_route_plan(i, 200000, 2, 4096, i, i, i, nullptr, 0, nullptr) == NERF_ERR_WORKSPACE);
    g_fail_malloc = false;
    CHECK(g_launches == before);
    g_fail_launch = true;  // a failed launch is reported, and the workspace freed all the same
    CHECK(nerf_route_plan(i, 200000, 2, 4096, i, i, i, nullptr, 0, nullptr) == NERF_ERR_HIP && g_live_allocs == 0);
    g_pending = true;  // another call's error is not this one's
    CHECK(nerf_route_plan(i, 100, 2, 8, i, i, i, nullptr, 0, nullptr) == NERF_OK);
    // rows
    for (int dt = 0; dt < 2; ++dt)
        for (int64_t ld : {(int64_t)0, (int64_t)9}) {
            CHECK(nerf_route_gather(f, dt, ld, 5, 2, 9, 3, i, i, f, nullptr) == NERF_OK);
            CHECK(nerf_route_combine(f, dt, 5, 2, 9, 3, i, i, nullptr, f, ld, nullptr) == NERF_OK);
            CHECK(nerf_route_combine_grad(f, ld, f, dt, 5, 2, 9, 3, i, i, f, f, nullptr, nullptr) == NERF_OK);
        }
    // layers: every k, every workspace size
    for (int k = 1; k <= NERF_MAX_CHOICES; ++k) {
        nerf_expert_layer L{NERF_BF16, 4, 16, 24, 0, k, 10, 0, 0};
        CHECK(nerf_expert_linear(&L, f, f, f, i, i, 10 * k, f, nullptr) == NERF_OK);
    }
    for (int64_t slots : {(int64_t)1, (int64_t)1000, (int64_t)1001, (int64_t)5000}) {
        nerf_expert_layer L{NERF_F32, 4, 16, 24, 0, 0, slots, 0, 0};
        CHECK(nerf_expert_linear_grad(&L, f, f, f, i, nullptr, slots, f, f, f, nullptr, 0, nullptr) == NERF_OK);
        CHECK(nerf_expert_linear_grad(&L, f, f, f, i, nullptr, slots, nullptr, f, nullptr, nullptr, 0, nullptr) ==
              NERF_OK);
        CHECK(g_live_allocs == 0);
        g_fail_launch = true;
        CHECK(nerf_expert_linear_grad(&L, f, f, f, i, nullptr, slots, f, f, f, nullptr, 0, nullptr) == NERF_ERR_HIP);
        CHECK(g_live_allocs == 0);
    }
    // distillation
    CHECK(nerf_distill_topk(f, 1, 0, 3, 5000, f, i, 4, 2.0f, nullptr, f + 8, nullptr, nullptr, 0, nullptr, 0, nullptr) ==
          NERF_OK);
    CHECK(g_live_allocs == 0);
    CHECK(nerf_distill_topk(f, 0, 0, 3000, 50, f, i, 4, 2.0f, f, f + 8, f, f + 16, 0, nullptr, 0, nullptr) == NERF_OK);
    CHECK(nerf_distill_topk_grad(f, 0, 60, 3000, 50, f, i, 4, 2.0f, f, f, f + 16, 70, nullptr) == NERF_OK);
    CHECK(nerf_distill_topk_grad(f, 0, 60, 3000, 50, f, i, 4, 2.0f, f, f, f, 70, nullptr) == NERF_ERR_INVALID_ARGUMENT);
    std::printf("all %d checks passed\n", g_checks);
    return 0;
}
