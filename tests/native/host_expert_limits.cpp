// Host-side checks of what the routed-field entry points hand to the launchers,
// without a GPU: the exact quotient that turns pairs into samples, and how large
// calls may be.  The real argument checks (experts_abi.cpp) with stand-ins for the
// launchers and HIP calls; nothing is dereferenced.
#include <hip/hip_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstdlib>

#include "abi_util.hpp"
#include "experts.hpp"
#include "nerf_mi355x.h"

extern "C" {
hipError_t hipMallocAsync(void** p, size_t, hipStream_t) {
    *p = reinterpret_cast<void*>(4096);
    return hipSuccess;
}
hipError_t hipFreeAsync(void*, hipStream_t) { return hipSuccess; }
hipError_t hipGetLastError(void) { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return ""; }
}

static char g_error[512];
nerf_status nerf_fail(nerf_status s, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    std::vsnprintf(g_error, sizeof(g_error), fmt, ap);
    va_end(ap);
    return s;
}

static long g_checks = 0;
#define CHECK(cond)                                                                              \
    do {                                                                                         \
        ++g_checks;                                                                              \
        if (!(cond)) {                                                                           \
            std::fprintf(stderr, "FAILED %s:%d: %s (%s)\n", __FILE__, __LINE__, #cond, g_error); \
            std::exit(1);                                                                        \
        }                                                                                        \
    } while (0)

static nerf::ExpertArgs g_args;
static int g_launches = 0;
namespace nerf {
void launch_route_plan(const int32_t*, int64_t, int, int32_t*, int32_t*, int32_t*, int32_t*, hipStream_t) {}
void launch_route_gather(bool, const RouteRows&, hipStream_t) {}
void launch_route_combine(bool, const RouteRows&, hipStream_t) {}
void launch_route_combine_grad(bool, const RouteRows&, hipStream_t) {}
int64_t expert_grad_chunk(int64_t, int, int, int) { return 0; }
void launch_expert_linear(bool, const ExpertArgs& a, hipStream_t) { g_args = a, ++g_launches; }
void launch_expert_grad_x(bool, const ExpertArgs& a, hipStream_t) { g_args = a, ++g_launches; }
void launch_expert_grad_w(bool, const ExpertArgs& a, hipStream_t) { g_args = a, ++g_launches; }
int distill_splits(int64_t, int64_t) { return 1; }
void launch_distill(bool, const DistillArgs&, hipStream_t) { ++g_launches; }
void launch_distill_grad(bool, const DistillArgs&, hipStream_t) { ++g_launches; }
}  // namespace nerf

static float* const F = reinterpret_cast<float*>(4096);
static int32_t* const I = reinterpret_cast<int32_t*>(4096);

static nerf_status forward(int dtype, int64_t slots, int experts, int d_in, int d_out, int k, const int32_t* order) {
    nerf_expert_layer L{dtype, experts, d_in, d_out, 0, k, slots, 0, 0};
    return nerf_expert_linear(&L, F, F, F, I, order, slots, F, nullptr);
}
static nerf_status backward(int dtype, int64_t slots, int experts, int d_in, int d_out) {
    nerf_expert_layer L{dtype, experts, d_in, d_out, 0, 1, slots, 0, 0};
    return nerf_expert_linear_grad(&L, F, F, F, I, nullptr, slots, F, F, F, nullptr, 0, nullptr);
}

int main() {
    // pair / k by multiplication: exact for each k at and around its multiples, to the last pair
    for (int64_t k = 1; k <= NERF_MAX_CHOICES; ++k) {
        CHECK(forward(NERF_BF16, 10 * k, 4, 16, 24, (int)k, I) == NERF_OK);
        const uint64_t mul = g_args.k_mul;
        const int shift = g_args.k_shift;
        const int64_t last = ((int64_t)1 << 31) - 1;
        auto exact = [&](int64_t p) { return p < 0 || p > last || (int64_t)(((uint64_t)p * mul) >> shift) == p / k; };
        for (int64_t m = 0; m <= 4096; ++m)
            for (int64_t d = -1; d <= 1; ++d) {
                CHECK(exact(m * k + d));                                  // the first multiples
                CHECK(exact((last / k - m) * k + d));                     // the last ones
                CHECK(exact((last / k * m >> 12) * k + d));               // and others between
            }
        CHECK(exact(last));
    }
    CHECK(forward(NERF_BF16, 10, 4, 16, 24, 7, nullptr) == NERF_OK);  // without an order a slot is its own row
    for (int64_t p : {(int64_t)0, (int64_t)1, (int64_t)7, ((int64_t)1 << 31) - 1})
        CHECK((int64_t)(((uint64_t)p * g_args.k_mul) >> g_args.k_shift) == p);

    // sizes that fit the card: none is refused
    int n = 0;
    for (int dt : {NERF_F32, NERF_BF16})
        for (int64_t slots : {(int64_t)1 << 20, (int64_t)1 << 22, (int64_t)5000000, (int64_t)1 << 24, (int64_t)1 << 27, (int64_t)1 << 30})
            for (int d : {1, 8, 32, 64, 65, 256, 1024, 4096, 16384, 65536})
                for (int e : {1, 64, 4096}) {
                    const double bytes = (double)(slots * (8 + d)) * (dt == NERF_F32 ? 4 : 2);
                    if (bytes > 250e9) continue;
                    CHECK(forward(dt, slots, e, 8, d, 1, nullptr) == NERF_OK);
                    CHECK(forward(dt, slots, e, d, 8, 1, nullptr) == NERF_OK);
                    if ((double)e * d * 8 * 4 < 20e9) CHECK(backward(dt, slots, e, d, 8) == NERF_OK);
                    ++n;
                }
    CHECK(n > 150);
    CHECK(forward(NERF_BF16, ((int64_t)1 << 31) - 1, 1, 8, 8, 1, nullptr) == NERF_ERR_UNSUPPORTED);
    // logits of many short rows and of few long ones
    for (int64_t rows : {(int64_t)1, (int64_t)1 << 20, (int64_t)16777216, (int64_t)100000000, (int64_t)1 << 32})
        for (int64_t classes : {(int64_t)1, (int64_t)10, (int64_t)1000, (int64_t)128000, ((int64_t)1 << 31) - 1}) {
            if ((double)rows * (double)classes * 2 > 250e9) continue;
            CHECK(nerf_distill_topk(F, NERF_BF16, 0, rows, classes, F, I, 1, 1.0f, nullptr, F, F, nullptr, 0, F, SIZE_MAX,
                                    nullptr) == NERF_OK);
            CHECK(nerf_distill_topk_grad(F, NERF_BF16, 0, rows, classes, F, I, 1, 1.0f, nullptr, F, F + 4, 0, nullptr) ==
                  NERF_OK);
        }
    CHECK(nerf_distill_topk_grad(F, NERF_BF16, 0, (int64_t)1 << 30, 4096, F, I, 1, 1.0f, nullptr, F, F + 4, 0, nullptr) ==
          NERF_ERR_UNSUPPORTED);
    std::printf("all %ld checks passed\n", g_checks);
    return 0;
}
