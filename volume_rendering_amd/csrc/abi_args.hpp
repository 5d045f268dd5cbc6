// Argument checks, launch status and workspaces shared by the routed- and
// streaming-field calls of the C ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "abi_util.hpp"
#include "nerf_mi355x.h"

namespace nerf {
namespace {

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

}  // namespace
}  // namespace nerf
