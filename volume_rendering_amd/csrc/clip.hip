// The norm of all gradients of a list of tensors, and the gradients scaled
// down to a largest norm, for gfx950:
//   norm = sqrt(sum over every element of every tensor of g^2)
//   out  = g min(1, max_norm / norm)
// Both are bound by memory: one read for the norm, one read and one write to
// scale.  The list travels as kernel arguments, kGroup tensors a launch, so
// there is no table to copy and a captured graph holds it.  Squares are summed
// in float64 (which neither overflows nor loses small gradients beside large
// ones, and still reads 403 MB in 71 us, 5.7 TB/s); each
// workgroup writes one partial sum, and whoever needs the norm adds all of them
// up in the same order, so results are the same from run to run.
// Measured: 403 MB of gradients of float32 and bfloat16 normed and scaled in 207 us,
// 3.9 TB/s of the least traffic (806 MB) and 5.9 of what it moves, as it reads twice; 48
// tensors of two networks, 4.8 MB, in 11.7 us, the two kernels 4.6 and 4.8 at least; of
// many small tensors the launches count (2000 of 20000 elements, 160 MB: 197 us, 33 launches).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "common.hpp"
#include "fields.hpp"
#include "rowio.hpp"

namespace nerf {

namespace {

constexpr int kGroup = 128;            // tensors a launch (kernel arguments hold 4 KiB)
constexpr int kClipThreads = 256;
constexpr int kPiecesAhead = 8;        // 16-byte loads in flight per lane
constexpr int kChunkPieces = kClipThreads * kPiecesAhead;  // 32 KiB
constexpr int kNormGrid = 2048;        // workgroups of a launch at most

struct TensorGroup {
    const void* src[kGroup];
    void* dst[kGroup];
    int64_t count[kGroup];
    int32_t first[kGroup + 1];  // chunks of the tensors before (fewer than 2^31: 2^41 elements at most)
    uint32_t bf16[kGroup / 32]; // bit i: tensor i is bfloat16
    int n;
};
static_assert(sizeof(TensorGroup) + 32 <= 4096, "kernel arguments");

__host__ __device__ inline int64_t chunks_of(int64_t count, bool bf16) {
    const int64_t per = (int64_t)kChunkPieces * (bf16 ? 8 : 4);
    return (count + per - 1) / per;
}

// The tensor of chunk c, and the elements [lo, hi) of the chunk.
struct Chunk {
    int t;
    int64_t lo, hi;
    bool bf16;
};
__device__ __forceinline__ Chunk chunk_at(const TensorGroup& g, int64_t c) {
    int lo = 0, hi = g.n - 1;  // the last tensor that starts at or before c (those after it start later)
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (g.first[mid] <= c)
            lo = mid;
        else
            hi = mid - 1;
    }
    Chunk r;
    r.t = lo;
    r.bf16 = (g.bf16[lo / 32] >> lo % 32) & 1;
    const int64_t per = (int64_t)kChunkPieces * (r.bf16 ? 8 : 4);
    r.lo = (c - g.first[lo]) * per;
    r.hi = r.lo + per < g.count[lo] ? r.lo + per : g.count[lo];
    return r;
}

__device__ __forceinline__ double block_sum(double v, double* scratch) {  // scratch: [kClipThreads / 64]
    v = wave_sum_f64(v);
    if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
    __syncthreads();
    v = scratch[0];
#pragma unroll
    for (int w = 1; w < kClipThreads / 64; ++w) v += scratch[w];
    __syncthreads();
    return v;
}

template <class T>
__device__ __forceinline__ void chunk_squares(double (&s)[2], const Chunk& c, const T* src) {
    using IO = RowIO<T>;
    if (c.hi - c.lo == (int64_t)kChunkPieces * IO::PER) {
        typename IO::Vec v[kPiecesAhead];
#pragma unroll
        for (int u = 0; u < kPiecesAhead; ++u)
            v[u] = IO::load_whole(src + c.lo + ((int64_t)u * kClipThreads + threadIdx.x) * IO::PER);
#pragma unroll
        for (int u = 0; u < kPiecesAhead; ++u)
#pragma unroll
            for (int i = 0; i < IO::PER; ++i) {
                const double d = IO::get(v[u], i);
                s[i & 1] = fma(d, d, s[i & 1]);
            }
        return;
    }
    for (int64_t k = c.lo + threadIdx.x * IO::PER; k < c.hi; k += kClipThreads * IO::PER) {
        const typename IO::Vec v = IO::load(src, k, c.hi);  // (zeros past the end)
#pragma unroll
        for (int i = 0; i < IO::PER; ++i) {
            const double d = IO::get(v, i);
            s[i & 1] = fma(d, d, s[i & 1]);
        }
    }
}

__global__ void __launch_bounds__(kClipThreads) k_grad_squares(TensorGroup g, double* partial) {
    __shared__ double scratch[kClipThreads / 64];
    double s[2] = {0.0, 0.0};
    const int64_t chunks = g.first[g.n];
    for (int64_t i = blockIdx.x; i < chunks; i += gridDim.x) {
        const Chunk c = chunk_at(g, i);
        if (c.bf16)
            chunk_squares(s, c, (const __bf16*)g.src[c.t]);
        else
            chunk_squares(s, c, (const float*)g.src[c.t]);
    }
    const double v = block_sum(s[0] + s[1], scratch);
    if (threadIdx.x == 0) partial[blockIdx.x] = v;
}

// The norm stays in float64 until the factor is known: float32 would not hold
// that of many gradients near the type's largest.
__device__ __forceinline__ double norm_of(const double* partial, int n, double* scratch) {
    double s = 0.0;
#pragma unroll 8
    for (int i = threadIdx.x; i < n; i += kClipThreads) s += partial[i];
    return sqrt(block_sum(s, scratch));
}

// partial[n], if kept, is the norm for the launches that follow.
__global__ void __launch_bounds__(kClipThreads) k_grad_norm(double* partial, int n, float* norm, int keep) {
    __shared__ double scratch[kClipThreads / 64];
    const double v = norm_of(partial, n, scratch);
    if (threadIdx.x == 0) {
        norm[0] = (float)v;
        if (keep) partial[n] = v;
    }
}

template <class T>
__device__ __forceinline__ void chunk_scale(const Chunk& c, const T* src, T* dst, float down, float f) {
    using IO = RowIO<T>;
    auto scaled = [&](const typename IO::Vec& v) {
        float o[IO::PER];
#pragma unroll
        for (int i = 0; i < IO::PER; ++i) o[i] = IO::get(v, i) * down * f;
        return IO::pack(o);
    };
    if (c.hi - c.lo == (int64_t)kChunkPieces * IO::PER) {
        typename IO::Vec v[kPiecesAhead];
#pragma unroll
        for (int u = 0; u < kPiecesAhead; ++u)
            v[u] = IO::load_whole(src + c.lo + ((int64_t)u * kClipThreads + threadIdx.x) * IO::PER);
#pragma unroll
        for (int u = 0; u < kPiecesAhead; ++u)
            IO::stream(dst, c.lo + ((int64_t)u * kClipThreads + threadIdx.x) * IO::PER, c.hi, scaled(v[u]));
        return;
    }
    for (int64_t k = c.lo + threadIdx.x * IO::PER; k < c.hi; k += kClipThreads * IO::PER)
        IO::stream(dst, k, c.hi, scaled(IO::load(src, k, c.hi)));
}

// Chunks are taken in the opposite order of the norm's, so that the last ones
// it read are still in the caches.  A factor of 1 leaves tensors that are
// scaled in place as they are.  Without `norm` the norm is partial[n].
__global__ void __launch_bounds__(kClipThreads) k_grad_scale(TensorGroup g, const double* partial, int n,
                                                             float max_norm, float* norm) {
    __shared__ double scratch[kClipThreads / 64];
    const double v = norm ? norm_of(partial, n, scratch) : partial[n];
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = (float)v;
    // (a NaN norm makes every gradient NaN); a factor that float32 holds with fewer
    // bits is applied in two steps, of which the first is exact
    const double factor = v <= max_norm ? 1.0 : max_norm / v;
    const float down = factor < 0x1p-100 ? 0x1p-60f : 1.0f, f = (float)(factor < 0x1p-100 ? factor * 0x1p60 : factor);
    const int64_t chunks = g.first[g.n];
    for (int64_t i = chunks - 1 - blockIdx.x; i >= 0; i -= gridDim.x) {
        const Chunk c = chunk_at(g, i);
        if (factor == 1.0 && g.src[c.t] == g.dst[c.t]) continue;
        if (c.bf16)
            chunk_scale(c, (const __bf16*)g.src[c.t], (__bf16*)g.dst[c.t], down, f);
        else
            chunk_scale(c, (const float*)g.src[c.t], (float*)g.dst[c.t], down, f);
    }
}

// The group of tensors list[0 .. n) that are not empty, from i on; returns the
// next i.
int next_group(TensorGroup& g, const nerf_tensor* list, int n, int i) {
    g.n = 0;
    for (uint32_t& bits : g.bf16) bits = 0;
    g.first[0] = 0;
    for (; i < n && g.n < kGroup; ++i) {
        if (list[i].count == 0) continue;
        const bool bf16 = list[i].dtype == NERF_BF16;
        g.src[g.n] = list[i].src;
        g.dst[g.n] = list[i].dst;
        g.count[g.n] = list[i].count;
        g.bf16[g.n / 32] |= (uint32_t)bf16 << g.n % 32;
        g.first[g.n + 1] = g.first[g.n] + (int32_t)chunks_of(list[i].count, bf16);
        ++g.n;
    }
    return i;
}

unsigned group_grid(const TensorGroup& g) { return (unsigned)std::min<int64_t>(g.first[g.n], kNormGrid); }

int launch_squares(const nerf_tensor* list, int n, double* partials, hipStream_t s) {
    int used = 0;
    TensorGroup g;
    for (int i = 0; i < n;) {
        i = next_group(g, list, n, i);
        if (g.n == 0) break;
        k_grad_squares<<<group_grid(g), kClipThreads, 0, s>>>(g, partials + used);
        used += (int)group_grid(g);
    }
    return used;
}

}  // namespace

size_t grad_norm_partials(const nerf_tensor* list, int n) {
    size_t used = 0;
    TensorGroup g;
    for (int i = 0; i < n;) {
        i = next_group(g, list, n, i);
        if (g.n) used += group_grid(g);
    }
    return used + 1;
}

void launch_grad_norm(const nerf_tensor* list, int n, double* partials, float* norm, hipStream_t s) {
    const int used = launch_squares(list, n, partials, s);
    k_grad_norm<<<1, kClipThreads, 0, s>>>(partials, used, norm, 0);
}

// With the partial sums of one launch every workgroup adds them up itself,
// which is cheaper than a kernel between the two; with more that kernel does.
void launch_grad_clip(const nerf_tensor* list, int n, float max_norm, double* partials, float* norm, hipStream_t s) {
    const int used = launch_squares(list, n, partials, s);
    const bool joined = used > 0 && used <= kNormGrid;
    if (!joined) k_grad_norm<<<1, kClipThreads, 0, s>>>(partials, used, norm, 1);
    TensorGroup g;
    for (int i = 0; i < n;) {
        i = next_group(g, list, n, i);
        if (g.n == 0) break;
        // (every launch writes the same norm)
        if (joined)
            k_grad_scale<<<group_grid(g), kClipThreads, 0, s>>>(g, partials, used, max_norm, norm);
        else
            k_grad_scale<<<group_grid(g), kClipThreads, 0, s>>>(g, partials, used, max_norm, nullptr);
    }
}

}  // namespace nerf
