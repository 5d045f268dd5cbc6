// Routing of sample-expert pairs for gfx950: a stable sort of the pairs by
// expert, rows copied into that order and summed back with weights, and the
// gradients of both.  Pair p = t k + j is choice j of sample t.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "experts.hpp"
#include "rowio.hpp"

namespace nerf {

namespace {

// ---------------------------------------------------------------------------
// The plan: a counting sort.  A workgroup owns route_chunk() consecutive
// pairs, each of its waves a consecutive part of them.  k_route_count writes
// every workgroup's counts per expert; in k_route_place each workgroup adds
// up the counts of all (the offsets) and of those before it (its base), and
// its waves then walk their pairs in order, 64 at a time: the lanes with the
// same expert find each other by one ballot per bit of the expert's number, a
// lane's rank among them is the number of lower ones, and the lowest advances
// the wave's counter.  Equal experts therefore keep the pairs' order and
// nothing depends on the order of atomics.  Pairs without an expert (id
// outside [0, E)) are expert E, after all others.
// ---------------------------------------------------------------------------
constexpr int kRT = 64 * kRouteWaves;

__device__ __forceinline__ int route_id(const int32_t* ids, int64_t p, int E) {
    const int e = ids[p];
    return (unsigned)e < (unsigned)E ? e : E;
}

__global__ void __launch_bounds__(kRT) k_route_count(const int32_t* __restrict__ ids, int64_t pairs, int64_t chunk,
                                                     int E, int32_t* __restrict__ counts) {
    extern __shared__ int32_t cnt[];  // [E + 1]
    for (int e = threadIdx.x; e <= E; e += kRT) cnt[e] = 0;
    __syncthreads();
    const int64_t p0 = (int64_t)blockIdx.x * chunk, p1 = p0 + chunk < pairs ? p0 + chunk : pairs;
    for (int64_t p = p0 + threadIdx.x; p < p1; p += kRT) atomicAdd(&cnt[route_id(ids, p, E)], 1);
    __syncthreads();
    for (int e = threadIdx.x; e <= E; e += kRT) counts[(int64_t)blockIdx.x * (E + 1) + e] = cnt[e];
}

// LDS: start[waves][E + 1], base[E + 1], scan scratch.
__global__ void __launch_bounds__(kRT) k_route_place(const int32_t* __restrict__ ids, int64_t pairs, int64_t chunk,
                                                     int E, int bits, const int32_t* __restrict__ counts,
                                                     int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                                                     int32_t* __restrict__ place) {
    extern __shared__ int32_t lds[];
    const int n1 = E + 1;
    int32_t* start = lds;                     // [waves][n1]
    int32_t* before = lds + kRouteWaves * n1; // [n1] pairs of this expert in earlier workgroups
    __shared__ int32_t wsum[kRouteWaves];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nb = gridDim.x, me = blockIdx.x;
    const int64_t p0 = (int64_t)me * chunk, p1 = p0 + chunk < pairs ? p0 + chunk : pairs;
    const int64_t per = chunk / kRouteWaves;
    const int64_t w0 = p0 + wave * per, w1 = w0 + per < p1 ? w0 + per : p1;
    for (int i = tid; i < kRouteWaves * n1; i += kRT) start[i] = 0;
    __syncthreads();
    int32_t* mine = start + wave * n1;
    for (int64_t p = w0 + lane; p < w1; p += 64) atomicAdd(&mine[route_id(ids, p, E)], 1);
    __syncthreads();
    // this expert's pairs in all workgroups, and in those before this one:
    // `cols` experts at a time, the workgroups dealt to kRT / cols threads each
    int cols = 1;
    while (cols < n1 && cols < kRT) cols <<= 1;
    const int parts = kRT / cols, part = tid / cols;
    int run = 0;  // slots of the experts of earlier rounds
    for (int e0 = 0; e0 < n1; e0 += cols) {
        const int e = e0 + (tid & (cols - 1));
        int tot = 0, pre = 0;
        if (e < n1) {
            if (nb == 1) {
                if (part == 0)
                    for (int w = 0; w < kRouteWaves; ++w) tot += start[w * n1 + e];
            } else {
#pragma unroll 4
                for (int b = part; b < nb; b += parts) {
                    const int c = counts[(int64_t)b * n1 + e];
                    tot += c;
                    pre += b < me ? c : 0;
                }
            }
        }
        // sum over the threads of one expert (a power-of-two stride apart)
        __shared__ int32_t st[kRT], sp[kRT];
        st[tid] = tot;
        sp[tid] = pre;
        for (int h = parts / 2; h >= 1; h >>= 1) {
            __syncthreads();
            if (part < h) {
                st[tid] += st[tid + h * cols];
                sp[tid] += sp[tid + h * cols];
            }
        }
        __syncthreads();
        tot = tid < cols ? st[tid] : 0;
        pre = tid < cols ? sp[tid] : 0;
        // exclusive scan of the totals over the experts of this round
        int inc = tot;
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
            const int o = __shfl_up(inc, off, 64);
            if (lane >= off) inc += o;
        }
        if (lane == 63) wsum[wave] = inc;
        __syncthreads();
        int add = 0, all = 0;
        for (int w = 0; w < kRouteWaves; ++w) {
            if (w < wave) add += wsum[w];
            all += wsum[w];
        }
        if (tid < cols && e < n1) {
            const int off = run + add + inc - tot;
            if (me == 0) offsets[e] = off;
            before[e] = off + pre;
        }
        run += all;
        __syncthreads();
    }
    for (int e = tid; e < n1; e += kRT) {
        int at = before[e];
        for (int w = 0; w < kRouteWaves; ++w) {
            const int c = start[w * n1 + e];
            start[w * n1 + e] = at;
            at += c;
        }
    }
    __syncthreads();
    for (int64_t q = w0; q < w1; q += 64) {
        const int64_t p = q + lane;
        const bool in = p < w1;
        const int e = in ? route_id(ids, p, E) : n1;  // lanes past the end match only each other
        uint64_t same = ~0ull;
        for (int b = 0; b < bits; ++b) {
            const uint64_t m = __ballot((e >> b) & 1);
            same &= (e >> b) & 1 ? m : ~m;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        const int at = in ? mine[e] : 0;
        wave_lds_sync();
        if (in) {
            if (rank == 0) mine[e] = at + __popcll(same);
            const int slot = at + rank;
            NERF_DCHECK(slot >= 0 && slot < pairs, kCheckRouteSlot);
            order[slot] = (int32_t)p;
            place[p] = slot;
        }
        wave_lds_sync();
    }
}

// ---------------------------------------------------------------------------
// Row movement.  One group of G lanes per sample, 16 bytes a lane: a sample's
// row is read (or summed) once for all its k choices, so each kernel moves
// every row once.  All are bound by memory; nothing is shared, so there is no
// LDS.
// ---------------------------------------------------------------------------
constexpr int kRowThreads = 256;
constexpr int64_t kRowGrid = (int64_t)1 << 22;  // workgroups at most: further samples go round again
// for each sample t of this group of G lanes
#define NERF_EACH_SAMPLE(t)                                                                   \
    for (int64_t t = (int64_t)blockIdx.x * (kRowThreads / G) + threadIdx.x / G; t < r.n;      \
         t += (int64_t)gridDim.x * (kRowThreads / G))

// Slots in use, read from the device and kept within the slots there are.
__device__ __forceinline__ int slots_used(const RouteRows& r) {
    const int64_t pairs = r.n * r.k;
    const int v = r.offsets[r.n_experts];
    NERF_DCHECK(v >= 0 && v <= pairs, kCheckRouteOffset);
    return v < 0 ? 0 : v > pairs ? (int)pairs : v;
}

template <class T, int G>
__global__ void __launch_bounds__(kRowThreads) k_route_gather(RouteRows r) {
    using IO = RowIO<T>;
    const int g = threadIdx.x % G;
    const int live = slots_used(r);
    NERF_EACH_SAMPLE(t) {
        const T* src = (const T*)r.a + t * r.lda;
        const int32_t* pl = r.place + t * r.k;
        for (int c = g * IO::PER; c < r.d; c += G * IO::PER) {
            const typename IO::Vec v = IO::load(src, c, r.d);
            for (int j = 0; j < r.k; ++j) {
                const int slot = pl[j];
                NERF_DCHECK(slot >= 0 && slot < r.n * r.k, kCheckRouteSlot);
                if ((unsigned)slot >= (uint64_t)(r.n * r.k)) continue;
                IO::store((T*)r.out + (int64_t)slot * r.d, c, r.d, slot < live ? v : IO::zero());
            }
        }
    }
}

template <class T, int G>
__global__ void __launch_bounds__(kRowThreads) k_route_combine(RouteRows r) {
    using IO = RowIO<T>;
    const int g = threadIdx.x % G;
    const int live = slots_used(r);
    NERF_EACH_SAMPLE(t) {
        const int32_t* pl = r.place + t * r.k;
        const float* w = r.weights ? r.weights + t * r.k : nullptr;
        for (int c = g * IO::PER; c < r.d; c += G * IO::PER) {
            float acc[IO::PER] = {};
            for (int j = 0; j < r.k; ++j) {
                const int slot = pl[j];
                if ((unsigned)slot >= (unsigned)live) continue;  // no expert: its row and weight count for nothing
                const typename IO::Vec v = IO::load((const T*)r.y + (int64_t)slot * r.d, c, r.d);
                const float wj = w ? w[j] : 1.0f;
    #pragma unroll
                for (int i = 0; i < IO::PER; ++i) acc[i] = fmaf(wj, IO::get(v, i), acc[i]);
            }
            IO::store((T*)r.out + t * r.ldo, c, r.d, IO::pack(acc));
        }
    }
}

template <class T, int G>
__global__ void __launch_bounds__(kRowThreads) k_route_combine_grad(RouteRows r) {
    using IO = RowIO<T>;
    const int g = threadIdx.x % G;
    const int live = slots_used(r);
    NERF_EACH_SAMPLE(t) {
        const T* go = (const T*)r.a + t * r.lda;
        const int32_t* pl = r.place + t * r.k;
        for (int j = 0; j < r.k; ++j) {
            const int slot = pl[j];
            NERF_DCHECK(slot >= 0 && slot < r.n * r.k, kCheckRouteSlot);
            const bool in = (unsigned)slot < (uint64_t)(r.n * r.k), used = in && slot < live;
            const float wj = r.weights ? r.weights[t * r.k + j] : 1.0f;
            float dot = 0.0f;
            if (in) {
                const int64_t row = (int64_t)slot * r.d;
                for (int c = g * IO::PER; c < r.d; c += G * IO::PER) {
                    if (!used) {
                        IO::store((T*)r.out + row, c, r.d, IO::zero());
                        continue;
                    }
                    const typename IO::Vec v = IO::load(go, c, r.d), y = IO::load((const T*)r.y + row, c, r.d);
                    float o[IO::PER];
    #pragma unroll
                    for (int i = 0; i < IO::PER; ++i) {
                        o[i] = wj * IO::get(v, i);
                        dot = fmaf(IO::get(v, i), IO::get(y, i), dot);  // columns past d are zero in both
                    }
                    IO::store((T*)r.out + row, c, r.d, IO::pack(o));
                }
            }
            if (r.dweights) {
    #pragma unroll
                for (int off = G / 2; off >= 1; off >>= 1) dot += __shfl_xor(dot, off, 64);
                if (g == 0) r.dweights[t * r.k + j] = used ? dot : 0.0f;
            }
        }
    }
}

// Lanes per row: enough for one 16-byte piece each, at most a wave.
int row_lanes(bool bf16, int d) {
    const int units = (d + (bf16 ? 7 : 3)) / (bf16 ? 8 : 4);
    int g = 1;
    while (g < units && g < 64) g <<= 1;
    return g;
}

template <class F>
void by_lanes(int g, F&& f) {
    switch (g) {
        case 1: f(std::integral_constant<int, 1>{}); break;
        case 2: f(std::integral_constant<int, 2>{}); break;
        case 4: f(std::integral_constant<int, 4>{}); break;
        case 8: f(std::integral_constant<int, 8>{}); break;
        case 16: f(std::integral_constant<int, 16>{}); break;
        case 32: f(std::integral_constant<int, 32>{}); break;
        default: f(std::integral_constant<int, 64>{}); break;
    }
}

unsigned row_grid(int64_t n, int g) {
    const int64_t blocks = (n + kRowThreads / g - 1) / (kRowThreads / g);
    return (unsigned)(blocks < kRowGrid ? blocks : kRowGrid);
}

}  // namespace

void launch_route_plan(const int32_t* ids, int64_t pairs, int n_experts, int32_t* offsets, int32_t* order,
                       int32_t* place, int32_t* counts, hipStream_t s) {
    const int64_t chunk = route_chunk(pairs);
    const unsigned nb = pairs > 0 ? (unsigned)route_blocks(pairs) : 1u;  // (no pairs: the offsets are still written)
    const int n1 = n_experts + 1;
    int bits = 1;
    while ((n1 + 1) > (1 << bits)) ++bits;  // ids 0 .. E + 1
    if (nb > 1)
        k_route_count<<<nb, kRT, n1 * sizeof(int32_t), s>>>(ids, pairs, chunk, n_experts, counts);
    k_route_place<<<nb, kRT, (kRouteWaves + 1) * (size_t)n1 * sizeof(int32_t), s>>>(
        ids, pairs, chunk, n_experts, bits, counts, offsets, order, place);
}

#define NERF_ROW_LAUNCH(KERNEL)                                                                  \
    by_lanes(row_lanes(bf16, r.d), [&](auto g) {                                                 \
        constexpr int G = decltype(g)::value;                                                    \
        if (bf16)                                                                                \
            KERNEL<__bf16, G><<<row_grid(r.n, G), kRowThreads, 0, s>>>(r);                       \
        else                                                                                     \
            KERNEL<float, G><<<row_grid(r.n, G), kRowThreads, 0, s>>>(r);                        \
    })

void launch_route_gather(bool bf16, const RouteRows& r, hipStream_t s) { NERF_ROW_LAUNCH(k_route_gather); }
void launch_route_combine(bool bf16, const RouteRows& r, hipStream_t s) { NERF_ROW_LAUNCH(k_route_combine); }
void launch_route_combine_grad(bool bf16, const RouteRows& r, hipStream_t s) { NERF_ROW_LAUNCH(k_route_combine_grad); }

}  // namespace nerf
