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
// every workgroup's counts per expert; k_route_scan turns them into the number
// of the expert's pairs in earlier workgroups, and their totals; k_route_place
// scans the totals into offsets, and its waves walk their pairs in order, 64 at
// a time: the lanes with the same expert find each other by one ballot per bit
// of the expert's number, a lane's rank among them is the number of lower ones,
// and the lowest advances the wave's counter.  Equal experts therefore keep the
// pairs' order and nothing depends on the order of atomics.  Pairs without an
// expert (id outside [0, E)) are expert E, after all others.  One workgroup's
// pairs need the last kernel only.
//
// Bound by latency, not by the 12 bytes a pair moves: for 524,288 pairs of 8
// experts 4.6 + 5.3 + 6.1 us, for 150,001 pairs of 4096 experts 5 + 4 + 18 us
// (the last kernel clears, sums and rewrites 8 x 4097 counters in LDS per
// workgroup, and only 37 workgroups have pairs).  Eight waves with eight pairs
// a lane: the whole passes of both with row movement take
// 159.4 and 54.3 us; with four pairs a lane 158.9 and 51.9, but 1,572,864 pairs
// of 4096 experts then take 159 instead of 148; four waves of eight pairs a
// lane: 59.8 for the 150,001.
// ---------------------------------------------------------------------------
constexpr int kRT = 64 * kRouteWaves;

// Experts of the 64 kRouteBatch pairs from p on, one 64 after the other (n1: past the end).
__device__ __forceinline__ void route_ids(int (&e)[kRouteBatch], const int32_t* ids, int64_t p, int64_t end, int E) {
    const int lane = lane_id();
#pragma unroll
    for (int i = 0; i < kRouteBatch; ++i) {
        const int64_t q = p + 64 * i + lane;
        e[i] = q < end ? ids[q] : -2;
    }
#pragma unroll
    for (int i = 0; i < kRouteBatch; ++i) {
        const bool in = p + 64 * i + lane < end;
        e[i] = !in ? E + 1 : (unsigned)e[i] < (unsigned)E ? e[i] : E;
    }
}

// This wave's part of its workgroup's pairs.
struct WavePairs {
    int64_t lo, hi;
};
__device__ __forceinline__ WavePairs wave_pairs(int64_t pairs, int64_t chunk, int wave) {
    const int64_t per = chunk / kRouteWaves, lo = (int64_t)blockIdx.x * chunk + wave * per;
    return WavePairs{lo, lo + per < pairs ? lo + per : pairs};
}

__global__ void __launch_bounds__(kRT) k_route_count(const int32_t* __restrict__ ids, int64_t pairs, int64_t chunk,
                                                     int E, int32_t* __restrict__ counts) {
    extern __shared__ int32_t cnt[];  // [E + 1]
    const WavePairs w = wave_pairs(pairs, chunk, threadIdx.x >> 6);
    int e[kRouteBatch];
    route_ids(e, ids, w.lo, w.hi, E);
    for (int i = threadIdx.x; i <= E; i += kRT) cnt[i] = 0;
    __syncthreads();
    for (int64_t p = w.lo; p < w.hi; p += 64 * kRouteBatch) {
        if (p > w.lo) route_ids(e, ids, p, w.hi, E);
#pragma unroll
        for (int i = 0; i < kRouteBatch; ++i)
            if (e[i] <= E) atomicAdd(&cnt[e[i]], 1);
    }
    __syncthreads();
    for (int i = threadIdx.x; i <= E; i += kRT) counts[(int64_t)blockIdx.x * (E + 1) + i] = cnt[i];
}

// counts[b][e] -> sum of counts[b'][e], b' < b; row nb: the totals.  A workgroup
// has kScanCols experts, the rows dealt to kScanParts threads each.
constexpr int kScanCols = 32, kScanParts = 16;
__global__ void __launch_bounds__(kScanCols* kScanParts) k_route_scan(int32_t* __restrict__ counts, int nb, int n1) {
    __shared__ int32_t sums[kScanParts][kScanCols];
    const int col = threadIdx.x % kScanCols, part = threadIdx.x / kScanCols;
    const int e = blockIdx.x * kScanCols + col;
    const int per = (nb + kScanParts - 1) / kScanParts, b0 = part * per, b1 = b0 + per < nb ? b0 + per : nb;
    int sum = 0;
    if (e < n1)
#pragma unroll 8
        for (int b = b0; b < b1; ++b) sum += counts[(int64_t)b * n1 + e];
    sums[part][col] = sum;
    __syncthreads();
    int run = 0, all = 0;
#pragma unroll
    for (int p = 0; p < kScanParts; ++p) {
        run += p < part ? sums[p][col] : 0;
        all += sums[p][col];
    }
    if (e >= n1) return;
#pragma unroll 8
    for (int b = b0; b < b1; ++b) {
        const int c = counts[(int64_t)b * n1 + e];
        counts[(int64_t)b * n1 + e] = run;
        run += c;
    }
    if (part == 0) counts[(int64_t)nb * n1 + e] = all;
}

// LDS: start[waves][E + 1], before[E + 1].
__global__ void __launch_bounds__(kRT) k_route_place(const int32_t* __restrict__ ids, int64_t pairs, int64_t chunk,
                                                     int E, int bits, const int32_t* __restrict__ counts,
                                                     int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                                                     int32_t* __restrict__ place) {
    extern __shared__ int32_t lds[];
    __shared__ int32_t wsum[kRouteWaves];
    const int n1 = E + 1;
    int32_t* start = lds;                      // [waves][n1]
    int32_t* before = lds + kRouteWaves * n1;  // [n1]
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int nb = gridDim.x, me = blockIdx.x;
    const WavePairs w = wave_pairs(pairs, chunk, wave);
    int e[kRouteBatch];
    route_ids(e, ids, w.lo, w.hi, E);
    for (int i = tid; i < kRouteWaves * n1; i += kRT) start[i] = 0;
    if (nb > 1)
        for (int i = tid; i < n1; i += kRT) before[i] = counts[(int64_t)nb * n1 + i];
    __syncthreads();
    int32_t* mine = start + wave * n1;
    for (int64_t p = w.lo; p < w.hi; p += 64 * kRouteBatch) {
        if (p > w.lo) route_ids(e, ids, p, w.hi, E);
#pragma unroll
        for (int i = 0; i < kRouteBatch; ++i)
            if (e[i] <= E) atomicAdd(&mine[e[i]], 1);
    }
    __syncthreads();
    // offsets: exclusive scan of the totals, `per` consecutive experts a thread
    const int per = (n1 + kRT - 1) / kRT, i0 = tid * per < n1 ? tid * per : n1, i1 = i0 + per < n1 ? i0 + per : n1;
    int sum = 0;
    for (int i = i0; i < i1; ++i) {
        if (nb == 1) {
            int tot = 0;
            for (int v = 0; v < kRouteWaves; ++v) tot += start[v * n1 + i];
            before[i] = tot;
        }
        sum += before[i];
    }
    int inc = sum;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(inc, off, 64);
        if (lane >= off) inc += o;
    }
    if (lane == 63) wsum[wave] = inc;
    __syncthreads();
    int run = inc - sum;
    for (int v = 0; v < wave; ++v) run += wsum[v];
    for (int i = i0; i < i1; ++i) {
        const int c = before[i];
        before[i] = run;
        run += c;
    }
    __syncthreads();
    for (int i = tid; i < n1; i += kRT) {
        int at = before[i];
        if (me == 0) offsets[i] = at;
        if (nb > 1) at += counts[(int64_t)me * n1 + i];
        for (int v = 0; v < kRouteWaves; ++v) {
            const int c = start[v * n1 + i];
            start[v * n1 + i] = at;
            at += c;
        }
    }
    __syncthreads();
    const bool one = w.hi - w.lo <= 64 * kRouteBatch;
    for (int64_t p = w.lo; p < w.hi; p += 64 * kRouteBatch) {
        if (!one) route_ids(e, ids, p, w.hi, E);
#pragma unroll
        for (int i = 0; i < kRouteBatch; ++i) {
            const int64_t q = p + 64 * i + lane;
            const bool in = e[i] <= E;  // (lanes past the end match only each other)
            uint64_t same = ~0ull;
            for (int b = 0; b < bits; ++b) {
                const uint64_t m = __ballot((e[i] >> b) & 1);
                same &= (e[i] >> b) & 1 ? m : ~m;
            }
            const int rank = __popcll(same & ((1ull << lane) - 1));
            const int at = in ? mine[e[i]] : 0;
            wave_lds_sync();
            if (in) {
                if (rank == 0) mine[e[i]] = at + __popcll(same);
                const int slot = at + rank;
                NERF_DCHECK(slot >= 0 && slot < pairs, kCheckRouteSlot);
                order[slot] = (int32_t)q;
                place[q] = slot;
            }
            wave_lds_sync();
        }
    }
}

// ---------------------------------------------------------------------------
// Row movement.  One group of G lanes per sample, 16 bytes a lane: a sample's
// row is read (or summed) once for all its k choices, so each kernel moves
// every row once.  All are bound by memory; nothing is shared, so there is no
// LDS.  Outputs are stored nontemporally: nobody reads them again from this
// kernel.  262,144 samples x 2 of 256 bfloat16: plan, gather and combine 159 us
// for 814 MB (5.1 TB/s; a 2 GiB copy reaches 4.9), 169 with ordinary stores; the
// combination's gradient and the gather's 194 us (204).
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

// Pieces of a row of d elements: whole 16-byte pieces, of which the last is moved
// back to end with the row (its first elements are then the previous piece's
// too, and are written twice with the same values); a row shorter than a piece
// is one partial piece.
template <class T>
struct Piece {
    int c, skip;  // first element; elements that belong to the previous piece
    __device__ __forceinline__ Piece(int c0, int d) {
        c = c0 + RowIO<T>::PER <= d || d < RowIO<T>::PER ? c0 : d - RowIO<T>::PER;
        skip = c0 - c;
    }
};

// Choices of a sample whose rows are in flight together (16 bytes each a lane).
constexpr int kRowsAhead = 4;

template <class T, int G>
__global__ void __launch_bounds__(kRowThreads) k_route_gather(RouteRows r) {
    using IO = RowIO<T>;
    const int g = threadIdx.x % G;
    const int live = slots_used(r);
    NERF_EACH_SAMPLE(t) {
        const T* src = (const T*)r.a + t * r.lda;
        const int32_t* pl = r.place + t * r.k;
        for (int c0 = g * IO::PER; c0 < r.d; c0 += G * IO::PER) {
            const Piece<T> p(c0, r.d);
            const typename IO::Vec v = IO::load(src, p.c, r.d);
            for (int j = 0; j < r.k; ++j) {
                const int slot = pl[j];
                NERF_DCHECK(slot >= 0 && slot < r.n * r.k, kCheckRouteSlot);
                if ((unsigned)slot >= (uint64_t)(r.n * r.k)) continue;
                IO::stream((T*)r.out + (int64_t)slot * r.d, p.c, r.d, slot < live ? v : IO::zero());
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
        for (int c0 = g * IO::PER; c0 < r.d; c0 += G * IO::PER) {
            const Piece<T> p(c0, r.d);
            float acc[IO::PER] = {};
            for (int j0 = 0; j0 < r.k; j0 += kRowsAhead) {
                typename IO::Vec v[kRowsAhead];
                float wj[kRowsAhead];
                bool used[kRowsAhead];
#pragma unroll
                for (int u = 0; u < kRowsAhead; ++u) {
                    const int j = j0 + u;
                    const int slot = j < r.k ? pl[j] : -1;
                    used[u] = (unsigned)slot < (unsigned)live;  // (else its row and weight count for nothing)
                    wj[u] = j < r.k && w ? w[j] : 1.0f;
                    v[u] = used[u] ? IO::load((const T*)r.y + (int64_t)slot * r.d, p.c, r.d) : IO::zero();
                }
#pragma unroll
                for (int u = 0; u < kRowsAhead; ++u)
                    if (used[u])
#pragma unroll
                        for (int i = 0; i < IO::PER; ++i) acc[i] = fmaf(wj[u], IO::get(v[u], i), acc[i]);
            }
            IO::stream((T*)r.out + t * r.ldo, p.c, r.d, IO::pack(acc));
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
        for (int j0 = 0; j0 < r.k; j0 += kRowsAhead) {
            int64_t row[kRowsAhead];
            float wj[kRowsAhead], dot[kRowsAhead];
            bool in[kRowsAhead], used[kRowsAhead];
#pragma unroll
            for (int u = 0; u < kRowsAhead; ++u) {
                const int j = j0 + u;
                const int slot = j < r.k ? pl[j] : -1;
                NERF_DCHECK(j >= r.k || (slot >= 0 && slot < r.n * r.k), kCheckRouteSlot);
                in[u] = (unsigned)slot < (uint64_t)(r.n * r.k);
                used[u] = in[u] && slot < live;
                row[u] = (int64_t)slot * r.d;
                wj[u] = j < r.k && r.weights ? r.weights[t * r.k + j] : 1.0f;
                dot[u] = 0.0f;
            }
            for (int c0 = g * IO::PER; c0 < r.d; c0 += G * IO::PER) {
                const Piece<T> p(c0, r.d);
                const typename IO::Vec v = IO::load(go, p.c, r.d);
                typename IO::Vec y[kRowsAhead];
#pragma unroll
                for (int u = 0; u < kRowsAhead; ++u)
                    y[u] = used[u] ? IO::load((const T*)r.y + row[u], p.c, r.d) : IO::zero();
#pragma unroll
                for (int u = 0; u < kRowsAhead; ++u) {
                    if (!in[u]) continue;
                    float o[IO::PER];
#pragma unroll
                    for (int i = 0; i < IO::PER; ++i) {
                        const float f = IO::get(v, i);
                        o[i] = used[u] ? wj[u] * f : 0.0f;
                        // (columns past d are zero in both, those of the previous piece are counted there)
                        if (used[u] && i >= p.skip) dot[u] = fmaf(f, IO::get(y[u], i), dot[u]);
                    }
                    IO::stream((T*)r.out + row[u], p.c, r.d, IO::pack(o));
                }
            }
            if (r.dweights)
#pragma unroll
                for (int u = 0; u < kRowsAhead; ++u) {
#pragma unroll
                    for (int off = G / 2; off >= 1; off >>= 1) dot[u] += __shfl_xor(dot[u], off, 64);
                    if (g == 0 && j0 + u < r.k) r.dweights[t * r.k + j0 + u] = used[u] ? dot[u] : 0.0f;
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
    if (nb > 1) {
        k_route_count<<<nb, kRT, n1 * sizeof(int32_t), s>>>(ids, pairs, chunk, n_experts, counts);
        k_route_scan<<<(n1 + kScanCols - 1) / kScanCols, kScanCols * kScanParts, 0, s>>>(counts, (int)nb, n1);
    }
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
