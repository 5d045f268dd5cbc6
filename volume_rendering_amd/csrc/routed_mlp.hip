// The whole two-layer routed field for a few samples, for gfx950:
//   out_t = sum_j w_tj (W2_e act(W1_e x_t + b1_e) + b2_e),   e = ids_tj,
// in two kernels.  Every weight of an expert that some pair (sample, choice)
// uses is read from memory once; that read bounds both kernels, and for one
// sample the launches and one chain of dependent loads each.  Up to 64 pairs are
// sorted by expert by every workgroup itself, in LDS, which is cheaper than a
// kernel in front; more (the work grows with their square) by a kernel of their
// own.  First the hidden layer: workgroups take tiles of one expert's W1 and apply
// them to all its pairs.  Then the output: workgroups own columns, for all
// experts, so that a sample's k terms meet in LDS and are added in the order of
// its choices, without atomics.
// Up to two pairs per expert (on average) are dot products, whose weights a wave
// reads in whole lines; more go through the matrix units, 16 pairs at a time, as
// the vector units would take longer than the read (one expert 1024 -> 4096 ->
// 1024, 128 samples).  Hidden values keep 24 bits between the kernels (rounding
// them to bfloat16 would add an error as large as the output's own rounding, and
// saves only L2 traffic).
#include <hip/hip_runtime.h>

#include <cfloat>
#include <type_traits>

#include "common.hpp"
#include "fields.hpp"
#include "rowio.hpp"

namespace nerf {

namespace {

constexpr int kSelf = kMlpSelfSorted;  // pairs that a workgroup sorts itself
constexpr int kGroup = 64;             // pairs of one expert that a weight tile is applied to at once

// ---------------------------------------------------------------------------
// Pairs sorted by expert, stably: pair[s] for s < used, and the experts that
// have any: expert[u] owns slots head[u] .. head[u + 1] - 1.  group: the slots that
// start kGroup (or the last few) of one expert.
// ---------------------------------------------------------------------------
constexpr int kKeyBits = 9;
static_assert(NERF_FEW_PAIRS <= 1 << kKeyBits, "a pair's number fits its key");
template <int N>
struct Pairs {
    int key[N];     // of a pair: its expert (E: none), then its number
    int pair[N];    // of a slot
    int of[N];      // expert of a slot
    int slot[N];    // of a pair, -1 without an expert
    int expert[N];
    int head[N + 1];
    int group[N];
    int experts, groups, used;
};
using Plan = Pairs<NERF_FEW_PAIRS>;
static_assert(sizeof(Plan) <= kMlpPlanBytes, "room in the workspace");

// Pairs first .. first + pairs - 1 of the call, by every thread of the workgroup.
// A pair's slot is the number of smaller keys; the slots that start an expert or a
// group are counted by the first wave.
template <int N>
__device__ __forceinline__ void sort_pairs(Pairs<N>& s, const MlpArgs& a, int first, int pairs, int threads) {
    const int padded = (pairs + 3) & ~3;
    if (threadIdx.x == 0) s.used = 0;
    for (int p = threadIdx.x; p < padded; p += threads) {
        const int id = p < pairs ? a.ids[first + p] : -1;
        s.key[p] = ((unsigned)id < (unsigned)a.n_experts ? id : a.n_experts) << kKeyBits | p;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += threads) {
        const int key = s.key[p], e = key >> kKeyBits;
        int slot = 0;
#pragma unroll 4
        for (int q = 0; q < padded; q += 4) {
            const int4 o = *(const int4*)&s.key[q];
            slot += (o.x < key) + (o.y < key) + (o.z < key) + (o.w < key);
        }
        const bool live = e < a.n_experts;
        s.slot[p] = live ? slot : -1;
        if (live) {
            s.pair[slot] = p;
            s.of[slot] = e;
            atomicAdd(&s.used, 1);
        }
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        int experts = 0, groups = 0, head = 0;  // (head: of the last expert so far)
        for (int i0 = 0; i0 < s.used; i0 += 64) {
            const int i = i0 + threadIdx.x;
            const bool in = i < s.used, starts = in && (i == 0 || s.of[i - 1] != s.of[i]);
            const uint64_t self = (uint64_t)1 << threadIdx.x, lower = self - 1;
            const uint64_t heads = __ballot(starts), mine = heads & (lower | self);
            const int from = mine ? i0 + 63 - __clzll(mine) : head;
            const bool full = in && (i - from) % kGroup == 0;
            const uint64_t fulls = __ballot(full);
            if (starts) {
                const int u = experts + __popcll(heads & lower);
                s.expert[u] = s.of[i];
                s.head[u] = i;
            }
            if (full) s.group[groups + __popcll(fulls & lower)] = i;
            experts += __popcll(heads);
            groups += __popcll(fulls);
            if (heads) head = i0 + 63 - __clzll(heads);
        }
        if (threadIdx.x == 0) {
            s.experts = experts;
            s.groups = groups;
            s.head[experts] = s.used;
        }
    }
    __syncthreads();
}

constexpr int kSortThreads = NERF_FEW_PAIRS;
__global__ void __launch_bounds__(kSortThreads) k_mlp_sort(MlpArgs a) {
    __shared__ __attribute__((aligned(16))) Plan s;
    sort_pairs(s, a, 0, a.n * a.k, kSortThreads);
    const int* const from = (const int*)&s;
    for (int i = threadIdx.x; i < (int)(sizeof(Plan) / 4); i += kSortThreads) ((int*)a.plan)[i] = from[i];
}

// ---------------------------------------------------------------------------
// Dot products of R weight rows with M vectors over [k0, k1), by G lanes of a
// wave (lane g of them), a piece of PER elements each at a time.
// ---------------------------------------------------------------------------
template <class T, class X, int R, int M, int G>
__device__ __forceinline__ void dots(float (&acc)[R * M], const T* const (&w)[R], const X* const (&x)[M], int64_t k0,
                                     int64_t k1, int g) {
    constexpr int PER = RowIO<T>::PER, XP = PER / RowIO<X>::PER;
    auto step = [&](const typename RowIO<T>::Vec (&fw)[R], const typename RowIO<X>::Vec (&fx)[M][XP], int skip) {
        float wf[R][PER];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int i = 0; i < PER; ++i) wf[r][i] = i >= skip ? RowIO<T>::get(fw[r], i) : 0.0f;
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const float xf = i >= skip ? RowIO<X>::get(fx[m][i / RowIO<X>::PER], i % RowIO<X>::PER) : 0.0f;
#pragma unroll
                for (int r = 0; r < R; ++r) acc[r * M + m] = fmaf(wf[r][i], xf, acc[r * M + m]);
            }
    };
    int64_t k = k0 + g * PER;
    typename RowIO<T>::Vec fw[R];
    typename RowIO<X>::Vec fx[M][XP];
    // whole pieces
#pragma unroll 2
    for (; k + PER <= k1; k += G * PER) {
#pragma unroll
        for (int r = 0; r < R; ++r) fw[r] = RowIO<T>::load_whole(w[r] + k);
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int j = 0; j < XP; ++j) fx[m][j] = RowIO<X>::load_whole(x[m] + k + j * RowIO<X>::PER);
        step(fw, fx, 0);
    }
    if (k >= k1) return;
    if (k1 - k0 >= PER) {  // the last piece starts earlier, without what the one before has
#pragma unroll
        for (int r = 0; r < R; ++r) fw[r] = RowIO<T>::load_whole(w[r] + k1 - PER);
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int j = 0; j < XP; ++j) fx[m][j] = RowIO<X>::load_whole(x[m] + k1 - PER + j * RowIO<X>::PER);
        step(fw, fx, (int)(k - (k1 - PER)));
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) fw[r] = RowIO<T>::load(w[r], k, k1);
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
            for (int j = 0; j < XP; ++j) {
                fx[m][j] = RowIO<X>::zero();
                if (k + j * RowIO<X>::PER < k1) fx[m][j] = RowIO<X>::load(x[m], k + j * RowIO<X>::PER, k1);
            }
        step(fw, fx, 0);
    }
}

// Sums of N values (a power of two) over G lanes: while N halves, a lane keeps
// one half of the values and hands over the other, so lane g ends up with value
// g / (G / N).  (With fewer lanes than values it keeps N / G of them: not used.)
template <int N, int G>
__device__ __forceinline__ float sum_lanes(float (&v)[N], int g) {
    static_assert(N <= G, "a lane for every value");
    int off = G / 2;
#pragma unroll
    for (int n = N; n > 1; n /= 2, off /= 2) {
        const bool up = g & off;
#pragma unroll
        for (int i = 0; i < n / 2; ++i) {
            const float give = up ? v[i] : v[i + n / 2], keep = up ? v[i + n / 2] : v[i];
            v[i] = keep + __shfl_xor(give, off, 64);
        }
    }
    for (; off >= 1; off /= 2) v[0] += __shfl_xor(v[0], off, 64);
    return v[0];
}

// ---------------------------------------------------------------------------
// The same for up to 16 NG vectors by the matrix units: 16 weight rows (lane l
// holds row l % 16 of the operand) times NG sets of 16 vectors (likewise) over
// [k0, k1), straight from memory to registers; lane l gets rows 4 (l / 16) .. + 3
// of vector l % 16.  Float32 vectors of bfloat16 weights are taken as three
// bfloat16 parts of eight bits each, which hold them exactly: split here, or
// (PLANES: elements of `plane` apart) by whoever wrote them.
// ---------------------------------------------------------------------------
template <class T>
__device__ __forceinline__ f32x4 multiply(const typename RowIO<T>::Vec& w, const typename RowIO<T>::Vec& x, f32x4 acc) {
    if constexpr (sizeof(T) == 2) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.u), __builtin_bit_cast(bf16x8, x.u),
                                                       acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(w.e[j], x.e[j], acc, 0, 0, 0);
        return acc;
    }
}

// The leading eight bits of what is left, three times (an infinity or NaN: itself, then 0).
__device__ __forceinline__ void three_parts(float v, __bf16 (&part)[3]) {
    const bool finite = fabsf(v) <= FLT_MAX;
    const float top = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
    part[0] = (__bf16)(finite ? top : v);
    v = finite ? v - top : 0.0f;
    const float mid = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u);
    part[1] = (__bf16)mid;
    part[2] = (__bf16)(v - mid);
}

template <class T, class X, bool PLANES, int NG>
__device__ __forceinline__ void matrix_dots(f32x4 (&acc)[NG], const T* w, const X* const (&x)[NG], int64_t plane,
                                            int64_t k0, int64_t k1, int lane) {
    using WV = typename RowIO<T>::Vec;
    using XV = typename RowIO<X>::Vec;
    constexpr int PER = RowIO<T>::PER, BK = 4 * PER, AHEAD = 4 / NG;
    constexpr int XP = PLANES ? 3 : PER / RowIO<X>::PER;  // loads of a vector's piece
    const int64_t kx = PLANES ? 0 : RowIO<X>::PER;
#pragma unroll
    for (int n = 0; n < NG; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t kk = k0; kk < k1; kk += AHEAD * BK) {
        WV fw[AHEAD];
        XV fx[AHEAD][NG][XP];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int64_t k = kk + u * BK + (lane >> 4) * PER;
            fw[u] = RowIO<T>::zero();
            if (k < k1) fw[u] = RowIO<T>::load(w, k, k1);
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int j = 0; j < XP; ++j) {
                    fx[u][n][j] = RowIO<X>::zero();
                    if (k + j * kx < k1) fx[u][n][j] = RowIO<X>::load(x[n] + (PLANES ? j * plane : 0), k + j * kx, k1);
                }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
#pragma unroll
            for (int n = 0; n < NG; ++n) {
                if constexpr (PLANES) {
#pragma unroll
                    for (int t = 2; t >= 0; --t) acc[n] = multiply<T>(fw[u], fx[u][n][t], acc[n]);
                } else if constexpr (sizeof(T) == sizeof(X)) {
                    acc[n] = multiply<T>(fw[u], fx[u][n][0], acc[n]);
                } else {
                    WV part[3];
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        __bf16 p[3];
                        three_parts(fx[u][n][i / RowIO<X>::PER].e[i % RowIO<X>::PER], p);
#pragma unroll
                        for (int t = 0; t < 3; ++t) part[t].e[i] = p[t];
                    }
#pragma unroll
                    for (int t = 2; t >= 0; --t) acc[n] = multiply<T>(fw[u], part[t], acc[n]);
                }
            }
    }
}

// Calls f with the number of 16-vector sets that `count` (at most kGroup) pairs take: 1, 2 or 4.
template <class F>
__device__ __forceinline__ void by_sets(int count, F&& f) {
    if (count <= 16)
        f(std::integral_constant<int, 1>{});
    else if (count <= 32)
        f(std::integral_constant<int, 2>{});
    else
        f(std::integral_constant<int, 4>{});
}

// ---------------------------------------------------------------------------
// Hidden layer.  A workgroup takes 16 rows of one expert's W1 (gated: 8 of either
// half) after the other, or 64 of rows that 16 lanes hold.  Dot products: G lanes
// and kHidden rows each (a wave of 1024-wide bfloat16 rows has eight weight loads
// in flight per lane), two pairs at once.  Matrix products: kGroup pairs at once,
// the waves sharing the width.
// ---------------------------------------------------------------------------
constexpr int kHiddenThreads = 256;
constexpr int kHiddenGrid = 1024;
template <bool GATED>
constexpr int kHidden = GATED ? 2 : 4;

template <bool GATED>
__device__ __forceinline__ float activate(const MlpArgs& a, float v, float up) {
    if constexpr (GATED) return v / (1.0f + expf(-v)) * up;
    return a.act == NERF_ACT_RELU && v <= 0.0f ? 0.0f : v;  // (a NaN stays)
}

__device__ __forceinline__ void store_hidden(const MlpArgs& a, int pair, int64_t row, float v) {
    const int64_t at = (int64_t)pair * a.ld_h + row;
    if (a.plane) {
        __bf16 p[3];
        three_parts(v, p);
#pragma unroll
        for (int t = 0; t < 3; ++t) ((__bf16*)a.h)[t * a.plane + at] = p[t];
    } else {
        a.h[at] = v;
    }
}

template <class T, int G, bool GATED, int M, class P>
__device__ __forceinline__ void hidden_rows(const MlpArgs& a, const P& s, int e, int at, int64_t row0, int g) {
    constexpr int H = kHidden<GATED>, R = GATED ? 2 * H : H;
    const int64_t up = GATED ? 2 * (int64_t)a.hidden : a.hidden;
    const T* const base = (const T*)a.w1 + (int64_t)e * up * a.d_in;
    const T* w[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const int64_t row = row0 + i % H < a.hidden ? row0 + i % H : a.hidden - 1;
        w[i] = base + (row + (i / H) * (int64_t)a.hidden) * a.d_in;
    }
    const T* x[M];
    int pair[M];
#pragma unroll
    for (int m = 0; m < M; ++m) {
        pair[m] = s.pair[at + m];
        x[m] = (const T*)a.x + (int64_t)(pair[m] / a.k) * a.ld_x;
    }
    // this lane's value: row and pair i = g / (G / (R M)); the lanes that share it agree
    const int i = g / (G / (R * M)), r = i / M, m = i % M;
    const int64_t row = row0 + r % H;
    const float bias = a.b1 && row < a.hidden ? a.b1[(int64_t)e * up + row + (r / H) * (int64_t)a.hidden] : 0.0f;
    float acc[R * M] = {};
    dots<T, T, R, M, G>(acc, w, x, 0, a.d_in, g);
    float v = sum_lanes<R * M, G>(acc, g) + bias;
    // (gated: the second half's row is in the lanes' upper half)
    v = activate<GATED>(a, v, GATED ? __shfl_xor(v, G / 2, 64) : 0.0f);
    if (r < H && row < a.hidden && g % (G / (R * M)) == 0) {
        int p = pair[0];
#pragma unroll
        for (int j = 1; j < M; ++j) p = m == j ? pair[j] : p;
        store_hidden(a, p, row, v);
    }
}

// Pairs at .. at + count - 1 (at most 16 NG) of expert e.  part: a wave's 16 rows
// x 16 pairs; rows of 64 lanes: each wave takes a quarter of the width, else 16
// rows.
template <class T, int G, bool GATED, int NG, class P>
__device__ __forceinline__ void hidden_matrix(const MlpArgs& a, const P& s, int e, int at, int count, int64_t tile0,
                                              float (*part)[16][17]) {
    constexpr int SHARE = G == 64 ? 4 : 1, H = GATED ? 8 : 16, STEP = 4 * RowIO<T>::PER;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15;
    const int64_t up = GATED ? 2 * (int64_t)a.hidden : a.hidden;
    const int64_t want = tile0 + (wave / SHARE) * H + i % H, row = want < a.hidden ? want : a.hidden - 1;
    const T* const w = (const T*)a.w1 + ((int64_t)e * up + row + (i / H) * (int64_t)a.hidden) * a.d_in;
    const T* x[NG];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        const int j = 16 * n + i < count ? 16 * n + i : count - 1;
        x[n] = (const T*)a.x + (int64_t)(s.pair[at + j] / a.k) * a.ld_x;
    }
    const int64_t per = ((int64_t)a.d_in + SHARE * STEP - 1) / (SHARE * STEP) * STEP;
    const int64_t k0 = wave % SHARE * per, k1 = k0 + per < a.d_in ? k0 + per : a.d_in;
    const int r = threadIdx.x / 16, m = threadIdx.x % 16;
    float bv[4 / SHARE], bu[4 / SHARE];
#pragma unroll
    for (int slab = 0; slab < 4 / SHARE; ++slab) {
        const int64_t hid = tile0 + slab * H + r;
        const bool in = a.b1 && r < H && hid < a.hidden;
        bv[slab] = in ? a.b1[(int64_t)e * up + hid] : 0.0f;
        bu[slab] = in && GATED ? a.b1[(int64_t)e * up + a.hidden + hid] : 0.0f;
    }
    f32x4 d[NG];
    matrix_dots<T, T, false, NG>(d, w, x, 0, k0, k1, lane);
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
        for (int q = 0; q < 4; ++q) part[wave][(lane >> 4) * 4 + q][i] = d[n][q];
        __syncthreads();
#pragma unroll
        for (int slab = 0; slab < 4 / SHARE; ++slab) {
            const int64_t hid = tile0 + slab * H + r;
            if (r >= H || 16 * n + m >= count || hid >= a.hidden) continue;
            float v = bv[slab], u = bu[slab];
#pragma unroll
            for (int p = 0; p < SHARE; ++p) {
                v += part[slab * SHARE + p][r][m];
                if constexpr (GATED) u += part[slab * SHARE + p][r + H][m];
            }
            store_hidden(a, s.pair[at + 16 * n + m], hid, activate<GATED>(a, v, u));
        }
        __syncthreads();
    }
}

template <class T, int G, bool GATED, bool MATRIX, class P>
__device__ __forceinline__ void hidden_tiles(const MlpArgs& a, const P& s, int tiles, float (*part)[16][17]) {
    const int g = threadIdx.x % G;
    for (int it = blockIdx.x; it < (MATRIX ? s.groups : s.experts) * tiles; it += gridDim.x) {
        const int u = it / tiles;
        const int64_t tile0 = (int64_t)(it % tiles) * (kHiddenThreads / G) * kHidden<GATED>;
        if constexpr (MATRIX) {
            const int at = s.group[u], e = s.of[at];
            const int count = (u + 1 < s.groups ? s.group[u + 1] : s.used) - at;
            by_sets(count, [&](auto n) { hidden_matrix<T, G, GATED, decltype(n)::value>(a, s, e, at, count, tile0, part); });
        } else {
            const int e = s.expert[u], end = s.head[u + 1];
            const int64_t row0 = tile0 + threadIdx.x / G * kHidden<GATED>;
            // (a wave passes as a whole)
            if (row0 - (int64_t)((threadIdx.x & 63) / G) * kHidden<GATED> >= a.hidden) continue;
            int at = s.head[u];
            for (; at + 2 <= end; at += 2) hidden_rows<T, G, GATED, 2>(a, s, e, at, row0, g);
            if (at < end) hidden_rows<T, G, GATED, 1>(a, s, e, at, row0, g);
        }
    }
}

template <class T, int G, bool GATED, bool MATRIX, bool PLANNED>
__global__ void __launch_bounds__(kHiddenThreads) k_mlp_hidden(MlpArgs a, int tiles) {
    __shared__ float part[MATRIX ? 4 : 1][16][17];
    if constexpr (PLANNED) {
        hidden_tiles<T, G, GATED, MATRIX>(a, *(const Plan*)a.plan, tiles, part);
    } else {
        __shared__ __attribute__((aligned(16))) Pairs<kSelf> s;
        sort_pairs(s, a, 0, a.n * a.k, kHiddenThreads);
        hidden_tiles<T, G, GATED, MATRIX>(a, s, tiles, part);
    }
}

// ---------------------------------------------------------------------------
// Output layer.  A workgroup owns OT columns of n samples; its waves share the
// (expert, part of the hidden width) items, and the parts [split][slot][OT] meet
// in LDS.  Dot products: OT is up to four, an item a wave's.  Matrix products: 16
// columns, an item up to kGroup pairs; as that is few columns a workgroup, the
// samples are shared out over several, which read the same weights through one
// XCD's L2 (workgroups 8 apart are on the same XCD).
// ---------------------------------------------------------------------------
constexpr int kPartFloats = 16 * NERF_FEW_PAIRS;  // of partial sums
constexpr int kOutGroups = 256;
template <int OT>
constexpr int kOutWaves = OT == 16 ? 16 : 8;

template <class T, int OT, int M, class P>
__device__ __forceinline__ void out_rows(const MlpArgs& a, const P& s, const T* const (&w)[OT], int at, int64_t k0,
                                         int64_t k1, int lane, int first, float* part) {
    const float* x[M];
#pragma unroll
    for (int m = 0; m < M; ++m) x[m] = a.h + (int64_t)(first + s.pair[at + m]) * a.ld_h;
    float acc[OT * M] = {};
    dots<T, float, OT, M, 64>(acc, w, x, k0, k1, lane);
    const float v = sum_lanes<OT * M, 64>(acc, lane);
    const int i = lane / (64 / (OT * M));
    if (lane % (64 / (OT * M)) == 0) part[(at + i % M) * OT + i / M] = v;
}

template <class T, int OT, bool PLANES, class P>
__device__ __forceinline__ void out_columns(const MlpArgs& a, const P& s, int64_t c0, int t0, int n, int room, float* part) {
    constexpr bool WIDE = OT == 16;
    constexpr int STEP = (WIDE ? 4 : 64) * RowIO<T>::PER, WAVES = kOutWaves<OT>;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int first = t0 * a.k, pairs = n * a.k;
    // fewer items than waves: the waves share the hidden width too
    const int whole = WIDE ? s.groups : s.experts, steps = (a.hidden + STEP - 1) / STEP;
    int splits = whole > 0 && whole < WAVES ? WAVES / whole : 1;
    splits = splits < steps ? splits : steps;
    while (splits > 1 && splits * pairs * OT > room) --splits;
    const int64_t per = (int64_t)(steps + splits - 1) / splits * STEP;
    for (int it = wave; it < whole * splits; it += WAVES) {
        const int u = it / splits, ks = it % splits;
        const int64_t k0 = ks * per < a.hidden ? ks * per : a.hidden, k1 = k0 + per < a.hidden ? k0 + per : a.hidden;
        float* const mine = part + (size_t)ks * pairs * OT;
        if constexpr (WIDE) {
            using X = std::conditional_t<PLANES, __bf16, float>;
            const int at = s.group[u], i = lane & 15;
            const int e = s.of[at], count = (u + 1 < s.groups ? s.group[u + 1] : s.used) - at;
            const int64_t col = c0 + i < a.d_out ? c0 + i : a.d_out - 1;
            const T* const w = (const T*)a.w2 + ((int64_t)e * a.d_out + col) * a.hidden;
            by_sets(count, [&](auto sets) {
                constexpr int NG = decltype(sets)::value;
                const X* x[NG];
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    const int j = 16 * g + i < count ? 16 * g + i : count - 1;
                    x[g] = (const X*)a.h + (int64_t)(first + s.pair[at + j]) * a.ld_h;
                }
                f32x4 d[NG];
                matrix_dots<T, X, PLANES, NG>(d, w, x, a.plane, k0, k1, lane);
#pragma unroll
                for (int g = 0; g < NG; ++g)
                    if (16 * g + i < count)
#pragma unroll
                        for (int r = 0; r < 4; ++r) mine[(at + 16 * g + i) * OT + (lane >> 4) * 4 + r] = d[g][r];
            });
        } else {
            const int e = s.expert[u];
            const T* w[OT];
#pragma unroll
            for (int i = 0; i < OT; ++i)
                w[i] = (const T*)a.w2 + ((int64_t)e * a.d_out + (c0 + i < a.d_out ? c0 + i : a.d_out - 1)) * a.hidden;
            int at = s.head[u];
            const int end = s.head[u + 1];
            for (; at + 2 <= end; at += 2) out_rows<T, OT, 2>(a, s, w, at, k0, k1, lane, first, mine);
            if (at < end) out_rows<T, OT, 1>(a, s, w, at, k0, k1, lane, first, mine);
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * OT; i += 64 * WAVES) {
        const int t = i / OT, c = i % OT;
        if (c0 + c >= a.d_out) continue;
        float sum = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int p = t * a.k + j, slot = s.slot[p];
            if (slot < 0) continue;
            float y = a.b2 ? a.b2[(int64_t)(s.key[p] >> kKeyBits) * a.d_out + c0 + c] : 0.0f;
            for (int ks = 0; ks < splits; ++ks) y += part[((size_t)ks * pairs + slot) * OT + c];
            sum = fmaf(a.weights ? a.weights[first + p] : 1.0f, y, sum);
        }
        ((T*)a.out)[(int64_t)(t0 + t) * a.ld_out + c0 + c] = (T)sum;
    }
}

template <class T, int OT, bool PLANNED, bool PLANES>
__global__ void __launch_bounds__(64 * kOutWaves<OT>) k_mlp_out(MlpArgs a, int tiles, int samples, int groups, int room) {
    extern __shared__ float part[];  // `room` floats
    // tiles in steps of 8, each step's 8 groups of samples after one another
    const int step = blockIdx.x / (8 * groups), in = blockIdx.x % (8 * groups);
    const int tile = 8 * step + in % 8;
    if (tile >= tiles) return;
    if constexpr (PLANNED) {
        out_columns<T, OT, PLANES>(a, *(const Plan*)a.plan, (int64_t)tile * OT, 0, a.n, room, part);
    } else {
        __shared__ __attribute__((aligned(16))) Pairs<kSelf> s;
        const int t0 = in / 8 * samples, n = t0 + samples < a.n ? samples : a.n - t0;
        sort_pairs(s, a, t0 * a.k, n * a.k, 64 * kOutWaves<OT>);
        out_columns<T, OT, PLANES>(a, s, (int64_t)tile * OT, t0, n, room, part);
    }
}

template <class T, int G, bool MATRIX>
void launch_hidden(const MlpArgs& a, hipStream_t s) {
    const int pairs = a.n * a.k, experts = pairs < a.n_experts ? pairs : a.n_experts;
    const bool gated = a.act == NERF_ACT_GATED;
    const int per = kHiddenThreads / G * (gated ? kHidden<true> : kHidden<false>);
    const int tiles = (a.hidden + per - 1) / per;
    // workgroups that stay sort the pairs once for several tiles
    const int64_t items = (int64_t)(experts + pairs / kGroup) * tiles;
    const unsigned grid = (unsigned)(items < kHiddenGrid ? items : kHiddenGrid);
    auto go = [&](auto gate, auto planned) {
        k_mlp_hidden<T, G, decltype(gate)::value, MATRIX, decltype(planned)::value>
            <<<grid, kHiddenThreads, 0, s>>>(a, tiles);
    };
    using std::false_type;
    using std::true_type;
    if (pairs > kSelf)
        gated ? go(true_type{}, true_type{}) : go(false_type{}, true_type{});
    else
        gated ? go(true_type{}, false_type{}) : go(false_type{}, false_type{});
}

template <class T, int OT>
void launch_out(const MlpArgs& a, hipStream_t s) {
    constexpr bool MATRIX = OT == 16;
    const int tiles = (a.d_out + OT - 1) / OT;
    // few columns: the samples are shared out too, until there is a workgroup for every CU
    // (and, for matrix products, as many as a workgroup sorts itself)
    int groups = kOutGroups / tiles;
    groups = groups < 1 ? 1 : groups > a.n ? a.n : groups;
    int samples = (a.n + groups - 1) / groups;
    if (MATRIX && samples * a.k > kSelf) samples = kSelf / a.k;
    const bool planned = samples * a.k > kSelf;
    if (planned) samples = a.n;
    groups = (a.n + samples - 1) / samples;
    // (512 pairs of 16 columns fit once)
    const int all = samples * a.k * OT * kOutWaves<OT>, room = all < kPartFloats ? all : kPartFloats;
    const unsigned grid = (unsigned)((tiles + 7) / 8 * 8 * groups);
    auto go = [&](auto plan, auto planes) {
        k_mlp_out<T, OT, decltype(plan)::value, decltype(planes)::value>
            <<<grid, 64 * kOutWaves<OT>, room * sizeof(float), s>>>(a, tiles, samples, groups, room);
    };
    using std::false_type;
    using std::true_type;
    if constexpr (MATRIX) {
        if constexpr (sizeof(T) == 2) {
            if (a.plane) return go(false_type{}, true_type{});
        }
        go(false_type{}, false_type{});
    } else {
        planned ? go(true_type{}, false_type{}) : go(false_type{}, false_type{});
    }
}

template <class T, bool MATRIX>
void launch_layers(const MlpArgs& a, hipStream_t s) {
    if (a.d_in <= 16 * RowIO<T>::PER)
        launch_hidden<T, 16, MATRIX>(a, s);
    else
        launch_hidden<T, 64, MATRIX>(a, s);
    if constexpr (MATRIX) {
        launch_out<T, 16>(a, s);
    } else {
        if (a.d_out >= 1024)
            launch_out<T, 4>(a, s);
        else if (a.d_out >= 512)
            launch_out<T, 2>(a, s);
        else
            launch_out<T, 1>(a, s);
    }
}

template <class T>
void launch(MlpArgs a, hipStream_t s) {
    const int pairs = a.n * a.k;
    const bool matrix = pairs > 2 * a.n_experts;
    // the hidden values' three parts are written once if many pairs are read again and again
    a.plane = matrix && pairs > kSelf && sizeof(T) == 2 ? pairs * a.ld_h : 0;
    if (pairs > kSelf) k_mlp_sort<<<1, kSortThreads, 0, s>>>(a);
    if (matrix)
        launch_layers<T, true>(a, s);
    else
        launch_layers<T, false>(a, s);
}

}  // namespace

void launch_routed_mlp(bool bf16, const MlpArgs& a, hipStream_t s) {
    if (bf16)
        launch<__bf16>(a, s);
    else
        launch<float>(a, s);
}

}  // namespace nerf
