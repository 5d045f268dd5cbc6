// The whole two-layer routed field for a few samples, for gfx950:
//   out_t = sum_j w_tj (W2_e act(W1_e x_t + b1_e) + b2_e),   e = ids_tj.
// Every weight of an expert that some pair (sample, choice) uses is read from
// memory once; with few pairs per expert that read bounds the kernels, and for one
// sample the launches and one chain of dependent loads each.  Up to 64 pairs are sorted by expert by every
// workgroup itself, in LDS, which is cheaper than a kernel in front; more (the work
// grows with their square) by a kernel of their own.
// With up to two pairs per expert, on average over all of them, two kernels of dot
// products, whose weights a wave reads in whole lines.  First the hidden layer: workgroups take
// tiles of one expert's W1 and apply them to all its pairs.  Then the output:
// workgroups own columns, for all experts, so that a sample's k terms meet in LDS
// and are added in the order of its choices, without atomics.  An expert's pairs go
// through a tile two at a time, so ids that collapse onto one of many experts make
// it as many reads of that expert from the caches (bfloat16 1024 -> 1024 -> 1024, 512
// pairs over 256 experts 279 us, all of one 775).
// With more pairs the vector units would take longer than the read, and a column's
// owner would have too much of it: either layer goes through the matrix units, 16
// pairs at a time, and a third kernel adds up the samples' terms.  There the pairs'
// vectors, read again for every 16 rows of weights and three parts each in the
// second bfloat16 layer, cost more than the weights.
// Hidden values keep 24 bits between the kernels (rounding them to bfloat16 would
// add an error as large as the output's own rounding, and saves only L2 traffic).
// Measured, weights from memory: one sample through 2 of 16 experts 1024 -> 4096 ->
// 1024, bfloat16, 13.2 us (32.6 MB, 2.5 TB/s); 16 samples through 4 of 64 gated experts
// of 1024, 66 us (256 MB, 3.9 TB/s); 64 through 2 of 8 experts 1024 -> 4096 -> 1024, 81 us
// (134 MB; kernels of 5, 29, 47 and 5).
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
    float weight[N];  // of a pair
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
        const float weight = p < pairs && a.weights ? a.weights[first + p] : 1.0f;
        s.key[p] = ((unsigned)id < (unsigned)a.n_experts ? id : a.n_experts) << kKeyBits | p;
        s.weight[p] = weight;
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
    // whole pieces; a second step in flight costs bfloat16 more in registers than it hides (16 streams through 4 of
    // 64 gated experts 62 us with one, 71 with two; 128 float32 samples through 4 of 256 experts 161 and 145)
    constexpr int STEPS = sizeof(T) == 2 ? 1 : 2;
#pragma unroll STEPS
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

// Sums of N values (a power of two, G at most) over G lanes: while N halves, a lane
// keeps one half of the values and hands over the other, so lane g ends up with
// value g / (G / N).
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
// of vector l % 16.  PARTS: the vectors are sums of so many, `plane` elements
// apart.
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

template <class T, int PARTS, int NG>
__device__ __forceinline__ void matrix_dots(f32x4 (&acc)[NG], const T* w, const T* const (&x)[NG], int64_t plane,
                                            int64_t k0, int64_t k1, int lane) {
    using Vec = typename RowIO<T>::Vec;
    // loads in flight, as far as registers go
    constexpr int PER = RowIO<T>::PER, BK = 4 * PER, AHEAD = PARTS == 1 ? (NG == 1 ? 6 : NG == 2 ? 4 : 3) : NG == 1 ? 4 : 2;
#pragma unroll
    for (int n = 0; n < NG; ++n) acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int64_t kk = k0; kk < k1; kk += AHEAD * BK) {
        Vec fw[AHEAD], fx[AHEAD][NG][PARTS];
#pragma unroll
        for (int u = 0; u < AHEAD; ++u) {
            const int64_t k = kk + u * BK + (lane >> 4) * PER;
            fw[u] = RowIO<T>::zero();
            if (k < k1) fw[u] = RowIO<T>::load(w, k, k1);
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int t = 0; t < PARTS; ++t) {
                    fx[u][n][t] = RowIO<T>::zero();
                    if (k < k1) fx[u][n][t] = RowIO<T>::load(x[n] + t * plane, k, k1);
                }
        }
#pragma unroll
        for (int u = 0; u < AHEAD; ++u)
#pragma unroll
            for (int n = 0; n < NG; ++n)
#pragma unroll
                for (int t = PARTS - 1; t >= 0; --t) acc[n] = multiply<T>(fw[u], fx[u][n][t], acc[n]);
    }
}

// The leading eight bits of what is left, three times: bfloat16 numbers that add
// up to a float32 one.  A part of 0 beside others would make NaN of an infinite
// weight's product, so where nothing is left the part before is shared out (from
// 2^-96 on halves and quarters of eight bits are exact and normal; below, such a
// product is infinite or NaN), and an infinity or NaN is all three parts.
__device__ __forceinline__ void three_parts(float v, __bf16 (&part)[3]) {
    const float top = __uint_as_float(__float_as_uint(v) & 0xFFFF0000u), rest = v - top;
    const float mid = __uint_as_float(__float_as_uint(rest) & 0xFFFF0000u), low = rest - mid;
    float p[3] = {top, mid, low};
    if (!(fabsf(v) <= FLT_MAX)) {
        p[0] = p[1] = p[2] = v;
    } else if (fabsf(v) >= 0x1p-96f) {
        if (rest == 0.0f) {
            p[0] = 0.5f * top;
            p[1] = p[2] = 0.25f * top;
        } else if (low == 0.0f) {
            p[1] = p[2] = 0.5f * mid;
        }
    }
#pragma unroll
    for (int t = 0; t < 3; ++t) part[t] = (__bf16)p[t];
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
// Hidden layer by dot products.  A workgroup takes 16 rows of one expert's W1
// (gated: 8 of either half) after the other, more of rows that fewer than 64 lanes
// hold; G lanes take kHidden rows (a wave of 1024-wide bfloat16 rows has eight
// weight loads in flight per lane) and two pairs at once.
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
        a.h[(int64_t)p * a.ld_h + row] = v;
    }
}

template <class T, int G, bool GATED, class P>
__device__ __forceinline__ void hidden_tiles(const MlpArgs& a, const P& s, int tiles) {
    const int g = threadIdx.x % G;
    for (int it = blockIdx.x; it < s.experts * tiles; it += gridDim.x) {
        const int u = it / tiles, e = s.expert[u], end = s.head[u + 1];
        const int64_t row0 = ((int64_t)(it % tiles) * (kHiddenThreads / G) + threadIdx.x / G) * kHidden<GATED>;
        // (a wave passes as a whole)
        if (row0 - (int64_t)((threadIdx.x & 63) / G) * kHidden<GATED> >= a.hidden) continue;
        int at = s.head[u];
        for (; at + 2 <= end; at += 2) hidden_rows<T, G, GATED, 2>(a, s, e, at, row0, g);
        if (at < end) hidden_rows<T, G, GATED, 1>(a, s, e, at, row0, g);
    }
}

template <class T, int G, bool GATED, bool PLANNED>
__global__ void __launch_bounds__(kHiddenThreads) k_mlp_hidden(MlpArgs a, int tiles) {
    if constexpr (PLANNED) {
        hidden_tiles<T, G, GATED>(a, *(const Plan*)a.plan, tiles);
    } else {
        __shared__ __attribute__((aligned(16))) Pairs<kSelf> s;
        sort_pairs(s, a, 0, a.n * a.k, kHiddenThreads);
        hidden_tiles<T, G, GATED>(a, s, tiles);
    }
}

// ---------------------------------------------------------------------------
// Either layer by matrix products: a workgroup takes 16 rows of one expert's
// weights and up to kGroup of its pairs, its four waves a quarter of the width each
// (rows that 16 lanes hold: 64 rows, 16 a wave).  The hidden layer's values go out
// in bfloat16 parts (FIRST), the output layer's per pair, to be summed by
// k_mlp_combine.
// ---------------------------------------------------------------------------
template <class T, bool FIRST, int SHARE, bool GATED, int NG, class P>
__device__ __forceinline__ void matrix_tile(const MlpArgs& a, const P& s, int e, int at, int count, int64_t tile0,
                                            float (*part)[16][17]) {
    constexpr int H = GATED ? 8 : 16, STEP = 4 * RowIO<T>::PER, PARTS = FIRST || sizeof(T) == 4 ? 1 : 3;
    constexpr int SLABS = SHARE == 1 ? 4 : 1;  // of 16 rows
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i = lane & 15;
    const int64_t rows = FIRST ? a.hidden : a.d_out, width = FIRST ? a.d_in : a.hidden, all = GATED ? 2 * rows : rows;
    const float* const bias = FIRST ? a.b1 : a.b2;
    const int64_t want = tile0 + (wave / SHARE) * H + i % H, row = want < rows ? want : rows - 1;
    const T* const w = (const T*)(FIRST ? a.w1 : a.w2) + ((int64_t)e * all + row + (i / H) * rows) * width;
    const T* x[NG];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
        const int pair = s.pair[at + (16 * n + i < count ? 16 * n + i : count - 1)];
        x[n] = FIRST ? (const T*)a.x + (int64_t)(pair / a.k) * a.ld_x : (const T*)a.h + (int64_t)pair * a.ld_h;
    }
    const int64_t per = (width + SHARE * STEP - 1) / (SHARE * STEP) * STEP;
    const int64_t k0 = wave % SHARE * per, k1 = k0 + per < width ? k0 + per : width;
    const int r = threadIdx.x / 16, m = threadIdx.x % 16;
    float bv[SLABS], bu[SLABS];
#pragma unroll
    for (int slab = 0; slab < SLABS; ++slab) {
        const int64_t out = tile0 + slab * H + r;
        const bool in = bias && r < H && out < rows;
        bv[slab] = in ? bias[(int64_t)e * all + out] : 0.0f;
        bu[slab] = in && GATED ? bias[(int64_t)e * all + rows + out] : 0.0f;
    }
    f32x4 d[NG];
    matrix_dots<T, PARTS, NG>(d, w, x, a.plane, k0, k1, lane);
#pragma unroll
    for (int n = 0; n < NG; ++n) {
#pragma unroll
        for (int q = 0; q < 4; ++q) part[wave][(lane >> 4) * 4 + q][i] = d[n][q];
        __syncthreads();
#pragma unroll
        for (int slab = 0; slab < SLABS; ++slab) {
            const int64_t out = tile0 + slab * H + r;
            if (r >= H || 16 * n + m >= count || out >= rows) continue;
            float v = bv[slab], u = bu[slab];
#pragma unroll
            for (int p = 0; p < SHARE; ++p) {
                v += part[slab * SHARE + p][r][m];
                if constexpr (GATED) u += part[slab * SHARE + p][r + H][m];
            }
            const int pair = s.pair[at + 16 * n + m];
            if constexpr (!FIRST) {
                a.y[(int64_t)pair * a.d_out + out] = v;
            } else if constexpr (sizeof(T) == 4) {
                a.h[(int64_t)pair * a.ld_h + out] = activate<GATED>(a, v, u);
            } else {
                __bf16 parts[3];
                three_parts(activate<GATED>(a, v, u), parts);
#pragma unroll
                for (int t = 0; t < 3; ++t) ((__bf16*)a.h)[t * a.plane + (int64_t)pair * a.ld_h + out] = parts[t];
            }
        }
        __syncthreads();
    }
}

template <class T, bool FIRST, int SHARE, bool GATED, class P>
__device__ __forceinline__ void matrix_tiles(const MlpArgs& a, const P& s, int tiles, float (*part)[16][17]) {
    for (int it = blockIdx.x; it < s.groups * tiles; it += gridDim.x) {
        const int u = it / tiles, at = s.group[u], e = s.of[at];
        const int count = (u + 1 < s.groups ? s.group[u + 1] : s.used) - at;
        const int64_t tile0 = (int64_t)(it % tiles) * (SHARE == 1 ? 4 : 1) * (GATED ? 8 : 16);
        by_sets(count, [&](auto n) {
            matrix_tile<T, FIRST, SHARE, GATED, decltype(n)::value>(a, s, e, at, count, tile0, part);
        });
    }
}

template <class T, bool FIRST, int SHARE, bool GATED, bool PLANNED>
__global__ void __launch_bounds__(kHiddenThreads) k_mlp_matrix(MlpArgs a, int tiles) {
    __shared__ float part[4][16][17];
    if constexpr (PLANNED) {
        matrix_tiles<T, FIRST, SHARE, GATED>(a, *(const Plan*)a.plan, tiles, part);
    } else {
        __shared__ __attribute__((aligned(16))) Pairs<kSelf> s;
        sort_pairs(s, a, 0, a.n * a.k, kHiddenThreads);
        matrix_tiles<T, FIRST, SHARE, GATED>(a, s, tiles, part);
    }
}

// out[t] = sum_j weights_tj y_tj, j ascending, over the choices with an expert.
template <class T>
__global__ void __launch_bounds__(256) k_mlp_combine(MlpArgs a) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t t = i / a.d_out, c = i % a.d_out;
    if (t >= a.n) return;
    float sum = 0.0f;
#pragma unroll 4
    for (int j = 0; j < a.k; ++j) {
        const int64_t p = t * a.k + j;
        const float w = a.weights ? a.weights[p] : 1.0f, y = a.y[p * a.d_out + c];
        sum = (unsigned)a.ids[p] < (unsigned)a.n_experts ? fmaf(w, y, sum) : sum;
    }
    ((T*)a.out)[t * a.ld_out + c] = (T)sum;
}

// ---------------------------------------------------------------------------
// Output layer by dot products.  A workgroup owns OT columns of n samples; its
// waves share the (expert, part of the hidden width) items, and the parts
// [split][slot][OT] meet in LDS.
// ---------------------------------------------------------------------------
constexpr int kOutWaves = 8, kOutThreads = 64 * kOutWaves;
constexpr int kPartFloats = 16 * NERF_FEW_PAIRS;  // of partial sums
constexpr int kOutGroups = 256;

template <class T, int OT, int G, int M, class P>
__device__ __forceinline__ void out_rows(const MlpArgs& a, const P& s, const T* const (&w)[OT], const float* bias, int at,
                                         int64_t k0, int64_t k1, int g, int first, float* part) {
    const float* x[M];
#pragma unroll
    for (int m = 0; m < M; ++m) x[m] = a.h + (int64_t)(first + s.pair[at + m]) * a.ld_h;
    const int i = g / (G / (OT * M));
    const float b = bias ? bias[i / M] : 0.0f;
    float acc[OT * M] = {};
    dots<T, float, OT, M, G>(acc, w, x, k0, k1, g);
    const float v = sum_lanes<OT * M, G>(acc, g) + b;
    if (g % (G / (OT * M)) == 0) part[(at + i % M) * OT + i / M] = v;
}

template <class T, int OT, int G, class P>
__device__ __forceinline__ void out_columns(const MlpArgs& a, const P& s, int64_t c0, int t0, int n, int room, float* part) {
    constexpr int STEP = G * RowIO<T>::PER, SUB = 64 / G, GROUPS = kOutWaves * SUB;
    const int g = threadIdx.x % G, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int first = t0 * a.k, pairs = n * a.k;
    // fewer experts than waves: the waves share the hidden width too
    const int steps = (a.hidden + STEP - 1) / STEP;
    int splits = s.experts > 0 && s.experts < GROUPS ? GROUPS / s.experts : 1;
    splits = splits < steps ? splits : steps;
    while (splits > 1 && splits * pairs * OT > room) --splits;
    const int64_t per = (int64_t)(steps + splits - 1) / splits * STEP;
    const bool all = c0 + OT <= a.d_out;  // (else the last column's bias is read for those past it)
    for (int it = wave * SUB + (SUB > 1 ? threadIdx.x % 64 / G : 0); it < s.experts * splits; it += GROUPS) {
        const int u = it / splits, ks = it % splits, e = s.expert[u];
        const T* w[OT];
#pragma unroll
        for (int i = 0; i < OT; ++i)
            w[i] = (const T*)a.w2 + ((int64_t)e * a.d_out + (c0 + i < a.d_out ? c0 + i : a.d_out - 1)) * a.hidden;
        const int64_t k0 = ks * per < a.hidden ? ks * per : a.hidden, k1 = k0 + per < a.hidden ? k0 + per : a.hidden;
        float* const mine = part + (size_t)ks * pairs * OT;
        const float* const bias = a.b2 && ks == 0 && all ? a.b2 + (int64_t)e * a.d_out + c0 : nullptr;
        int at = s.head[u];
        const int end = s.head[u + 1];
        for (; at + 2 <= end; at += 2) out_rows<T, OT, G, 2>(a, s, w, bias, at, k0, k1, g, first, mine);
        if (at < end) out_rows<T, OT, G, 1>(a, s, w, bias, at, k0, k1, g, first, mine);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * OT; i += kOutThreads) {
        const int t = i / OT, c = i % OT;
        if (c0 + c >= a.d_out) continue;
        float sum = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int p = t * a.k + j, slot = s.slot[p];
            if (slot < 0) continue;
            float y = a.b2 && !all ? a.b2[(int64_t)(s.key[p] >> kKeyBits) * a.d_out + c0 + c] : 0.0f;
            for (int ks = 0; ks < splits; ++ks) y += part[((size_t)ks * pairs + slot) * OT + c];
            sum = fmaf(s.weight[p], y, sum);
        }
        ((T*)a.out)[(int64_t)(t0 + t) * a.ld_out + c0 + c] = (T)sum;
    }
}

template <class T, int OT, int G, bool PLANNED>
__global__ void __launch_bounds__(kOutThreads) k_mlp_out(MlpArgs a, int tiles, int samples, int room) {
    extern __shared__ float part[];  // `room` floats
    const int64_t c0 = (int64_t)(blockIdx.x % tiles) * OT;
    if constexpr (PLANNED) {
        out_columns<T, OT, G>(a, *(const Plan*)a.plan, c0, 0, a.n, room, part);
    } else {
        __shared__ __attribute__((aligned(16))) Pairs<kSelf> s;
        const int t0 = blockIdx.x / tiles * samples, n = t0 + samples < a.n ? samples : a.n - t0;
        sort_pairs(s, a, t0 * a.k, n * a.k, kOutThreads);
        out_columns<T, OT, G>(a, s, c0, t0, n, room, part);
    }
}

template <class F>
void by_flags(bool gated, bool planned, F&& f) {
    using std::false_type;
    using std::true_type;
    if (planned)
        gated ? f(true_type{}, true_type{}) : f(false_type{}, true_type{});
    else
        gated ? f(true_type{}, false_type{}) : f(false_type{}, false_type{});
}

// Workgroups that stay sort the pairs once for several tiles.
unsigned staying_grid(const MlpArgs& a, int tiles) {
    const int pairs = a.n * a.k, experts = pairs < a.n_experts ? pairs : a.n_experts;
    const int64_t items = (int64_t)(experts + pairs / kGroup) * tiles;
    return (unsigned)(items < kHiddenGrid ? items : kHiddenGrid);
}

template <class T, int G>
void launch_hidden(const MlpArgs& a, hipStream_t s) {
    const bool gated = a.act == NERF_ACT_GATED;
    const int per = kHiddenThreads / G * (gated ? kHidden<true> : kHidden<false>);
    const int tiles = (a.hidden + per - 1) / per;
    by_flags(gated, a.n * a.k > kSelf, [&](auto gate, auto planned) {
        k_mlp_hidden<T, G, decltype(gate)::value, decltype(planned)::value>
            <<<staying_grid(a, tiles), kHiddenThreads, 0, s>>>(a, tiles);
    });
}

template <class T, int OT, int G = 64>
void launch_out(const MlpArgs& a, hipStream_t s) {
    const int tiles = (a.d_out + OT - 1) / OT;
    // few columns: the samples are shared out too, until there is a workgroup for every CU
    int groups = kOutGroups / tiles;
    groups = groups < 1 ? 1 : groups > a.n ? a.n : groups;
    int samples = (a.n + groups - 1) / groups;
    const bool planned = samples * a.k > kSelf;
    if (planned) samples = a.n;
    groups = (a.n + samples - 1) / samples;
    const int all = samples * a.k * OT * kOutWaves, room = all < kPartFloats ? all : kPartFloats;
    const unsigned grid = (unsigned)(tiles * groups);
    if (planned)
        k_mlp_out<T, OT, G, true><<<grid, kOutThreads, room * sizeof(float), s>>>(a, tiles, samples, room);
    else
        k_mlp_out<T, OT, G, false><<<grid, kOutThreads, room * sizeof(float), s>>>(a, tiles, samples, room);
}

template <class T, bool FIRST, int SHARE>
void launch_matrix(const MlpArgs& a, hipStream_t s) {
    const bool gated = FIRST && a.act == NERF_ACT_GATED;
    const int per = (SHARE == 1 ? 4 : 1) * (gated ? 8 : 16), rows = FIRST ? a.hidden : a.d_out;
    const int tiles = (rows + per - 1) / per;
    by_flags(gated, a.n * a.k > kSelf, [&](auto gate, auto planned) {
        k_mlp_matrix<T, FIRST, SHARE, FIRST && decltype(gate)::value, decltype(planned)::value>
            <<<staying_grid(a, tiles), kHiddenThreads, 0, s>>>(a, tiles);
    });
}

template <class T, bool FIRST>
void launch_matrix_layer(const MlpArgs& a, hipStream_t s) {
    // (16 waves a tile: 64 samples through two of 8 experts 1024 -> 4096 -> 1024 74 to 83 us instead of 69)
    if ((FIRST ? a.d_in : a.hidden) <= 16 * RowIO<T>::PER)
        launch_matrix<T, FIRST, 1>(a, s);
    else
        launch_matrix<T, FIRST, 4>(a, s);
}

template <class T>
void launch(MlpArgs a, hipStream_t s) {
    const int pairs = a.n * a.k;
    if (pairs > kSelf) k_mlp_sort<<<1, kSortThreads, 0, s>>>(a);
    if (pairs > 2 * a.n_experts) {
        a.plane = pairs * a.ld_h;
        launch_matrix_layer<T, true>(a, s);
        launch_matrix_layer<T, false>(a, s);
        k_mlp_combine<T><<<(unsigned)(((int64_t)a.n * a.d_out + 255) / 256), 256, 0, s>>>(a);
        return;
    }
    // rows of few pieces take few lanes
    const int in = (a.d_in + RowIO<T>::PER - 1) / RowIO<T>::PER, hidden = (a.hidden + RowIO<T>::PER - 1) / RowIO<T>::PER;
    if (in <= 8)
        launch_hidden<T, 8>(a, s);
    else if (in <= 16)
        launch_hidden<T, 16>(a, s);
    else if (in <= 32)
        launch_hidden<T, 32>(a, s);
    else
        launch_hidden<T, 64>(a, s);
    // columns a workgroup: the more, the fewer reads of the hidden values; the fewer, the more workgroups (16
    // streams through 4 of 64 experts 1024 -> 1024: four 78 us, two 71; one sample through 4096 -> 1024: 11.6, 11.9)
    if (hidden <= 16)
        launch_out<T, 4, 16>(a, s);
    else if (hidden <= 32)
        launch_out<T, 4, 32>(a, s);
    else if (a.d_out >= 4096)
        launch_out<T, 4>(a, s);
    else if (a.d_out >= 512)
        launch_out<T, 2>(a, s);
    else
        launch_out<T, 1>(a, s);
}

}  // namespace

void launch_routed_mlp(bool bf16, const MlpArgs& a, hipStream_t s) {
    if (bf16)
        launch<__bf16>(a, s);
    else
        launch<float>(a, s);
}

}  // namespace nerf
