// The whole two-layer routed field for a few samples, for gfx950:
//   out_t = sum_j w_tj (W2_e act(W1_e x_t + b1_e) + b2_e),   e = ids_tj,
// in two kernels.  Every weight of an expert that some pair (sample, choice)
// uses is read from memory once; that read bounds both kernels, and for one
// sample the launches and one chain of dependent loads each.  A workgroup sorts
// the (at most 512) pairs by expert itself, in LDS, which is cheaper than a
// kernel in front.  k_mlp_hidden: workgroups own rows of one expert's W1 and
// apply them to all its pairs.  k_mlp_out: workgroups own columns of the
// output, for all experts, so that a sample's k terms meet in LDS and are added
// in the order of its choices, without atomics.  The hidden values stay in
// float32 between the two (rounding them to bfloat16 would add an error as
// large as the output's own rounding, and saves only L2 traffic).  Products are
// scalar: with few pairs per weight the matrix units would wait for memory all
// the same, at 16 columns of which most are empty.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "fields.hpp"
#include "rowio.hpp"

namespace nerf {

namespace {

constexpr int kPairs = NERF_FEW_PAIRS;

// ---------------------------------------------------------------------------
// Pairs sorted by expert, stably: pair[s] for s < used, and the experts that
// have any: expert[u] owns slots head[u] .. head[u + 1] - 1.
// ---------------------------------------------------------------------------
struct Pairs {
    int id[kPairs];      // expert of a pair (E: none)
    int pair[kPairs];    // of a slot
    int of[kPairs];      // expert of a slot
    int slot[kPairs];    // of a pair, -1 without an expert
    int expert[kPairs];
    int head[kPairs + 1];
    int experts, used;
};

// (Every thread of the workgroup; a pair's slot is the number of pairs with a
// smaller expert, or the same and earlier.)
__device__ __forceinline__ void sort_pairs(Pairs& s, const MlpArgs& a, int pairs, int threads) {
    const int padded = (pairs + 3) & ~3;
    if (threadIdx.x == 0) s.experts = s.used = 0;
    for (int p = threadIdx.x; p < padded; p += threads) {
        const int id = p < pairs ? a.ids[p] : -1;
        s.id[p] = (unsigned)id < (unsigned)a.n_experts ? id : a.n_experts;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += threads) {
        const int e = s.id[p];
        int slot = 0, before = 0;
        for (int q = 0; q < padded; q += 4) {
            const int4 o = *(const int4*)&s.id[q];
            const int v[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int same = v[i] == e && q + i < p;
                slot += v[i] < e || same;
                before += same;
            }
        }
        const bool live = e < a.n_experts;
        s.slot[p] = live ? slot : -1;
        if (live) {
            s.pair[slot] = p;
            s.of[slot] = e;
            atomicAdd(&s.used, 1);
            if (before == 0) atomicAdd(&s.experts, 1);
        }
    }
    __syncthreads();
    // a slot that starts an expert finds how many do before it
    for (int i = threadIdx.x; i < s.used; i += threads) {
        if (i > 0 && s.of[i - 1] == s.of[i]) continue;
        int u = 0;
        for (int j = 1; j <= i; ++j) u += s.of[j] != s.of[j - 1];
        s.expert[u] = s.of[i];
        s.head[u] = i;
    }
    if (threadIdx.x == 0) s.head[s.experts] = s.used;
    __syncthreads();
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
// Hidden layer.  grid: [experts touched at most][row tiles]; each group of G
// lanes takes kHidden rows of W1 (gated: as many of either half), so a wave of
// 1024-wide bfloat16 rows has eight weight loads in flight per lane.
// ---------------------------------------------------------------------------
constexpr int kHiddenThreads = 256;
template <bool GATED>
constexpr int kHidden = GATED ? 2 : 4;

template <class T, int G, bool GATED, int M>
__device__ __forceinline__ void hidden_rows(const MlpArgs& a, const Pairs& s, int e, int at, int64_t row0, int g) {
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
    float acc[R * M] = {};
    dots<T, T, R, M, G>(acc, w, x, 0, a.d_in, g);
    float v = sum_lanes<R * M, G>(acc, g);
    // this lane's value: row and pair i = g / (G / (R M)); the lanes that share it agree
    const int i = g / (G / (R * M)), r = i / M, m = i % M;
    const int64_t row = row0 + r % H;
    if (a.b1 && row < a.hidden) v += a.b1[(int64_t)e * up + row + (r / H) * (int64_t)a.hidden];
    if constexpr (GATED) {
        const float other = __shfl_xor(v, G / 2, 64);  // the second half's row, in the lanes' upper half
        v = v / (1.0f + expf(-v)) * other;
    } else if (a.act == NERF_ACT_RELU) {
        v = v <= 0.0f ? 0.0f : v;  // (a NaN stays)
    }
    if (r < H && row < a.hidden && g % (G / (R * M)) == 0) {
        int p = pair[0];
#pragma unroll
        for (int j = 1; j < M; ++j) p = m == j ? pair[j] : p;
        a.h[(int64_t)p * a.ld_h + row] = v;
    }
}

template <class T, int G, bool GATED>
__global__ void __launch_bounds__(kHiddenThreads) k_mlp_hidden(MlpArgs a, int tiles) {
    __shared__ __attribute__((aligned(16))) Pairs s;
    sort_pairs(s, a, a.n * a.k, kHiddenThreads);
    const int u = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    if (u >= s.experts) return;
    const int e = s.expert[u], g = threadIdx.x % G;
    const int64_t row0 = ((int64_t)tile * (kHiddenThreads / G) + threadIdx.x / G) * kHidden<GATED>;
    if (row0 - (int64_t)((threadIdx.x & 63) / G) * kHidden<GATED> >= a.hidden) return;  // (a wave leaves as a whole)
    int at = s.head[u];
    const int end = s.head[u + 1];
    for (; at + 4 <= end; at += 4) hidden_rows<T, G, GATED, 4>(a, s, e, at, row0, g);
    if (at + 2 <= end) {
        hidden_rows<T, G, GATED, 2>(a, s, e, at, row0, g);
        at += 2;
    }
    if (at < end) hidden_rows<T, G, GATED, 1>(a, s, e, at, row0, g);
}

// ---------------------------------------------------------------------------
// Output layer.  A workgroup owns OT columns; its waves share the (expert, part
// of the hidden width) items.  part: [split][slot][OT].
// ---------------------------------------------------------------------------
constexpr int kOutWaves = 8, kOutThreads = 64 * kOutWaves;
constexpr size_t kPartBytes = 32768;

template <class T, int OT, int M>
__device__ __forceinline__ void out_rows(const MlpArgs& a, const Pairs& s, const T* const (&w)[OT], int at, int64_t k0,
                                         int64_t k1, int lane, float* part) {
    const float* x[M];
#pragma unroll
    for (int m = 0; m < M; ++m) x[m] = a.h + (int64_t)s.pair[at + m] * a.ld_h;
    float acc[OT * M] = {};
    dots<T, float, OT, M, 64>(acc, w, x, k0, k1, lane);
    const float v = sum_lanes<OT * M, 64>(acc, lane);
    const int i = lane / (64 / (OT * M));
    if (lane % (64 / (OT * M)) == 0) part[(at + i % M) * OT + i / M] = v;
}

template <class T, int OT>
__global__ void __launch_bounds__(kOutThreads) k_mlp_out(MlpArgs a, int splits, int64_t per) {
    __shared__ __attribute__((aligned(16))) Pairs s;
    extern __shared__ float part[];
    const int pairs = a.n * a.k, lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    sort_pairs(s, a, pairs, kOutThreads);
    const int64_t c0 = (int64_t)blockIdx.x * OT;
    for (int it = wave; it < s.experts * splits; it += kOutWaves) {
        const int u = it / splits, ks = it % splits;
        const int e = s.expert[u];
        const T* w[OT];
#pragma unroll
        for (int i = 0; i < OT; ++i)
            w[i] = (const T*)a.w2 + ((int64_t)e * a.d_out + (c0 + i < a.d_out ? c0 + i : a.d_out - 1)) * a.hidden;
        const int64_t k0 = ks * per < a.hidden ? ks * per : a.hidden, k1 = k0 + per < a.hidden ? k0 + per : a.hidden;
        float* const mine = part + (size_t)ks * pairs * OT;
        int at = s.head[u];
        const int end = s.head[u + 1];
        for (; at + 4 <= end; at += 4) out_rows<T, OT, 4>(a, s, w, at, k0, k1, lane, mine);
        if (at + 2 <= end) {
            out_rows<T, OT, 2>(a, s, w, at, k0, k1, lane, mine);
            at += 2;
        }
        if (at < end) out_rows<T, OT, 1>(a, s, w, at, k0, k1, lane, mine);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < a.n * OT; i += kOutThreads) {
        const int t = i / OT, c = i % OT;
        if (c0 + c >= a.d_out) continue;
        float sum = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            const int p = t * a.k + j, slot = s.slot[p];
            if (slot < 0) continue;
            float y = a.b2 ? a.b2[(int64_t)s.id[p] * a.d_out + c0 + c] : 0.0f;
            for (int ks = 0; ks < splits; ++ks) y += part[((size_t)ks * pairs + slot) * OT + c];
            sum = fmaf(a.weights ? a.weights[p] : 1.0f, y, sum);
        }
        ((T*)a.out)[(int64_t)t * a.ld_out + c0 + c] = (T)sum;
    }
}

template <class T, int G>
void launch_hidden(const MlpArgs& a, hipStream_t s) {
    const int pairs = a.n * a.k, experts = pairs < a.n_experts ? pairs : a.n_experts;
    const bool gated = a.act == NERF_ACT_GATED;
    const int per = kHiddenThreads / G * (gated ? kHidden<true> : kHidden<false>);
    const int tiles = (a.hidden + per - 1) / per;
    const unsigned grid = (unsigned)experts * (unsigned)tiles;
    if (gated)
        k_mlp_hidden<T, G, true><<<grid, kHiddenThreads, 0, s>>>(a, tiles);
    else
        k_mlp_hidden<T, G, false><<<grid, kHiddenThreads, 0, s>>>(a, tiles);
}

template <class T, int OT>
void launch_out(const MlpArgs& a, hipStream_t s) {
    constexpr int STEP = 64 * RowIO<T>::PER;
    const int pairs = a.n * a.k, experts = pairs < a.n_experts ? pairs : a.n_experts;
    // fewer experts than waves: the waves share the hidden width too
    int splits = experts < kOutWaves ? kOutWaves / experts : 1;
    const int steps = (a.hidden + STEP - 1) / STEP;
    if (splits > steps) splits = steps;
    while (splits > 1 && (size_t)splits * pairs * OT * sizeof(float) > kPartBytes) --splits;
    const int64_t per = (int64_t)(steps + splits - 1) / splits * STEP;
    const size_t lds = (size_t)splits * pairs * OT * sizeof(float);
    k_mlp_out<T, OT><<<(unsigned)((a.d_out + OT - 1) / OT), kOutThreads, lds, s>>>(a, splits, per);
}

template <class T>
void launch(const MlpArgs& a, hipStream_t s) {
    if (a.d_in <= 16 * RowIO<T>::PER)
        launch_hidden<T, 16>(a, s);
    else
        launch_hidden<T, 64>(a, s);
    if (a.d_out >= 1024)
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
