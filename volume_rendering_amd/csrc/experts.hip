// The experts' products for gfx950: one linear layer per expert on rows
// sorted by expert, and its gradients.
//   forward          y[s][o]     = act(sum_i x[s][i] W_e[o][i] + b_e[o])
//   input gradient   dx[s][i]    = sum_o dz[s][o] W_e[o][i]   (times [x > 0])
//   weight gradient  dW_e[o][i]  = sum_s dz[s][o] x[s][i],  db_e[o] = sum_s dz[s][o]
// with e the expert of slot s.  All three are one tile scheme,
// C[m][n] = sum_k M[m][k] N[k][n], on the matrix cores (bfloat16 operands or
// float32 throughout, float32 accumulators), that differs in which index of
// an operand is contiguous in memory.
#include <hip/hip_runtime.h>

#include "common.hpp"
#include "experts.hpp"
#include "rowio.hpp"

namespace nerf {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

// ---------------------------------------------------------------------------
// Which expert a workgroup works for.  Experts' row counts are known on the
// device only, so workgroups are numbered by "virtual tiles": expert e starts
// at tile offsets[e] / B + e.  That number never decreases, leaves room for
// all ceil(rows / B) tiles of e, and needs no table: the expert of a tile is
// found by a 64-way search over the offsets (one step for up to 64 experts,
// two for up to 4096).  At most one tile an expert is empty.
// ---------------------------------------------------------------------------
template <class F>
__device__ __forceinline__ int last_where(int n, F&& holds) {  // largest e < n with holds(e); holds(0) is true
    const int lane = lane_id();
    int lo = 0, len = n;
    while (len > 1) {
        const int step = (len + 63) / 64;
        const int e = lo + lane * step;
        const bool ok = e < lo + len && holds(e);
        const int c = __popcll(__ballot(ok));
        const int end = lo + len;
        lo += (c > 0 ? c - 1 : 0) * step;
        len = step < end - lo ? step : end - lo;
    }
    return __builtin_amdgcn_readfirstlane(lo);
}

struct Group {
    int e;           // expert, or n_experts: the slots without one
    int64_t lo, hi;  // its slots that this workgroup works on
};

__device__ __forceinline__ int64_t clamp_slot(int64_t v, int64_t slots) { return v < 0 ? 0 : v > slots ? slots : v; }

// Slots [lo, hi) of virtual tile v of B slots each; `groups` experts, the last
// of which may be the slots without one.
__device__ __forceinline__ Group find_group(const ExpertArgs& a, int64_t v, int64_t B, int groups) {
    const int32_t* off = a.offsets;
    Group g;
    g.e = last_where(groups, [&](int e) { return off[e] / B + e <= v; });
    const int64_t o0 = off[g.e], o1 = g.e < a.n_experts ? off[g.e + 1] : a.slots;
    NERF_DCHECK(o0 >= 0 && o0 <= o1 && o1 <= a.slots, kCheckRouteOffset);
    const int64_t lo = o0 + (v - (o0 / B + g.e)) * B;
    g.hi = clamp_slot(lo + B < o1 ? lo + B : o1, a.slots);
    g.lo = clamp_slot(lo, a.slots);
    return g;
}

// Row of x of slot s (-1: none).
__device__ __forceinline__ int64_t x_row(const ExpertArgs& a, int64_t s) {
    if (!a.order) return s < a.x_rows ? s : -1;
    const int p = a.order[s];
    const int64_t t = (unsigned)p / (unsigned)a.k;
    NERF_DCHECK(p >= 0 && t < a.x_rows, kCheckRouteSlot);
    return p >= 0 && t < a.x_rows ? t : -1;
}

// ---------------------------------------------------------------------------
// Tiles in LDS.  A k-step is 128 bytes of k (64 bfloat16 or 32 float32).
//  k contiguous: a row is 128 bytes, its eight 16-byte pieces XOR-swizzled by
//    row, so that a read of 32 rows at one piece falls on distinct banks.
//  k outermost (k-major): a row is the tile's width at one k; bfloat16 pieces
//    are swizzled by k in pairs (the transposing read takes 32 bytes of four
//    consecutive k).
// Every fragment is 16 bytes a lane: lanes 0..31 and 32..63 take the two
// 16-byte pieces of a 32-byte step of k for their row.  For float32 that
// permutes k within a step, the same way for both operands.
// ---------------------------------------------------------------------------
constexpr int kStepBytes = 128;

template <class T>
struct Elt {
    static constexpr int PER = 16 / (int)sizeof(T);
    static constexpr int BK = kStepBytes / (int)sizeof(T);
    union Frag {
        u32x4 u;
        T e[PER];
        s16x4 h[2];
    };
};

__device__ __forceinline__ int swz_row(int row) { return row & 7; }
template <class T, int C>
__device__ __forceinline__ int swz_k(int k) {
    return sizeof(T) == 2 ? ((k & 3) << 2) & (C / 8 - 1) & ~1 : 0;
}

// Fragment of k-contiguous rows: row (lane % 32) + r0, 32-byte step q.
template <class T>
__device__ __forceinline__ typename Elt<T>::Frag frag_rows(const char* tile, int r0, int q, int lane) {
    typename Elt<T>::Frag f;
    const int r = r0 + (lane & 31);
    f.u = *reinterpret_cast<const u32x4*>(tile + r * kStepBytes + (((2 * q + (lane >> 5)) ^ swz_row(r)) << 4));
    return f;
}

// Fragment of a k-major tile of C columns: column (lane % 32) + c0.
template <class T, int C>
__device__ __forceinline__ typename Elt<T>::Frag frag_cols(const char* tile, int c0, int q, int lane) {
    typename Elt<T>::Frag f;
    if constexpr (sizeof(T) == 2) {
        // each 16 lanes read 4 k x 16 columns and get them transposed
        const int i = lane & 15, c = c0 + (lane & 16) + 4 * (i & 3);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int k = 16 * q + 8 * (lane >> 5) + 4 * t + (i >> 2);
            const char* p = tile + k * (C * 2) + (((c >> 3) ^ swz_k<T, C>(k)) << 4) + ((c & 7) << 1);
            f.h[t] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((s16x4 NERF_LDS_PTR)p);
        }
    } else {
        const int c = c0 + (lane & 31);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            f.e[j] = *reinterpret_cast<const float*>(tile + ((8 * q + 4 * (lane >> 5) + j) * C + c) * 4);
    }
    return f;
}

// acc[a's row][b's row] += over one 32-byte step of k.  A lane's accumulator r
// holds a's row 8 (r / 4) + 4 (lane / 32) + r % 4 and b's row lane % 32.
template <class T>
__device__ __forceinline__ void mma(f32x16& acc, const typename Elt<T>::Frag& a, const typename Elt<T>::Frag& b) {
    if constexpr (sizeof(T) == 2) {
        acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a.u), __builtin_bit_cast(bf16x8, b.u),
                                                      acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a.e[j], b.e[j], acc, 0, 0, 0);
    }
}

// ---------------------------------------------------------------------------
// Register-staged tile copies: any width, stride and alignment.  Elements past
// the matrix are zero, so a step past k or a row past the group adds nothing.
// ---------------------------------------------------------------------------
template <class T, int R, int NT>
struct StageRows {  // R rows, k contiguous
    static constexpr int UNITS = R * 8, UPT = (UNITS + NT - 1) / NT;
    typename RowIO<T>::Vec v[UPT];
    // row_of(r): pointer to row r, or NULL (a zero row)
    template <class F>
    __device__ __forceinline__ void load(F&& row_of, int64_t k0, int64_t K, int tid) {
#pragma unroll
        for (int q = 0; q < UPT; ++q) {
            const int u = tid + NT * q;
            v[q] = RowIO<T>::zero();
            if (UNITS % NT == 0 || u < UNITS) {
                const T* p = row_of(u >> 3);
                if (p) v[q] = RowIO<T>::load(p, k0 + (u & 7) * RowIO<T>::PER, K);
            }
        }
    }
    __device__ __forceinline__ void store(char* tile, int tid) const {
#pragma unroll
        for (int q = 0; q < UPT; ++q) {
            const int u = tid + NT * q, r = u >> 3;
            if (UNITS % NT == 0 || u < UNITS)
                *reinterpret_cast<u32x4*>(tile + r * kStepBytes + (((u & 7) ^ swz_row(r)) << 4)) = v[q].u;
        }
    }
};

template <class T, int C, int NT>
struct StageCols {  // one k-step of a k-major matrix, C columns
    static constexpr int PIECES = C / RowIO<T>::PER, UNITS = Elt<T>::BK * PIECES, UPT = (UNITS + NT - 1) / NT;
    typename RowIO<T>::Vec v[UPT];
    // row_of(k): pointer to the matrix row at k of this step, or NULL
    template <class F>
    __device__ __forceinline__ void load(F&& row_of, int64_t c0, int64_t width, int tid) {
#pragma unroll
        for (int q = 0; q < UPT; ++q) {
            const int u = tid + NT * q;
            v[q] = RowIO<T>::zero();
            if (UNITS % NT == 0 || u < UNITS) {
                const T* p = row_of(u / PIECES);
                if (p) v[q] = RowIO<T>::load(p, c0 + (u % PIECES) * RowIO<T>::PER, width);
            }
        }
    }
    __device__ __forceinline__ void store(char* tile, int tid) const {
#pragma unroll
        for (int q = 0; q < UPT; ++q) {
            const int u = tid + NT * q, k = u / PIECES;
            if (UNITS % NT == 0 || u < UNITS)
                *reinterpret_cast<u32x4*>(tile + k * (C * (int)sizeof(T)) + (((u % PIECES) ^ swz_k<T, C>(k)) << 4)) =
                    v[q].u;
        }
    }
};

// ---------------------------------------------------------------------------
// A wave's accumulators to memory, through LDS so that rows leave in 16-byte
// pieces along n.  One 32-row block of m at a time; `st` is the wave's own
// 32 x (WN elements + 16 bytes).
// ---------------------------------------------------------------------------
template <class O, int WN>
constexpr int epilogue_bytes() { return 32 * (WN * (int)sizeof(O) + 16); }

template <class O, int WN, class V, class S>
__device__ __forceinline__ void epilogue_block(char* st, const f32x16 (&acc)[WN / 32], int lane, V&& value, S&& store) {
    constexpr int PITCH = WN * (int)sizeof(O) + 16, PER = 16 / (int)sizeof(O), PIECES = WN / PER;
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < WN / 32; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int n = 32 * i + 8 * g + 4 * (lane >> 5);
            O* p = reinterpret_cast<O*>(st + (lane & 31) * PITCH) + n;
            O o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = (O)value(acc[i][4 * g + e], n + e);
            __builtin_memcpy(__builtin_assume_aligned(p, 4 * sizeof(O)), o, 4 * sizeof(O));
        }
    wave_lds_sync();
#pragma unroll
    for (int u = lane; u < 32 * PIECES; u += 64) {
        const int m = u / PIECES, n = (u % PIECES) * PER;
        typename RowIO<O>::Vec v;
        v.u = *reinterpret_cast<const u32x4*>(st + m * PITCH + n * (int)sizeof(O));
        store(m, n, v);
    }
}

// ---------------------------------------------------------------------------
// Forward and input gradient: a workgroup owns BM slots of one expert and BN
// columns.  GRAD: weights are read k-major (k = outputs), rows are dz.
// ---------------------------------------------------------------------------
template <class T, bool GRAD, int BM, int BN, int WM, int WN>
struct RowsTile {
    static constexpr int NT = 64 * (BM / WM) * (BN / WN);
    static constexpr int A_BYTES = BM * kStepBytes, STAGE = A_BYTES + BN * kStepBytes;
    static constexpr int EPI = (NT / 64) * epilogue_bytes<T, WN>();
    static constexpr int LDS = 2 * STAGE > EPI ? 2 * STAGE : EPI;
};

template <class T, bool GRAD, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__((RowsTile<T, GRAD, BM, BN, WM, WN>::NT))
    k_expert_rows(ExpertArgs a, int n_tiles) {
    using L = RowsTile<T, GRAD, BM, BN, WM, WN>;
    constexpr int NT = L::NT;
    __shared__ __attribute__((aligned(1024))) char lds[L::LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave % (BM / WM), wn = wave / (BM / WM);
    const int nt = blockIdx.x % n_tiles;
    const Group g = find_group(a, blockIdx.x / n_tiles, BM, a.n_experts + 1);
    const int rows = (int)(g.hi - g.lo);
    if (rows <= 0) return;
    const int64_t n0 = (int64_t)nt * BN;
    const int64_t K = GRAD ? a.d_out : a.d_in, N = GRAD ? a.d_in : a.d_out;
    T* const y = (T*)a.y + g.lo * a.ld_y;
    if (g.e == a.n_experts) {  // slots without an expert: zero rows
        constexpr int PIECES = BN / RowIO<T>::PER;
        for (int u = tid; u < rows * PIECES; u += NT)
            if (n0 + (u % PIECES) * RowIO<T>::PER < N)
                RowIO<T>::store(y + (int64_t)(u / PIECES) * a.ld_y, n0 + (u % PIECES) * RowIO<T>::PER, N,
                                RowIO<T>::zero());
        return;
    }
    const T* const w = (const T*)a.w + (int64_t)g.e * a.d_in * a.d_out;

    StageRows<T, BM, NT> sa;
    StageRows<T, BN, NT> sb;  // forward: rows of W
    StageCols<T, BN, NT> sc;  // gradient: W is k-major
    auto load = [&](int64_t k0) {
        sa.load(
            [&](int r) -> const T* {
                if (r >= rows) return nullptr;
                if (GRAD) return (const T*)a.dz + (g.lo + r) * a.ld_dz;
                const int64_t t = x_row(a, g.lo + r);
                return t < 0 ? nullptr : (const T*)a.x + t * a.ld_x;
            },
            k0, K, tid);
        if constexpr (GRAD)
            sc.load([&](int k) { return k0 + k < K ? w + (k0 + k) * N : nullptr; }, n0, N, tid);
        else
            sb.load([&](int r) { return n0 + r < N ? w + (n0 + r) * K : nullptr; }, k0, K, tid);
    };
    auto store = [&](char* stage) {
        sa.store(stage, tid);
        if constexpr (GRAD)
            sc.store(stage + L::A_BYTES, tid);
        else
            sb.store(stage + L::A_BYTES, tid);
    };

    f32x16 acc[WM / 32][WN / 32];
#pragma unroll
    for (int j = 0; j < WM / 32; ++j)
#pragma unroll
        for (int i = 0; i < WN / 32; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;

    load(0);
    store(lds);
    __syncthreads();
    int buf = 0;
    for (int64_t k0 = 0; k0 < K; k0 += Elt<T>::BK) {
        const bool more = k0 + Elt<T>::BK < K;
        if (more) load(k0 + Elt<T>::BK);
        const char *ta = lds + buf * L::STAGE, *tb = ta + L::A_BYTES;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            typename Elt<T>::Frag fm[WM / 32], fn[WN / 32];
#pragma unroll
            for (int j = 0; j < WM / 32; ++j) fm[j] = frag_rows<T>(ta, wm * WM + 32 * j, q, lane);
#pragma unroll
            for (int i = 0; i < WN / 32; ++i)
                fn[i] = GRAD ? frag_cols<T, BN>(tb, wn * WN + 32 * i, q, lane)
                             : frag_rows<T>(tb, wn * WN + 32 * i, q, lane);
#pragma unroll
            for (int j = 0; j < WM / 32; ++j)
#pragma unroll
                for (int i = 0; i < WN / 32; ++i) mma<T>(acc[j][i], fn[i], fm[j]);
        }
        if (more) store(lds + (buf ^ 1) * L::STAGE);
        __syncthreads();
        buf ^= 1;
    }

    char* st = lds + wave * epilogue_bytes<T, WN>();
    const int64_t nw = n0 + wn * WN;
    const float* bias = !GRAD && a.bias ? a.bias + (int64_t)g.e * N : nullptr;
#pragma unroll
    for (int j = 0; j < WM / 32; ++j) {
        epilogue_block<T, WN>(
            st, acc[j], lane,
            [&](float v, int n) {
                if (GRAD) return v;
                if (bias && nw + n < N) v += bias[nw + n];
                return a.relu && v < 0.0f ? 0.0f : v;  // (a NaN stays)
            },
            [&](int m, int n, typename RowIO<T>::Vec v) {
                const int r = wm * WM + 32 * j + m;
                if (r >= rows || nw + n >= N) return;
                if (GRAD && a.relu) {
                    const int64_t t = x_row(a, g.lo + r);
                    const typename RowIO<T>::Vec x =
                        t < 0 ? RowIO<T>::zero() : RowIO<T>::load((const T*)a.x + t * a.ld_x, nw + n, N);
#pragma unroll
                    for (int e = 0; e < RowIO<T>::PER; ++e)
                        if (!(RowIO<T>::get(x, e) > 0.0f)) v.e[e] = (T)0.0f;
                }
                RowIO<T>::store(y + (int64_t)r * a.ld_y, nw + n, N, v);
            });
    }
}

// ---------------------------------------------------------------------------
// Weight gradient: k runs over an expert's slots, both operands are k-major.
// A workgroup owns BM outputs x BN inputs of one expert and, with a.chunk,
// one range of its slots (partial sums, added in order by k_expert_sum).
// Bias gradients are one more product, with a column of ones.
// ---------------------------------------------------------------------------
template <class T, int BM, int BN, int WM, int WN>
struct WeightTile {
    static constexpr int NT = 64 * (BM / WM) * (BN / WN);
    static constexpr int A_BYTES = BM * kStepBytes, STAGE = A_BYTES + BN * kStepBytes;
    static constexpr int EPI = (NT / 64) * epilogue_bytes<float, WN>();
    static constexpr int LDS = 2 * STAGE > EPI ? 2 * STAGE : EPI;
};

template <class T, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__((WeightTile<T, BM, BN, WM, WN>::NT))
    k_expert_weights(ExpertArgs a, int m_tiles, int n_tiles) {
    using L = WeightTile<T, BM, BN, WM, WN>;
    constexpr int NT = L::NT, BK = Elt<T>::BK;
    __shared__ __attribute__((aligned(1024))) char lds[L::LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave % (BM / WM), wn = wave / (BM / WM);
    const int tile = blockIdx.x % (m_tiles * n_tiles);
    const int64_t v = blockIdx.x / (m_tiles * n_tiles);
    const int64_t M = a.d_out, N = a.d_in;
    const int64_t m0 = (int64_t)(tile / n_tiles) * BM, n0 = (int64_t)(tile % n_tiles) * BN;
    Group g;
    if (a.chunk) {
        g = find_group(a, v, a.chunk, a.n_experts);
        if (g.hi <= g.lo) return;
    } else {
        g.e = (int)v;
        g.lo = clamp_slot(a.offsets[v], a.slots);
        g.hi = clamp_slot(a.offsets[v + 1], a.slots);
    }
    float* const out = a.chunk ? a.part + v * M * N : a.dw + g.e * M * N;
    float* const bout = a.chunk ? a.bpart + v * M : a.db ? a.db + g.e * M : nullptr;
    const bool ones_tile = a.db && n0 == 0 && wn == 0;

    StageCols<T, BM, NT> sa;
    StageCols<T, BN, NT> sb;
    auto load = [&](int64_t s0) {
        sa.load([&](int k) { return s0 + k < g.hi ? (const T*)a.dz + (s0 + k) * a.ld_dz : nullptr; }, m0, M, tid);
        sb.load(
            [&](int k) -> const T* {
                if (s0 + k >= g.hi) return nullptr;
                const int64_t t = x_row(a, s0 + k);
                return t < 0 ? nullptr : (const T*)a.x + t * a.ld_x;
            },
            n0, N, tid);
    };
    f32x16 acc[WM / 32][WN / 32], bacc[WM / 32];
#pragma unroll
    for (int j = 0; j < WM / 32; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            bacc[j][r] = 0.0f;
#pragma unroll
            for (int i = 0; i < WN / 32; ++i) acc[j][i][r] = 0.0f;
        }
    typename Elt<T>::Frag ones;
#pragma unroll
    for (int e = 0; e < Elt<T>::PER; ++e) ones.e[e] = (T)1.0f;

    if (g.lo < g.hi) {
        load(g.lo);
        sa.store(lds, tid);
        sb.store(lds + L::A_BYTES, tid);
    }
    __syncthreads();
    int buf = 0;
    for (int64_t s0 = g.lo; s0 < g.hi; s0 += BK) {
        const bool more = s0 + BK < g.hi;
        if (more) load(s0 + BK);
        const char *ta = lds + buf * L::STAGE, *tb = ta + L::A_BYTES;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            typename Elt<T>::Frag fm[WM / 32], fn[WN / 32];
#pragma unroll
            for (int j = 0; j < WM / 32; ++j) fm[j] = frag_cols<T, BM>(ta, wm * WM + 32 * j, q, lane);
#pragma unroll
            for (int i = 0; i < WN / 32; ++i) fn[i] = frag_cols<T, BN>(tb, wn * WN + 32 * i, q, lane);
#pragma unroll
            for (int j = 0; j < WM / 32; ++j)
#pragma unroll
                for (int i = 0; i < WN / 32; ++i) mma<T>(acc[j][i], fn[i], fm[j]);
            if (ones_tile)
#pragma unroll
                for (int j = 0; j < WM / 32; ++j) mma<T>(bacc[j], ones, fm[j]);
        }
        if (more) {
            char* next = lds + (buf ^ 1) * L::STAGE;
            sa.store(next, tid);
            sb.store(next + L::A_BYTES, tid);
        }
        __syncthreads();
        buf ^= 1;
    }

    char* st = lds + wave * epilogue_bytes<float, WN>();
    const int64_t mw = m0 + wm * WM, nw = n0 + wn * WN;
#pragma unroll
    for (int j = 0; j < WM / 32; ++j) {
        if (ones_tile && lane < 32 && mw + 32 * j + lane < M) bout[mw + 32 * j + lane] = bacc[j][0];
        epilogue_block<float, WN>(
            st, acc[j], lane, [](float x, int) { return x; },
            [&](int m, int n, typename RowIO<float>::Vec x) {
                const int64_t r = mw + 32 * j + m;
                if (r < M && nw + n < N) RowIO<float>::store(out + r * N, nw + n, N, x);
            });
    }
}

// dW_e (and db_e) from the partial sums of its ranges, in their order.
__global__ void __launch_bounds__(256) k_expert_sum(ExpertArgs a) {
    const int64_t MN = (int64_t)a.d_out * a.d_in, per = MN + (a.db ? a.d_out : 0);
    const int e = blockIdx.y;
    const int64_t o0 = clamp_slot(a.offsets[e], a.slots), o1 = clamp_slot(a.offsets[e + 1], a.slots);
    const int64_t v0 = o0 / a.chunk + e, nv = o1 > o0 ? (o1 - o0 + a.chunk - 1) / a.chunk : 0;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= per) return;
    const bool is_w = i < MN;
    const float* p = is_w ? a.part + v0 * MN + i : a.bpart + v0 * a.d_out + (i - MN);
    const int64_t stride = is_w ? MN : a.d_out;
    float sum = 0.0f;
#pragma unroll 4
    for (int64_t c = 0; c < nv; ++c) sum += p[c * stride];
    if (is_w)
        a.dw[e * MN + i] = sum;
    else
        a.db[(int64_t)e * a.d_out + (i - MN)] = sum;
}

template <class T, bool GRAD, int BM, int BN, int WM, int WN>
void run_rows(const ExpertArgs& a, hipStream_t s) {
    const int64_t N = GRAD ? a.d_in : a.d_out;
    const int n_tiles = (int)((N + BN - 1) / BN);
    const int64_t tiles = a.slots / BM + a.n_experts + 1;
    k_expert_rows<T, GRAD, BM, BN, WM, WN>
        <<<(unsigned)(tiles * n_tiles), RowsTile<T, GRAD, BM, BN, WM, WN>::NT, 0, s>>>(a, n_tiles);
}

template <class T, bool GRAD>
void pick_rows(const ExpertArgs& a, hipStream_t s) {
    const int64_t N = GRAD ? a.d_in : a.d_out;
    if (a.slots / a.n_experts < 64 || N <= 32)
        run_rows<T, GRAD, 32, 32, 32, 32>(a, s);
    else
        run_rows<T, GRAD, 128, 128, 64, 64>(a, s);
}

template <class T, int BM, int BN, int WM, int WN>
void run_weights(const ExpertArgs& a, hipStream_t s) {
    const int mt = (a.d_out + BM - 1) / BM, nt = (a.d_in + BN - 1) / BN;
    const int64_t items = a.chunk ? a.slots / a.chunk + a.n_experts : a.n_experts;
    k_expert_weights<T, BM, BN, WM, WN>
        <<<(unsigned)(items * mt * nt), WeightTile<T, BM, BN, WM, WN>::NT, 0, s>>>(a, mt, nt);
}

template <class T>
void pick_weights(const ExpertArgs& a, hipStream_t s) {
    if (a.d_out <= 32 || a.d_in <= 32)
        run_weights<T, 32, 64, 32, 64>(a, s);
    else
        run_weights<T, 128, 128, 64, 64>(a, s);
    if (a.chunk) {
        const int64_t per = (int64_t)a.d_out * a.d_in + (a.db ? a.d_out : 0);
        k_expert_sum<<<dim3((unsigned)((per + 255) / 256), a.n_experts), 256, 0, s>>>(a);
    }
}

}  // namespace

int64_t expert_grad_chunk(int64_t slots, int n_experts, int d_in, int d_out) {
    const int64_t tiles = (int64_t)n_experts * ((d_in + 127) / 128) * ((d_out + 127) / 128);
    if (tiles >= 512 || slots <= 2048) return 0;
    return 2048;
}

void launch_expert_linear(bool bf16, const ExpertArgs& a, hipStream_t s) {
    if (bf16)
        pick_rows<__bf16, false>(a, s);
    else
        pick_rows<float, false>(a, s);
}
void launch_expert_grad_x(bool bf16, const ExpertArgs& a, hipStream_t s) {
    if (bf16)
        pick_rows<__bf16, true>(a, s);
    else
        pick_rows<float, true>(a, s);
}
void launch_expert_grad_w(bool bf16, const ExpertArgs& a, hipStream_t s) {
    if (bf16)
        pick_weights<__bf16>(a, s);
    else
        pick_weights<float>(a, s);
}

}  // namespace nerf
