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

constexpr int64_t kDirectBytes = ((int64_t)1 << 32) - 65536;  // extent one buffer resource may cover

// The same value, which the compiler takes for a new one: what depends on it is
// computed where it is used, once a tile, and not kept in registers across the
// loop over k.
__device__ __forceinline__ int again(int v) {
    asm volatile("" : "+v"(v));
    return v;
}
// Values that are the same in every lane, kept in scalar registers.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint64_t uniform(const void* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    return (uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v);
}
// base and bytes uniform; bytes as an unsigned number
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc_of(uint64_t base, int bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(base), (short)0, bytes, kBufferWord3);
}
// ---------------------------------------------------------------------------
// Which expert a workgroup works for.  Experts' row counts are known on the
// device only, so workgroups are numbered by "virtual tiles": expert e starts
// at tile offsets[e] / B + e.  That number never decreases, leaves room for
// all ceil(rows / B) tiles of e, and needs no table: the expert of a tile is
// found by a 64-way search over the offsets of the experts and of the slots
// without one (one step for up to 63 experts, two for up to 4095, three for
// 4096).  At most one tile an expert is empty.
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
    int e;       // expert, or n_experts: the slots without one
    int lo, hi;  // its slots that this workgroup works on
};

__device__ __forceinline__ int clamp_slot(int64_t v, int64_t slots) {
    return v < 0 ? 0 : v > slots ? (int)slots : (int)v;
}

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

// Row of x of pair p (-1: none).
__device__ __forceinline__ int64_t row_of_pair(const ExpertArgs& a, int p) {
    const int64_t t = (int64_t)(((uint64_t)(uint32_t)p * a.k_mul) >> a.k_shift);  // p / k
    NERF_DCHECK(p < 0 || t < a.x_rows, kCheckRouteSlot);
    return p >= 0 && t < a.x_rows ? t : -1;
}

// Row of x of slot s (-1: none).
__device__ __forceinline__ int64_t x_row(const ExpertArgs& a, int64_t s) {
    if (!a.order) return s < a.x_rows ? s : -1;
    const int p = a.order[s];
    NERF_DCHECK(p >= 0, kCheckRouteSlot);
    return row_of_pair(a, p);
}

// ---------------------------------------------------------------------------
// Tiles in LDS.  A k-step is 128 bytes of k (64 bfloat16 or 32 float32).
//  k contiguous: a row is 128 bytes, its eight 16-byte pieces XOR-swizzled by
//    row, so that a read of 32 rows at one piece falls on distinct banks
//    (whether 8 or 16 lanes are served at a time).
//  k outermost (k-major): a row is the tile's width at one k; bfloat16 pieces
//    are swizzled by k in pairs: the transposing read takes 32 bytes of four
//    consecutive k per 16 lanes, and of two neighbouring 32 bytes per 32 lanes,
//    which fall on distinct banks whether it serves 16 or 32 lanes at a time.
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

__device__ __forceinline__ int swz_row(int row) { return (row ^ (row >> 3)) & 7; }
template <class T, int C>
__device__ __forceinline__ int swz_k(int k) {
    return sizeof(T) == 2 ? (((k & 3) << 1) | ((k & 1) << 3)) & (C / 8 - 1) : 0;
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
// A row's last, partial piece is loaded as the last whole one and shifted into
// place when it goes to LDS: loads then hold nothing that waits for one.
// ---------------------------------------------------------------------------
// Two LDS stages; one in a workgroup of a single wave, which has nobody to wait
// for and lives from many workgroups on a CU (k-steps are few there).
constexpr int staged_stages(int NT) { return NT == 64 ? 1 : 2; }

// Elements c .. of a row of `width`, to be settled (below) before use.
template <class T>
__device__ __forceinline__ typename RowIO<T>::Vec load_ahead(const T* row, int64_t c, int64_t width) {
    if (width < RowIO<T>::PER) return RowIO<T>::load(row, c, width);  // (the same for every lane)
    return RowIO<T>::load_whole(row + (c + RowIO<T>::PER <= width ? c : width - RowIO<T>::PER));
}
template <class T>
__device__ __forceinline__ u32x4 settle(const typename RowIO<T>::Vec& v, int64_t c, int64_t width) {
    const int64_t past = c + RowIO<T>::PER - width;
    u32x4 u = v.u;
    if (past > 0 && width >= RowIO<T>::PER) {
        uint64_t lo = (uint64_t)u[1] << 32 | u[0], hi = (uint64_t)u[3] << 32 | u[2];
        const int s = past < RowIO<T>::PER ? (int)past * 8 * (int)sizeof(T) : 128;  // bits of earlier elements
        const uint64_t over = s < 64 ? hi << (64 - s) : 0;                           // (s is at least 16)
        lo = s < 64 ? lo >> s | over : s < 128 ? hi >> (s - 64) : 0;
        hi = s < 64 ? hi >> s : 0;
        u = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
    return u;
}

template <class T, int R, int NT>
struct StageRows {  // R rows, k contiguous
    static constexpr int UNITS = R * 8, UPT = (UNITS + NT - 1) / NT;
    const T* row[UPT];  // of each unit; NULL: a zero row
    typename RowIO<T>::Vec v[UPT];
    // row_of(r): pointer to row r, or NULL
    template <class F>
    __device__ __forceinline__ void init(F&& row_of, int tid) {
#pragma unroll
        for (int q = 0; q < UPT; ++q) {
            const int u = tid + NT * q;
            row[q] = UNITS % NT == 0 || u < UNITS ? row_of(u >> 3) : nullptr;
        }
    }
    __device__ __forceinline__ void load(int64_t k0, int64_t K, int tid) {
#pragma unroll
        for (int q = 0; q < UPT; ++q) {
            v[q] = RowIO<T>::zero();
            if (row[q]) v[q] = load_ahead<T>(row[q], k0 + ((tid + NT * q) & 7) * RowIO<T>::PER, K);
        }
    }
    __device__ __forceinline__ void store(char* tile, int64_t k0, int64_t K, int tid) const {
#pragma unroll
        for (int q = 0; q < UPT; ++q) {
            const int u = tid + NT * q, r = u >> 3;
            if (UNITS % NT == 0 || u < UNITS)
                *reinterpret_cast<u32x4*>(tile + r * kStepBytes + (((u & 7) ^ swz_row(r)) << 4)) =
                    settle<T>(v[q], k0 + (u & 7) * RowIO<T>::PER, K);
        }
    }
};

template <class T, int C, int NT>
struct StageCols {  // one k-step of a k-major matrix, C columns
    static constexpr int PIECES = C / RowIO<T>::PER, UNITS = Elt<T>::BK * PIECES, UPT = (UNITS + NT - 1) / NT;
    static_assert(UNITS % NT == 0, "whole units");
    typename RowIO<T>::Vec v[UPT];
    static __device__ __forceinline__ int k_of(int q, int tid) { return (tid + NT * q) / PIECES; }
    // row_of(q): pointer to the matrix row at unit q's k of this step, or NULL
    template <class F>
    __device__ __forceinline__ void load(F&& row_of, int64_t c0, int64_t width, int tid) {
#pragma unroll
        for (int q = 0; q < UPT; ++q) {
            v[q] = RowIO<T>::zero();
            const T* p = row_of(q);
            if (p) v[q] = load_ahead<T>(p, c0 + ((tid + NT * q) % PIECES) * RowIO<T>::PER, width);
        }
    }
    __device__ __forceinline__ void store(char* tile, int64_t c0, int64_t width, int tid) const {
#pragma unroll
        for (int q = 0; q < UPT; ++q) {
            const int u = tid + NT * q, k = u / PIECES, c = u % PIECES;
            *reinterpret_cast<u32x4*>(tile + k * (C * (int)sizeof(T)) + ((c ^ swz_k<T, C>(k)) << 4)) =
                settle<T>(v[q], c0 + c * RowIO<T>::PER, width);
        }
    }
};

// ---------------------------------------------------------------------------
// A wave's accumulators to memory, through LDS so that rows leave in 16-byte
// pieces along n.  One 32-row block of m at a time; `st` is the wave's own
// 32 rows of WN elements, pieces swizzled by row (no padding: LDS is full).
// ---------------------------------------------------------------------------
template <class O, int WN>
constexpr int epilogue_bytes() { return 32 * WN * (int)sizeof(O); }

template <class O, int WN, class V, class S>
__device__ __forceinline__ void epilogue_block(char* st, const f32x16 (&acc)[WN / 32], int lane, V&& value, S&& store) {
    constexpr int PER = 16 / (int)sizeof(O), PIECES = WN / PER, PITCH = PIECES * 16, MASK = PIECES < 8 ? PIECES - 1 : 7;
    wave_lds_sync();
#pragma unroll
    for (int i = 0; i < WN / 32; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const int n = 32 * i + 8 * g + 4 * (lane >> 5), m = lane & 31;
            char* p = st + m * PITCH + (((n / PER) ^ (m & MASK)) << 4) + (n % PER) * (int)sizeof(O);
            O o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = (O)value(acc[i][4 * g + e]);
            __builtin_memcpy(__builtin_assume_aligned(p, 4 * sizeof(O)), o, 4 * sizeof(O));
        }
    wave_lds_sync();
#pragma unroll
    for (int k = 0; k < PIECES / 2; ++k) {
        const int u = 64 * k + lane, m = u / PIECES, c = u % PIECES;
        typename RowIO<O>::Vec v;
        v.u = *reinterpret_cast<const u32x4*>(st + m * PITCH + ((c ^ (m & MASK)) << 4));
        store(m, c * PER, v);
    }
}

// Columns n0 .. n0 + BN - 1 of `rows` rows of y to zero.
template <class T, int BN, int NT>
__device__ __forceinline__ void zero_rows(T* y, int64_t ld, int rows, int64_t n0, int64_t N, int tid) {
    constexpr int PIECES = BN / RowIO<T>::PER;
    for (int u = tid; u < rows * PIECES; u += NT) {
        const int64_t n = n0 + (u % PIECES) * RowIO<T>::PER;
        if (n < N) RowIO<T>::store(y + (int64_t)(u / PIECES) * ld, n, N, RowIO<T>::zero());
    }
}

// Accumulators start at the bias (0 without one, and past the last column).
template <bool GRAD, int WM, int WN>
__device__ __forceinline__ void rows_start(const ExpertArgs& a, int e, f32x16 (&acc)[WM / 32][WN / 32], int64_t nw,
                                           int64_t N, int lane) {
#pragma unroll
    for (int i = 0; i < WN / 32; ++i) {
        f32x16 b;
#pragma unroll
        for (int r = 0; r < 16; ++r) b[r] = 0.0f;
        if (!GRAD && a.bias) {
            const float* bias = a.bias + (int64_t)e * N;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int64_t n = nw + 32 * i + 8 * (r / 4) + 4 * (lane >> 5) + r % 4;
                b[r] = bias[n < N ? n : N - 1];
            }
        }
#pragma unroll
        for (int j = 0; j < WM / 32; ++j) acc[j][i] = b;
    }
}

// A wave's WM x WN block of y (ReLU) or dx (the mask of x), from row r0 of the
// group's `rows` and column nw.  DIRECT: 16-byte aligned rows of whole pieces,
// stored through a buffer resource, lanes outside the tile out of its range:
// every wave then issues exactly WM / 32 * WN / 16 stores, which the product
// loop counts.
template <class T, bool GRAD, int WM, int WN, bool DIRECT = false>
__device__ __forceinline__ void rows_epilogue(const ExpertArgs& a, const Group& g, char* st,
                                              const f32x16 (&acc)[WM / 32][WN / 32], T* y, int rows, int r0,
                                              int64_t nw, int64_t N, int lane) {
    const float floor = !GRAD && a.relu ? 0.0f : -INFINITY;
    const __amdgpu_buffer_rsrc_t ry =
        rsrc_of(uniform(y), uniform((int)(uint32_t)((rows - 1) * a.ld_y * (int)sizeof(T) + N * (int)sizeof(T))));
#pragma unroll
    for (int j = 0; j < WM / 32; ++j) {
        epilogue_block<T, WN>(
            st, acc[j], lane, [&](float v) { return v < floor ? floor : v; },  // (a NaN stays)
            [&](int m, int n, typename RowIO<T>::Vec v) {
                const int r = r0 + 32 * j + m;
                const bool in = r < rows && nw + n < N;
                if constexpr (!DIRECT)
                    if (!in) return;
                if (GRAD && a.relu) {
                    const int64_t t = in ? x_row(a, g.lo + r) : -1;
                    const typename RowIO<T>::Vec x =
                        t < 0 ? RowIO<T>::zero()
                              : RowIO<T>::load((const T*)a.x + t * a.ld_x, nw + n, DIRECT ? INT64_MAX : N);
#pragma unroll
                    for (int e = 0; e < RowIO<T>::PER; ++e)
                        if (!(RowIO<T>::get(x, e) > 0.0f)) v.e[e] = (T)0.0f;
                }
                if constexpr (DIRECT)
                    __builtin_amdgcn_raw_buffer_store_b128(
                        v.u, ry, in ? (uint32_t)((r * a.ld_y + nw + n) * (int)sizeof(T)) : kBufferOutOfRange, 0, 2);
                else
                    RowIO<T>::store(y + (int64_t)r * a.ld_y, nw + n, N, v);
            });
    }
}

// ---------------------------------------------------------------------------
// Forward and input gradient: a workgroup owns BM slots of one expert and BN
// columns.  GRAD: weights are read k-major (k = outputs), rows are dz.  This
// kernel serves every type, width, stride and alignment.  128 x 128 tiles: 8
// experts 1024 -> 1024, 16,384 slots, float32: 384 us, 90 TF/s (a library product
// of 4096 cubed: 142), two waves a SIMD being too few to hide each other's
// barriers; 32 experts 333 -> 517, 131,072 slots, bfloat16: 201 us, 225 TF/s,
// bound by the copies through registers.  32-slot tiles (one wave each) are bound
// by the latency of one chain of load, store, read and multiplication, of which a
// CU runs many side by side: 90,000 slots of 4096 experts 63 -> 32, float32, the
// input gradient 30 us.
// ---------------------------------------------------------------------------
template <class T, bool GRAD, int BM, int BN, int WM, int WN>
struct RowsTile {
    static constexpr int NT = 64 * (BM / WM) * (BN / WN), STAGES = staged_stages(NT);
    static constexpr int A_BYTES = BM * kStepBytes, STAGE = A_BYTES + BN * kStepBytes;
    static constexpr int EPI = (NT / 64) * epilogue_bytes<T, WN>();
    static constexpr int LDS = STAGES * STAGE > EPI ? STAGES * STAGE : EPI;
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
        zero_rows<T, BN, NT>(y, a.ld_y, rows, n0, N, tid);
        return;
    }
    const T* const w = (const T*)a.w + (int64_t)g.e * a.d_in * a.d_out;

    StageRows<T, BM, NT> sa;
    StageRows<T, BN, NT> sb;  // forward: rows of W
    StageCols<T, BN, NT> sc;  // gradient: W is k-major
    sa.init(
        [&](int r) -> const T* {
            if (r >= rows) return nullptr;
            if (GRAD) return (const T*)a.dz + (g.lo + r) * a.ld_dz;
            const int64_t t = x_row(a, g.lo + r);
            return t < 0 ? nullptr : (const T*)a.x + t * a.ld_x;
        },
        tid);
    if constexpr (!GRAD) sb.init([&](int r) { return n0 + r < N ? w + (n0 + r) * K : nullptr; }, tid);
    auto load = [&](int64_t k0) {
        sa.load(k0, K, tid);
        if constexpr (GRAD)
            sc.load(
                [&](int q) {
                    const int64_t k = k0 + sc.k_of(q, tid);
                    return k < K ? w + k * N : nullptr;
                },
                n0, N, tid);
        else
            sb.load(k0, K, tid);
    };
    auto store = [&](char* stage, int64_t k0) {
        sa.store(stage, k0, K, tid);
        if constexpr (GRAD)
            sc.store(stage + L::A_BYTES, n0, N, tid);
        else
            sb.store(stage + L::A_BYTES, k0, K, tid);
    };

    f32x16 acc[WM / 32][WN / 32];
    rows_start<GRAD, WM, WN>(a, g.e, acc, n0 + wn * WN, N, lane);

    load(0);
    store(lds, 0);
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
        if (L::STAGES == 1) __syncthreads();
        buf = L::STAGES == 1 ? 0 : buf ^ 1;
        if (more) store(lds + buf * L::STAGE, k0 + Elt<T>::BK);
        __syncthreads();
    }

    rows_epilogue<T, GRAD, WM, WN>(a, g, lds + wave * epilogue_bytes<T, WN>(), acc, y, rows, wm * WM, n0 + wn * WN, N,
                                   lane);
}

// ---------------------------------------------------------------------------
// Forward for few slots (serving): bound by the read of the touched experts'
// weights, and for one sample by launch and latency (1024 -> 4096 bfloat16
// through two experts: 16.8 MB, 3.4 us at 4.9 TB/s, 8.5 us a call).  A workgroup
// owns 16 slots of an expert and 16 outputs; its four waves take a quarter of k
// each, straight from memory to registers (each weight is used once, so LDS would
// only add a step), eight loads in flight, and their partial sums are added up in
// LDS in a fixed order.
// Slots are found like tiles, or, with fewer slots than tiles, one workgroup
// row per slot, of which those that start a tile work.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 4, kFewAhead = 8;
constexpr int kFewSlots = 256;

template <class T>
__global__ void __launch_bounds__(64 * kFewWaves) k_expert_few(ExpertArgs a, int n_tiles, int by_slot) {
    using IO = RowIO<T>;
    constexpr int BK = 4 * IO::PER;  // k per load: four lane groups of a piece
    __shared__ float part[kFewWaves][16][17];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nt = blockIdx.x % n_tiles, v = blockIdx.x / n_tiles;
    Group g;
    if (by_slot) {
        g.e = last_where(a.n_experts + 1, [&](int e) { return a.offsets[e] <= v; });
        const int o0 = clamp_slot(a.offsets[g.e], a.slots);
        const int o1 = g.e < a.n_experts ? clamp_slot(a.offsets[g.e + 1], a.slots) : (int)a.slots;
        if (v < o0 || v >= o1 || (v - o0) % 16) return;
        g.lo = v;
        g.hi = o1 - v > 16 ? v + 16 : o1;
    } else {
        g = find_group(a, v, 16, a.n_experts + 1);
    }
    const int rows = g.hi - g.lo;
    if (rows <= 0) return;
    const int64_t K = a.d_in, N = a.d_out, n0 = 16 * (int64_t)nt;
    if (g.e < a.n_experts) {
        const int64_t n = n0 + (lane & 15);
        const T* const w = (const T*)a.w + ((int64_t)g.e * N + (n < N ? n : N - 1)) * K;
        const int64_t t = (lane & 15) < rows ? x_row(a, g.lo + (lane & 15)) : -1;
        const T* const x = (const T*)a.x + (t < 0 ? 0 : t) * a.ld_x;
        const int64_t per = (K + kFewWaves * BK - 1) / (kFewWaves * BK) * BK;
        const int64_t k1 = (wave + 1) * per < K ? (wave + 1) * per : K;
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int64_t k0 = wave * per; k0 < k1; k0 += kFewAhead * BK) {
            typename IO::Vec fw[kFewAhead], fx[kFewAhead];
#pragma unroll
            for (int u = 0; u < kFewAhead; ++u) {
                const int64_t k = k0 + u * BK + (lane >> 4) * IO::PER;
                fw[u] = fx[u] = IO::zero();
                if (k < k1) {
                    fw[u] = IO::load(w, k, k1);
                    if (t >= 0) fx[u] = IO::load(x, k, k1);
                }
            }
#pragma unroll
            for (int u = 0; u < kFewAhead; ++u) {
                if constexpr (sizeof(T) == 2)
                    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fx[u].u),
                                                                  __builtin_bit_cast(bf16x8, fw[u].u), acc, 0, 0, 0);
                else
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        acc = __builtin_amdgcn_mfma_f32_16x16x4f32(fx[u].e[j], fw[u].e[j], acc, 0, 0, 0);
            }
        }
        // (a lane holds slots 4 (lane / 16) + r of output lane % 16)
#pragma unroll
        for (int r = 0; r < 4; ++r) part[wave][4 * (lane >> 4) + r][lane & 15] = acc[r];
    }
    __syncthreads();
    const int m = tid >> 4, n = tid & 15;
    if (m >= rows || n0 + n >= N) return;
    float y = 0.0f;
    if (g.e < a.n_experts) {
        if (a.bias) y = a.bias[(int64_t)g.e * N + n0 + n];
#pragma unroll
        for (int i = 0; i < kFewWaves; ++i) y += part[i][m][n];
        if (a.relu && y < 0.0f) y = 0.0f;
    }
    ((T*)a.y)[(g.lo + m) * a.ld_y + n0 + n] = (T)y;
}

// ---------------------------------------------------------------------------
// Direct copies global -> LDS (no registers): bfloat16 with every row 16-byte
// aligned.  Each instruction fills 1 KB of LDS in lane order, so the swizzle
// is in the source: a lane fetches the piece that belongs where it writes.
// Pieces past the matrix get an offset out of the buffer's range, which copies
// zeros.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t r, char* dst, uint32_t off) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (void NERF_LDS_PTR)dst, 16, (int)off, 0, 0, 0);
}
// All but the wave's N latest copies have arrived, and its LDS reads are done;
// then all waves'.
template <int N>
__device__ __forceinline__ void wait_copies_barrier() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));  // vmcnt(N) lgkmcnt(0)
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
}

template <int R, int NT>
struct CopyRows {  // R rows, k contiguous
    static constexpr int NW = NT / 64, Q = R * 8 / NT, APART = 8 * NW;  // rows between a wave's copies
    static_assert(R * 8 % NT == 0, "whole copies");
    static __device__ __forceinline__ int row(int q, int wave, int lane) {
        return (q * NW + wave) * 8 + (lane >> 3);
    }
    // byte of a lane's piece within a k-step
    static __device__ __forceinline__ uint32_t piece(int q, int wave, int lane) {
        return (uint32_t)((lane & 7) ^ swz_row(row(q, wave, lane))) << 4;
    }
    // copy q, whose row starts at byte `off` (its lane's piece included), of
    // the k-step at byte kb of rows of `width` bytes; `inside`: the piece is
    // inside a last, partial step
    static __device__ __forceinline__ void issue(int q, __amdgpu_buffer_rsrc_t rs, char* tile, uint32_t off,
                                                 uint32_t kb, uint32_t width, bool inside, int wave) {
        uint32_t o = __builtin_elementwise_add_sat(off, kb);  // (out of range stays so)
        if (kb + kStepBytes > width) o = kb < width && inside ? o : kBufferOutOfRange;
        copy16(rs, tile + (q * NW + wave) * 1024, o);
    }
};

template <int C, int NT>
struct CopyCols {  // one k-step (64 rows) of a k-major matrix, C columns
    static constexpr int P = C / 8, Q = 64 * P / NT;
    static_assert(64 * P % NT == 0, "whole copies");
    uint32_t off[Q];  // bytes from the step's first row and the tile's first column; or out of range
    static __device__ __forceinline__ int k_of(int q, int wave, int lane) { return ((wave * Q + q) * 64 + lane) / P; }
    static __device__ __forceinline__ int piece(int q, int wave, int lane) {
        return (((wave * Q + q) * 64 + lane) % P) ^ swz_k<__bf16, C>(k_of(q, wave, lane));
    }
    // rows `pitch` bytes apart, `cols` columns of the tile inside the matrix
    __device__ __forceinline__ void init(uint32_t pitch, int cols, int wave, int lane) {
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int c = piece(q, wave, lane);
            off[q] = 8 * c < cols ? k_of(q, wave, lane) * pitch + 16 * c : kBufferOutOfRange;
        }
    }
    // copy q of a step: rows past the matrix lie past the resource's end
    __device__ __forceinline__ void issue(int q, __amdgpu_buffer_rsrc_t rs, char* tile, int wave) const {
        copy16(rs, tile + (wave * Q + q) * 1024, off[q]);
    }
};

// k-steps of 64 rows of a k-major matrix: `rows` rows `pitch` bytes apart from
// base on, which is `c0` bytes into the first.
struct ColsSource {
    uint64_t base;
    int pitch, c0, rows;
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t step(int t) const {
        const int left = rows - 64 * t;
        const int kl = left < 0 ? 0 : left < 64 ? left : 64;
        const int bytes = kl * pitch - c0;
        const uint64_t p = base + (uint64_t)(64 * (int64_t)t * pitch);
        return rsrc_of(uniform(reinterpret_cast<const void*>(p)), uniform(bytes < 0 ? 0 : bytes));
    }
};

// ---------------------------------------------------------------------------
// One k-step of 64 of a product, in two LDS stages (an array for each stage of
// each operand: the compiler then sees that reads need not wait for copies in
// flight, which go into other arrays).  The fragments of the next 16 k are read
// while the current ones multiply, a read or a copy between each two matrix
// instructions.  In a step's last quarter every wave has its fragments in
// registers, so after one barrier the stage is free: the copies of the step
// after next start there and have a step's multiplications to arrive in.  (Four
// stages of 32 k, three of them in flight, took the same time.)
//   stores: at that barrier the STORES rows stored since the awaited copies may
//   still be in flight;
//   read(r, next, q, fm, fn): piece r of NM + NN of the fragments of quarter q
//   of this step or (next) of quarter 0 of the next one;
//   ready(): a step's copies are about to start (called before the barrier with
//   EARLY: its work then overlaps the wait, but holds registers across it);
//   copy(c): copy c of them;
//   extra(fm): further use of a quarter's fragments.
// ---------------------------------------------------------------------------
template <int NM, int NN>
struct Frags {
    Elt<__bf16>::Frag m[2][NM], n[2][NN];
};

template <int COPIES, int STORES, bool EARLY, int NM, int NN, class RD, class RY, class CP, class EX>
__device__ __forceinline__ void product_step(f32x16 (&acc)[NM][NN], Frags<NM, NN>& f, bool stores, RD&& read,
                                             RY&& ready, CP&& copy, EX&& extra) {
    constexpr int CPM = (COPIES + NM * NN - 1) / (NM * NN), RPM = (NM + NN + NM * NN - 1) / (NM * NN);
    auto part = [&](auto qc) {
        constexpr int q = decltype(qc)::value;
        constexpr bool last = q == 3;
        if constexpr (last) {
            if constexpr (EARLY) {
                ready();
                __builtin_amdgcn_sched_barrier(0);
            }
            if (STORES > 0 && stores)
                wait_copies_barrier<STORES>();
            else
                wait_copies_barrier<0>();
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (!EARLY) ready();
        }
#pragma unroll
        for (int m = 0; m < NM * NN; ++m) {
#pragma unroll
            for (int u = 0; u < RPM; ++u)
                if (m * RPM + u < NM + NN)
                    read(m * RPM + u, std::integral_constant<bool, last>{}, last ? 0 : q + 1, f.m[(q + 1) & 1],
                         f.n[(q + 1) & 1]);
            if constexpr (last)
#pragma unroll
                for (int u = 0; u < CPM; ++u)
                    if (m * CPM + u < COPIES) copy(m * CPM + u);
            mma<__bf16>(acc[m / NN][m % NN], f.n[q & 1][m % NN], f.m[q & 1][m / NN]);
            __builtin_amdgcn_sched_barrier(0);
        }
        extra(f.m[q & 1]);
    };
    part(std::integral_constant<int, 0>{});
    part(std::integral_constant<int, 1>{});
    part(std::integral_constant<int, 2>{});
    part(std::integral_constant<int, 3>{});
}

template <int BM, int BN, int WM, int WN, class O>
struct DirectTile {
    static constexpr int NT = 64 * (BM / WM) * (BN / WN);
    static constexpr int A_BYTES = BM * kStepBytes, B_BYTES = BN * kStepBytes;  // a stage of each operand
    static constexpr int EPI = (NT / 64) * epilogue_bytes<O, WN>();
    static constexpr int QA = BM * 8 / NT, QB = BN * 8 / NT;  // copies of each operand per wave and step
    static constexpr int COPIES = QA + QB;
};

// ---------------------------------------------------------------------------
// The tiles of a rows product, dealt out to a grid that stays: workgroup b
// runs on XCD b % 8, each XCD gets a contiguous eighth of the tiles, and its
// workgroups walk it side by side, kGroupTiles slot tiles at a time, so that
// what its L2 holds of rows and weights is used by its neighbours.  With up to
// 63 experts the tiles are counted exactly (each lane holds an expert);
// otherwise they are virtual tiles and the empty ones are skipped.
// ---------------------------------------------------------------------------
constexpr int kCus = 256;  // workgroups of a grid that stays: one per CU
constexpr int kGroupTiles = 4;

struct TileWalk {
    int BM;  // slots per tile
    int l, end, v_tiles, step, n_tiles;
    int off, upto;  // lane e: first slot of expert e; tiles of experts 0 .. e

    __device__ __forceinline__ void start(const ExpertArgs& a, int height, int n) {
        BM = height;
        n_tiles = n;
        const int groups = a.n_experts + 1;
        if (groups <= 64) {
            const int e = lane_id();
            off = e < groups ? clamp_slot(a.offsets[e], a.slots) : (int)a.slots;
            const int o1 = e < a.n_experts ? clamp_slot(a.offsets[e + 1], a.slots) : (int)a.slots;
            upto = o1 > off ? (o1 - off + BM - 1) / BM : 0;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int o = __shfl_up(upto, d, 64);
                if (e >= d) upto += o;
            }
            v_tiles = __builtin_amdgcn_readlane(upto, 63);
        } else {
            v_tiles = (int)(a.slots / BM) + groups;
        }
        const int part = blockIdx.x & 7;  // (fewer than 2^31 tiles: the host has checked)
        l = (int)((int64_t)v_tiles * n_tiles * part / 8) + (int)(blockIdx.x >> 3);
        end = (int)((int64_t)v_tiles * n_tiles * (part + 1) / 8);
        step = gridDim.x >> 3;
    }
    // The next tile with slots; false: none is left.
    __device__ __forceinline__ bool next(const ExpertArgs& a, Group& g, int& nt) {
        while (l < end) {
            const int group = (unsigned)l / (unsigned)(kGroupTiles * n_tiles), in = l - group * kGroupTiles * n_tiles;
            const int left = v_tiles - group * kGroupTiles, wide = left < kGroupTiles ? left : kGroupTiles;
            nt = (unsigned)in / (unsigned)wide;
            const int v = group * kGroupTiles + in - nt * wide;
            l += step;
            if (a.n_experts + 1 <= 64) {
                g.e = __popcll(__ballot(upto <= v));
                const int before = g.e ? __builtin_amdgcn_readlane(upto, g.e - 1) : 0;
                const int o1 = g.e < a.n_experts ? __builtin_amdgcn_readlane(off, g.e + 1) : (int)a.slots;
                g.lo = __builtin_amdgcn_readlane(off, g.e) + (v - before) * BM;
                g.hi = o1 - g.lo > BM ? g.lo + BM : o1;
            } else {
                g = find_group(a, v, BM, a.n_experts + 1);
            }
            if (g.lo < g.hi) return true;
        }
        return false;
    }
};

// Bound by the matrix cores and what feeds them from LDS.  16 experts
// 1024 -> 4096, 32,768 slots: 294 us, 930 TF/s.  Of these the multiplications
// alone take 175 us (copies of the kernel with the rest taken out), with the
// fragments' reads 210, with the stores 233; the copies into LDS, which share
// its ports, bring the rest, and 8.5 tiles a CU run as 9.  A library product of
// 4096 x 4096 x 4096 without routing reaches 1320 TF/s here.  256 x 256 tiles of
// eight 128 x 64 waves (251 registers, two waves a SIMD) read least from LDS a
// multiplication of the shapes timed; four 128 x 128 waves would read a third less
// and have not been.  Fewer rows a tile where that fills the last round of the grid
// (tile_height).
// 8 experts 256 -> 256, 262,144 slots: 74 us, bound by memory (268 MB, 55 us).
template <bool GRAD, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__((DirectTile<BM, BN, WM, WN, __bf16>::NT))
    k_expert_rows_direct(ExpertArgs a, int tile_rows, int n_tiles) {
    using T = __bf16;
    using L = DirectTile<BM, BN, WM, WN, T>;
    using F = Elt<T>::Frag;
    constexpr int NT = L::NT, NM = WM / 32, NN = WN / 32;
    __shared__ __attribute__((aligned(1024))) char m0[L::A_BYTES], m1[L::A_BYTES], w0[L::B_BYTES], w1[L::B_BYTES];
    __shared__ __attribute__((aligned(1024))) char epi[L::EPI];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % (BM / WM), wn = wave / (BM / WM);
    const int64_t K = GRAD ? a.d_out : a.d_in, N = GRAD ? a.d_in : a.d_out;
    const uint32_t width = (uint32_t)(K * 2);
    const bool through = !GRAD && a.order;
    const int64_t lda = GRAD ? a.ld_dz : a.ld_x;

    TileWalk walk;
    walk.start(a, tile_rows, n_tiles);
    struct Tile {
        Group g;
        int64_t n0;
        int rows, n_left;
    } cur, nxt;
    int pair[L::QA];  // through the order: the next tile's slots, loaded a tile ahead
    // the next tile with an expert; slots without one become zero rows on the way
    auto advance = [&](Tile& t) {
        int nt = 0;
        while (walk.next(a, t.g, nt)) {
            t.n0 = (int64_t)nt * BN;
            t.rows = uniform(t.g.hi - t.g.lo);
            t.n_left = (int)(N - t.n0 < BN ? N - t.n0 : BN);
            if (t.g.e < a.n_experts) {
                if (through)
#pragma unroll
                    for (int q = 0; q < L::QA; ++q) {
                        const int r = CopyRows<BM, NT>::row(q, wave, again(lane));
                        pair[q] = r < t.rows ? a.order[t.g.lo + r] : -1;
                    }
                return;
            }
            zero_rows<T, BN, NT>((T*)a.y + (int64_t)t.g.lo * a.ld_y, a.ld_y, t.rows, t.n0, N, tid);
        }
        t.rows = 0;
    };

    // sources of the tile that is being copied (none left: nothing in range);
    // rows past the tile's are past the end of its resource
    using CA = CopyRows<BM, NT>;
    using CB = CopyRows<BN, NT>;
    __amdgpu_buffer_rsrc_t ra, rb;
    uint32_t oa[L::QA], ob[2];    // forward: rows of W, the first two copies
    CopyCols<BN, NT> cc;   // gradient: its columns
    ColsSource wc;
    // (the swizzle of a wave's copies is the same in all of them, or alternates
    // between two)
    static_assert(CA::APART % 32 == 0, "one swizzle in every second copy");
    const bool inside[2] = {CA::piece(0, wave, lane) < width % kStepBytes,
                            CA::piece(1, wave, lane) < width % kStepBytes};
    auto source = [&](const Tile& t) {
        const int ln = again(lane);
        const T* const w = (const T*)a.w + (t.rows ? (int64_t)t.g.e * a.d_in * a.d_out : 0);
        const int64_t lo = t.rows ? (int64_t)t.g.lo : 0;
        const T* const base = GRAD ? (const T*)a.dz + lo * lda : through ? (const T*)a.x : (const T*)a.x + lo * lda;
        const int64_t bytes = ((through ? a.x_rows : t.rows) - 1) * lda * 2 + K * 2;
        ra = rsrc_of(uniform(base), uniform(t.rows ? (int)(uint32_t)bytes : 0));
#pragma unroll
        for (int q = 0; q < L::QA; ++q) {
            const int64_t row = through ? row_of_pair(a, pair[q]) : CA::row(q, wave, ln);
            oa[q] = row < 0 ? kBufferOutOfRange : (uint32_t)(row * lda * 2) + CA::piece(q, wave, ln);
        }
        const int cols = t.rows ? t.n_left : 0;
        if (GRAD) {
            wc = ColsSource{uniform(w + t.n0), (int)(N * 2), (int)(t.n0 * 2), cols ? (int)K : 0};
            cc.init((uint32_t)(N * 2), cols, wave, ln);
        } else {
            rb = rsrc_of(uniform(w + t.n0 * K), uniform((int)(cols * K * 2)));
#pragma unroll
            for (int q = 0; q < 2; ++q)
                ob[q] = (uint32_t)(CB::row(q, wave, ln) * K * 2) + CB::piece(q, wave, ln);
        }
    };
    auto copy = [&](int c, char* ms, char* ws, int t) {
        const uint32_t kb = (uint32_t)t * kStepBytes;
        const int q = c < L::QA ? c : c - L::QA;
        if (c < L::QA)
            CA::issue(q, ra, ms, oa[q], kb, width, inside[q & 1], wave);
        else if constexpr (!GRAD)
            CB::issue(q, rb, ws, ob[q & 1] + (uint32_t)((q & ~1) * CB::APART * K * 2), kb, width, inside[q & 1], wave);
        else
            cc.issue(c - L::QA, rb, ws, wave);
    };
    auto ready = [&](int t) {
        if (GRAD) rb = wc.step(t);
    };
    auto read = [&](int r, const char* ms, const char* ws, int q, F(&fm)[NM], F(&fn)[NN]) {
        if (r < NM)
            fm[r] = frag_rows<T>(ms, wm * WM + 32 * r, q, lane);
        else
            fn[r - NM] = GRAD ? frag_cols<T, BN>(ws, wn * WN + 32 * (r - NM), q, lane)
                              : frag_rows<T>(ws, wn * WN + 32 * (r - NM), q, lane);
    };

    // steps, rounded up to whole rounds of both stages (a step past K is zeros)
    const int nk = 2 * (int)((K + 127) / 128);
    advance(cur);
    if (cur.rows == 0) return;
    source(cur);
    ready(0);
#pragma unroll
    for (int c = 0; c < L::COPIES; ++c) copy(c, m0, w0, 0);
    ready(1);
#pragma unroll
    for (int c = 0; c < L::COPIES; ++c) copy(c, m1, w1, 1);
    wait_copies_barrier<L::COPIES>();
    Frags<NM, NN> f;
#pragma unroll
    for (int r = 0; r < NM + NN; ++r) read(r, m0, w0, 0, f.m[0], f.n[0]);

    // tile after tile without a pause: the last two steps of one copy the first
    // two of the next, which is in flight while the one's rows are stored
    bool stored = false;
    while (true) {
        advance(nxt);
        f32x16 acc[NM][NN];
        rows_start<GRAD, WM, WN>(a, cur.g.e, acc, cur.n0 + wn * WN, N, again(lane));
        int done = 0;  // steps of the copied tile's predecessor
        for (int t = 0; t < nk; t += 2) {
            // (a tile's first step waits for copies issued before the last
            // tile's rows were stored)
            int fresh = uniform(t == 0 && stored);
            asm volatile("" : "+s"(fresh));  // (one loop, not one for each value)
            product_step<L::COPIES, NM * WN / 16, GRAD>(
                acc, f, fresh != 0,
                [&](int r, auto next, int q, F(&fm)[NM], F(&fn)[NN]) {
                    if constexpr (decltype(next)::value)
                        read(r, m1, w1, q, fm, fn);
                    else
                        read(r, m0, w0, q, fm, fn);
                },
                [&]() {
                    if (t + 2 == nk) {
                        source(nxt);
                        done = nk;
                    }
                    ready(t + 2 - done);
                },
                [&](int c) { copy(c, m0, w0, t + 2 - done); }, [](const F(&)[NM]) {});
            product_step<L::COPIES, 0, GRAD>(
                acc, f, false,
                [&](int r, auto next, int q, F(&fm)[NM], F(&fn)[NN]) {
                    if constexpr (decltype(next)::value)
                        read(r, m0, w0, q, fm, fn);
                    else
                        read(r, m1, w1, q, fm, fn);
                },
                [&]() { ready(t + 3 - done); }, [&](int c) { copy(c, m1, w1, t + 3 - done); }, [](const F(&)[NM]) {});
        }
        rows_epilogue<T, GRAD, WM, WN, true>(a, cur.g, epi + wave * epilogue_bytes<T, WN>(), acc,
                                             (T*)a.y + (int64_t)cur.g.lo * a.ld_y, cur.rows, wm * WM, cur.n0 + wn * WN, N,
                                             again(lane));
        if (nxt.rows == 0) break;
        cur = nxt;
        stored = !(GRAD && a.relu);  // (else loads are among the stores: all are waited for)
    }
    wait_copies_barrier<0>();  // (no copy outlives its workgroup)
}

// ---------------------------------------------------------------------------
// Weight gradient: k runs over an expert's slots, both operands are k-major.
// A workgroup owns BM outputs x BN inputs of one expert and, with a.chunk,
// one range of its slots (partial sums, added in order by k_expert_sum).
// This kernel serves every type, width, stride and alignment; which rows of x a
// step copies is read a step ahead.  16 experts 512 -> 512, 32,768 slots, float32:
// 276 us, 62 TF/s; 32 experts 333 -> 517, 131,072 slots, bfloat16: 480 us, 94 TF/s;
// 4096 experts 63 -> 32, 90,000 slots, float32: 29 us.  All bound by latency, as
// k_expert_rows.
// ---------------------------------------------------------------------------
template <class T, int BM, int BN, int WM, int WN>
struct WeightTile {
    static constexpr int NT = 64 * (BM / WM) * (BN / WN), STAGES = staged_stages(NT);
    static constexpr int A_BYTES = BM * kStepBytes, STAGE = A_BYTES + BN * kStepBytes;
    static constexpr int EPI = (NT / 64) * epilogue_bytes<float, WN>();
    static constexpr int LDS = STAGES * STAGE > EPI ? STAGES * STAGE : EPI;
};

// The expert with the v-th most slots, for up to 64 experts (v beyond): the
// longest sums start first, so that none starts when the others are done.
__device__ __forceinline__ int longest_first(const ExpertArgs& a, int v) {
    if (a.n_experts > 64) return v;
    const int lane = lane_id();
    const int mine = lane < a.n_experts ? a.offsets[lane + 1] - a.offsets[lane] : INT32_MIN;
    int rank = 0;
    for (int e = 0; e < a.n_experts; ++e) {
        const int o = __builtin_amdgcn_readlane(mine, e);
        rank += o > mine || (o == mine && e < lane);
    }
    return __ffsll((unsigned long long)__ballot(lane < a.n_experts && rank == v)) - 1;
}

// One workgroup's share of the weight gradients.
struct WeightWork {
    Group g;
    int64_t m0, n0;
    float* out;   // [d_out][d_in]
    float* bout;  // [d_out], or NULL
    bool any;
};
__device__ __forceinline__ WeightWork weight_work(const ExpertArgs& a, int64_t b, int m_tiles, int n_tiles, int BM,
                                                  int BN) {
    // Workgroup b runs on XCD b % 8.  Each XCD gets an eighth of every item's
    // tiles, neighbouring ones (they read the same columns of dz, and few of
    // x), and the items in the same order; which eighth rotates.
    WeightWork w;
    w.any = false;
    const int tiles = m_tiles * n_tiles, most = (tiles + 7) / 8;
    const int64_t M = a.d_out, N = a.d_in;
    int64_t v;
    int tile;
    if (tiles < 8) {  // (fewer tiles than XCDs: nothing to share)
        v = b / tiles;
        tile = (int)(b % tiles);
    } else {
        v = (b >> 3) / most;
        const int part = (int)((b + v) & 7);
        tile = part * tiles / 8 + (int)((b >> 3) % most);
        if (tile >= (part + 1) * tiles / 8) return w;
    }
    w.m0 = (int64_t)(tile / n_tiles) * BM;
    w.n0 = (int64_t)(tile % n_tiles) * BN;
    if (a.chunk) {
        w.g = find_group(a, v, a.chunk, a.n_experts);
        w.any = w.g.hi > w.g.lo;
    } else {  // (an expert without slots gets zeros)
        w.g.e = longest_first(a, (int)v);
        w.g.lo = clamp_slot(a.offsets[w.g.e], a.slots);
        w.g.hi = clamp_slot(a.offsets[w.g.e + 1], a.slots);
        w.any = true;
    }
    w.out = a.chunk ? a.part + v * M * N : a.dw + w.g.e * M * N;
    w.bout = !a.db || w.n0 ? nullptr : a.chunk ? a.bpart + v * M : a.db + w.g.e * M;
    return w;
}

// A wave's WM x WN block of the weight gradient, and the bias gradients of its rows.
template <int WM, int WN>
__device__ __forceinline__ void weights_epilogue(const ExpertArgs& a, const WeightWork& w, char* st,
                                                 const f32x16 (&acc)[WM / 32][WN / 32], const float (&bsum)[WM / 32],
                                                 int64_t mw, int64_t nw, bool with_bias, int lane) {
    const int64_t M = a.d_out, N = a.d_in;
#pragma unroll
    for (int j = 0; j < WM / 32; ++j) {
        if (with_bias) {
            const float b = bsum[j] + __shfl_xor(bsum[j], 32, 64);
            if (lane < 32 && mw + 32 * j + lane < M) w.bout[mw + 32 * j + lane] = b;
        }
        epilogue_block<float, WN>(
            st, acc[j], lane, [](float x) { return x; },
            [&](int m, int n, typename RowIO<float>::Vec x) {
                const int64_t r = mw + 32 * j + m;
                if (r < M && nw + n < N) RowIO<float>::store(w.out + r * N, nw + n, N, x);
            });
    }
}

template <int NM, int NN>
__device__ __forceinline__ void clear(f32x16 (&acc)[NM][NN]) {
#pragma unroll
    for (int j = 0; j < NM; ++j)
#pragma unroll
        for (int i = 0; i < NN; ++i)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[j][i][r] = 0.0f;
}

// Bias gradients are sums of the same fragments: a lane adds up its k of column lane % 32.
template <class T, int NM>
__device__ __forceinline__ void add_bias(float (&bsum)[NM], const typename Elt<T>::Frag (&fm)[NM]) {
#pragma unroll
    for (int j = 0; j < NM; ++j)
#pragma unroll
        for (int e = 0; e < Elt<T>::PER; ++e) bsum[j] += (float)fm[j].e[e];
}

template <class T, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__((WeightTile<T, BM, BN, WM, WN>::NT))
    k_expert_weights(ExpertArgs a, int m_tiles, int n_tiles) {
    using L = WeightTile<T, BM, BN, WM, WN>;
    constexpr int NT = L::NT, BK = Elt<T>::BK;
    __shared__ __attribute__((aligned(1024))) char lds[L::LDS];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wm = wave % (BM / WM), wn = wave / (BM / WM);
    const WeightWork w = weight_work(a, blockIdx.x, m_tiles, n_tiles, BM, BN);
    if (!w.any) return;
    const Group g = w.g;
    const bool with_bias = w.bout && wn == 0;

    StageCols<T, BM, NT> sa;
    StageCols<T, BN, NT> sb;
    int64_t from[sb.UPT];  // the next step's rows of x (-1: none), read a step ahead
    auto before = [&](int64_t s0) {
#pragma unroll
        for (int q = 0; q < sb.UPT; ++q) {
            const int64_t s = s0 + sb.k_of(q, tid);
            from[q] = s < g.hi ? x_row(a, s) : -1;
        }
    };
    auto load = [&](int64_t s0) {
        sa.load(
            [&](int q) {
                const int64_t s = s0 + sa.k_of(q, tid);
                return s < g.hi ? (const T*)a.dz + s * a.ld_dz : nullptr;
            },
            w.m0, a.d_out, tid);
        sb.load([&](int q) { return from[q] < 0 ? nullptr : (const T*)a.x + from[q] * a.ld_x; }, w.n0, a.d_in, tid);
    };
    auto store = [&](char* stage) {
        sa.store(stage, w.m0, a.d_out, tid);
        sb.store(stage + L::A_BYTES, w.n0, a.d_in, tid);
    };
    f32x16 acc[WM / 32][WN / 32];
    float bsum[WM / 32] = {};
    clear(acc);

    if (g.lo < g.hi) {
        before(g.lo);
        load(g.lo);
        before(g.lo + BK);
        store(lds);
    }
    __syncthreads();
    int buf = 0;
    for (int64_t s0 = g.lo; s0 < g.hi; s0 += BK) {
        const bool more = s0 + BK < g.hi;
        if (more) {
            load(s0 + BK);
            before(s0 + 2 * BK);
        }
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
            if (with_bias) add_bias<T>(bsum, fm);
        }
        if (L::STAGES == 1) __syncthreads();
        buf = L::STAGES == 1 ? 0 : buf ^ 1;
        if (more) store(lds + buf * L::STAGE);
        __syncthreads();
    }
    weights_epilogue<WM, WN>(a, w, lds + wave * epilogue_bytes<float, WN>(), acc, bsum, w.m0 + wm * WM,
                             w.n0 + wn * WN, with_bias, lane);
}

// The same with direct copies (bfloat16).  THROUGH: x rows through the order.
// Bound like k_expert_rows_direct; both operands are read transposed, which
// takes two LDS reads a fragment: 16 experts 1024 -> 4096, 32,768 slots: 330 us,
// 833 TF/s.  Longest expert first and neighbouring tiles on one XCD: both
// gradients 1079 -> 651 us together with the rows kernel's persistent grid.
template <bool THROUGH, int BM, int BN, int WM, int WN>
__global__ void __launch_bounds__((DirectTile<BM, BN, WM, WN, float>::NT))
    k_expert_weights_direct(ExpertArgs a, int m_tiles, int n_tiles) {
    using T = __bf16;
    using L = DirectTile<BM, BN, WM, WN, float>;
    constexpr int NT = L::NT;
    using CB = CopyCols<BN, NT>;
    using F = Elt<T>::Frag;
    constexpr int NM = WM / 32, NN = WN / 32;
    static_assert(L::EPI <= 2 * L::A_BYTES, "rows leave through the first operand's stages");
    __shared__ __attribute__((aligned(1024))) char m0[L::A_BYTES], m1[L::A_BYTES], w0[L::B_BYTES], w1[L::B_BYTES];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave % (BM / WM), wn = wave / (BM / WM);
    const WeightWork w = weight_work(a, blockIdx.x, m_tiles, n_tiles, BM, BN);
    if (!w.any) return;
    const Group g = w.g;
    const bool with_bias = w.bout && wn == 0;
    const int rows = uniform(g.hi > g.lo ? g.hi - g.lo : 0);
    const int m_left = (int)(a.d_out - w.m0 < BM ? a.d_out - w.m0 : BM);
    const int n_left = (int)(a.d_in - w.n0 < BN ? a.d_in - w.n0 : BN);

    f32x16 acc[WM / 32][WN / 32];
    float bsum[WM / 32] = {};
    clear(acc);
    const ColsSource zs{uniform((const T*)a.dz + g.lo * a.ld_dz + w.m0), (int)(a.ld_dz * 2), (int)(w.m0 * 2), rows};
    const ColsSource xs{uniform((const T*)a.x + (THROUGH ? 0 : g.lo * a.ld_x) + w.n0), (int)(a.ld_x * 2),
                        (int)(w.n0 * 2), rows};
    const __amdgpu_buffer_rsrc_t all =  // through the order: every row of x
        rsrc_of(xs.base, uniform((int)(uint32_t)(((a.x_rows - 1) * a.ld_x + a.d_in - w.n0) * 2)));
    CopyCols<BM, NT> ca;
    CB cb;
    ca.init((uint32_t)zs.pitch, m_left, wave, lane);
    cb.init((uint32_t)xs.pitch, n_left, wave, lane);
    __amdgpu_buffer_rsrc_t rz = all, rx = all;
    int pair[CB::Q];  // through the order: the next copies' slots, loaded a step ahead
    auto before = [&](int t) {
        if constexpr (THROUGH)
#pragma unroll
            for (int q = 0; q < CB::Q; ++q) {
                const int s = 64 * t + CB::k_of(q, wave, lane);
                pair[q] = s < rows ? a.order[g.lo + s] : -1;
            }
    };
    auto ready = [&](int t) {
        rz = zs.step(t);
        if constexpr (THROUGH) {
#pragma unroll
            for (int q = 0; q < CB::Q; ++q) {
                const int64_t r = row_of_pair(a, pair[q]);
                const int c = CB::piece(q, wave, lane);
                cb.off[q] = r >= 0 && 8 * c < n_left ? (uint32_t)(r * a.ld_x * 2) + 16 * c : kBufferOutOfRange;
            }
        } else {
            rx = xs.step(t);
        }
    };
    auto copy = [&](int c, char* ms, char* ws) {
        if (c < L::QA)
            ca.issue(c, rz, ms, wave);
        else
            cb.issue(c - L::QA, rx, ws, wave);
    };
    auto read = [&](int r, const char* ms, const char* ws, int q, F(&fm)[NM], F(&fn)[NN]) {
        if (r < NM)
            fm[r] = frag_cols<T, BM>(ms, wm * WM + 32 * r, q, lane);
        else
            fn[r - NM] = frag_cols<T, BN>(ws, wn * WN + 32 * (r - NM), q, lane);
    };
    auto bias = [&](const F(&fm)[NM]) {
        if (with_bias) add_bias<T>(bsum, fm);
    };
    Frags<NM, NN> f;
    if (rows) {
        before(0);
        ready(0);
#pragma unroll
        for (int c = 0; c < L::COPIES; ++c) copy(c, m0, w0);
        before(1);
        ready(1);
#pragma unroll
        for (int c = 0; c < L::COPIES; ++c) copy(c, m1, w1);
    }
    wait_copies_barrier<L::COPIES>();
#pragma unroll
    for (int r = 0; r < NM + NN; ++r) read(r, m0, w0, 0, f.m[0], f.n[0]);
    // (steps past the last slot copy zeros)
    for (int t = 0; 64 * t < rows; t += 2) {
        before(t + 2);
        product_step<L::COPIES, 0, true>(
            acc, f, false,
            [&](int r, auto next, int q, F(&fm)[NM], F(&fn)[NN]) {
                if constexpr (decltype(next)::value)
                    read(r, m1, w1, q, fm, fn);
                else
                    read(r, m0, w0, q, fm, fn);
            },
            [&]() { ready(t + 2); }, [&](int c) { copy(c, m0, w0); }, bias);
        before(t + 3);
        product_step<L::COPIES, 0, true>(
            acc, f, false,
            [&](int r, auto next, int q, F(&fm)[NM], F(&fn)[NN]) {
                if constexpr (decltype(next)::value)
                    read(r, m0, w0, q, fm, fn);
                else
                    read(r, m1, w1, q, fm, fn);
            },
            [&]() { ready(t + 3); }, [&](int c) { copy(c, m1, w1); }, bias);
    }
    wait_copies_barrier<0>();
    constexpr int HALF = NT / 128;  // waves whose rows leave through one stage
    weights_epilogue<WM, WN>(a, w, (wave < HALF ? m0 : m1) + wave % HALF * epilogue_bytes<float, WN>(), acc, bsum,
                             w.m0 + wm * WM, w.n0 + wn * WN, with_bias, lane);
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

// tile_rows <= BM slots a tile, `per_cu` workgroups on a CU.
template <bool GRAD, int BM, int BN, int WM, int WN>
void run_rows_direct(const ExpertArgs& a, int tile_rows, int per_cu, hipStream_t s) {
    const int64_t N = GRAD ? a.d_in : a.d_out;
    const int n_tiles = (int)((N + BN - 1) / BN);
    const int64_t tiles = (a.slots / tile_rows + a.n_experts + 1) * n_tiles;
    const unsigned blocks = (unsigned)(tiles < per_cu * kCus ? (tiles + 7) / 8 * 8 : per_cu * kCus);
    k_expert_rows_direct<GRAD, BM, BN, WM, WN>
        <<<blocks, DirectTile<BM, BN, WM, WN, __bf16>::NT, 0, s>>>(a, tile_rows, n_tiles);
}

// The least tile height, a multiple of 16, at which the tiles of 256 columns
// still take no more rounds of the grid than at height 256; an expert's last
// tile is taken to be half full.  Tiles of 192 rows or fewer have a kernel of
// that many: forward of 64 experts 512 -> 512, 512 slots each, 45 us against 52
// with 256 rows; 16 experts 1024 -> 1024, 1024 each: 51 and 61.  Where 128 rows
// do, two workgroups of 128 x 128 share a CU: 8 experts 512 -> 1024, 512 slots
// each: 15.2 us against 17.8 with 192 rows and 20.6 with 256.
int tile_height(int64_t slots, int n_experts, int64_t n_tiles) {
    const int64_t part = n_experts / 2;
    const int64_t rounds = ((slots / 256 + part + 1) * n_tiles + kCus - 1) / kCus;
    for (int h = 16; h < 256; h += 16)
        if ((slots / h + part + 1) * n_tiles <= rounds * kCus) return h;
    return 256;
}

template <bool GRAD>
void pick_rows_direct(const ExpertArgs& a, hipStream_t s) {
    const int64_t N = GRAD ? a.d_in : a.d_out;
    const int h = tile_height(a.slots, a.n_experts, (N + 255) / 256);
    if (h <= 128)
        run_rows_direct<GRAD, 128, 128, 64, 64>(a, 128, 2, s);
    else if (h <= 192)
        run_rows_direct<GRAD, 192, 256, 96, 64>(a, h, 1, s);
    else
        run_rows_direct<GRAD, 256, 256, 128, 64>(a, h, 1, s);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Whether the rows kernels may copy directly: bfloat16 rows of whole 16-byte
// pieces, and a gathered x within one buffer resource.
bool direct_rows(const ExpertArgs& a, bool grad) {
    if (a.d_in % 8 || a.d_out % 8 || !aligned16(a.w)) return false;
    const int64_t ld = grad ? a.ld_dz : a.ld_x;
    if (ld % 8 || ld > 1 << 22) return false;  // (a tile of 256 such rows is within 2^31 bytes)
    if (a.ld_y % 8 || a.ld_y > 1 << 22 || !aligned16(a.y)) return false;
    if (grad) return aligned16(a.dz);
    return aligned16(a.x) && (!a.order || a.x_rows * a.ld_x * 2 < kDirectBytes);
}

template <class T>
void run_few(const ExpertArgs& a, hipStream_t s) {
    const int n_tiles = (a.d_out + 15) / 16;
    const int64_t tiles = a.slots / 16 + a.n_experts + 1;
    const bool by_slot = a.slots < tiles;
    k_expert_few<T><<<(unsigned)((by_slot ? a.slots : tiles) * n_tiles), 64 * kFewWaves, 0, s>>>(a, n_tiles, by_slot);
}

// Which rows kernel, by the slots an expert has on average (all bfloat16
// figures are of one call, us):
//  - below 16, for at most 256 slots: k_expert_few.  16 experts 1024 -> 4096, 64
//    slots: 31 against 35 with 32-slot tiles (float32, 1024 -> 2048: 37 against
//    64); 256 slots, 16 an expert: 49 against 38; 1024 slots, 4 an expert: 14
//    against 12.
//  - below 32: 32-slot tiles.  1024 experts 256 -> 256, 16 slots each: 42 against
//    51 with copied tiles; 64 experts 512 -> 512, 32 each: 18 against 16.
//  - also with at most 64 columns, of which the larger tiles leave half empty, and
//    at most 512 k in bfloat16: 8 experts, 32768 slots each, 64 -> 64: 32 against 44
//    (float32: 59 against 80), 512 -> 64: 97 against 97; 8192 each, 1024 -> 64: 61
//    against 56 (float32: 163 against 233), 2047 -> 63: 142 against 130 (float32: 322
//    against 463); 1024 experts, 256 each, 64 -> 64: 36 against 76; but with 128
//    columns, 8 experts, 32768 each, 64 -> 128: 58 against 45 (float32: 111 against
//    89).  These are forward.  The gradient follows the same rule; of both gradients
//    with 128 columns, 128 -> 128 bfloat16, one-wave tiles would take 140 against 169
//    (8 experts, 32768 slots each), 136 against 151 (32, 8000) and 91 against 144
//    (500, 300), float32 342 against 326, 333 against 315 and 298 against 306.
//  - also below 256 with more than 63 experts (whose tiles have to be searched
//    for) and at most 128 x 128 weights: 1024 experts, 64 slots each, 128 -> 128:
//    29 against 45, 256 -> 256: 76 against 71; 256 slots each, 128 -> 128: 79
//    against 79.
//  - 32 x 32 tiles for up to 32 columns: both gradients of 16 experts 32 -> 256,
//    8192 slots each, float32: 164 against 230 with wider ones, bfloat16: 7 less.
//  - else copied tiles where rows allow it, or staged ones (128 x 128).
template <class T, bool GRAD>
void pick_rows(const ExpertArgs& a, hipStream_t s) {
    const int64_t N = GRAD ? a.d_in : a.d_out, K = GRAD ? a.d_out : a.d_in, per = a.slots / a.n_experts;
    const bool small = N <= 64 && (K <= 512 || sizeof(T) == 4);
    const bool narrow = a.n_experts > 63 && (int64_t)a.d_in * a.d_out <= 128 * 128;
    if (!GRAD && a.slots <= kFewSlots && per < 16)
        run_few<T>(a, s);
    else if (N <= 32)
        run_rows<T, GRAD, 32, 32, 32, 32>(a, s);
    else if (small || per < (narrow ? 256 : 32))
        run_rows<T, GRAD, 32, 64, 32, 64>(a, s);
    else if (sizeof(T) == 2 && direct_rows(a, GRAD))
        pick_rows_direct<GRAD>(a, s);
    else
        run_rows<T, GRAD, 128, 128, 64, 64>(a, s);
}

// Workgroups of `items` weight gradients of `tiles` tiles (as weight_work deals them out).
int64_t weight_blocks(int64_t items, int tiles) { return tiles < 8 ? items * tiles : 8 * items * ((tiles + 7) / 8); }

template <class T, int BM, int BN, int WM, int WN>
void run_weights(const ExpertArgs& a, hipStream_t s) {
    const int mt = (a.d_out + BM - 1) / BM, nt = (a.d_in + BN - 1) / BN;
    const int64_t items = a.chunk ? a.slots / a.chunk + a.n_experts : a.n_experts;
    k_expert_weights<T, BM, BN, WM, WN>
        <<<(unsigned)weight_blocks(items, mt * nt), WeightTile<T, BM, BN, WM, WN>::NT, 0, s>>>(a, mt, nt);
}

template <int BM, int BN, int WM, int WN>
void run_weights_direct(const ExpertArgs& a, hipStream_t s) {
    const int mt = (a.d_out + BM - 1) / BM, nt = (a.d_in + BN - 1) / BN;
    const int64_t items = a.chunk ? a.slots / a.chunk + a.n_experts : a.n_experts;
    constexpr int NT = DirectTile<BM, BN, WM, WN, float>::NT;
    const unsigned blocks = (unsigned)weight_blocks(items, mt * nt);
    if (a.order)
        k_expert_weights_direct<true, BM, BN, WM, WN><<<blocks, NT, 0, s>>>(a, mt, nt);
    else
        k_expert_weights_direct<false, BM, BN, WM, WN><<<blocks, NT, 0, s>>>(a, mt, nt);
}

// Whether the weight kernels may copy directly.
bool direct_weights(const ExpertArgs& a) {
    if (a.d_in % 8 || a.d_out % 8 || a.ld_x % 8 || a.ld_dz % 8 || a.ld_x > 1 << 22 || a.ld_dz > 1 << 22) return false;
    return aligned16(a.x) && aligned16(a.dz) && (!a.order || a.x_rows * a.ld_x * 2 < kDirectBytes);
}

// 256 x 256 tiles of a weight gradient where an expert's sums are long (2048
// slots and more on average), else 128 x 128 (two workgroups on a CU).  The
// weight gradient alone, bfloat16, us with 256 and with 128, of even experts | of
// experts whose slots fall off by rank as rank^-0.7:
//   16 experts 1024 -> 4096, 512 slots each: 113, 138 | 119, 147; 1024: 176, 210 |
//     182, 227; 2048: 275, 344 | 284, 343;
//   64 experts 512 -> 512, 512: 37, 47 | 77, 57; 2048: 110, 127 | 347, 236;
//   16 experts 512 -> 512, 1024: 41, 24 | 40, 38; 2048: 52, 41 | 51, 68; 8192: 114,
//     143 | 117, 315;
//   8 experts 256 -> 256, 1024: 24, 15 | 23, 16; 4096: 25, 23 | 25, 24; 8192: 29, 34
//     | 30, 34;
//   8 experts 1024 -> 1024, 1024: 36, 31 | 47, 35; 4096: 105, 97 | 155, 121.
// No length alone is right for all: many tiles of even experts want 256 earlier, few
// tiles or uneven experts, whose longest decides, 128 for longer.
bool wide_weight_tiles(int64_t slots, int n_experts, int d_in, int d_out) {
    return slots / n_experts >= 2048 && d_in > 128 && d_out > 128;
}

// Copied tiles where rows allow it, also of narrow weights (both gradients of 16
// experts 32 -> 256, 8192 slots each, bfloat16: 50 us against 82 with 32 x 64
// staged ones; 1024 experts 32 -> 64, 128 slots each: 37 and 44).  Staged ones are
// 32 x 64 where a side has at most 64 (float32, 1024 experts, 128 slots each,
// 63 -> 32: 90 against 145 with 128 x 128, 64 -> 64: 102 and 151; 16 experts
// 64 -> 256, 8192 each: 235 and 241).
template <class T>
void pick_weights(const ExpertArgs& a, hipStream_t s) {
    if (sizeof(T) == 2 && direct_weights(a)) {
        if (wide_weight_tiles(a.slots, a.n_experts, a.d_in, a.d_out))
            run_weights_direct<256, 256, 128, 64>(a, s);
        else
            run_weights_direct<128, 128, 64, 64>(a, s);
    } else if (a.d_out <= 64 || a.d_in <= 64) {
        run_weights<T, 32, 64, 32, 64>(a, s);
    } else {
        run_weights<T, 128, 128, 64, 64>(a, s);
    }
    if (a.chunk) {
        const int64_t per = (int64_t)a.d_out * a.d_in + (a.db ? a.d_out : 0);
        k_expert_sum<<<dim3((unsigned)((per + 255) / 256), a.n_experts), 256, 0, s>>>(a);
    }
}

}  // namespace

// With fewer tiles than half the workgroups that fit on the card, experts' slots
// are split into ranges so that the items fill it once; every range costs a
// write and a read of a float32 weight gradient, so none is below 512 slots.
int64_t expert_grad_chunk(int64_t slots, int n_experts, int d_in, int d_out) {
    const bool wide = wide_weight_tiles(slots, n_experts, d_in, d_out);
    const int64_t side = wide ? 256 : 128, fit = wide ? kCus : 2 * kCus;
    const int64_t tiles = ((d_in + side - 1) / side) * ((d_out + side - 1) / side);
    if (n_experts * tiles >= fit / 2 || slots <= 1024) return 0;
    const int64_t items = fit / tiles - n_experts > 1 ? fit / tiles - n_experts : 1;
    const int64_t chunk = ((slots + items - 1) / items + 63) / 64 * 64;
    return chunk > 512 ? chunk : 512;
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
