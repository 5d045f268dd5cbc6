// The gate of a routed field for gfx950: each sample's k largest logits of E,
// their softmax weights, and the logits' gradient.  For a row z, with the
// chosen experts i_1 .. i_k (largest first, the lowest index among equals):
//   w_j = e^(z_ij - m) / sum,  m = z_i1,  the sum over the chosen (renorm) or over all E
//   renorm:  dz_v = sum_{j: i_j = v} w_j (dw_j - S),          S = sum_j w_j dw_j
//   else:    dz_v = sum_{j: i_j = v} w_j dw_j - p_v S,        p = softmax over all E
// An expert whose logit is -inf is never chosen; a choice without an expert
// has id -1 and weight 0.
// A row is read once and stays in registers: k rounds of a maximum over its lanes,
// which bound the kernel (in a graph of calls, 262144 rows of 16 bfloat16 logits, 2
// chosen, 12.6 MB: 6.2 us, 2.0 TB/s; 16384 of 256, 8 chosen: 10.9 us; 4096 of 4096:
// 28 us, four times the read, as every round looks at all of a lane's keys), and a
// launch's latency for few rows (one: 2.6 us).  The gradient reads a row at most once:
// 20011 of 61 float32 logits, 10.5 MB, in 4.8 us, 2.2 TB/s.
#include <hip/hip_runtime.h>

#include <cmath>
#include <type_traits>

#include "common.hpp"
#include "fields.hpp"
#include "rowio.hpp"

namespace nerf {

namespace {

constexpr int kGateThreads = 256;
constexpr int kGateGrid = 1 << 16;  // workgroups at most; each takes every 2^16th group of rows

// A row belongs to G lanes of a wave, which hold it in NP 16-byte pieces each:
// piece p of lane g is number p G + g of the row.  Small E take few lanes (16
// bfloat16 logits two), so that a wave has many rows.
template <class T, int G, int NP>
struct GateRow {
    static constexpr int PER = RowIO<T>::PER;
    float z[NP * PER];

    static __device__ __forceinline__ int column(int g, int i) { return ((i / PER) * G + g) * PER + i % PER; }

    __device__ __forceinline__ void load(const T* row, int E, int g) {
#pragma unroll
        for (int p = 0; p < NP; ++p) {
            const int c = (p * G + g) * PER;
            typename RowIO<T>::Vec v = RowIO<T>::zero();
            if (c < E) v = RowIO<T>::load(row, c, E);
#pragma unroll
            for (int e = 0; e < PER; ++e) z[p * PER + e] = c + e < E ? RowIO<T>::get(v, e) : -INFINITY;
        }
    }
    // e^(z - m) summed over the row (every lane gets the sum)
    __device__ __forceinline__ float exp_sum(float m) const {
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NP * PER; ++i) s += expf(z[i] - m);
#pragma unroll
        for (int off = G / 2; off >= 1; off >>= 1) s += __shfl_xor(s, off, 64);
        return s;
    }
};

// Order of logits as unsigned numbers: -inf is kNoExpert and everything above it
// larger, 0 and -0 alike, NaN above all (its row's weights become NaN).
constexpr uint32_t kNoExpert = 0x007FFFFFu;
__device__ __forceinline__ uint32_t order_key(float z) {
    const uint32_t u = __float_as_uint(z + 0.0f);
    return z != z ? ~0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t key) {
    return key == ~0u ? __uint_as_float(0x7FC00000u) : __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// The largest of G lanes' values, in each of them.  Up to 16 lanes exchange
// within the vector units (pairs, fours, mirrored halves and rows of 16).
template <int CONTROL>
__device__ __forceinline__ uint32_t max_across(uint32_t v) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CONTROL, 0xF, 0xF, true);
    return o > v ? o : v;
}
template <int G>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
    if constexpr (G >= 2) v = max_across<0xB1>(v);    // lane ^ 1
    if constexpr (G >= 4) v = max_across<0x4E>(v);    // lane ^ 2
    if constexpr (G >= 8) v = max_across<0x141>(v);   // 7 - lane, of 8
    if constexpr (G >= 16) v = max_across<0x140>(v);  // 15 - lane, of 16
#pragma unroll
    for (int off = 16; off < G; off <<= 1) {
        const uint32_t o = __shfl_xor(v, off, 64);
        v = o > v ? o : v;
    }
    return v;
}

// The rows' keys.  Those of bfloat16 logits have 16 bits and leave 12 for the
// column, lowest first among equals, so that a maximum finds both.
constexpr int kColumnBits = 12;
static_assert(NERF_MAX_EXPERTS <= 1 << kColumnBits, "a column fits its key");
constexpr uint32_t kLastColumn = (1u << kColumnBits) - 1;

// Bound by instructions, not by memory: k rounds over the row's keys in
// registers, each a maximum over the lane's own and log2 G exchanges.
template <class T, int G, int NP>
__global__ void __launch_bounds__(kGateThreads) k_gate(GateArgs a) {
    using Row = GateRow<T, G, NP>;
    constexpr int N = NP * Row::PER, ROWS = kGateThreads / G;
    constexpr bool JOINT = sizeof(T) == 2;
    extern __shared__ char lds[];
    const int g = threadIdx.x % G, group = threadIdx.x / G;
    int* const ids = (int*)lds + group * a.k;
    float* const zs = (float*)lds + ROWS * a.k + group * a.k;
    // (whole waves stay in the loop: a wave's groups exchange under one mask)
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.n; r0 += (int64_t)gridDim.x * ROWS) {
        const int64_t r = r0 + group < a.n ? r0 + group : a.n - 1;
        Row row;
        row.load((const T*)a.logits + r * a.ld, a.n_experts, g);
        uint32_t key[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            key[i] = order_key(row.z[i]);
            if constexpr (JOINT) key[i] = (key[i] >> 16) << kColumnBits | (kLastColumn - Row::column(g, i));
        }
        float m = 0.0f, total = 0.0f;
        for (int j = 0; j < a.k; ++j) {
            uint32_t best = 0, mine = 0;
            int at = 0;
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (key[i] > mine) {
                    mine = key[i];
                    if constexpr (!JOINT) at = Row::column(g, i);
                }
            best = group_max<G>(mine);
            if constexpr (JOINT) {
                at = (int)(kLastColumn - (best & kLastColumn));
#pragma unroll
                for (int i = 0; i < N; ++i) key[i] = key[i] == best ? 0u : key[i];
                best = best >> kColumnBits << 16;
                // (the bits that a float32 number has more: those of the numbers' complement are ones)
                if (!(best & 0x80000000u) || best == 0xFFFF0000u) best |= 0xFFFFu;
            } else {
                at = (int)(kLastColumn - group_max<G>(mine == best ? kLastColumn - at : 0u));
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (Row::column(g, i) == at) key[i] = 0;
            }
            const bool some = best > kNoExpert;
            const float z = key_value(best);
            if (j == 0) {
                m = z;
                if (!a.renorm && some) total = row.exp_sum(m);
            }
            if (a.renorm && some) total += expf(z - m);
            if (g == 0) {
                ids[j] = some ? at : -1;
                zs[j] = some ? z : -INFINITY;
            }
        }
        wave_lds_sync();
        if (r0 + group < a.n)
            for (int j = g; j < a.k; j += G) {
                const int id = ids[j];
                a.ids[r * a.k + j] = id;
                a.weights[r * a.k + j] = id >= 0 ? expf(zs[j] - m) / total : 0.0f;
            }
        wave_lds_sync();
    }
}

template <class T, int G, int NP, bool RENORM>
__global__ void __launch_bounds__(kGateThreads) k_gate_grad(GateArgs a) {
    using Row = GateRow<T, G, NP>;
    using IO = RowIO<T>;
    constexpr int ROWS = kGateThreads / G;
    extern __shared__ char lds[];
    const int g = threadIdx.x % G, group = threadIdx.x / G;
    int* const ids = (int*)lds + group * a.k;
    float* const gs = (float*)lds + ROWS * a.k + group * a.k;
    for (int64_t r0 = (int64_t)blockIdx.x * ROWS; r0 < a.n; r0 += (int64_t)gridDim.x * ROWS) {
        const int64_t r = r0 + group < a.n ? r0 + group : a.n - 1;
        Row row;
        if constexpr (!RENORM) row.load((const T*)a.logits + r * a.ld, a.n_experts, g);
        // choices without an expert count for nothing, whatever their weights
        float sum = 0.0f;
        for (int j = g; j < a.k; j += G) {
            const int id = a.ids[r * a.k + j];
            const bool live = (unsigned)id < (unsigned)a.n_experts;
            const float w = live ? a.weights[r * a.k + j] : 0.0f, wd = live ? w * a.dweights[r * a.k + j] : 0.0f;
            ids[j] = live ? id : -1;
            gs[j] = RENORM ? w : wd;
            sum += wd;
        }
#pragma unroll
        for (int off = G / 2; off >= 1; off >>= 1) sum += __shfl_xor(sum, off, 64);
        if constexpr (RENORM)
            for (int j = g; j < a.k; j += G)
                if (ids[j] >= 0) gs[j] *= a.dweights[r * a.k + j] - sum;
        float dz[NP * Row::PER];
        if constexpr (RENORM) {
#pragma unroll
            for (int i = 0; i < NP * Row::PER; ++i) dz[i] = 0.0f;
        } else {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < NP * Row::PER; ++i) m = fmaxf(m, row.z[i]);
#pragma unroll
            for (int off = G / 2; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
            if (m == -INFINITY) m = 0.0f;  // (no expert: every p is 0, or NaN)
            const float total = row.exp_sum(m);
            const float f = total != 0.0f ? -sum / total : 0.0f;
#pragma unroll
            for (int i = 0; i < NP * Row::PER; ++i) dz[i] = f * expf(row.z[i] - m);
        }
        wave_lds_sync();
        for (int j = 0; j < a.k; ++j) {
            const int id = ids[j];
            const float v = gs[j];
#pragma unroll
            for (int i = 0; i < NP * Row::PER; ++i)
                if (Row::column(g, i) == id) dz[i] += v;
        }
        wave_lds_sync();
        if (r0 + group < a.n)
#pragma unroll
            for (int p = 0; p < NP; ++p) {
                const int c = (p * G + g) * Row::PER;
                if (c >= a.n_experts) continue;
                float o[Row::PER];
#pragma unroll
                for (int e = 0; e < Row::PER; ++e) o[e] = dz[p * Row::PER + e];
                IO::store((T*)a.dlogits + r * a.ld_d, c, a.n_experts, IO::pack(o));
            }
    }
}

// Calls f(G, NP) with the fewest lanes that hold a row in one piece each, or
// all 64 with up to 16 pieces (4096 float32).
template <class F>
void by_width(int pieces, F&& f) {
    using std::integral_constant;
    auto lanes = [&](auto g) { f(g, integral_constant<int, 1>{}); };
    auto deep = [&](auto np) { f(integral_constant<int, 64>{}, np); };
    if (pieces <= 1) lanes(integral_constant<int, 1>{});
    else if (pieces <= 2) lanes(integral_constant<int, 2>{});
    else if (pieces <= 4) lanes(integral_constant<int, 4>{});
    else if (pieces <= 8) lanes(integral_constant<int, 8>{});
    else if (pieces <= 16) lanes(integral_constant<int, 16>{});
    else if (pieces <= 32) lanes(integral_constant<int, 32>{});
    else if (pieces <= 64) lanes(integral_constant<int, 64>{});
    else if (pieces <= 128) deep(integral_constant<int, 2>{});
    else if (pieces <= 256) deep(integral_constant<int, 4>{});
    else if (pieces <= 512) deep(integral_constant<int, 8>{});
    else deep(integral_constant<int, 16>{});
}

unsigned gate_grid(int64_t n, int rows) {
    const int64_t blocks = (n + rows - 1) / rows;
    return (unsigned)(blocks < kGateGrid ? blocks : kGateGrid);
}

template <class T>
void launch(const GateArgs& a, hipStream_t s) {
    by_width((a.n_experts + RowIO<T>::PER - 1) / RowIO<T>::PER, [&](auto g, auto np) {
        constexpr int G = decltype(g)::value, NP = decltype(np)::value, ROWS = kGateThreads / G;
        if constexpr (NP * RowIO<T>::PER * 64 <= 4096) {
            const size_t lds = (size_t)ROWS * a.k * 8;
            k_gate<T, G, NP><<<gate_grid(a.n, ROWS), kGateThreads, lds, s>>>(a);
        }
    });
}

template <class T>
void launch_grad(const GateArgs& a, hipStream_t s) {
    by_width((a.n_experts + RowIO<T>::PER - 1) / RowIO<T>::PER, [&](auto g, auto np) {
        constexpr int G = decltype(g)::value, NP = decltype(np)::value, ROWS = kGateThreads / G;
        if constexpr (NP * RowIO<T>::PER * 64 <= 4096) {
            const size_t lds = (size_t)ROWS * a.k * 8;
            if (a.renorm)
                k_gate_grad<T, G, NP, true><<<gate_grid(a.n, ROWS), kGateThreads, lds, s>>>(a);
            else
                k_gate_grad<T, G, NP, false><<<gate_grid(a.n, ROWS), kGateThreads, lds, s>>>(a);
        }
    });
}

}  // namespace

void launch_gate(bool bf16, const GateArgs& a, hipStream_t s) {
    if (bf16)
        launch<__bf16>(a, s);
    else
        launch<float>(a, s);
}

void launch_gate_grad(bool bf16, const GateArgs& a, hipStream_t s) {
    if (bf16)
        launch_grad<__bf16>(a, s);
    else
        launch_grad<float>(a, s);
}

}  // namespace nerf
