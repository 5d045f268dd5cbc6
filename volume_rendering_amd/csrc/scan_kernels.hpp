// The gated linear recurrence and its gradient for gfx950.  Along a sequence,
// per channel,
//   h_t = a_t h_{t-1} + b_t,      b_t = x_t, or (1 - a_t) x_t  (mix)
// and, with D_t = dh_t + a_{t+1} D_{t+1} the whole gradient at h_t (D_T has
// dh_last added),
//   dx_t = D_t [(1 - a_t)],   da_t = sum over the gate's channels D_t (h_{t-1} [- x_t]),   dh0 = a_1 D_1.
// Both are recurrences s' = A s + B: the forward one with (a_t, b_t), the
// gradient against the sequence with (a_t, a_t dh_t) on what flows into h_t
// from behind.  n steps are again such a step, with the product of their A and
// the state that they reach from 0; so a wave's lanes take runs of S
// consecutive steps each, join the runs by a scan of those pairs, and then walk
// their own steps from the true state before them.  Products of gates only
// carry states from run to run; within a run the recurrence itself is applied.
//
// Bound by memory: x, a and h once each (the gradient: dh, a, h and the
// outputs), 65536 rays of 64 steps of 16 float32 channels in 109 us, 5.1 TB/s.
// A workgroup walks one sequence for a block of channels, tile by tile, with the
// tile's loads all in flight at once.  When sequences are too few for that to fill
// the card they are split into chunks of one tile, which hand the state on in one
// pass, looking back at the chunks in front (the published decoupled look-back of
// prefix sums, here of affine steps, with words that mark themselves ready): 2 of
// 32768 steps of 1024 bfloat16 channels in 122 us, 4.4 TB/s, the gradient in 236,
// 4.0 TB/s (chunks' sums first, the states between them and then the chunks, with
// every input read twice: 164 and 243).
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "common.hpp"
#include "fields.hpp"

namespace nerf {

namespace {

constexpr int kScanGrid = 1 << 20;

// V consecutive elements at any element alignment (global memory takes wide
// accesses at any address here), held as the 32-bit words they are loaded in:
// as elements the compiler gives each bfloat16 a register of its own.
template <class T, int V>
struct Some {
    static constexpr int WORDS = (V * (int)sizeof(T) + 3) / 4;
    struct Raw {
        uint32_t w[WORDS];
    };
    struct __attribute__((packed, aligned(sizeof(T)))) Memory {
        T e[V];
    };
    static __device__ __forceinline__ Raw raw(const T* p) {
        Raw r = {};
        if constexpr (V * sizeof(T) % 4 == 0) {
            struct __attribute__((packed, aligned(sizeof(T)))) Words {
                uint32_t w[WORDS];
            };
            const Words m = *reinterpret_cast<const Words*>(p);
#pragma unroll
            for (int i = 0; i < WORDS; ++i) r.w[i] = m.w[i];
        } else {
            r.w[0] = __builtin_bit_cast(uint16_t, p[0]);
        }
        return r;
    }
    static __device__ __forceinline__ float get(const Raw& r, int v) {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(r.w[v]);
        else
            return __uint_as_float((v & 1) ? r.w[v / 2] & 0xFFFF0000u : r.w[v / 2] << 16);
    }
    static __device__ __forceinline__ void load(float (&f)[V], const T* p) {
        const Raw r = raw(p);
#pragma unroll
        for (int v = 0; v < V; ++v) f[v] = get(r, v);
    }
    // Elements from `skip` on.  STREAM: past the caches, which are left to the inputs.
    template <bool STREAM = false>
    static __device__ __forceinline__ void store(T* p, const float (&f)[V], int skip) {
        Memory m;
#pragma unroll
        for (int v = 0; v < V; ++v) m.e[v] = (T)f[v];
        if (skip == 0) {
            constexpr int BYTES = V * (int)sizeof(T);
            if constexpr (STREAM && BYTES >= 8) {
                typedef uint32_t Vec __attribute__((ext_vector_type(BYTES / 4)));
                typedef uint32_t Loose __attribute__((ext_vector_type(BYTES / 4), aligned(sizeof(T))));
                __builtin_nontemporal_store(__builtin_bit_cast(Vec, m), reinterpret_cast<Loose*>(p));
                return;
            }
            *reinterpret_cast<Memory*>(p) = m;
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (v >= skip) p[v] = m.e[v];
        }
    }
};

// What a workgroup (or, of single waves, a wave) works on: steps [c0, c1) of a
// sequence of `len`, whose step i is row first + i step, for channels from
// block on.
struct ScanUnit {
    int64_t seq, first, len, c0, c1;
    int step, block;
};

__device__ __forceinline__ int64_t clamp_row(int64_t v, int64_t rows) { return v < 0 ? 0 : v > rows ? rows : v; }

__device__ __forceinline__ void sequence_rows(const ScanArgs& a, int64_t seq, int64_t& lo, int64_t& len) {
    if (a.offsets) {
        const int64_t o0 = a.offsets[seq], o1 = a.offsets[seq + 1];
        NERF_DCHECK(o0 >= 0 && o1 >= o0 && o1 <= a.rows, kCheckScanOffset);
        lo = clamp_row(o0, a.rows);
        const int64_t hi = clamp_row(o1, a.rows);
        len = hi > lo ? hi - lo : 0;
    } else {
        lo = seq * a.len;
        len = a.len;
    }
}

// Quotient and remainder of numbers that mostly fit 32 bits.
__device__ __forceinline__ int64_t quotient(int64_t u, int64_t by, int64_t& rest) {
    if (((uint64_t)u | (uint64_t)by) >> 32) {
        rest = u % by;
        return u / by;
    }
    const uint32_t q = (uint32_t)u / (uint32_t)by;
    rest = (uint32_t)u - q * (uint32_t)by;
    return q;
}

// First chunk of a sequence of given offsets: at most one more than the whole
// chunks in front for each (room for every sequence's partial one).
__device__ __forceinline__ int64_t first_slot(const ScanArgs& a, int64_t seq) {
    return (uint32_t)clamp_row(a.offsets[seq], a.rows) / (uint32_t)a.p.chunk + seq;
}

// Unit `u` of a call that walks whole sequences (chunk 0), or of one chunk
// each, of which every sequence has one at least; false if there is nothing to
// do.  By whole waves.
__device__ __forceinline__ bool scan_unit(const ScanArgs& a, int64_t u, bool against, ScanUnit& r) {
    int64_t lo, rest = 0;
    if (a.p.blocks > 1) u = quotient(u, a.p.blocks, rest);
    r.block = (int)rest;
    if (a.p.chunk == 0) {
        r.seq = u;
        sequence_rows(a, u, lo, r.len);
        r.c0 = 0;
        r.c1 = r.len;
    } else {
        int64_t i;
        if (a.offsets) {
            // the last sequence whose first chunk is at or before u; there are few (kScanMaxSplit), so
            // the lanes look at all of them at once
            int before = 0;
#pragma unroll
            for (int j = 0; j < kScanMaxSplit / 64; ++j) {
                const int64_t seq = 64 * j + lane_id();
                before += __popcll(__ballot(seq < a.n_seq && first_slot(a, seq < a.n_seq ? seq : 0) <= u));
            }
            r.seq = before - 1;
            if (r.seq < 0) return false;
            i = u - first_slot(a, r.seq);
        } else {
            i = quotient(u, a.n_seq, r.seq);  // (sequences side by side)
        }
        sequence_rows(a, r.seq, lo, r.len);
        r.c0 = i * a.p.chunk;
        if (i < 0 || (i > 0 && r.c0 >= r.len)) return false;
        r.c1 = r.c0 + a.p.chunk < r.len ? r.c0 + a.p.chunk : r.len;
    }
    r.step = (a.reverse != 0) != against ? -1 : 1;
    r.first = r.step > 0 ? lo : lo + r.len - 1;
    return true;
}

// A lane's channels.  It has V of them from `c` on, of which those before
// `skip` belong to its neighbour (the last lane of a width that is no multiple
// of V starts earlier); none of them if !live.
struct ScanLane {
    int c, gate, skip;
    bool live, gate_live;  // gate_live: the lane's gate exists
};
template <int V, bool GROUPED>
__device__ __forceinline__ ScanLane scan_lane(const ScanArgs& a, int block, int cl) {
    ScanLane r;
    if constexpr (GROUPED) {
        const int m = a.d / a.gates, lg = a.p.lg, per = a.p.cl / lg;  // gates side by side in a block
        const int in = cl % lg + block % a.p.parts * lg;              // lane of the gate's channels
        r.gate = block / a.p.parts * per + cl / lg;
        const int want = in * V;
        r.live = r.gate < a.gates && want < m;
        const int c = want + V <= m ? want : m - V;
        r.skip = r.live ? want - c : V;
        r.gate_live = r.gate < a.gates;
        if (!r.gate_live) r.gate = a.gates - 1;
        r.c = r.gate * m + c;
    } else {
        const int64_t want = ((int64_t)block * a.p.cl + cl) * V;
        r.live = want < a.d;
        r.c = want + V <= a.d ? (int)want : a.d - V;
        r.skip = r.live ? (int)want - r.c : V;
        r.gate = r.c;
        r.gate_live = r.live;
    }
    return r;
}

// s' = A s + B for a lane's channels: NA is V, or 1 where they share a gate.
template <int NA, int V>
struct Affine {
    float A[NA], B[V];
};
// Products of gates.  One of gates that are not 0 stays so when it leaves
// float32's range, as an infinite state stays infinite behind it; a finite state
// gets 2^-149 of itself at most, half of which such a product is off by anyway.
__device__ __forceinline__ float not_zero(float p, bool zero) {
    return p == 0.0f && !zero ? copysignf(0x1p-149f, p) : p;
}
__device__ __forceinline__ float times(float a, float b) { return not_zero(a * b, a == 0.0f || b == 0.0f); }
template <int NA, int V>
__device__ __forceinline__ Affine<NA, V> after(const Affine<NA, V>& first, const Affine<NA, V>& then) {
    Affine<NA, V> r;
#pragma unroll
    for (int v = 0; v < V; ++v) r.B[v] = fmaf(then.A[NA == 1 ? 0 : v], first.B[v], then.B[v]);
#pragma unroll
    for (int v = 0; v < NA; ++v) r.A[v] = times(then.A[v], first.A[v]);
    return r;
}

// ---------------------------------------------------------------------------
// Chunks of one sequence, worked on at once.  A chunk's workgroup leaves the
// chunk as one step (A, B) for those behind it, takes the state before it from
// the nearest workgroup in front that has left the state after its chunk, and
// steps over the chunks between; then it leaves the state after its own.  Those
// steps are always taken one by one in order, so the result does not depend on
// how far back the nearest state was.
// The words carry their own readiness: kNotYet, a NaN that nothing computed is
// left as, stands in all of them at first.  So no order among them matters, and
// plain device-wide atomic words do, without fences.
// Workgroups take their chunks from a counter: whoever waits waits for one that
// took its chunk earlier, so runs already, and every one leaves its words whatever
// its offsets are.  Only another call in the same workspace at the same time can
// take words away; the wait then ends with NaN.
// ---------------------------------------------------------------------------
constexpr uint32_t kNotYet = 0xFFFFFFFFu;
constexpr int kLooks = 1 << 21;  // at least a second of a running wave, however long it was set aside

__device__ __forceinline__ void leave(uint32_t* p, float f) {
    const uint32_t w = __float_as_uint(f);
    __hip_atomic_store(p, w == kNotYet ? 0x7FC00000u : w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ uint32_t look(const uint32_t* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// Looks again until the words of all lanes are there.
__device__ __forceinline__ float wait_for(const uint32_t* p, uint32_t w, int& looks) {
    while (!__all(w != kNotYet) && --looks > 0) {
        __builtin_amdgcn_s_sleep(1);
        w = look(p);
    }
    return __uint_as_float(w);
}

// How many chunks in front the nearest state is (of the channel whose word is
// `first`): 1 to `most`.  By a wave.
__device__ __forceinline__ int nearest_state(const uint32_t* first, int64_t back, int most, int lane, int& looks) {
    for (;;) {
        const bool in = lane < most;
        const uint64_t have = __ballot(in && look(first - (in ? lane + 1 : 1) * back) != kNotYet);
        if (have) return __builtin_ctzll(have) + 1;
        if (--looks <= 0) return 1;
        __builtin_amdgcn_s_sleep(1);
    }
}

constexpr int kScanLooked = 4096;  // words of the chunks between, at most

// Sums over lg lanes (a power of two) of N values each, a power of two.  While
// values are left to halve, a lane keeps one half of them and hands over the
// other, so that ten exchanges do for eight values and 64 lanes; lane g of the
// lg ends up with value g / (lg / N) (fewer lanes than values: with those from
// g N / lg on).
template <int H, int N>
__device__ __forceinline__ void sum_halves(float (&v)[N], int off, int lane) {
    if constexpr (H >= 1) {
        if (off < 1) return;
        const bool up = lane & off;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const float give = up ? v[i] : v[i + H], keep = up ? v[i + H] : v[i];
            v[i] = keep + __shfl_xor(give, off, 64);
        }
        sum_halves<H / 2>(v, off / 2, lane);
    } else {
        for (; off >= 1; off >>= 1) v[0] += __shfl_xor(v[0], off, 64);
    }
}

// The gradient of a lane's gate at S steps from row `first` on, of which it has
// `mine`: the sum over the gate's lanes.
template <class TA, int S>
__device__ __forceinline__ void store_gate_sums(const ScanArgs& a, const ScanLane& ch, float (&sum)[S], int block, int cl,
                                                int lane, int64_t first, int step, int mine) {
    const int lg = a.p.lg, g = cl % lg;
    sum_halves<S / 2>(sum, lg / 2, lane);
    const int have = lg >= S ? 1 : S / lg, each = lg >= S ? lg / S : 1;
    if (g % each != 0 || !ch.gate_live) return;
#pragma unroll
    for (int i = 0; i < S; ++i) {
        const int j = g / each * have + i;
        if (i >= have || j >= mine) break;
        const int64_t r = first + (int64_t)j * step;
        if (a.p.parts > 1)
            a.part_da[((int64_t)(block % a.p.parts) * a.rows + r) * a.gates + ch.gate] = sum[i];
        else
            ((TA*)a.da)[r * a.gates + ch.gate] = (TA)sum[i];
    }
}

// TA, T: types of the gates and of the rows; V channels a lane; W waves share a
// unit (1: each wave has its own); S steps a lane; BACK: the gradient; STREAM:
// outputs are stored past the caches; CHAIN: units are chunks of one tile (two
// workgroups a CU for bfloat16 rows, so that one loads while the other waits:
// 125 us against 146 in 175 registers; float32 rows would spill too much of
// theirs: 83 us against 106).
template <class TA, class T, int V, bool GROUPED, int W, int S, bool BACK, bool STREAM, bool CHAIN>
__global__ void __launch_bounds__(W == 1 ? 256 : 64 * W, CHAIN && sizeof(T) == 2 ? 4 : 1) k_scan(ScanArgs a, int64_t units) {
    constexpr int NA = GROUPED ? 1 : V;
    using Aff = Affine<NA, V>;
    __shared__ Aff total[W == 1 || CHAIN ? 1 : 2][W][W == 1 ? 1 : 64];
    __shared__ float handed[CHAIN ? 64 : 1][V];
    __shared__ float between_a[CHAIN ? kScanLooked : 1], between_b[CHAIN ? kScanLooked : 1];
    __shared__ int64_t taken;
    __shared__ int nearest;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int CL = a.p.cl, TL = 64 / CL, cl = lane % CL, tl = lane / CL;
    const int run = TL * S;  // steps of a wave's tile
    const T* const in = (const T*)(BACK ? a.dh : a.x);
    const int64_t ld_in = BACK ? a.ld_dh : a.ld_x;
    int turn = 0;
    for (int64_t u = W == 1 ? (int64_t)blockIdx.x * 4 + wave : blockIdx.x; u < units;
         u += W == 1 ? (int64_t)gridDim.x * 4 : gridDim.x) {
        ScanUnit q;
        int64_t unit = u;
        if constexpr (CHAIN) {
            if (threadIdx.x == 0) taken = (int64_t)atomicAdd((unsigned long long*)a.ticket, 1ull);
            __syncthreads();
            unit = (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(taken >> 32)) << 32 |
                             (uint32_t)__builtin_amdgcn_readfirstlane((int)taken));
        }
        // a chunk's words, and how far in front those of the chunk before are
        const int64_t words = unit * CL * V, back = (a.offsets ? 1 : a.n_seq) * (int64_t)a.p.blocks * CL * V;
        if (!scan_unit(a, unit, BACK, q)) {
            if constexpr (CHAIN) {
                if ((int)threadIdx.x < CL * V) {
                    leave(a.sum_a + words + threadIdx.x, 0.0f);
                    leave(a.sum_b + words + threadIdx.x, 0.0f);
                    leave(a.state + words + threadIdx.x, 0.0f);
                }
                __syncthreads();
            }
            continue;
        }
        const ScanLane ch = scan_lane<V, GROUPED>(a, q.block, cl);
        // the state before the unit's first step
        float s[V];
        {
            const float* const from = BACK ? a.dh_last : a.h0;
#pragma unroll
            for (int v = 0; v < V; ++v) s[v] = 0.0f;
            if (from && !CHAIN) Some<float, V>::load(s, from + q.seq * a.d + ch.c);
        }
        float first_h[V];  // gradient: the state before the sequence
        if constexpr (BACK) {
#pragma unroll
            for (int v = 0; v < V; ++v) first_h[v] = 0.0f;
            if (a.h0) Some<float, V>::load(first_h, a.h0 + q.seq * a.d + ch.c);
        }

        // What a lane has loaded of a tile (kept as loaded until it is used: bfloat16 rows take half the registers).
        struct Rows {
            typename Some<TA, NA>::Raw a[S];
            typename Some<T, V>::Raw in[S], h[BACK ? S : 1], x[BACK ? S : 1];
        };
        auto steps_of = [&](int64_t t0) {  // the wave's steps of a tile: at most `run`, none if <= 0
            const int64_t w0 = t0 + (W == 1 ? 0 : wave * run);
            return q.c1 - w0 < run ? (int)(q.c1 - w0) : run;
        };
        // Addresses are 32-bit offsets of lanes from bases that are the wave's.  Where every
        // lane has all its steps (and the row after each) a lane has one for all of them; else
        // steps past the end repeat the last one's loads and are left out.
        auto whole_tile = [&](int64_t t0) {
            const int64_t w0 = t0 + (W == 1 ? 0 : wave * run);
            return steps_of(t0) == run && (!BACK || w0 + run < q.len);
        };
        auto fetch = [&](Rows& f, int64_t t0, auto whole) {
            constexpr bool WHOLE = decltype(whole)::value;
            const int64_t w0 = t0 + (W == 1 ? 0 : wave * run), row0 = q.first + w0 * q.step;
            const int left = steps_of(t0);
            {
                const bool up = q.step > 0;
                // the lowest row that the wave reads, as offsets are not negative
                const int64_t low = up ? row0 : row0 - (WHOLE ? run - S : left - 1);
                const uint32_t lane_row = (uint32_t)(up ? tl * S : run - S - tl * S);
                auto at = [&](auto* base, int64_t ld, int c, int j, int more) {
                    using P = decltype(base);
                    int64_t row = low;
                    uint32_t rel = lane_row;
                    if constexpr (WHOLE) {
                        row += (int64_t)(j + more) * q.step;
                    } else {
                        int i = tl * S + j;
                        i = i < left ? i : left - 1;
                        if (more) {
                            if (w0 + i + 1 < q.len) ++i;
                            row -= up ? 0 : 1;
                        }
                        rel = (uint32_t)(up ? i : left - 1 + more - i);
                    }
                    return (P)((const char*)(base + row * ld) +
                               (rel * (uint32_t)ld + (uint32_t)c) * (uint32_t)sizeof(*base));
                };
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    f.a[j] = Some<TA, NA>::raw(at((const TA*)a.a, a.ld_a, ch.gate, j, 0));
                    f.in[j] = Some<T, V>::raw(at(in, ld_in, ch.c, j, 0));
                }
                if constexpr (BACK) {
#pragma unroll
                    for (int j = 0; j < S; ++j) f.h[j] = Some<T, V>::raw(at((const T*)a.h, a.ld_h, ch.c, j, 1));
                    if (a.mix)
#pragma unroll
                        for (int j = 0; j < S; ++j) f.x[j] = Some<T, V>::raw(at((const T*)a.x, a.ld_x, ch.c, j, 0));
                }
            }
        };

        // With few workgroups (eight waves each) the next tile's loads are in flight while one is worked on.
        constexpr bool AHEAD = W == 8 && !CHAIN;
        Rows next;
        auto fetch_next = [&](int64_t t0) {
            if (whole_tile(t0))
                fetch(next, t0, std::true_type{});
            else if (steps_of(t0) > 0)
                fetch(next, t0, std::false_type{});
        };
        if constexpr (AHEAD) fetch_next(q.c0);
        for (int64_t t0 = q.c0; t0 < q.c1 || (CHAIN && t0 == q.c0); t0 += (int64_t)W * run) {
            const int64_t w0 = t0 + (W == 1 ? 0 : wave * run);  // the wave's first step
            const int left = steps_of(t0);
            const int mine = left - tl * S;              // this lane's steps: min(mine, S)
            const int64_t row0 = q.first + w0 * q.step;  // row of the wave's first step
            Rows f;
            auto gate_of = [&](int j, int v) { return Some<TA, NA>::get(f.a[j], NA == 1 ? 0 : v); };
            auto in_of = [&](int j, int v) {
                const float in = Some<T, V>::get(f.in[j], v);
                return !BACK && a.mix ? in * (1.0f - gate_of(j, v)) : in;
            };
            Aff lanes;         // the lane's run as one step
            float least[NA];  // the smallest gate's magnitude
#pragma unroll
            for (int v = 0; v < NA; ++v) lanes.A[v] = least[v] = 1.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) lanes.B[v] = 0.0f;
            auto fold = [&](auto whole) {
#pragma unroll
                for (int j = 0; j < S; ++j)
                    if (decltype(whole)::value || j < mine) {
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            const float A = gate_of(j, v), in = in_of(j, v);
                            lanes.B[v] = BACK ? A * (lanes.B[v] + in) : fmaf(A, lanes.B[v], in);
                        }
#pragma unroll
                        for (int v = 0; v < NA; ++v) {
                            lanes.A[v] *= gate_of(j, v);
                            least[v] = fminf(least[v], fabsf(gate_of(j, v)));
                        }
                    }
#pragma unroll
                for (int v = 0; v < NA; ++v) lanes.A[v] = not_zero(lanes.A[v], least[v] == 0.0f);
            };
            if constexpr (AHEAD) {
                f = next;
                fetch_next(t0 + (int64_t)W * run);
                fold(std::false_type{});
            } else if (whole_tile(t0)) {
                fetch(f, t0, std::true_type{});
                fold(std::true_type{});
            } else if (left > 0) {
                fetch(f, t0, std::false_type{});
                fold(std::false_type{});
            }

            // runs of the wave's lanes of the same channels, in order
            Aff all = lanes, before;  // the wave's steps; those of the lanes before
#pragma unroll
            for (int v = 0; v < NA; ++v) before.A[v] = 1.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) before.B[v] = 0.0f;
            if (TL > 1) {
                for (int off = CL; off < 64; off <<= 1) {
                    Aff o;
#pragma unroll
                    for (int v = 0; v < NA; ++v) o.A[v] = __shfl_up(lanes.A[v], off, 64);
#pragma unroll
                    for (int v = 0; v < V; ++v) o.B[v] = __shfl_up(lanes.B[v], off, 64);
                    if (lane >= off) lanes = after(o, lanes);
                }
#pragma unroll
                for (int v = 0; v < NA; ++v) {
                    all.A[v] = __shfl(lanes.A[v], 64 - CL + cl, 64);
                    const float A = __shfl_up(lanes.A[v], CL, 64);
                    if (tl > 0) before.A[v] = A;
                }
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    all.B[v] = __shfl(lanes.B[v], 64 - CL + cl, 64);
                    const float B = __shfl_up(lanes.B[v], CL, 64);
                    if (tl > 0) before.B[v] = B;
                }
            }
            // the state before the wave's first step, and after the tile
            float st[V];
            if constexpr (W == 1) {
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    st[v] = s[v];
                    s[v] = fmaf(all.A[NA == 1 ? 0 : v], s[v], all.B[v]);
                }
            } else if constexpr (CHAIN) {
                if (tl == 0) total[0][wave][cl] = all;
                __syncthreads();
                // a lane to a channel, by as many waves as that takes
                const int width = CL * V, groups = (width + 63) / 64;
                const bool joins = wave < groups;
                const int word = wave * 64 + lane < width ? wave * 64 + lane : 0, cw = word / V, v = word % V;
                float A = 1.0f, B = 0.0f, s1 = 0.0f;
                if (joins) {
                    float least = 1.0f;
#pragma unroll
                    for (int w = 0; w < W; ++w) {
                        const float m = total[0][w][cw].A[NA == 1 ? 0 : v];
                        B = fmaf(m, B, total[0][w][cw].B[v]);
                        A *= m;
                        least = fminf(least, fabsf(m));
                    }
                    A = not_zero(A, least == 0.0f);
                    leave(a.sum_a + words + word, A);
                    leave(a.sum_b + words + word, B);
                }
                if (q.c0 > 0) {
                    int looks = kLooks;
                    if (wave == 0) {
                        const uint32_t front = (uint32_t)q.c0 / (uint32_t)a.p.chunk, window = kScanLooked / width;
                        const int most = front < 64 && front < window ? (int)front : window < 64 ? (int)window : 64;
                        nearest = nearest_state(a.state + words, back, most, lane, looks);
                    }
                    __syncthreads();
                    const int k = __builtin_amdgcn_readfirstlane(nearest);
                    uint32_t w = joins ? look(a.state + (words - k * back) + word) : 0;
                    // the chunks between, the farthest first
                    const int in = lane < width ? lane : 0, all_of = (k - 1) * groups;
                    for (int p = wave; p < all_of; p += W) {
                        const int64_t at = words - (k - 1 - p / groups) * back + (p % groups) * 64;
                        const uint32_t wa = look(a.sum_a + at + in), wb = look(a.sum_b + at + in);
                        const int to = p / groups * width + p % groups * 64 + in;
                        between_a[to] = wait_for(a.sum_a + at + in, wa, looks);
                        between_b[to] = wait_for(a.sum_b + at + in, wb, looks);
                    }
                    if (k > 1) __syncthreads();
                    if (joins) s1 = wait_for(a.state + (words - k * back) + word, w, looks);
                    if (joins)
#pragma unroll 4
                        for (int p = 0; p < k - 1; ++p) s1 = fmaf(between_a[p * width + word], s1, between_b[p * width + word]);
                }
                if (joins) {
                    const ScanLane own = scan_lane<V, GROUPED>(a, q.block, cw);
                    const int64_t c = q.seq * a.d + own.c + v;
                    if (q.c0 == 0) {
                        const float* const from = BACK ? a.dh_last : a.h0;
                        s1 = from ? from[c] : 0.0f;
                    }
                    handed[cw][v] = s1;
                    s1 = fmaf(A, s1, B);
                    leave(a.state + words + word, s1);
                    float* const last = BACK ? a.dh0 : a.h_last;
                    if (last && q.c1 == q.len && own.live && v >= own.skip) last[c] = s1;
                }
                __syncthreads();
#pragma unroll
                for (int v = 0; v < V; ++v) st[v] = handed[cl][v];
                for (int w = 0; w < wave; ++w) {
                    const Aff o = total[0][w][cl];
#pragma unroll
                    for (int v = 0; v < V; ++v) st[v] = fmaf(o.A[NA == 1 ? 0 : v], st[v], o.B[v]);
                }
            } else {
                // (two buffers in turn: a wave is at most one tile ahead of the slowest)
                if (tl == 0) total[turn][wave][cl] = all;
                __syncthreads();
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const Aff o = total[turn][w][cl];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        if (w == wave) st[v] = s[v];
                        s[v] = fmaf(o.A[NA == 1 ? 0 : v], s[v], o.B[v]);
                    }
                }
                turn ^= 1;
            }
            if (left <= 0) continue;
#pragma unroll
            for (int v = 0; v < V; ++v) st[v] = fmaf(before.A[NA == 1 ? 0 : v], st[v], before.B[v]);
            // the steps themselves
            const int64_t lane0 = row0 + (int64_t)(tl * S) * q.step;
            if constexpr (!BACK) {
                T* out = (T*)a.h + lane0 * a.ld_h + ch.c;
#pragma unroll
                for (int j = 0; j < S; ++j, out += q.step * a.ld_h) {
#pragma unroll
                    for (int v = 0; v < V; ++v) st[v] = fmaf(gate_of(j, v), st[v], in_of(j, v));
                    if (j < mine && ch.live) Some<T, V>::template store<STREAM>(out, st, ch.skip);
                }
            } else {
                float sum[S];
                T* out = (T*)a.dx + lane0 * a.d + ch.c;
                TA* gate = (TA*)a.da + lane0 * a.gates + ch.c;
#pragma unroll
                for (int j = 0; j < S; ++j, out += (int64_t)q.step * a.d, gate += (int64_t)q.step * a.gates) {
                    float dx[V], da[V];
                    const bool begins = w0 + tl * S + j + 1 == q.len;  // the sequence's first step
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float A = gate_of(j, v), D = in_of(j, v) + st[v];
                        float before = begins ? first_h[v] : Some<T, V>::get(f.h[j], v);
                        if (a.mix) before -= Some<T, V>::get(f.x[j], v);
                        dx[v] = a.mix ? (1.0f - A) * D : D;
                        da[v] = D * before;
                        st[v] = A * D;
                    }
                    if (j < mine && ch.live) {
                        Some<T, V>::template store<STREAM>(out, dx, ch.skip);
                        if constexpr (!GROUPED) Some<TA, V>::template store<STREAM>(gate, da, ch.skip);
                    }
                    if constexpr (GROUPED) {
                        sum[j] = 0.0f;
#pragma unroll
                        for (int v = 0; v < V; ++v) sum[j] += ch.live && v >= ch.skip ? da[v] : 0.0f;
                    }
                }
                if constexpr (GROUPED) store_gate_sums<TA, S>(a, ch, sum, q.block, cl, lane, lane0, q.step, mine);
            }
        }
        if constexpr (!CHAIN) {
            // (every wave has the state after the last tile)
            float* const last = BACK ? a.dh0 : a.h_last;
            if (last && ch.live && tl == 0 && (W == 1 || wave == 0))
                Some<float, V>::store(last + q.seq * a.d + ch.c, s, ch.skip);
        }
        if constexpr (CHAIN) __syncthreads();  // (before the next chunk's number is written)
    }
}

// Many sequences of few steps: a lane of a wave's 64 / CL time lanes has one of its
// own, and walks it run by run; nothing is exchanged but the sums of a gate's
// gradient.
template <class TA, class T, int V, bool GROUPED, int S, bool BACK>
__global__ void __launch_bounds__(256) k_scan_short(ScanArgs a, int64_t waves) {
    constexpr int NA = GROUPED ? 1 : V;
    const int lane = threadIdx.x & 63;
    const int CL = a.p.cl, cl = lane % CL, each = 64 / CL;
    const T* const in = (const T*)(BACK ? a.dh : a.x);
    const int64_t ld_in = BACK ? a.ld_dh : a.ld_x;
    for (int64_t w = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); w < waves; w += (int64_t)gridDim.x * 4) {
        int64_t block = 0;
        const int64_t group = a.p.blocks > 1 ? quotient(w, a.p.blocks, block) : w;
        const int64_t seq = group * each + lane / CL;
        if (seq >= a.n_seq) continue;  // (its lanes leave together, and exchange only among themselves)
        const ScanLane ch = scan_lane<V, GROUPED>(a, (int)block, cl);
        int64_t lo, len;
        sequence_rows(a, seq, lo, len);
        const int step = (a.reverse != 0) != BACK ? -1 : 1;
        const int64_t first = step > 0 ? lo : lo + len - 1;
        float st[V], first_h[V];
        const float* const from = BACK ? a.dh_last : a.h0;
#pragma unroll
        for (int v = 0; v < V; ++v) st[v] = first_h[v] = 0.0f;
        if (from) Some<float, V>::load(st, from + seq * a.d + ch.c);
        if (BACK && a.h0) Some<float, V>::load(first_h, a.h0 + seq * a.d + ch.c);
        for (int64_t t0 = 0; t0 < len; t0 += S) {
            const int left = len - t0 < S ? (int)(len - t0) : S;
            typename Some<TA, NA>::Raw ra[S];
            typename Some<T, V>::Raw ri[S], rh[BACK ? S : 1], rx[BACK ? S : 1];
            // (steps past the end repeat the last one's loads)
            auto row = [&](int j) { return first + (t0 + (j < left ? j : left - 1)) * step; };
#pragma unroll
            for (int j = 0; j < S; ++j) {
                ra[j] = Some<TA, NA>::raw((const TA*)a.a + row(j) * a.ld_a + ch.gate);
                ri[j] = Some<T, V>::raw(in + row(j) * ld_in + ch.c);
            }
            if constexpr (BACK) {
#pragma unroll
                for (int j = 0; j < S; ++j) {
                    const int64_t r = row(j), before = t0 + (j < left ? j : left - 1) + 1 < len ? r + step : r;
                    rh[j] = Some<T, V>::raw((const T*)a.h + before * a.ld_h + ch.c);
                    if (a.mix) rx[j] = Some<T, V>::raw((const T*)a.x + r * a.ld_x + ch.c);
                }
            }
            float sum[S];
#pragma unroll
            for (int j = 0; j < S; ++j) {
                const bool has = j < left;
                const int64_t r = first + (t0 + j) * step;
                if constexpr (!BACK) {
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float A = Some<TA, NA>::get(ra[j], NA == 1 ? 0 : v), x = Some<T, V>::get(ri[j], v);
                        const float now = fmaf(A, st[v], a.mix ? x * (1.0f - A) : x);
                        st[v] = has ? now : st[v];
                    }
                    if (has && ch.live) Some<T, V>::store((T*)a.h + r * a.ld_h + ch.c, st, ch.skip);
                } else {
                    float dx[V], da[V];
                    const bool begins = t0 + j + 1 == len;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float A = Some<TA, NA>::get(ra[j], NA == 1 ? 0 : v), D = Some<T, V>::get(ri[j], v) + st[v];
                        float before = begins ? first_h[v] : Some<T, V>::get(rh[j], v);
                        if (a.mix) before -= Some<T, V>::get(rx[j], v);
                        dx[v] = a.mix ? (1.0f - A) * D : D;
                        da[v] = D * before;
                        st[v] = has ? A * D : st[v];
                    }
                    if (has && ch.live) {
                        Some<T, V>::store((T*)a.dx + r * a.d + ch.c, dx, ch.skip);
                        if constexpr (!GROUPED)
                            Some<TA, V>::store((TA*)a.da + r * a.gates + ch.c, da, ch.skip);
                    }
                    sum[j] = 0.0f;
#pragma unroll
                    for (int v = 0; v < V; ++v) sum[j] += ch.live && v >= ch.skip ? da[v] : 0.0f;
                }
            }
            if constexpr (BACK && GROUPED) store_gate_sums<TA, S>(a, ch, sum, (int)block, cl, lane, first + t0 * step, step, left);
        }
        float* const last = BACK ? a.dh0 : a.h_last;
        if (last && ch.live) Some<float, V>::store(last + seq * a.d + ch.c, st, ch.skip);
    }
}

// Whole sequences, alone or by waves, or chunks of them.
template <class TA, class T, int V, bool GROUPED, bool BACK>
void run_scan(const ScanArgs& a, hipStream_t s) {
    using std::integral_constant;
    // (the gradient of float32 rows holds twice the registers a step)
    constexpr int kSteps = scan_steps(BACK);
    if (a.p.alone) {
        const int64_t each = 64 / a.p.cl, waves = (a.n_seq + each - 1) / each * a.p.blocks, blocks = (waves + 3) / 4;
        const unsigned grid = (unsigned)(blocks < kScanGrid ? blocks : kScanGrid);
        if (!a.offsets && a.len <= 1)
            k_scan_short<TA, T, V, GROUPED, 1, BACK><<<grid, 256, 0, s>>>(a, waves);
        else
            k_scan_short<TA, T, V, GROUPED, kSteps, BACK><<<grid, 256, 0, s>>>(a, waves);
        return;
    }
    const int64_t units = (a.p.chunk ? a.p.slots : a.n_seq) * a.p.blocks;
    auto go = [&](auto waves, auto chain) {
        constexpr int W = decltype(waves)::value;
        constexpr bool CHAIN = decltype(chain)::value;
        const int64_t blocks = W == 1 ? (units + 3) / 4 : units;
        const unsigned grid = (unsigned)(blocks < kScanGrid ? blocks : kScanGrid), threads = W == 1 ? 256 : 64 * W;
        if constexpr (V > 1) {
            if (a.p.stream) {
                k_scan<TA, T, V, GROUPED, W, kSteps, BACK, true, CHAIN><<<grid, threads, 0, s>>>(a, units);
                return;
            }
        }
        k_scan<TA, T, V, GROUPED, W, kSteps, BACK, false, CHAIN><<<grid, threads, 0, s>>>(a, units);
    };
    if (a.p.chunk) {
        launch_scan_reset(a, s);
        go(integral_constant<int, kScanChainWaves>{}, std::true_type{});
    } else if (a.p.waves == 1) {
        go(integral_constant<int, 1>{}, std::false_type{});
    } else if (a.p.waves == 4) {
        go(integral_constant<int, 4>{}, std::false_type{});
    } else {
        go(integral_constant<int, 8>{}, std::false_type{});
    }
}

template <class TA, class T, bool BACK>
void pick_scan(const ScanArgs& a, hipStream_t s) {
    constexpr int V = 4;
    if (a.p.grouped) {
        if (a.p.vec)
            run_scan<TA, T, V, true, BACK>(a, s);
        else
            run_scan<TA, T, 1, true, BACK>(a, s);
    } else {
        if (a.p.vec)
            run_scan<TA, T, V, false, BACK>(a, s);
        else
            run_scan<TA, T, 1, false, BACK>(a, s);
    }
}

}  // namespace

}  // namespace nerf
