// Distillation from a teacher's K largest logits for gfx950.  Per row, with
// z = s / T the student's scaled logits and t_j the teacher's logit of class
// i_j:
//   p_j = softmax_j(t / T) over the row's entries,  q = softmax(z) over all classes
//   loss = T^2 sum_j p_j (ln p_j - ln q_{i_j}),     ln q_v = z_v - lse,  lse = ln sum_v e^{z_v}
//   d loss / d s_v = T (P q_v - sum_{j: i_j = v} p_j),   P = sum_j p_j
// P is 1, or 0 for a row without entries (loss and gradient 0).  The student's
// logits are read once for the running maximum and sum of e^(z - max), and
// once more for the gradient; both are bound by memory.  An exponential is
// 2^((s - m) c), c = log2(e) / T: subtracting the maximum before scaling keeps
// the exponent's error relative to s - m, however large the logits are.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>

#include "common.hpp"
#include "experts.hpp"
#include "rowio.hpp"

namespace nerf {

namespace {

constexpr float kLog2e = 1.44269504088896341f;

// Running maximum m of logits and sum s of 2^((x - m) c).  m is -inf as long as
// only -inf was seen, and then s is 0; a NaN (or +inf) logit makes s NaN.
struct MaxSum {
    float m, s;
};

// 1 / T and log2(e) / T, kept finite for the T (below 2^-127) that have none: a
// difference of logits above 2^-120 is then still past the range of an exponential.
__device__ __forceinline__ float over_t(float x, float temperature) { return fminf(x / temperature, FLT_MAX); }

// What to subtract for the maximum m: with m = -inf every logit is -inf (or NaN)
// and 2^((x - 0) c) is 0 (or NaN), as it has to be.
__device__ __forceinline__ float shift_of(float m) { return m == -INFINITY ? 0.0f : m; }
__device__ __forceinline__ float exp2_below(float x, float shift, float c) {
    return __builtin_amdgcn_exp2f((x - shift) * c);
}

__device__ __forceinline__ MaxSum join(const MaxSum& a, const MaxSum& b, float c) {
    MaxSum r;
    r.m = fmaxf(a.m, b.m);
    // a part that saw nothing, or only NaN, has m = -inf and keeps its sum
    const float fa = a.m == r.m || a.m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((a.m - r.m) * c);
    const float fb = b.m == r.m || b.m == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f((b.m - r.m) * c);
    r.s = a.s * fa + b.s * fb;
    return r;
}

template <int NT>
__device__ __forceinline__ MaxSum block_join(MaxSum v, float c, MaxSum* scratch) {  // scratch: [NT / 64]
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const MaxSum o{__shfl_xor(v.m, off, 64), __shfl_xor(v.s, off, 64)};
        v = join(v, o, c);
    }
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = v;
        __syncthreads();
        v = scratch[0];
#pragma unroll 4
        for (int w = 1; w < NT / 64; ++w) v = join(v, scratch[w], c);
        __syncthreads();
    }
    return v;
}

template <class T>
__device__ __forceinline__ void add_piece(MaxSum& a, const typename RowIO<T>::Vec& v, int n, float c) {
    float z[RowIO<T>::PER], m = -INFINITY;
#pragma unroll
    for (int i = 0; i < RowIO<T>::PER; ++i) {
        z[i] = i < n ? RowIO<T>::get(v, i) : -INFINITY;
        m = fmaxf(m, z[i]);
    }
    if (m > a.m) {
        if (a.m != -INFINITY) a.s *= __builtin_amdgcn_exp2f((a.m - m) * c);
        a.m = m;
    }
    const float shift = shift_of(a.m);
#pragma unroll
    for (int i = 0; i < RowIO<T>::PER; ++i) a.s += exp2_below(z[i], shift, c);
}

// Maximum and sum of classes [c0, c1) of a row, by NT threads.
template <class T, int NT>
__device__ __forceinline__ MaxSum scan_row(const T* row, int64_t c0, int64_t c1, float c, MaxSum* scratch) {
    constexpr int PER = RowIO<T>::PER;
    MaxSum a{-INFINITY, 0.0f};
    int64_t v = c0 + (int64_t)threadIdx.x * PER;
    for (; v + 3 * NT * PER + PER <= c1; v += 4 * NT * PER) {  // four loads in flight
        typename RowIO<T>::Vec x[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x[u] = RowIO<T>::load(row, v + (int64_t)u * NT * PER, c1);
#pragma unroll
        for (int u = 0; u < 4; ++u) add_piece<T>(a, x[u], PER, c);
    }
    for (; v < c1; v += NT * PER) {
        const int64_t left = c1 - v;
        add_piece<T>(a, RowIO<T>::load(row, v, c1), left < PER ? (int)left : PER, c);
    }
    return block_join<NT>(a, c, scratch);
}

// ---------------------------------------------------------------------------
// The teacher's side of a row, by the first wave of a workgroup (lane l holds
// entries l, l + 64, ...).  Entries whose class is outside [0, classes) do not
// exist; a row whose entries are all missing or -inf has p = 0.
// ---------------------------------------------------------------------------
constexpr int kTopPerLane = kDistillMaxTop / 64;

struct Teacher {
    int id[kTopPerLane];   // -1: no entry
    float p[kTopPerLane];
    float logp[kTopPerLane];
    float total;           // P
};

__device__ __forceinline__ Teacher teacher_row(const DistillArgs& a, int64_t row, int lane) {
    Teacher t;
    float z[kTopPerLane], m = -INFINITY, nan = 0.0f;
    const float inv_t = over_t(1.0f, a.temperature);
#pragma unroll
    for (int u = 0; u < kTopPerLane; ++u) {
        const int j = lane + 64 * u;
        t.id[u] = j < a.top ? a.t_ids[row * a.top + j] : -1;
        if ((unsigned)t.id[u] >= (uint64_t)a.classes) t.id[u] = -1;
        z[u] = t.id[u] >= 0 ? a.t_logits[row * a.top + j] : -INFINITY;
        m = fmaxf(m, z[u]);
        if (z[u] != z[u]) nan = z[u];
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off, 64));
    float s = nan;
#pragma unroll
    for (int u = 0; u < kTopPerLane; ++u) {
        z[u] = (z[u] - m) * inv_t;
        t.p[u] = m == -INFINITY ? 0.0f : expf(z[u]);
        s += t.p[u];
    }
    s = wave_sum(s);
    const float ls = logf(s);
#pragma unroll
    for (int u = 0; u < kTopPerLane; ++u) {
        t.logp[u] = z[u] - ls;
        if (s != s)
            t.p[u] = t.id[u] >= 0 ? s : 0.0f;
        else
            t.p[u] = s > 0.0f ? t.p[u] / s : 0.0f;
    }
    t.total = s != s ? s : s > 0.0f ? 1.0f : 0.0f;
    return t;
}

// Loss of a row from its maximum and sum, by one wave.  With ln q_v = (s_v - m) / T - ln sum,
//   loss = T sum_j p_j (T (ln p_j + ln sum) - (s_{i_j} - m)),
// which stays accurate however large the logits are, and in range where (s - m) / T
// or T^2 is not (a class of the type's lowest value, a temperature far from one).
template <class T>
__device__ __forceinline__ float row_loss(const DistillArgs& a, const Teacher& t, const T* row, const MaxSum& v) {
    float sum = 0.0f;
    const float log_s = logf(v.s);
#pragma unroll
    for (int u = 0; u < kTopPerLane; ++u)
        if (t.id[u] >= 0 && t.p[u] != 0.0f) {
            const float below = v.m == -INFINITY ? (v.s == 0.0f ? INFINITY : v.s)  // (no student, or NaN)
                                                 : a.temperature * (t.logp[u] + log_s) - ((float)row[t.id[u]] - v.m);
            sum += t.p[u] * below;
        }
    return a.temperature * wave_sum(sum);
}

// The gradient at the teacher's classes: after the sweep over the row has
// stored scale P q there, the entries' owners store scale (P q - p), with the
// masses of entries of one class added up.  Classes outside [c0, c1) belong to
// another workgroup.
struct TopLds {
    int id[kDistillMaxTop];
    float p[kDistillMaxTop];
    float total;
};

template <class T, int NT>
__device__ __forceinline__ void patch_top(const DistillArgs& a, const TopLds& t, const T* row, T* grad, int64_t c0,
                                          int64_t c1, float c, float shift, float inv, float scale) {
    for (int j = threadIdx.x; j < a.top; j += NT) {
        const int id = t.id[j];
        if (id < 0 || id < c0 || id >= c1) continue;
        float p = 0.0f;
        for (int i = 0; i < a.top; ++i) p += t.id[i] == id ? t.p[i] : 0.0f;
        const float q = exp2_below((float)row[id], shift, c) * inv;
        grad[id] = (T)(scale * (t.total * q - p));
    }
}

template <class T, int NT>
__device__ __forceinline__ void write_grad(const DistillArgs& a, const TopLds& t, const T* row, T* grad, int64_t c0,
                                           int64_t c1, float c, float shift, float inv, float scale) {
    constexpr int PER = RowIO<T>::PER;
    const float f = scale * t.total * inv;
    const int64_t v0 = c0 + (int64_t)threadIdx.x * PER;
    // a row without entries has gradient 0 whatever its logits
    if (__builtin_amdgcn_readfirstlane(t.total == 0.0f)) {
        for (int64_t v = v0; v < c1; v += NT * PER) RowIO<T>::stream(grad, v, c1, RowIO<T>::zero());
        return;
    }
    auto piece = [&](int64_t v, const typename RowIO<T>::Vec& x) {
        float g[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) g[i] = f * exp2_below(RowIO<T>::get(x, i), shift, c);
        RowIO<T>::stream(grad, v, c1, RowIO<T>::pack(g));  // (the row's logits stay in the cache for this sweep)
    };
    int64_t v = v0;
    for (; v + NT * PER + PER <= c1; v += 2 * NT * PER) {  // two loads in flight
        const typename RowIO<T>::Vec x0 = RowIO<T>::load(row, v, c1), x1 = RowIO<T>::load(row, v + NT * PER, c1);
        piece(v, x0);
        piece(v + NT * PER, x1);
    }
    for (; v < c1; v += NT * PER) piece(v, RowIO<T>::load(row, v, c1));
    __syncthreads();
    patch_top<T, NT>(a, t, row, grad, c0, c1, c, shift, inv, scale);
}

template <class T>
__device__ __forceinline__ void keep_top(TopLds& l, const Teacher& t, int top, int lane) {
#pragma unroll
    for (int u = 0; u < kTopPerLane; ++u)
        if (lane + 64 * u < top) {
            l.id[lane + 64 * u] = t.id[u];
            l.p[lane + 64 * u] = t.p[u];
        }
    if (lane == 0) l.total = t.total;
}

__device__ __forceinline__ float natural_lse(const MaxSum& v, float temperature) {
    return v.m == -INFINITY ? (v.s == 0.0f ? -INFINITY : v.s) : v.m / temperature + logf(v.s);
}

// ---------------------------------------------------------------------------
// One workgroup per row: loss, and the gradient if asked for.  Bound by memory:
// the second sweep finds in the caches what the first has read (the gradient is
// stored nontemporally for that: 4096 x 128000 bfloat16 with 1024 threads 521 us
// with ordinary stores, 471 without), which leaves one read and one write, 2.1
// GB at 4.45 TB/s; a copy of that size moves 4.9.  Keeping the row in registers
// between the sweeps spilled (582 us and more).
// ---------------------------------------------------------------------------
template <class T, int NT>
__global__ void __launch_bounds__(NT) k_distill_rows(DistillArgs a) {
    __shared__ MaxSum scratch[NT / 64];
    __shared__ TopLds top;
    const int64_t r = blockIdx.x;
    const T* row = (const T*)a.logits + r * a.ld;
    const float c = over_t(kLog2e, a.temperature);
    const int lane = threadIdx.x & 63;
    const MaxSum v = scan_row<T, NT>(row, 0, a.classes, c, scratch);
    if (threadIdx.x < 64) {
        const Teacher t = teacher_row(a, r, lane);
        const float lse = natural_lse(v, a.temperature), loss = row_loss<T>(a, t, row, v);
        if (lane == 0) {
            a.loss[r] = loss;
            if (a.lse) a.lse[r] = lse;
        }
        keep_top<T>(top, t, a.top, lane);
    }
    if (!a.grad) return;
    __syncthreads();
    const float scale = a.temperature * (a.row_scale ? a.row_scale[r] : 1.0f);
    write_grad<T, NT>(a, top, row, (T*)a.grad + r * a.ld_grad, 0, a.classes, c, shift_of(v.m),
                      v.s == 0.0f ? 0.0f : 1.0f / v.s, scale);
}

// ---------------------------------------------------------------------------
// Few rows: the classes of a row are split over `splits` workgroups, whose
// maxima and sums are joined by whoever needs them, in the same order.  Two
// launches; the loss of one row of 50,001 float32 takes 11.5 us a call, all of
// it launches and the chain of dependent steps (200 KB are read).
// ---------------------------------------------------------------------------
constexpr int kSplitThreads = 256;

__device__ __forceinline__ void split_range(int64_t classes, int splits, int i, int64_t& c0, int64_t& c1) {
    // whole 16-byte pieces of bfloat16, the widest piece in elements
    const int64_t per = ((classes + splits - 1) / splits + 7) & ~(int64_t)7;
    c0 = per * i < classes ? per * i : classes;
    c1 = c0 + per < classes ? c0 + per : classes;
}

template <class T>
__global__ void __launch_bounds__(kSplitThreads) k_distill_part(DistillArgs a, int splits) {
    __shared__ MaxSum scratch[kSplitThreads / 64];
    const int64_t r = blockIdx.x / splits;
    const int i = blockIdx.x % splits;
    int64_t c0, c1;
    split_range(a.classes, splits, i, c0, c1);
    const MaxSum v = scan_row<T, kSplitThreads>((const T*)a.logits + r * a.ld, c0, c1, over_t(kLog2e, a.temperature),
                                                scratch);
    if (threadIdx.x == 0) {
        a.part[2 * (r * splits + i)] = v.m;
        a.part[2 * (r * splits + i) + 1] = v.s;
    }
}

__device__ __forceinline__ MaxSum joined_parts(const DistillArgs& a, int64_t r, int splits, int lane) {
    MaxSum v{-INFINITY, 0.0f};
    for (int i = lane; i < splits; i += 64) {
        const MaxSum o{a.part[2 * (r * splits + i)], a.part[2 * (r * splits + i) + 1]};
        v = join(v, o, over_t(kLog2e, a.temperature));
    }
    return block_join<64>(v, over_t(kLog2e, a.temperature), nullptr);
}

// grid: [n][max(gsplits, 1)]; the first workgroup of a row writes its loss.
template <class T>
__global__ void __launch_bounds__(kSplitThreads) k_distill_join(DistillArgs a, int splits, int gsplits) {
    __shared__ TopLds top;
    __shared__ MaxSum all;
    const int64_t r = blockIdx.x / gsplits;
    const int i = blockIdx.x % gsplits, lane = threadIdx.x & 63;
    const T* row = (const T*)a.logits + r * a.ld;
    if (threadIdx.x < 64) {
        const MaxSum v = joined_parts(a, r, splits, lane);
        const Teacher t = teacher_row(a, r, lane);
        if (i == 0) {
            const float lse = natural_lse(v, a.temperature), loss = row_loss<T>(a, t, row, v);
            if (lane == 0) {
                a.loss[r] = loss;
                if (a.lse) a.lse[r] = lse;
            }
        }
        if (lane == 0) all = v;
        keep_top<T>(top, t, a.top, lane);
    }
    if (!a.grad) return;
    __syncthreads();
    int64_t c0, c1;
    split_range(a.classes, gsplits, i, c0, c1);
    const float scale = a.temperature * (a.row_scale ? a.row_scale[r] : 1.0f);
    write_grad<T, kSplitThreads>(a, top, row, (T*)a.grad + r * a.ld_grad, c0, c1, over_t(kLog2e, a.temperature),
                                 shift_of(all.m), all.s == 0.0f ? 0.0f : 1.0f / all.s, scale);
}

// Gradient from a saved log-sum-exp: q = e^(z - lse).  Rounding lse, one float32
// of the size of the largest z, and its product with T is a relative error of up
// to |lse| 2^-23 of q: 2^-17 for the |lse| < 64 of logits a softmax is meant for.
// A row beyond (shifted, or all masked with the type's lowest value, where ln of
// the sum is lost beside the maximum, or lse not finite) is done whole by one of
// its workgroups (in turn, so that all XCDs have some), which finds the maximum
// and the sum again: the same error as with the loss, for one more read of the row
// (8192 x 4096 bfloat16: 41 us if all rows are such, 28 if none; 4096 x 128000:
// 1027 and 394).
constexpr float kLseLargest = 64.0f;

template <class T>
__global__ void __launch_bounds__(kSplitThreads) k_distill_grad(DistillArgs a, int gsplits) {
    __shared__ MaxSum scratch[kSplitThreads / 64];
    __shared__ TopLds top;
    const int64_t r = blockIdx.x / gsplits;
    const int i = blockIdx.x % gsplits, lane = threadIdx.x & 63;
    const T* row = (const T*)a.logits + r * a.ld;
    const float c = over_t(kLog2e, a.temperature), lse = a.lse[r];
    if (threadIdx.x < 64) keep_top<T>(top, teacher_row(a, r, lane), a.top, lane);
    int64_t c0, c1;
    split_range(a.classes, gsplits, i, c0, c1);
    __syncthreads();
    float m = lse * a.temperature, inv = 1.0f;
    if (!(fabsf(lse) < kLseLargest && fabsf(m) < INFINITY)) {  // (the same for all of a row's workgroups)
        if (i != r % gsplits) return;
        c0 = 0;
        c1 = a.classes;
        const MaxSum v = scan_row<T, kSplitThreads>(row, 0, c1, c, scratch);
        m = v.m;
        inv = v.s == 0.0f ? 0.0f : 1.0f / v.s;
    }
    const float scale = a.temperature * (a.row_scale ? a.row_scale[r] : 1.0f);
    write_grad<T, kSplitThreads>(a, top, row, (T*)a.grad + r * a.ld_grad, c0, c1, c, shift_of(m), inv, scale);
}

// Workgroups per row of a gradient sweep: ranges of 16384 classes (64 x 128000
// bfloat16: 9.7 us, 14.2 with ranges of 65536; 4096 x 128000: 388, 404; ranges of
// 4096: 9.8 and 391).  Bound by memory: 5.4 TB/s.
int grad_splits(int64_t classes) { return (int)((classes + 16383) / 16384); }

// Rows r0 .. r0 + n - 1 of a call.
template <class T>
DistillArgs rows_from(DistillArgs a, int64_t r0, int64_t n) {
    a.logits = (const T*)a.logits + r0 * a.ld;
    a.n = n;
    a.t_logits += r0 * a.top;
    a.t_ids += r0 * a.top;
    if (a.row_scale) a.row_scale += r0;
    if (a.loss) a.loss += r0;
    if (a.lse) a.lse += r0;
    if (a.grad) a.grad = (T*)a.grad + r0 * a.ld_grad;
    return a;
}

// A launch for as many rows of `items` work items each as it holds.
template <class T, class F>
void by_launches(const DistillArgs& a, int64_t items, F&& launch) {
    const int64_t most = kMaxWorkItems / items;
    for (int64_t r = 0; r < a.n; r += most) launch(rows_from<T>(a, r, a.n - r < most ? a.n - r : most));
}

template <class T, int NT>
void run_rows(const DistillArgs& all, hipStream_t s) {
    by_launches<T>(all, NT, [&](const DistillArgs& a) { k_distill_rows<T, NT><<<(unsigned)a.n, NT, 0, s>>>(a); });
}

// Threads by the length of a row, so that the rows in flight on the card stay
// few enough to be cached between the sweeps, and short ones keep no idle waves.
// Loss and gradient of bfloat16 rows, us:
//   16384 x 1024: 28 with 64 threads, 55 with 256;  8192 x 4096: 36 and 41;
//   8192 x 8000: 78 and 72;  8192 x 32000: 244 with 256 threads, 283 with 1024;
//   2048 x 65536: 139 and 127;  4096 x 128000: 600 and 465.
template <class T>
void run_distill(const DistillArgs& a, hipStream_t s) {
    const int splits = distill_splits(a.n, a.classes);
    if (splits > 1) {  // (fewer than 256 rows, and about 1024 workgroups)
        k_distill_part<T><<<(unsigned)(a.n * splits), kSplitThreads, 0, s>>>(a, splits);
        const int gs = a.grad ? splits : 1;
        k_distill_join<T><<<(unsigned)(a.n * gs), kSplitThreads, 0, s>>>(a, splits, gs);
    } else if (a.classes <= 4096) {
        run_rows<T, 64>(a, s);
    } else if (a.classes * sizeof(T) <= 65536) {
        run_rows<T, 256>(a, s);
    } else {
        run_rows<T, 1024>(a, s);
    }
}

template <class T>
void run_grad(const DistillArgs& all, hipStream_t s) {
    const int gs = grad_splits(all.classes);
    by_launches<T>(all, (int64_t)gs * kSplitThreads, [&](const DistillArgs& a) {
        k_distill_grad<T><<<(unsigned)(a.n * gs), kSplitThreads, 0, s>>>(a, gs);
    });
}

}  // namespace

// Rows are split when there are fewer than CUs, into parts of at least 2048 classes
// and about 1024 workgroups (512 of them: the same).  Loss and gradient, bfloat16,
// us: 64 x 128000: 16.6 split, 23.4 not; 128 x 262144: 39 and 43; 200 x 50000: 18.3
// and 17.0 (with nearly as many rows as CUs a split loses a little); 700 x 8000:
// 16.4 and 12.2; 1000 x 128000: 138 and 126.
int distill_splits(int64_t n, int64_t classes) {
    if (n >= 256 || classes <= 4096) return 1;
    const int64_t most = classes / 2048, want = (1024 + n - 1) / n;
    return (int)(want < most ? want : most);
}

void launch_distill(bool bf16, const DistillArgs& a, hipStream_t s) {
    if (bf16)
        run_distill<__bf16>(a, s);
    else
        run_distill<float>(a, s);
}

void launch_distill_grad(bool bf16, const DistillArgs& a, hipStream_t s) {
    if (bf16)
        run_grad<__bf16>(a, s);
    else
        run_grad<float>(a, s);
}

}  // namespace nerf
