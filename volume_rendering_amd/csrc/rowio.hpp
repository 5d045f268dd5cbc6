// 16-byte pieces of rows of float32 or bfloat16 elements at any element
// alignment.  Global memory takes 16-byte accesses at any address here, so
// rows of odd widths or strides use the same wide accesses; only a row's last,
// partial piece goes element by element.
#pragma once

#include "common.hpp"

namespace nerf {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_loose __attribute__((ext_vector_type(4), aligned(2)));

template <class T>
struct RowIO {
    static constexpr int PER = 16 / (int)sizeof(T);  // elements of a piece
    union Vec {
        u32x4 u;
        T e[PER];
    };
    struct __attribute__((packed, aligned(sizeof(T)))) Loose {
        u32x4 u;
    };
    static __device__ __forceinline__ Vec zero() {
        Vec v;
        v.u = u32x4{0u, 0u, 0u, 0u};
        return v;
    }
    // A whole piece from p on.
    static __device__ __forceinline__ Vec load_whole(const T* p) {
        Vec v;
        v.u = reinterpret_cast<const Loose*>(p)->u;
        return v;
    }
    // Elements c .. c + PER - 1 of a row of `width` (those past it: zero).
    static __device__ __forceinline__ Vec load(const T* row, int64_t c, int64_t width) {
        Vec v = zero();
        if (c + PER <= width)
            v.u = reinterpret_cast<const Loose*>(row + c)->u;
        else
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (c + i < width) v.e[i] = row[c + i];
        return v;
    }
    static __device__ __forceinline__ void store(T* row, int64_t c, int64_t width, const Vec& v) {
        if (c + PER <= width)
            reinterpret_cast<Loose*>(row + c)->u = v.u;
        else
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (c + i < width) row[c + i] = v.e[i];
    }
    // A store that is not to be read again soon: it leaves the caches to data
    // that is (nontemporal).
    static __device__ __forceinline__ void stream(T* row, int64_t c, int64_t width, const Vec& v) {
        if (c + PER <= width)
            __builtin_nontemporal_store(v.u, reinterpret_cast<u32x4_loose*>(row + c));
        else
            store(row, c, width, v);
    }
    static __device__ __forceinline__ float get(const Vec& v, int i) { return (float)v.e[i]; }
    static __device__ __forceinline__ Vec pack(const float (&f)[PER]) {
        Vec v;
#pragma unroll
        for (int i = 0; i < PER; ++i) v.e[i] = (T)f[i];  // bfloat16: nearest even
        return v;
    }
};

}  // namespace nerf
