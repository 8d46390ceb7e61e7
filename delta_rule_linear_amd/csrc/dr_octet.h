// dr_octet.h -- eight consecutive channels of a row, as the elementwise kernels
// load, convert and store them.
//
// A lane has eight channels.  Rows start anywhere (any width, stride or slice), so
// the accesses are 16 bytes wide at the alignment of one element, which global
// memory takes; no kernel needs a slower form for odd widths.  Where the width is
// no multiple of 8 the last lane's window is moved back to the row's last eight
// channels: it computes some of its neighbour's channels again, and stores its
// own alone.  Rows of fewer than eight channels (SMALL) are read one channel at a
// time, the last one repeated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dr {

template <bool F32>
struct Oct {
    unsigned w[F32 ? 8 : 4];
};

typedef unsigned oct_u32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned oct_u16x8 __attribute__((ext_vector_type(4), aligned(2)));   // eight 16-bit values
typedef float oct_f32x4 __attribute__((ext_vector_type(4), aligned(4)));
typedef unsigned oct_u8x8 __attribute__((ext_vector_type(2), aligned(1)));    // eight 8-bit values

// Where a lane's eight channels are: it reads [at, at + 8) of a row and owns the
// last `own` of them (0: a lane behind the row, which reads what is there).
struct OctPlace {
    int at, own;
};
__device__ __forceinline__ OctPlace oct_place(int group, int C) {
    const int left = C - 8 * group;
    return {left >= 8 ? 8 * group : C > 8 ? C - 8 : 0, left >= 8 ? 8 : left > 0 ? left : 0};
}

// The channel that value e of a lane's window is.
template <bool SMALL>
__device__ __forceinline__ int oct_channel(int group, int e, int C) {
    return SMALL ? min(e, C - 1) : oct_place(group, C).at + e;
}

// row: the row's first channel.  SMALL converts to fp32 at once, of either type
// (one kernel serves all types); the others take F32's.  ONCE: bf16 values are
// not read again soon, and leave the caches to others (fp32's 32 bytes a lane are two
// accesses to the same line, which then comes twice).
template <bool F32, bool SMALL, bool ONCE = false>
__device__ __forceinline__ void oct_load(const void* row, bool f32, int at, int C, Oct<F32>& r) {
    if constexpr (SMALL) {
        static_assert(F32, "small rows are held in fp32");
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = min(e, C - 1);
            r.w[e] = f32 ? static_cast<const unsigned*>(row)[c]
                         : (unsigned)static_cast<const unsigned short*>(row)[c] << 16;
        }
    } else if constexpr (F32) {
        const oct_u32x4* p = reinterpret_cast<const oct_u32x4*>(static_cast<const float*>(row) + at);
        const oct_u32x4 a = p[0], b = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r.w[i] = a[i];
            r.w[4 + i] = b[i];
        }
    } else {
        const oct_u16x8* p = reinterpret_cast<const oct_u16x8*>(static_cast<const uint16_t*>(row) + at);
        const oct_u16x8 a = ONCE ? __builtin_nontemporal_load(p) : *p;
#pragma unroll
        for (int i = 0; i < 4; ++i) r.w[i] = a[i];
    }
}

// Forgets what the compiler knows of the values, so that what was made of them is made
// again instead of kept in registers.
template <bool F32>
__device__ __forceinline__ void oct_forget(Oct<F32>& r) {
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) asm volatile("" : "+v"(r.w[i]));
}

template <bool F32>
__device__ __forceinline__ float oct_value(const Oct<F32>& r, int e) {
    if constexpr (F32) return __uint_as_float(r.w[e]);
    else return __uint_as_float(e % 2 ? r.w[e / 2] & 0xffff0000u : r.w[e / 2] << 16);
}

// Whether channel e of the window is the lane's own.
template <bool SMALL>
__device__ __forceinline__ bool oct_own(const OctPlace& p, int e) {
    return SMALL ? e < p.own : e >= 8 - p.own;
}

template <bool SMALL>
__device__ __forceinline__ void oct_store(void* row, bool f32, const OctPlace& p, const float (&x)[8]) {
    typedef float f4 __attribute__((ext_vector_type(4)));
    typedef float f8 __attribute__((ext_vector_type(8)));
    typedef __bf16 b8 __attribute__((ext_vector_type(8)));
    typedef __bf16 b8u __attribute__((ext_vector_type(8), aligned(2)));
    const bool whole = !SMALL && p.own == 8;
    if (f32) {
        float* to = static_cast<float*>(row) + p.at;
        if (whole) {
            reinterpret_cast<oct_f32x4*>(to)[0] = f4{x[0], x[1], x[2], x[3]};
            reinterpret_cast<oct_f32x4*>(to)[1] = f4{x[4], x[5], x[6], x[7]};
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (oct_own<SMALL>(p, e)) to[e] = x[e];
        }
    } else {
        const b8 y = __builtin_convertvector((f8{x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]}), b8);
        __bf16* to = static_cast<__bf16*>(row) + p.at;
        if (whole) {
            *reinterpret_cast<b8u*>(to) = y;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (oct_own<SMALL>(p, e)) to[e] = y[e];
        }
    }
}

}  // namespace dr
