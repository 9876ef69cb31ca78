// encoder_dev.h -- device helpers shared by the embedding head's kernels:
// vectors of 8 values of any type at any element alignment, reductions over
// 16 and 64 lanes, and the rule for values held in 8 bits.
#pragma once

#include <hip/hip_runtime.h>

#include "encoder.h"

namespace maxsim {
namespace {

constexpr int kVec = 8;  // values a lane handles at a time; 16 lanes make one block of 128

struct F16 {
    typedef _Float16 type;
};
struct BF16 {
    typedef __bf16 type;
};
struct F32 {
    typedef float type;
};

// 8 values, aligned as one of them: the hardware loads and stores 16 bytes at
// any 2-byte address, so odd pitches and offsets need no path of their own.
template <typename T>
struct Pack8 {
    typedef T V __attribute__((ext_vector_type(8), aligned(sizeof(T))));
};

__device__ __forceinline__ uint32_t fbits(float v) { return __float_as_uint(v); }

// 8 values of a row from column c on; zeros at and past width n.
template <typename T>
__device__ __forceinline__ typename Pack8<T>::V load8(const T* row, int c, int n) {
    typename Pack8<T>::V v;
    if (c + kVec <= n) {
        v = *reinterpret_cast<const typename Pack8<T>::V*>(row + c);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = c + i < n ? row[c + i] : (T)0.f;
    }
    return v;
}
// The same in two parts, for many loads at once: near() reads 8 values without a
// branch (the row's last 8 where c is past them), so that all of a row's loads are
// on their way together; fit() then moves a last vector that does not fit down
// into place.  (With the branch in the load, rows of 769 took 40 % longer.)
// TOGETHER false: near() is the whole load (threads that hold long rows have no
// registers for them all).
template <typename T, bool TOGETHER = true>
__device__ __forceinline__ typename Pack8<T>::V near8(const T* row, int c, int n) {
    if (!TOGETHER || n < kVec) return load8<T>(row, c, n);  // the same for the whole launch
    return *reinterpret_cast<const typename Pack8<T>::V*>(row + min(c, n - kVec));
}
template <typename T, bool TOGETHER = true>
__device__ __forceinline__ void fit8(typename Pack8<T>::V& v, int c, int n) {
    if (!TOGETHER || c + kVec <= n || n < kVec) return;
    const int down = min(c + kVec - n, (int)kVec);  // 1 to 7; all of them past the end
#pragma unroll
    for (int step = kVec; step > 0; step >>= 1) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = (down & step) ? (i + step < kVec ? v[i + step] : (T)0.f) : v[i];
    }
}

// 8 values to a row from column c on, those before width n.
template <typename T>
__device__ __forceinline__ void put8(T* row, int c, int n, const typename Pack8<T>::V& v) {
    if (c + kVec <= n) {
        *reinterpret_cast<typename Pack8<T>::V*>(row + c) = v;
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (c + i < n) row[c + i] = v[i];
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* row, int c, int n, const float* f) {
    typename Pack8<T>::V v;
#pragma unroll
    for (int i = 0; i < kVec; ++i) v[i] = (T)f[i];
    put8<T>(row, c, n, v);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef Pack8<uint8_t>::V u8x8;

__device__ __forceinline__ void store8_bytes(uint8_t* row, int c, int n, u32x2 bytes) {
    put8<uint8_t>(row, c, n, __builtin_bit_cast(u8x8, bytes));
}

// Maxima of magnitudes as integers: the order of non-negative floats is that of
// their bits, and an infinity or NaN (largest of all) is never lost.
__device__ __forceinline__ uint32_t mag(float v) { return fbits(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}

// Every lane gets the maximum / sum over its row of 16 lanes: neighbours, pairs
// (quad_perm), then the two halves and the whole mirrored.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = umax(v, dpp<0xB1>(v));
    v = umax(v, dpp<0x4E>(v));
    v = umax(v, dpp<0x141>(v));
    return umax(v, dpp<0x140>(v));
}
__device__ __forceinline__ float sum16(float v) {
    v += __uint_as_float(dpp<0xB1>(fbits(v)));
    v += __uint_as_float(dpp<0x4E>(fbits(v)));
    v += __uint_as_float(dpp<0x141>(fbits(v)));
    return v + __uint_as_float(dpp<0x140>(fbits(v)));
}
// The same over all 64 lanes.
__device__ __forceinline__ uint32_t max64(uint32_t v) {
    v = max16(v);
    auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = umax(r[0], r[1]);
    r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return umax(r[0], r[1]);
}
__device__ __forceinline__ float sum64(float v) {
    v = sum16(v);
    auto r = __builtin_amdgcn_permlane16_swap(fbits(v), fbits(v), false, false);
    v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
    r = __builtin_amdgcn_permlane32_swap(fbits(v), fbits(v), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// The scale of a block whose largest magnitude has the bits `top`, and what
// multiplies and corrects its values.
struct Scale {
    float s;     // as stored
    float inv;   // 1 / s to a unit in the last place
    bool zeros;  // the block is held as zeros (too small, or not finite)
};
// v / s in 3 operations (a division has ten), given inv = 1 / s to a unit in the
// last place: the product is within 3 units, and the correction by its remainder leaves
// the nearest value or, in about 1 of 10^7 pairs, its neighbour (the remainder of a product 3
// units off need not fit 24 bits).  For s = 127 with inv rounded to nearest all 2^23 mantissas
// of v give the nearest.
__device__ __forceinline__ float quotient(float v, float s, float inv) {
    const float q = v * inv;
    return __builtin_fmaf(__builtin_fmaf(-q, s, v), inv, q);
}
// e4m3's scale is one multiplication by the fp32 value next to 1 / 448, which is
// what torch's division of a tensor by a constant does on the device.  Divided,
// more than half of the scales were the neighbouring fp32 value, which moved the codes
// of values next to a tie (63,505 of 67 M in bf16 rows): a step of up to 1 / 8 in
// a code each, where a unit in the scale's last place is nothing by itself.
__device__ __forceinline__ Scale block_scale(uint32_t top, float largest) {
    Scale r;
    const bool tiny = top < 0x0D800000u;    // 2^-100
    const bool broken = top >= 0x7F800000u;  // infinity or NaN
    const float v = __uint_as_float(top);
    r.s = tiny ? 1.f : largest == 448.f ? v * (1.f / 448.f) : quotient(v, largest, 1.f / largest);
    if (broken) r.s = __uint_as_float(0x7FC00000u);
    r.inv = __builtin_amdgcn_rcpf(r.s);
    r.zeros = tiny || broken;
    return r;
}
__device__ __forceinline__ float scaled(float v, const Scale& k) { return quotient(v, k.s, k.inv); }
// 8 values in e4m3 (the conversion rounds to nearest even; |v / s| is at most
// 448 and a rounding error, which rounds to 448).
__device__ __forceinline__ u32x2 to_e4m3(const float* v, const Scale& k) {
    u32x2 out;
    int lo = 0, hi = 0;
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(scaled(v[0], k), scaled(v[1], k), lo, false);
    lo = __builtin_amdgcn_cvt_pk_fp8_f32(scaled(v[2], k), scaled(v[3], k), lo, true);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(scaled(v[4], k), scaled(v[5], k), hi, false);
    hi = __builtin_amdgcn_cvt_pk_fp8_f32(scaled(v[6], k), scaled(v[7], k), hi, true);
    out[0] = k.zeros ? 0u : (uint32_t)lo;
    out[1] = k.zeros ? 0u : (uint32_t)hi;
    return out;
}
// 8 values in int8 (|v / s| is at most 127 and a rounding error).
__device__ __forceinline__ u32x2 to_i8(const float* v, const Scale& k) {
    u32x2 out = {0u, 0u};
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        const int q = (int)__builtin_rintf(scaled(v[i], k)) & 255;
        out[i >> 2] |= (uint32_t)q << (8 * (i & 3));
    }
    if (k.zeros) out = u32x2{0u, 0u};
    return out;
}

}  // namespace
}  // namespace maxsim
