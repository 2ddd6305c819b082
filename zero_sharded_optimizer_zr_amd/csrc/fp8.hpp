// Helpers shared by the 8-bit floating-point operators (gfx950): 16-bit
// elements, e4m3 / e5m2 codes and E8M0 scales.
#pragma once

#include "zr_device.hpp"
#include "zr_fp8.h"
#include "zr_math.hpp"

namespace zr {

constexpr int kGroup = ZR_FP8_GROUP;  // elements that share a scale
constexpr int kVec = 8;               // 16-bit elements of one 16-byte access

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
// a vector that may start at any element, of two bytes or one
typedef uint32_t any_u32x4 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t any_u32x2 __attribute__((ext_vector_type(2), aligned(1)));

// The two element types, two elements to a word.  bf16 and fp16 widen exactly;
// narrowing rounds to nearest even (one hardware instruction per pair).
struct BF16 {
    static __device__ __forceinline__ float lo(uint32_t w) { return bf16_lo(w); }
    static __device__ __forceinline__ float hi(uint32_t w) { return bf16_hi(w); }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        typedef __bf16 pair __attribute__((ext_vector_type(2)));
        const pair p = {(__bf16)lo, (__bf16)hi};
        return __builtin_bit_cast(uint32_t, p);
    }
};

struct F16 {
    typedef _Float16 pair __attribute__((ext_vector_type(2)));
    static __device__ __forceinline__ float lo(uint32_t w) { return (float)__builtin_bit_cast(pair, w)[0]; }
    static __device__ __forceinline__ float hi(uint32_t w) { return (float)__builtin_bit_cast(pair, w)[1]; }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const pair p = {(_Float16)lo, (_Float16)hi};
        return __builtin_bit_cast(uint32_t, p);
    }
};

template <typename T>
__device__ __forceinline__ float widen(uint16_t x)
{
    return T::lo(x);
}

template <typename T>
__device__ __forceinline__ uint16_t narrow(float x)
{
    return (uint16_t)T::pack(x, 0.0f);
}

// Eight elements at p as four words; elements `n` and later are 0.  A whole vector is
// one access, wherever it starts: the hardware takes 16 bytes at any address, and rows of
// an odd length need no path of their own (2961 x 402 normed in 6 us, with single
// elements where rows do not start on 16 bytes 18; 16384 x 4095 in 167, 477; 2413 x 1915
// quantized both ways in 18, 26).  kStream, here and below: the access carries the
// non-temporal hint (the builtins themselves: load_stream and store_stream would take the
// vectors' full alignment for granted).
template <bool kStream = false>
__device__ __forceinline__ u32x4 load8(const uint16_t *p, int64_t n)
{
    if (n >= kVec)
        return kStream ? __builtin_nontemporal_load((global_ptr<const any_u32x4>)p) : *(global_ptr<const any_u32x4>)p;
    u32x4 w = {0, 0, 0, 0};
#pragma unroll
    for (int e = 0; e < kVec; ++e)
        if (e < n)
            w[e / 2] |= (uint32_t)load_global(p + e) << (16 * (e % 2));
    return w;
}

template <bool kStream = false>
__device__ __forceinline__ void store8(uint16_t *p, u32x4 w, int64_t n)
{
    if (n >= kVec) {
        if (kStream)
            __builtin_nontemporal_store((any_u32x4)w, (global_ptr<any_u32x4>)p);
        else
            *(global_ptr<any_u32x4>)p = w;
        return;
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e)
        if (e < n)
            *(global_ptr<uint16_t>)(p + e) = (uint16_t)(w[e / 2] >> (16 * (e % 2)));
}

// Eight codes at p, the first n of them.
template <bool kStream = true>
__device__ __forceinline__ void store_codes8(uint8_t *p, u32x2 w, int64_t n)
{
    if (n >= kVec) {
        if (kStream)
            __builtin_nontemporal_store((any_u32x2)w, (global_ptr<any_u32x2>)p);
        else
            *(global_ptr<any_u32x2>)p = w;
        return;
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e)
        if (e < n)
            *(global_ptr<uint8_t>)(p + e) = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
}

// Exponent of a format's largest value, 1.75 * 2^8 (e4m3) or 1.75 * 2^15 (e5m2).
template <int kFormat>
constexpr uint32_t kTopExponent = kFormat == ZR_E4M3 ? 8 : 15;

// E8M0 byte of a group whose largest magnitude has the fp32 pattern `amax`:
// with amax = m * 2^x, 1 <= m < 2, the smallest e with amax <= 1.75 * 2^top * 2^e is
// x - top, plus one where m > 1.75; a byte below 0 is held at 0 (subnormal
// amax included: its exponent field 0 stands for less than it says).
template <int kFormat>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax)
{
    const int32_t s = (int32_t)(amax >> 23) - (int32_t)kTopExponent<kFormat> + ((amax & 0x7fffffu) > 0x600000u);
    return amax >= 0x7f800000u ? 255u : s < 0 ? 0u : (uint32_t)s;
}

// 2^-(s - 127): the factor that turns elements into codes' values, exact for
// every s a finite group can have (0 ... 247).
__device__ __forceinline__ float inverse_scale(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// Codes of four products x * inv, rounded to nearest even; 0x7f for all when the
// group's scale byte is 255.  No value exceeds the format's range (the scale was
// chosen so), so the conversion's saturation never acts.
template <int kFormat>
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, float inv, uint32_t s)
{
    int w;
    if constexpr (kFormat == ZR_E4M3) {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(a * inv, b * inv, 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c * inv, d * inv, w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(a * inv, b * inv, 0, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c * inv, d * inv, w, true);
    }
    return s == 255u ? 0x7f7f7f7fu : (uint32_t)w;
}

template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_move(uint32_t a)
{
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, kCtrl, 0xf, 0xf, false);
}

// Every lane of each row of 16 lanes gets f over the row: swap neighbours, swap
// pairs, mirror halves of 8, mirror the row.
template <typename F>
__device__ __forceinline__ uint32_t row16_all(uint32_t a, F f)
{
    a = f(a, dpp_move<0xb1>(a));   // quad_perm [1, 0, 3, 2]
    a = f(a, dpp_move<0x4e>(a));   // quad_perm [2, 3, 0, 1]
    a = f(a, dpp_move<0x141>(a));  // row_half_mirror
    a = f(a, dpp_move<0x140>(a));  // row_mirror
    return a;
}

__device__ __forceinline__ uint32_t max_u32(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Maximum over a group held by a row of 16 lanes.
__device__ __forceinline__ uint32_t group_max(uint32_t a) { return row16_all(a, max_u32); }

// Sum over the wave, the same bits in every lane and on every call.
__device__ __forceinline__ float wave_sum(float a)
{
    const auto add = [](uint32_t x, uint32_t y) {
        return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
    };
    a = __uint_as_float(row16_all(__float_as_uint(a), add));
    a += __shfl_xor(a, 16, 64);
    a += __shfl_xor(a, 32, 64);
    return a;
}

// Per 16-bit lane maxima of magnitudes: the patterns of non-negative bf16 and
// fp16 values order as unsigned integers, NaN and infinity on top.
__device__ __forceinline__ uint32_t abs2(uint32_t w) { return w & 0x7fff7fffu; }
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b)
{
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a),
                                                                  __builtin_bit_cast(u16x2, b)));
}

// Byte offset of group g (of kb) of a row of codes that starts at byte `row`, for a load
// through a buffer descriptor; kNowhere, which is past the end of every buffer, for
// groups behind the row and for lanes whose row is kNowhere.
constexpr uint32_t kNowhere = 0xffffffffu;
__host__ __device__ __forceinline__ uint32_t group_of_row(uint32_t row, int32_t g, int32_t kb)
{
    return row != kNowhere && g < kb ? row + (uint32_t)g * kGroup : kNowhere;
}

// Host side: *bytes = address range of a matrix of `size`-byte elements, from its
// first to its last element (rows, cols > 0).  False if ld < cols or the range
// does not fit int64.
inline bool matrix_extent(int64_t rows, int64_t cols, int64_t ld, int64_t size, int64_t *bytes)
{
    int64_t n;
    return ld >= cols && !__builtin_mul_overflow(rows - 1, ld, &n) && !__builtin_add_overflow(n, cols, &n) &&
           !__builtin_mul_overflow(n, size, bytes);
}

}  // namespace zr
