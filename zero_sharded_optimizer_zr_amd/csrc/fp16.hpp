// fp16 elements and the loss-scale record, shared by the kernels that take fp16
// gradients (gfx950).
#pragma once

#include "zr_math.hpp"

namespace zr {

__device__ __forceinline__ float f16_to_f32(uint32_t h16)
{
    return (float)__builtin_bit_cast(_Float16, (uint16_t)h16);
}
__device__ __forceinline__ float f16_lo(uint32_t w) { return f16_to_f32(w & 0xffffu); }
__device__ __forceinline__ float f16_hi(uint32_t w) { return f16_to_f32(w >> 16); }

// fp32 -> fp16 bits, round to nearest even (hardware), NaN -> sign | 0x7e00.
__device__ __forceinline__ uint32_t f32_to_f16(float f)
{
    uint32_t h = __builtin_bit_cast(uint16_t, (_Float16)f);
    return (f != f) ? (((__float_as_uint(f) >> 16) & 0x8000u) | 0x7e00u) : h;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) { return f32_to_f16(lo) | (f32_to_f16(hi) << 16); }

inline zr_status check_ls(const char *who, const void *ls)
{
    if (!ls)
        return fail(ZR_EINVAL, "%s: loss-scale record is NULL", who);
    if (!aligned_to(ls, 4))
        return fail(ZR_EALIGN, "%s: loss-scale record must be 4-byte aligned", who);
    return ZR_OK;
}

}  // namespace zr
