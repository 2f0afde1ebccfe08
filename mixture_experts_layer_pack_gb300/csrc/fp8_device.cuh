// Device-side pieces of the dense layers in 8-bit floating point.
#pragma once

#include "device_common.cuh"

namespace moe {

// Scale of a block whose largest magnitude is `most`: E4M3's largest value, 448, stands for it; at least the smallest
// normal fp32, so that its reciprocal is finite (a block of zeros has zero codes then). A NaN is not seen by the maximum and
// becomes the NaN code, in its own place; an infinity makes the scale infinite and with it the whole block NaN.
__device__ __forceinline__ float block_scale(float most) { return fmaxf(__fdiv_rn(most, 448.0f), 0x1p-126f); }

// min(g, L) and clip(u, -L, L) that keep a NaN
__device__ __forceinline__ float clamp_top(float g, float limit) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(g), "f"(limit));
    return r;
}
__device__ __forceinline__ float clamp_both(float u, float limit) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(clamp_top(u, limit)), "f"(-limit));
    return r;
}

// two fp32 numbers in a register pair, and the operations on them of one instruction
__device__ __forceinline__ uint64_t pair(uint32_t a, uint32_t b) {
    uint64_t p;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "r"(a), "r"(b));
    return p;
}
__device__ __forceinline__ uint64_t pair(float a, float b) { return pair(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ void unpair(uint64_t p, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(p)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t p;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
    return p;
}
__device__ __forceinline__ uint64_t mad2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t p;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(c));
    return p;
}

// out[at] = x, or out[at] + x; bf16: both the addend and the sum are rounded, as the layer's main_grads
__device__ __forceinline__ void store_one(void* out, int64_t at, bool bf16, bool add, float x) {
    if (bf16) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(out) + at;
        const __nv_bfloat16 w = __float2bfloat16(x);
        *dst = add ? __float2bfloat16(__bfloat162float(*dst) + __bfloat162float(w)) : w;
    } else {
        float* dst = static_cast<float*>(out) + at;
        *dst = add ? *dst + x : x;
    }
}

}  // namespace moe
