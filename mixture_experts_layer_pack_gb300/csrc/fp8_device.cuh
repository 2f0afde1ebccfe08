// Device-side pieces of the dense layers in 8-bit floating point.
#pragma once

#include "device_common.cuh"

namespace moe {

// Scale of a block whose largest magnitude is `most`: E4M3's largest value, 448, stands for it; at least the smallest
// normal fp32, so that its reciprocal is finite (a block of zeros has zero codes then). A NaN is not seen by the maximum and
// becomes the NaN code, in its own place; an infinity makes the scale infinite and with it the whole block NaN.
__device__ __forceinline__ float block_scale(float most) { return fmaxf(__fdiv_rn(most, 448.0f), 0x1p-126f); }

// min(g, L) and clip(u, -L, L) that keep a NaN
__device__ __forceinline__ float clamp_top(float g, float limit) { return g > limit ? limit : g; }
__device__ __forceinline__ float clamp_both(float u, float limit) { return u > limit ? limit : (u < -limit ? -limit : u); }

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
