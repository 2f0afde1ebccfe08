// Device-side pieces of the dense layers in 8-bit floating point.
#pragma once

#include "device_common.cuh"

#include <type_traits>

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

// Results and what they are added to. In bf16 both the addend and the sum are rounded, as the layer's main_grads.
template <typename Y>
using Two = std::conditional_t<sizeof(Y) == 2, uint32_t, float2>;  // two adjacent ones, the first on the pair's alignment
__device__ __forceinline__ float load_one(const float* p) { return *p; }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float2 load_two(const float* p) { return *reinterpret_cast<const float2*>(p); }
__device__ __forceinline__ uint32_t load_two(const __nv_bfloat16* p) { return *reinterpret_cast<const uint32_t*>(p); }
__device__ __forceinline__ float2 load_first(const float* p) { return make_float2(*p, 0.0f); }
__device__ __forceinline__ uint32_t load_first(const __nv_bfloat16* p) { return __bfloat16_as_ushort(*p); }
__device__ __forceinline__ float first_of(float2 x) { return x.x; }
__device__ __forceinline__ float first_of(uint32_t x) { return __uint_as_float(x << 16); }
template <bool ADD>  // *p = x, or old + x
__device__ __forceinline__ void save_one(float* p, float x, float old) { *p = ADD ? old + x : x; }
template <bool ADD>
__device__ __forceinline__ void save_one(__nv_bfloat16* p, float x, float old) {
    const __nv_bfloat16 w = __float2bfloat16(x);
    *p = ADD ? __float2bfloat16(old + __bfloat162float(w)) : w;
}
template <bool ADD>
__device__ __forceinline__ void save_two(float* p, float x, float y, float2 old) {
    *reinterpret_cast<float2*>(p) = ADD ? make_float2(old.x + x, old.y + y) : make_float2(x, y);
}
template <bool ADD>
__device__ __forceinline__ void save_two(__nv_bfloat16* p, float x, float y, uint32_t old) {
    uint32_t w = pack_bf16x2(x, y);
    if (ADD) {
        float a, b, c, d;
        unpack_bf16x2(old, a, b), unpack_bf16x2(w, c, d);
        w = pack_bf16x2(a + c, b + d);
    }
    *reinterpret_cast<uint32_t*>(p) = w;
}
__device__ __forceinline__ void store_one(void* out, int64_t at, bool bf16, bool add, float x) {
    auto put = [&](auto* p) {
        if (add)
            save_one<true>(p, x, load_one(p));
        else
            save_one<false>(p, x, 0.0f);
    };
    if (bf16)
        put(static_cast<__nv_bfloat16*>(out) + at);
    else
        put(static_cast<float*>(out) + at);
}

}  // namespace moe
