// Dense layers in 8-bit floating point with one fp32 scale for a block of 128: the codes, the pieces between the
// products (fp8_gemm.cu), and the calls.
#include "fp8.h"
#include "fp8_device.cuh"
#include "internal.h"

#include <cuda_fp16.h>

#include <cmath>

namespace moe {

namespace {

constexpr int64_t kMostRows = int64_t(1) << 24, kMostCols = int64_t(1) << 20;
constexpr int kQuantThreads = 256;
constexpr int kGatedThreads = 512;

struct Codes {          // codes and compact scales; q null: not wanted
    uint8_t* q;
    int64_t ld;
    float* s;
};

// ---------------------------------------------------------------- reading and writing eight columns
// Bytes [o, o + 16) of the 32 of a and b, 0 <= o < 16
__device__ __forceinline__ uint4 bytes_from(uint4 a, uint4 b, int o) {
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (o & 8)
#pragma unroll
        for (int j = 0; j < 6; ++j) w[j] = w[j + 2];
    if (o & 4)
#pragma unroll
        for (int j = 0; j < 5; ++j) w[j] = w[j + 1];
    const int s = 8 * (o & 3);
    return make_uint4(__funnelshift_r(w[0], w[1], s), __funnelshift_r(w[1], w[2], s), __funnelshift_r(w[2], w[3], s), __funnelshift_r(w[3], w[4], s));
}

// 16 bytes at any address of which `bytes` (1 to 16) are the row's, the others as zeros: from the one or two aligned words that hold them
__device__ __forceinline__ uint4 load16(const void* p, int bytes) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const int o = int(at & 15);
    const uint4* src = reinterpret_cast<const uint4*>(at - o);
    const uint4 a = __ldg(src), b = o + bytes > 16 ? __ldg(src + 1) : make_uint4(0, 0, 0, 0);
    const uint4 v = bytes_from(a, b, o);
    auto own = [&](uint32_t w, int from) { return bytes >= from + 4 ? w : bytes <= from ? 0u : w & ((1u << 8 * (bytes - from)) - 1); };
    return make_uint4(own(v.x, 0), own(v.y, 4), own(v.z, 8), own(v.w, 12));
}

// Eight elements of a row as they were read, and the largest magnitudes of such: of bf16 two to a register, which the maximum
// keeps (a NaN is not taken)
template <typename X>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
    __nv_bfloat162 w[4];
    __device__ __forceinline__ void load(const __nv_bfloat16* p, int n, bool wide) {
        if (wide && n >= 8) {
            *reinterpret_cast<uint4*>(w) = __ldg(reinterpret_cast<const uint4*>(p));
        } else if (n > 0) {
            *reinterpret_cast<uint4*>(w) = load16(p, 2 * min(n, 8));
        } else {
            zero();
        }
    }
    __device__ __forceinline__ void zero() { *reinterpret_cast<uint4*>(w) = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void most(Eight& m) const {  // m: magnitudes
#pragma unroll
        for (int j = 0; j < 4; ++j) m.w[j] = __hmax2(m.w[j], __habs2(w[j]));
    }
    __device__ __forceinline__ float most() const {
        const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(w[0]), __habs2(w[1])), __hmax2(__habs2(w[2]), __habs2(w[3])));
        const float a = __low2float(m), b = __high2float(m);
        return fmaxf(fmaxf(a, b), 0.0f);  // two NaN are no maximum
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = __bfloat1622float2(w[j]);
            v[2 * j] = f.x, v[2 * j + 1] = f.y;
        }
    }
};
template <>
struct Eight<float> {
    float w[8];
    __device__ __forceinline__ void load(const float* p, int n, bool wide) {
        if (wide && n >= 8) {
            *reinterpret_cast<float4*>(w) = __ldg(reinterpret_cast<const float4*>(p));
            *reinterpret_cast<float4*>(w + 4) = __ldg(reinterpret_cast<const float4*>(p) + 1);
        } else if (n > 0) {
            *reinterpret_cast<uint4*>(w) = load16(p, 4 * min(n, 4));
            *reinterpret_cast<uint4*>(w + 4) = n > 4 ? load16(p + 4, 4 * min(n - 4, 4)) : make_uint4(0, 0, 0, 0);
        } else {
            zero();
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = 0.0f;
    }
    __device__ __forceinline__ void most(Eight& m) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) m.w[j] = fmaxf(m.w[j], fabsf(w[j]));
    }
    __device__ __forceinline__ float most() const {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(w[j]));
        return m;
    }
    __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = w[j];
    }
};

// eight codes of a row (8-byte aligned); its bytes past n are not ours
__device__ __forceinline__ void store8(uint8_t* p, int n, uint32_t lo, uint32_t hi) {
    if (n >= 8) {
        *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (j < n) p[j] = uint8_t((j < 4 ? lo : hi) >> (8 * (j & 3)));
    }
}

__device__ __forceinline__ void put8(uint8_t* p, int n, const float (&v)[8], const float (&r)[8]) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) unpair(mul2(pair(v[j], v[j + 1]), pair(r[j], r[j + 1])), q[j], q[j + 1]);
    store8(p, n, e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7]));
}
__device__ __forceinline__ void put8(uint8_t* p, int n, const float (&v)[8], float r) {
    const float r8[8] = {r, r, r, r, r, r, r, r};
    put8(p, n, v, r8);
}
__device__ __forceinline__ float most_of16(float m) {  // over the 16 lanes that share a row
#pragma unroll
    for (int d = 1; d < 16; d *= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    return m;
}

// Of N rows' (N = 4, 8) maxima over the 16 lanes that share them each lane gets one: that of row lane_row<N>(lane). Half of the rows go to the
// other half of the lanes at every step, so that the sum of the exchanges is N and not 4 N.
template <int N>
__device__ __forceinline__ float spread_max(float (&m)[N]) {
    const int lane = threadIdx.x & 15;
    int d = 8;
#pragma unroll
    for (int n = N / 2; n >= 1; n /= 2, d /= 2) {
        const bool high = lane & d;
#pragma unroll
        for (int j = 0; j < n; ++j) {
            const float other = __shfl_xor_sync(0xffffffffu, high ? m[j] : m[j + n], d);
            m[j] = fmaxf(high ? m[j + n] : m[j], other);
        }
    }
    for (; d >= 1; d /= 2) m[0] = fmaxf(m[0], __shfl_xor_sync(0xffffffffu, m[0], d));
    return m[0];
}
template <int N>  // the row of a lane, and the first lane that has a row (of 16)
__device__ __forceinline__ int lane_row(int lane) { return N == 8 ? lane >> 1 & 7 : lane >> 2 & 3; }
template <int N>
__device__ __forceinline__ int row_lane(int row) { return N == 8 ? row << 1 : row << 2; }

// ---------------------------------------------------------------- codes of a matrix
// A block takes 128 x 128 elements, which it reads once and holds in registers: 16 threads a row with eight columns
// each, a thread eight rows 16 apart. Rows' maxima go through 16 lanes, columns' through registers and shared memory.
// Memory bounds it once enough blocks share an SM: bf16 is held as it was read, two to a register (64 registers a thread instead
// of 116, 36 bytes of them spilled), and each scale's division is one lane's.
template <typename X>
__global__ void __launch_bounds__(kQuantThreads, sizeof(X) == 2 ? 4 : 2)
    fp8_quantize_kernel(const X* __restrict__ x, int64_t rows, int cols, int64_t ld, bool wide, Codes row, Codes col, Codes square) {
    constexpr int W = kQuantThreads / 32;
    __shared__ float part[W][128];
    __shared__ float scale[128], inv[128];
    pdl_wait();
    pdl_trigger();
    const int col_blocks = (cols + 127) >> 7;
    const int64_t rb = blockIdx.x / col_blocks;
    const int cb = int(blockIdx.x - rb * col_blocks);
    const int c8 = threadIdx.x & 15, rg = threadIdx.x >> 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = cb * 128 + c8 * 8, n = cols - c0;  // n columns of this thread's (8 or more: all)
    const int left = int(min(rows - rb * 128, int64_t(128)));
    Eight<X> e[8];
    const X* src = x + (rb * 128 + rg) * ld + c0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (rg + 16 * i < left && n > 0)
            e[i].load(src + 16 * i * ld, n, wide);
        else
            e[i].zero();
    }
    if (row.q) {
        float m[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = e[i].most();
        const float s = block_scale(spread_max(m)), r = __frcp_rn(s);
        const int mine = rg + 16 * lane_row<8>(c8);
        if ((c8 & 1) == 0 && mine < left) row.s[cb * rows + rb * 128 + mine] = s;
        uint8_t* dst = row.q + (rb * 128 + rg) * row.ld + c0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[8];
            e[i].values(v);
            const float ri = __shfl_sync(0xffffffffu, r, row_lane<8>(i), 16);
            if (rg + 16 * i < left && n > 0) put8(dst + 16 * i * row.ld, n, v, ri);
        }
    }
    if (!col.q && !square.q) return;
    Eight<X> most;
    most.zero();
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i].most(most);
    float m[8];
    most.values(m);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
        if (lane < 16) part[warp][c8 * 8 + j] = m[j];
    }
    __syncthreads();
    if (threadIdx.x < 128) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) t = fmaxf(t, part[w][threadIdx.x]);
        const float s = block_scale(t);
        scale[threadIdx.x] = s;
        inv[threadIdx.x] = __frcp_rn(s);
        if (col.q && cb * 128 + int(threadIdx.x) < cols) col.s[rb * cols + cb * 128 + threadIdx.x] = s;
    }
    __syncthreads();
    if (col.q) {
        float r8[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) r8[j] = inv[c8 * 8 + j];
        uint8_t* dst = col.q + (rb * 128 + rg) * col.ld + c0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[8];
            e[i].values(v);
            if (rg + 16 * i < left && n > 0) put8(dst + 16 * i * col.ld, n, v, r8);
        }
    }
    if (square.q) {
        float s = scale[lane];  // the columns' scales grow with their maxima
#pragma unroll
        for (int z = 1; z < 4; ++z) s = fmaxf(s, scale[lane + 32 * z]);
#pragma unroll
        for (int d = 1; d < 32; d *= 2) s = fmaxf(s, __shfl_xor_sync(0xffffffffu, s, d));
        if (threadIdx.x == 0) square.s[rb * col_blocks + cb] = s;
        const float rs = __frcp_rn(s);
        uint8_t* dst = square.q + (rb * 128 + rg) * square.ld + c0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v[8];
            e[i].values(v);
            if (rg + 16 * i < left && n > 0) put8(dst + 16 * i * square.ld, n, v, rs);
        }
    }
}

// ---------------------------------------------------------------- values of codes
__device__ __forceinline__ uint2 codes8(const uint8_t* p, int n) {
    if (n >= 8) return __ldg(reinterpret_cast<const uint2*>(p));
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (j < n) w[j >> 2] |= uint32_t(p[j]) << (8 * (j & 3));
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void values8(uint2 w, float (&v)[8]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t((j < 2 ? w.x : w.y) >> (16 * (j & 1))), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        v[2 * j] = f.x, v[2 * j + 1] = f.y;
    }
}

// Eight results of each of the 16 lanes of a row, n of this one's to be written (a lane that has less than eight is the last).
// Rows that do not start on 16 bytes are written in aligned words all the same: a lane's first word has the end of the lane before
// it; only what is before the row's first whole word and behind its last goes element by element. All 16 lanes call it.
template <typename Y>
__device__ __forceinline__ void store_row(Y* to, int n, int c8, const uint4* x) {
    constexpr int WORDS = sizeof(Y) / 2, PER = 16 / sizeof(Y);  // 16-byte words of eight results, results of a word
    const int o = int(reinterpret_cast<uintptr_t>(to) & 15);
    uint4 before;
    before.x = __shfl_up_sync(0xffffffffu, x[WORDS - 1].x, 1, 16), before.y = __shfl_up_sync(0xffffffffu, x[WORDS - 1].y, 1, 16);
    before.z = __shfl_up_sync(0xffffffffu, x[WORDS - 1].z, 1, 16), before.w = __shfl_up_sync(0xffffffffu, x[WORDS - 1].w, 1, 16);
    auto each = [&](int from, int end) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint4& w = x[j / PER];
            const uint32_t* half = &w.x;
            const uint32_t v = half[(j % PER) * sizeof(Y) / 4];
            if (j >= from && j < end) {
                if constexpr (sizeof(Y) == 2)
                    reinterpret_cast<unsigned short*>(to)[j] = static_cast<unsigned short>(j & 1 ? v >> 16 : v);
                else
                    reinterpret_cast<uint32_t*>(to)[j] = v;
            }
        }
    };
    if (n < 8) {
        each(0, n);
    } else if (o == 0) {
#pragma unroll
        for (int z = 0; z < WORDS; ++z) reinterpret_cast<uint4*>(to)[z] = x[z];
    } else {
        uint4* at = reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(to) - o);
        const int head = (16 - o) / int(sizeof(Y));  // results before the first whole word
        if (c8 == 0)
            each(0, head);
        else
            at[0] = bytes_from(before, x[0], 16 - o);
#pragma unroll
        for (int z = 1; z < WORDS; ++z) at[z] = bytes_from(x[z - 1], x[z], 16 - o);
        if (c8 == 15 || n < 16) each(8 - PER + head, 8);
    }
}

template <typename Y>
__global__ void __launch_bounds__(kQuantThreads) fp8_dequantize_kernel(const uint8_t* __restrict__ q, int64_t ldq, const float* __restrict__ s,
                                                                       int block, int64_t rows, int cols, Y* __restrict__ out, int64_t ld) {
    pdl_wait();
    pdl_trigger();
    const int col_blocks = (cols + 127) >> 7;
    const int64_t rb = blockIdx.x / col_blocks;
    const int cb = int(blockIdx.x - rb * col_blocks);
    const int c8 = threadIdx.x & 15, rg = threadIdx.x >> 4;
    const int c0 = cb * 128 + c8 * 8, n = cols - c0;
    const int left = int(min(rows - rb * 128, int64_t(128)));
    uint2 w[8];
    float rs[8], s8[8];
    const uint8_t* src = q + (rb * 128 + rg) * ldq + c0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const bool in = rg + 16 * i < left && n > 0;
        w[i] = in ? codes8(src + 16 * i * ldq, n) : make_uint2(0, 0);
        rs[i] = block == MOE_B_ROW && in ? __ldg(s + cb * rows + rb * 128 + rg + 16 * i) : 1.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        s8[j] = block == MOE_B_SQUARE ? __ldg(s + rb * col_blocks + cb) : block == MOE_B_COL && j < n ? __ldg(s + rb * cols + c0 + j) : 1.0f;
    Y* dst = out + (rb * 128 + rg) * ld + c0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float v[8];
        values8(w[i], v);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] *= block == MOE_B_ROW ? rs[i] : s8[j];
        Y* to = dst + 16 * i * ld;
        if constexpr (sizeof(Y) == 2) {
            const uint4 x = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
            store_row(to, rg + 16 * i < left ? n : 0, c8, &x);
        } else {
            const uint4 x[2] = {make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])),
                                make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]))};
            store_row(to, rg + 16 * i < left ? n : 0, c8, x);
        }
    }
}

// ---------------------------------------------------------------- the gate's backward pass
struct GatedBack {
    const float* dh;  // [T, I], row stride ld_dh
    int64_t ld_dh;
    Codes g, u;       // kept, row blocks
    Codes dg_row, du_row, dg_col, du_col, h_col;
    int64_t T;
    int I;
    float limit;
};

// dg, du and h of eight columns of a row, two columns an instruction
template <bool CLAMP>
__device__ __forceinline__ void gated_back8(const float (&dh)[8], const float (&gq)[8], float sg, const float (&uq)[8], float su,
                                            float limit, float (&dg)[8], float (&du)[8], float (&h)[8]) {
    const uint64_t sg2 = pair(sg, sg), su2 = pair(su, su), one = pair(1.0f, 1.0f), minus = pair(-1.0f, -1.0f);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const uint64_t g2 = mul2(pair(gq[j], gq[j + 1]), sg2), u2 = mul2(pair(uq[j], uq[j + 1]), su2), dh2 = pair(dh[j], dh[j + 1]);
        float g[2], u[2], gc[2], uc[2];
        unpair(g2, g[0], g[1]), unpair(u2, u[0], u[1]);
#pragma unroll
        for (int z = 0; z < 2; ++z) gc[z] = CLAMP ? clamp_top(g[z], limit) : g[z], uc[z] = CLAMP ? clamp_both(u[z], limit) : u[z];
        const uint64_t gc2 = pair(gc[0], gc[1]), uc2 = pair(uc[0], uc[1]);
        const uint64_t sig = pair(sigmoidf_(gc[0]), sigmoidf_(gc[1])), silu = mul2(gc2, sig);
        const uint64_t slope = mul2(sig, mad2(gc2, mad2(sig, minus, one), one));
        unpair(mul2(silu, uc2), h[j], h[j + 1]);
        unpair(mul2(mul2(dh2, uc2), slope), dg[j], dg[j + 1]);
        unpair(mul2(dh2, silu), du[j], du[j + 1]);
        if constexpr (CLAMP) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                dg[j + z] = g[z] > limit ? 0.0f : dg[j + z];
                du[j + z] = fabsf(u[z]) > limit ? 0.0f : du[j + z];
            }
        }
    }
}

// dh and the kept g, u -> dg and du as row blocks (for dx) and column blocks, h as column blocks (for the weights' gradients).
// 128 tokens x 128 columns a block. The results are computed twice, for the maxima and for the codes, from inputs that are
// read twice, the second time from L2: held in registers, they or the results leave room for one block an SM, whose reads,
// arithmetic and writes then wait for one another (8192 x 8192: 335 us). Two blocks an SM leave 64 registers a thread, of which 88 bytes are spilled (108
// with a clamp). Its instructions bound it: at 8192 x 8192 one column each 250 us and with
// a clamp 288; two columns each, and the clamp compiled apart, 216 and 272.
template <bool CLAMP>
__global__ void __launch_bounds__(kGatedThreads, 2) fp8_gated_back_kernel(const GatedBack a) {
    constexpr int W = kGatedThreads / 32, R = 128 * 16 / kGatedThreads, S = 128 / R;
    __shared__ float part[3][W][128];
    __shared__ float inv[3][128];
    pdl_wait();
    pdl_trigger();
    const int col_blocks = (a.I + 127) >> 7;
    const int64_t rb = blockIdx.x / col_blocks;
    const int cb = int(blockIdx.x - rb * col_blocks);
    const int c8 = threadIdx.x & 15, rg = threadIdx.x >> 4, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = cb * 128 + c8 * 8, n = a.I - c0;
    const int left = n > 0 ? int(min(a.T - rb * 128, int64_t(128))) : 0;  // rows of the block, for this thread
    const int64_t row0 = rb * 128 + rg;
    // dg, du, h of this thread's eight columns of its i-th row
    auto results = [&](int i, float (&dg)[8], float (&du)[8], float (&h)[8]) {
        const int64_t r = min(row0 + S * i, a.T - 1);  // a row past the last is read as that one, so that the rows' reads have no branch between them
        Eight<float> dh;
        dh.load(a.dh + r * a.ld_dh + c0, n, true);
        const uint2 gq = codes8(a.g.q + r * a.g.ld + c0, n), uq = codes8(a.u.q + r * a.u.ld + c0, n);
        const float sg = __ldg(a.g.s + cb * a.T + r), su = __ldg(a.u.s + cb * a.T + r);
        float g[8], u[8];
        values8(gq, g), values8(uq, u);
        gated_back8<CLAMP>(dh.w, g, sg, u, su, a.limit, dg, du, h);
    };
    float mg[R], mu[R], mc[3][8] = {};
#pragma unroll
    for (int i = 0; i < R; ++i) {
        float dg[8], du[8], h[8];
        results(i, dg, du, h);  // of a row past the last: the last one's, which change no maximum of a column
        mg[i] = mu[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            mg[i] = fmaxf(mg[i], fabsf(dg[j]));
            mu[i] = fmaxf(mu[i], fabsf(du[j]));
            mc[0][j] = fmaxf(mc[0][j], fabsf(dg[j]));
            mc[1][j] = fmaxf(mc[1][j], fabsf(du[j]));
            mc[2][j] = fmaxf(mc[2][j], fabsf(h[j]));
        }
    }
    const float s0 = block_scale(spread_max(mg)), s1 = block_scale(spread_max(mu));
    const float r0 = __frcp_rn(s0), r1 = __frcp_rn(s1);
    if (a.dg_row.q && (c8 & 3) == 0) {
        const int64_t mine = rb * 128 + rg + S * lane_row<R>(c8);
        if (mine < a.T) a.dg_row.s[cb * a.T + mine] = s0, a.du_row.s[cb * a.T + mine] = s1;
    }
#pragma unroll
    for (int z = 0; z < 3; ++z)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float m = fmaxf(mc[z][j], __shfl_xor_sync(0xffffffffu, mc[z][j], 16));
            if (lane < 16) part[z][warp][c8 * 8 + j] = m;
        }
    __syncthreads();
    if (threadIdx.x < 384) {
        const int z = threadIdx.x >> 7, c = threadIdx.x & 127;
        float m = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) m = fmaxf(m, part[z][w][c]);
        const float s = block_scale(m);
        inv[z][c] = __frcp_rn(s);
        float* to = z == 0 ? a.dg_col.s : z == 1 ? a.du_col.s : a.h_col.s;
        if (to && cb * 128 + c < a.I) to[rb * a.I + cb * 128 + c] = s;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < R; ++i) {
        const float q0 = __shfl_sync(0xffffffffu, r0, row_lane<R>(i), 16), q1 = __shfl_sync(0xffffffffu, r1, row_lane<R>(i), 16);
        const int64_t r = row0 + S * i;
        float dg[8], du[8], h[8];
        results(i, dg, du, h);
        if (rg + S * i >= left) continue;
        if (a.dg_row.q) {
            put8(a.dg_row.q + r * a.dg_row.ld + c0, n, dg, q0);
            put8(a.du_row.q + r * a.du_row.ld + c0, n, du, q1);
        }
        if (a.dg_col.q) {
            auto cols = [&](int z, const Codes& c, const float (&v)[8]) {
                float r8[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) r8[j] = inv[z][c8 * 8 + j];
                put8(c.q + r * c.ld + c0, n, v, r8);
            };
            cols(0, a.dg_col, dg), cols(1, a.du_col, du), cols(2, a.h_col, h);
        }
    }
}

// ---------------------------------------------------------------- the gate over partial sums
// h = silu(g) u from the partial sums of g and u, as row blocks, and g and u themselves where they are kept: 16 threads a block of 128
__global__ void __launch_bounds__(256) fp8_gated_sum_kernel(const __grid_constant__ F8Args a) {
    pdl_wait();
    pdl_trigger();
    const F8Out& o = a.o[0];
    const int64_t unit = int64_t(blockIdx.x) * 16 + (threadIdx.x >> 4);
    const int64_t row = min(unit / o.n_tiles, int64_t(o.M) - 1);
    const int block = int(unit % o.n_tiles), c8 = threadIdx.x & 15, c0 = block * 128 + c8 * 8, n = o.N - c0;
    const bool mine = unit < int64_t(o.M) * o.n_tiles;
    float v[2][8] = {};
    const int64_t plane = int64_t(o.M) * o.ld_partial;
    const float* src = o.partial + row * o.ld_partial + c0;
#pragma unroll 2
    for (int s = 0; s < a.splits; ++s) {  // the rows of the partial sums have room for whole blocks
        Eight<float> g, u;
        g.load(src + 2 * s * plane, 8, true);
        u.load(src + (2 * s + 1) * plane, 8, true);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[0][j] += g.w[j], v[1][j] += u.w[j];
    }
    auto put = [&](const float (&x)[8], uint8_t* q, int64_t ld, float* scales) {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[j]));
        const float s = block_scale(most_of16(m));
        if (!mine) return;
        if (c8 == 0) scales[int64_t(block) * o.M + row] = s;
        if (n > 0) put8(q + row * ld + c0, n, x, __frcp_rn(s));
    };
    if (a.g) put(v[0], a.g, a.ld_g, a.gs), put(v[1], a.u, a.ld_u, a.us);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        float g = v[0][j], u = v[1][j];
        if (a.limit > 0.0f) g = clamp_top(g, a.limit), u = clamp_both(u, a.limit);
        v[0][j] = g * sigmoidf_(g) * u;
    }
    put(v[0], a.h, a.ld_h, a.hs);
}

// ---------------------------------------------------------------- launches
int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t blocks(int64_t n) { return (n + 127) / 128; }

bool aligned(const void* p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool rows_on(const void* p, int64_t stride, size_t elem, size_t bytes) {
    return ((reinterpret_cast<uintptr_t>(p) | (size_t(stride) * elem)) & (bytes - 1)) == 0;
}
size_t size_of(int32_t type) { return type == MOE_T_BF16 ? 2 : 4; }
bool is_type(int32_t t) { return t == MOE_T_BF16 || t == MOE_T_FP32; }

cudaError_t quantize(const void* x, int32_t type, int64_t rows, int64_t cols, int64_t ld, Codes row, Codes col, Codes square,
                     cudaStream_t st) {
    const dim3 grid(unsigned(blocks(rows) * blocks(cols)));
    const bool wide = rows_on(x, ld, size_of(type), 16);
    count_launch();
    if (type == MOE_T_BF16)
        return launch_pdl(fp8_quantize_kernel<__nv_bfloat16>, grid, dim3(kQuantThreads), 0, st, static_cast<const __nv_bfloat16*>(x),
                          rows, int(cols), ld, wide, row, col, square);
    return launch_pdl(fp8_quantize_kernel<float>, grid, dim3(kQuantThreads), 0, st, static_cast<const float*>(x), rows, int(cols), ld,
                      wide, row, col, square);
}

int sm_count() {  // of the current device
    static std::atomic<int> known[64];
    int sms = 152, device = 0;
    if (cudaGetDevice(&device) != cudaSuccess) return sms;
    if (device < 64 && (sms = known[device].load(std::memory_order_relaxed)) > 0) return sms;
    sms = 152;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device) == cudaSuccess && device < 64) known[device].store(sms, std::memory_order_relaxed);
    return sms;
}

// Pieces of a workspace, or (base null) their size
struct Arena {
    char* base;
    size_t at = 0;
    explicit Arena(void* p) : base(static_cast<char*>(p)) {}
    void* take(int64_t bytes) {
        void* p = base ? base + at : nullptr;
        at += size_t(up(bytes, 256));
        return p;
    }
    Codes codes(int64_t rows, int64_t cols, bool by_row) {
        Codes c;
        c.ld = up(cols, 16);
        c.q = static_cast<uint8_t*>(take(rows * c.ld));
        c.s = static_cast<float*>(take(4 * (by_row ? blocks(cols) * rows : blocks(rows) * cols)));
        return c;
    }
};

// How a product is cut up
struct Plan {
    int bn, cg, splits;
};

// The cut with the least time, by what was measured of each (us): a round of tiles takes a start and an end (128 x 128 tiles 4, 128 x 256
// 5.5, pairs 6, the gate's results 3 more) and its blocks along K, a chain
// of copy, product, read and release that is nearly as long for a small tile as for a large one, and longer the more SMs
// work (128 columns 0.3 to 0.55 a block, 256 0.45 to 0.6, a pair's 0.42 to 0.5; a weight's gradient 0.35 more). K in parts fills the SMs of a few
// tiles and shortens the chain, for a launch that sums the parts (2.7) and their way through memory. E.g. 512 x 1024, K 4096: 14.9
// whole, 10.4 in four parts, pairs 18.5; 6788 x 324, K 2900: pairs 18.8, 128 x 128 23.9; three gradients of 1450 x 324, K 6788: 128 x 128 whole
// 72, 128 x 256 in two parts 58. It goes by the sizes alone, as the workspace's size does.
Plan plan(int op, const F8Args& a) {
    const int sms = sm_count();
    const bool gated = op == F8_GU;
    double elements = 0;
    int64_t small = 0, wide = 0, pairs = 0;  // tiles
    for (int p = 0; p < a.products; ++p) {
        const int64_t M = a.o[p].M, N = a.o[p].N, n = (N + 127) / 128, n2 = gated ? n : (N + 255) / 256;
        elements += double(M) * N;
        small += (M + 127) / 128 * n;
        wide += (M + 127) / 128 * n2;
        pairs += (M + 255) / 256 * n2;
    }
    Plan best = {256, 2, 1};
    double least = 1e30;
    auto look = [&](int bn, int cg, int splits) {
        const int units = sms / cg;
        const int64_t items = (cg == 2 ? pairs : bn == 256 ? wide : small) * splits;
        const double busy = items < units ? double(items) / units : 1.0;
        const double chain = (bn == 128 ? 0.3 + 0.25 * busy : cg == 2 ? 0.42 + 0.08 * busy : 0.45 + 0.15 * busy) + (op == F8_TN ? 0.35 : 0.0);
        const double ends = (bn == 128 ? 4.0 : cg == 2 ? 6.0 : 5.5) + (gated && splits == 1 ? 3.0 : 0.0);
        double us = double((items + units - 1) / units) * (ends + chain * ((a.k_blocks + splits - 1) / splits));
        if (splits > 1) us += 2.7 + (gated ? 1.5 : 0.0) + elements * (gated ? 2 : 1) * splits * 0.8e-6;
        if (us < least) least = us, best = {bn, cg, splits};
    };
    look(256, 2, 1);
    for (const int splits : {1, 2, 3, 4, 5, 6, 8, 10, 12, 16}) {
        if (splits > a.k_blocks || (splits > 1 && wide > sms)) break;
        if (gated || op == F8_TN || splits == 1) look(256, 1, splits);
        if (!gated) look(128, 1, splits);
    }
    return best;
}

void set_out(F8Out& o, void* out, int64_t ld, bool bf16, bool accumulate, int64_t M, int64_t N) {
    o = F8Out{out, ld, nullptr, up(N, 256), int(M), int(N), 0, 0, bf16 ? 1 : 0, accumulate ? 1 : 0};
}

// completes `a` and takes the partial sums' memory from `ws`
Plan prepare(int op, F8Args& a, Arena& ws) {
    const Plan pl = plan(op, a);
    const int tm = 128 * pl.cg, tn = op == F8_GU ? 128 : pl.bn;
    a.splits = pl.splits;
    for (int p = 0; p < a.products; ++p) {
        F8Out& o = a.o[p];
        o.m_tiles = (o.M + tm - 1) / tm;
        o.n_tiles = (o.N + tn - 1) / tn;
        if (pl.splits > 1) o.partial = static_cast<float*>(ws.take(4 * int64_t(pl.splits) * (op == F8_GU ? 2 : 1) * o.M * o.ld_partial));
    }
    return pl;
}

// boxes of 128 bytes (columns) x box_rows
bool map_of(CUtensorMap& m, const void* q, int64_t ld, int64_t rows, int64_t cols, uint32_t box_rows = 128) {
    const uint64_t dims[2] = {uint64_t(cols), uint64_t(rows)}, strides[1] = {uint64_t(ld)};
    const uint32_t box[2] = {128, box_rows};
    return encode_map(&m, q, 2, dims, strides, box, MAP_U8);
}

cudaError_t multiply(int op, const Plan& pl, const F8Maps& maps, const F8Args& a, cudaStream_t st) {
    const cudaError_t e = launch_f8_gemm(op, pl.bn, pl.cg, maps, a, sm_count(), st);
    if (e != cudaSuccess || pl.splits == 1) return e;
    if (op != F8_GU) return launch_f8_reduce(a, st);
    const int64_t units = int64_t(a.o[0].M) * a.o[0].n_tiles;  // blocks of 128 of a row, 16 threads each
    count_launch();
    return launch_pdl(fp8_gated_sum_kernel, dim3(unsigned((units + 15) / 16)), dim3(256), 0, st, a);
}

// A product of a linear layer. x, w: the operands' codes; sizes as in fp8.h. `run` false: its workspace alone.
cudaError_t product(int op, Codes x, int64_t xr, int64_t xc, Codes w, int64_t wr, int64_t wc, void* out, int64_t ld, bool bf16,
                    bool accumulate, Arena& ws, bool run, cudaStream_t st) {
    F8Args a = {};
    a.products = 1;
    const int64_t M = op == F8_TN ? xc : xr, N = op == F8_NT ? wr : wc, K = op == F8_TN ? xr : xc;
    a.k_blocks = a.k_part = int(blocks(K));
    set_out(a.o[0], out, ld, bf16, accumulate, M, N);
    a.s[0] = {x.s, w.s, op == F8_TN ? xc : xr, op == F8_TN ? wc : blocks(wc)};
    const Plan pl = prepare(op, a, ws);
    if (!run) return cudaSuccess;
    F8Maps m;
    if (!map_of(m.a[0], x.q, x.ld, xr, xc) || !map_of(m.b[0], w.q, w.ld, wr, wc)) return cudaErrorInvalidValue;
    return multiply(op, pl, m, a, st);
}

// ---------------------------------------------------------------- checks
bool ok_codes(const moe_fp8* v, int64_t cols) {
    return v && v->q && v->scales && v->ld >= cols && v->ld % 16 == 0 && aligned(v->q, 16) && aligned(v->scales, 4);
}
Codes codes_of(const moe_fp8& v) { return {static_cast<uint8_t*>(v.q), v.ld, v.scales}; }
constexpr Codes kNone = {nullptr, 0, nullptr};

bool ok_size(int64_t T, int64_t a, int64_t b) {
    return T >= 0 && T <= kMostRows && a >= 1 && a <= kMostCols && b >= 1 && b <= kMostCols;
}
bool ok_rows(const void* p, int32_t type, int64_t stride, int64_t cols) { return p && aligned(p, size_of(type)) && stride >= cols; }
bool ok_workspace(const void* p, size_t have, size_t need) { return need == 0 || (p && have >= need && aligned(p, 256)); }
bool ok_linear(const moe_linear_config* c, int64_t T) {
    return c && ok_size(T, c->in_features, c->out_features) && is_type(c->x_type) && is_type(c->y_type);
}
bool ok_ffn(const moe_ffn_config* c, int64_t T) {
    return c && ok_size(T, c->hidden, c->inter) && std::isfinite(c->swiglu_limit) && c->swiglu_limit >= 0.0f;
}
bool ok_grad(int32_t g_type, int32_t accumulate) {
    return (g_type == MOE_G_FP32 || g_type == MOE_G_BF16) && (accumulate == 0 || accumulate == 1);
}
moe_status answer(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

// gradients of no rows: nothing to add, or zeros
cudaError_t no_rows(void* out, int64_t ld, int64_t rows, int64_t cols, int32_t g_type, int32_t accumulate, cudaStream_t st) {
    if (!out || accumulate) return cudaSuccess;
    const size_t es = g_type == MOE_G_BF16 ? 2 : 4;
    return cudaMemset2DAsync(out, size_t(ld) * es, 0, size_t(cols) * es, size_t(rows), st);
}

// ---------------------------------------------------------------- the calls' work; `run` false: the workspace alone
struct LinearCall {
    const moe_linear_config* c;
    int64_t T;
    const void* in;  // x or dy
    int64_t in_stride;
    Codes w, kept;
    void* out;  // y or dx
    int64_t out_stride;
    void* dw;
    int64_t dw_stride;
    int32_t g_type, accumulate;
};

// y = x W^T for a few tokens
F8Few few(const Codes& w, const void* x, int64_t ld_x, int32_t x_type, void* out, int64_t ld_out, bool bf16, int64_t T, int64_t N, int64_t K) {
    F8Few a = {};
    a.w[0] = w.q, a.ld_w[0] = w.ld, a.ws[0] = w.s;
    a.x = x, a.ld_x = ld_x, a.wide = rows_on(x, ld_x, size_of(x_type), 16);
    a.out = out, a.ld_out = ld_out, a.bf16 = bf16;
    a.T = int(T), a.N = int(N), a.K = int(K);
    return a;
}

cudaError_t linear_forward(const LinearCall& k, Arena& ws, bool run, cudaStream_t st) {
    const int64_t T = k.T, K = k.c->in_features, N = k.c->out_features;
    if (f8_few_fits(T, N, K, false, sm_count())) {
        if (!run) return cudaSuccess;
        if (k.kept.q) {
            const cudaError_t e = quantize(k.in, k.c->x_type, T, K, k.in_stride, kNone, k.kept, kNone, st);
            if (e != cudaSuccess) return e;
        }
        F8Few a = few(k.w, k.in, k.in_stride, k.c->x_type, k.out, k.out_stride, k.c->y_type == MOE_T_BF16, T, N, K);
        a.early = k.kept.q != nullptr;
        return launch_f8_few(a, k.c->x_type == MOE_T_BF16, sm_count(), st);
    }
    const Codes xq = ws.codes(T, K, true);
    if (run) {
        const cudaError_t e = quantize(k.in, k.c->x_type, T, K, k.in_stride, xq, k.kept, kNone, st);
        if (e != cudaSuccess) return e;
    }
    return product(F8_NT, xq, T, K, k.w, N, K, k.out, k.out_stride, k.c->y_type == MOE_T_BF16, false, ws, run, st);
}

cudaError_t linear_backward(const LinearCall& k, Arena& ws, bool run, cudaStream_t st) {
    const int64_t T = k.T, K = k.c->in_features, N = k.c->out_features;
    const bool x = !run || k.out, w = !run || k.dw;
    const Codes row = x ? ws.codes(T, N, true) : kNone, col = w ? ws.codes(T, N, false) : kNone;
    cudaError_t e = cudaSuccess;
    if (run && (x || w)) e = quantize(k.in, k.c->y_type, T, N, k.in_stride, row, col, kNone, st);
    if (x && e == cudaSuccess)
        e = product(F8_NN, row, T, N, k.w, N, K, k.out, k.out_stride, k.c->x_type == MOE_T_BF16, false, ws, run, st);
    if (w && e == cudaSuccess)
        e = product(F8_TN, col, T, N, k.kept, T, K, k.dw, k.dw_stride, k.g_type == MOE_G_BF16, k.accumulate, ws, run, st);
    return e;
}

struct FfnCall {
    const moe_ffn_config* c;
    int64_t T;
    const void* in;
    int64_t in_stride;
    Codes gate, up, down;
    Codes kx, kg, ku;
    void* out;
    int64_t out_stride;
    const moe_ffn_grads* grads;
    int32_t g_type, accumulate;
};

// Few tokens and nothing kept: h passes in fp32 from the first launch to the second, which quantises it
cudaError_t ffn_few(const FfnCall& k, Arena& ws, bool run, cudaStream_t st) {
    const int64_t T = k.T, H = k.c->hidden, I = k.c->inter, ld_h = up(I, 4);
    float* h = static_cast<float*>(ws.take(4 * T * ld_h));
    if (!run) return cudaSuccess;
    F8Few g = few(k.gate, k.in, k.in_stride, MOE_T_BF16, h, ld_h, false, T, I, H);
    g.w[1] = k.up.q, g.ld_w[1] = k.up.ld, g.ws[1] = k.up.s;
    g.limit = k.c->swiglu_limit;
    const cudaError_t e = launch_f8_few(g, true, sm_count(), st);
    if (e != cudaSuccess) return e;
    F8Few d = few(k.down, h, ld_h, MOE_T_FP32, k.out, k.out_stride, true, T, H, I);
    d.early = 1;
    return launch_f8_few(d, false, sm_count(), st);
}

cudaError_t ffn_forward(const FfnCall& k, Arena& ws, bool run, cudaStream_t st) {
    const int64_t T = k.T, H = k.c->hidden, I = k.c->inter;
    if (!k.kx.q && f8_few_fits(T, I, H, true, sm_count()) && f8_few_fits(T, H, I, false, sm_count())) return ffn_few(k, ws, run, st);
    const Codes xq = ws.codes(T, H, true), h = ws.codes(T, I, true);
    F8Args a = {};
    a.products = 1;
    a.k_blocks = a.k_part = int(blocks(H));
    set_out(a.o[0], nullptr, 0, false, false, T, I);
    const Plan pl = prepare(F8_GU, a, ws);
    if (run) {
        cudaError_t e = quantize(k.in, MOE_T_BF16, T, H, k.in_stride, xq, k.kx, kNone, st);
        if (e != cudaSuccess) return e;
        a.s[0] = {xq.s, k.gate.s, T, blocks(H)};
        a.s[1] = {xq.s, k.up.s, T, blocks(H)};
        a.h = h.q, a.hs = h.s, a.ld_h = h.ld;
        a.g = k.kg.q, a.gs = k.kg.s, a.ld_g = k.kg.ld;
        a.u = k.ku.q, a.us = k.ku.s, a.ld_u = k.ku.ld;
        a.limit = k.c->swiglu_limit;
        F8Maps m;
        if (!map_of(m.a[0], xq.q, xq.ld, T, H) || !map_of(m.b[0], k.gate.q, k.gate.ld, I, H, 64) ||
            !map_of(m.b[1], k.up.q, k.up.ld, I, H, 64))
            return cudaErrorInvalidValue;
        e = multiply(F8_GU, pl, m, a, st);
        if (e != cudaSuccess) return e;
    }
    return product(F8_NT, h, T, I, k.down, H, I, k.out, k.out_stride, true, false, ws, run, st);
}

cudaError_t ffn_backward(const FfnCall& k, Arena& ws, bool run, cudaStream_t st) {
    const int64_t T = k.T, H = k.c->hidden, I = k.c->inter;
    const bool x = !run || k.out, w = !run || k.grads;
    if (!x && !w) return cudaSuccess;
    const Codes dy = ws.codes(T, H, true), dyc = w ? ws.codes(T, H, false) : kNone;
    const int64_t ld_dh = up(I, 4);
    float* dh = static_cast<float*>(ws.take(4 * T * ld_dh));
    GatedBack b = {dh, ld_dh, k.kg, k.ku, kNone, kNone, kNone, kNone, kNone, T, int(I), k.c->swiglu_limit};
    if (x) b.dg_row = ws.codes(T, I, true), b.du_row = ws.codes(T, I, true);
    if (w) b.dg_col = ws.codes(T, I, false), b.du_col = ws.codes(T, I, false), b.h_col = ws.codes(T, I, false);
    cudaError_t e = cudaSuccess;
    if (run) e = quantize(k.in, MOE_T_BF16, T, H, k.in_stride, dy, dyc, kNone, st);
    if (e == cudaSuccess) e = product(F8_NN, dy, T, H, k.down, H, I, dh, ld_dh, false, false, ws, run, st);
    if (e != cudaSuccess) return e;
    if (run) {
        count_launch();
        e = launch_pdl(b.limit > 0.0f ? fp8_gated_back_kernel<true> : fp8_gated_back_kernel<false>, dim3(unsigned(blocks(T) * blocks(I))), dim3(kGatedThreads), 0, st, b);
        if (e != cudaSuccess) return e;
    }
    if (x) {
        F8Args a = {};
        a.products = 1;
        a.k_part = int(blocks(I));
        a.k_blocks = 2 * a.k_part;
        set_out(a.o[0], k.out, k.out_stride, true, false, T, H);
        a.s[0] = {b.dg_row.s, k.gate.s, T, blocks(H)};
        a.s[1] = {b.du_row.s, k.up.s, T, blocks(H)};
        const Plan pl = prepare(F8_NN, a, ws);
        if (run) {
            F8Maps m;
            if (!map_of(m.a[0], b.dg_row.q, b.dg_row.ld, T, I) || !map_of(m.a[1], b.du_row.q, b.du_row.ld, T, I) ||
                !map_of(m.b[0], k.gate.q, k.gate.ld, I, H) || !map_of(m.b[1], k.up.q, k.up.ld, I, H))
                return cudaErrorInvalidValue;
            e = multiply(F8_NN, pl, m, a, st);
            if (e != cudaSuccess) return e;
        }
    }
    if (w) {
        F8Args a = {};
        a.products = 3;
        a.k_blocks = a.k_part = int(blocks(T));
        const moe_ffn_grads none = {};
        const moe_ffn_grads& g = k.grads ? *k.grads : none;
        const bool bf = k.g_type == MOE_G_BF16, add = k.accumulate;
        set_out(a.o[0], g.gate, g.gate_stride, bf, add, I, H);
        set_out(a.o[1], g.up, g.up_stride, bf, add, I, H);
        set_out(a.o[2], g.down, g.down_stride, bf, add, H, I);
        a.s[0] = {b.dg_col.s, k.kx.s, I, H};
        a.s[1] = {b.du_col.s, k.kx.s, I, H};
        a.s[2] = {dyc.s, b.h_col.s, H, I};
        const Plan pl = prepare(F8_TN, a, ws);
        if (run) {
            F8Maps m;
            if (!map_of(m.a[0], b.dg_col.q, b.dg_col.ld, T, I) || !map_of(m.a[1], b.du_col.q, b.du_col.ld, T, I) ||
                !map_of(m.a[2], dyc.q, dyc.ld, T, H) || !map_of(m.b[0], k.kx.q, k.kx.ld, T, H) ||
                !map_of(m.b[2], b.h_col.q, b.h_col.ld, T, I))
                return cudaErrorInvalidValue;
            m.b[1] = m.b[0];
            e = multiply(F8_TN, pl, m, a, st);
        }
    }
    return e;
}

}  // namespace

}  // namespace moe

extern "C" {

moe_status moe_fp8_quantize(const void* x, int32_t x_type, int64_t rows, int64_t cols, int64_t x_stride,
                            const moe_fp8* row, const moe_fp8* col, const moe_fp8* square, void* stream) {
    using namespace moe;
    if (!is_type(x_type) || !ok_size(rows, cols, 1) || x_stride < cols) return MOE_ERR_INVALID_ARG;
    if (rows == 0 || (!row && !col && !square)) return MOE_OK;
    if (!ok_rows(x, x_type, x_stride, cols)) return MOE_ERR_INVALID_ARG;
    for (const moe_fp8* v : {row, col, square})
        if (v && !ok_codes(v, cols)) return MOE_ERR_INVALID_ARG;
    auto of = [](const moe_fp8* v) { return v ? codes_of(*v) : kNone; };
    return answer(quantize(x, x_type, rows, cols, x_stride, of(row), of(col), of(square), static_cast<cudaStream_t>(stream)));
}

moe_status moe_fp8_dequantize(const moe_fp8* v, int32_t block, int64_t rows, int64_t cols, void* out, int32_t out_type,
                              int64_t out_stride, void* stream) {
    using namespace moe;
    if (!is_type(out_type) || !ok_size(rows, cols, 1) || out_stride < cols || block < MOE_B_ROW || block > MOE_B_SQUARE)
        return MOE_ERR_INVALID_ARG;
    if (rows == 0) return MOE_OK;
    if (!ok_codes(v, cols) || !ok_rows(out, out_type, out_stride, cols)) return MOE_ERR_INVALID_ARG;
    const dim3 grid(unsigned(blocks(rows) * blocks(cols)));
    const uint8_t* q = static_cast<const uint8_t*>(v->q);
    const float* s = v->scales;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    count_launch();
    if (out_type == MOE_T_BF16)
        return answer(launch_pdl(fp8_dequantize_kernel<__nv_bfloat16>, grid, dim3(kQuantThreads), 0, st, q, v->ld, s, block, rows, int(cols),
                                 static_cast<__nv_bfloat16*>(out), out_stride));
    return answer(launch_pdl(fp8_dequantize_kernel<float>, grid, dim3(kQuantThreads), 0, st, q, v->ld, s, block, rows, int(cols),
                             static_cast<float*>(out), out_stride));
}

moe_status moe_linear_size(const moe_linear_config* cfg, int64_t T, int32_t backward, size_t* bytes) {
    using namespace moe;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = 0;
    if (!ok_linear(cfg, T) || (backward != 0 && backward != 1)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    LinearCall k = {};
    k.c = cfg, k.T = T;
    Arena ws(nullptr);
    (void)(backward ? linear_backward(k, ws, false, nullptr) : linear_forward(k, ws, false, nullptr));
    *bytes = ws.at;
    return MOE_OK;
}

moe_status moe_linear_forward(const moe_linear_config* cfg, int64_t T, const void* x, int64_t x_stride, const moe_fp8* w, void* y,
                              int64_t y_stride, const moe_fp8* kept, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace moe;
    size_t need = 0;
    const moe_status s = moe_linear_size(cfg, T, 0, &need);
    if (s != MOE_OK) return s;
    if (x_stride < cfg->in_features || y_stride < cfg->out_features) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!ok_rows(x, cfg->x_type, x_stride, cfg->in_features) || !ok_rows(y, cfg->y_type, y_stride, cfg->out_features) ||
        !ok_codes(w, cfg->in_features) || (kept && !ok_codes(kept, cfg->in_features)) || !ok_workspace(workspace, workspace_bytes, need))
        return MOE_ERR_INVALID_ARG;
    const LinearCall k = {cfg, T, x, x_stride, codes_of(*w), kept ? codes_of(*kept) : kNone, y, y_stride, nullptr, 0, 0, 0};
    Arena ws(workspace);
    return answer(linear_forward(k, ws, true, static_cast<cudaStream_t>(stream)));
}

moe_status moe_linear_backward(const moe_linear_config* cfg, int64_t T, const void* dy, int64_t dy_stride, const moe_fp8* w,
                               const moe_fp8* kept, void* dx, int64_t dx_stride, void* dweight, int64_t dweight_stride, int32_t g_type,
                               int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace moe;
    size_t need = 0;
    const moe_status s = moe_linear_size(cfg, T, 1, &need);
    if (s != MOE_OK) return s;
    const int64_t K = cfg->in_features, N = cfg->out_features;
    const int32_t gt = g_type == MOE_G_BF16 ? MOE_T_BF16 : MOE_T_FP32;
    if (!ok_grad(g_type, accumulate) || dy_stride < N || (dx && dx_stride < K)) return MOE_ERR_INVALID_ARG;
    if (dweight && !ok_rows(dweight, gt, dweight_stride, K)) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) return answer(no_rows(dweight, dweight_stride, N, K, g_type, accumulate, st));
    if (!ok_rows(dy, cfg->y_type, dy_stride, N) || (dx && (!ok_rows(dx, cfg->x_type, dx_stride, K) || !ok_codes(w, K))) ||
        (dweight && !ok_codes(kept, K)) || !ok_workspace(workspace, workspace_bytes, need))
        return MOE_ERR_INVALID_ARG;
    const LinearCall k = {cfg, T, dy, dy_stride, w ? codes_of(*w) : kNone, kept ? codes_of(*kept) : kNone, dx, dx_stride,
                          dweight, dweight_stride, g_type, accumulate};
    Arena ws(workspace);
    return answer(linear_backward(k, ws, true, st));
}

moe_status moe_ffn_size(const moe_ffn_config* cfg, int64_t T, int32_t backward, size_t* bytes) {
    using namespace moe;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = 0;
    if (!ok_ffn(cfg, T) || (backward != 0 && backward != 1)) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    FfnCall k = {};
    k.c = cfg, k.T = T;
    Arena ws(nullptr);
    (void)(backward ? ffn_backward(k, ws, false, nullptr) : ffn_forward(k, ws, false, nullptr));
    *bytes = ws.at;
    if (!backward) {  // the way of a call that keeps
        k.kx.q = reinterpret_cast<uint8_t*>(bytes);
        Arena keeping(nullptr);
        (void)ffn_forward(k, keeping, false, nullptr);
        *bytes = keeping.at > ws.at ? keeping.at : ws.at;
    }
    return MOE_OK;
}

moe_status moe_ffn_forward(const moe_ffn_config* cfg, int64_t T, const void* x, int64_t x_stride, const moe_ffn_weights* w, void* y,
                           int64_t y_stride, const moe_ffn_kept* kept, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace moe;
    size_t need = 0;
    const moe_status s = moe_ffn_size(cfg, T, 0, &need);
    if (s != MOE_OK) return s;
    const int64_t H = cfg->hidden, I = cfg->inter;
    if (x_stride < H || y_stride < H) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!ok_rows(x, MOE_T_BF16, x_stride, H) || !ok_rows(y, MOE_T_BF16, y_stride, H) || !w || !ok_codes(&w->gate, H) ||
        !ok_codes(&w->up, H) || !ok_codes(&w->down, I) || !ok_workspace(workspace, workspace_bytes, need))
        return MOE_ERR_INVALID_ARG;
    if (kept && (!ok_codes(&kept->x, H) || !ok_codes(&kept->gate, I) || !ok_codes(&kept->up, I))) return MOE_ERR_INVALID_ARG;
    FfnCall k = {cfg, T, x, x_stride, codes_of(w->gate), codes_of(w->up), codes_of(w->down), kNone, kNone, kNone, y, y_stride, nullptr, 0, 0};
    if (kept) k.kx = codes_of(kept->x), k.kg = codes_of(kept->gate), k.ku = codes_of(kept->up);
    Arena ws(workspace);
    return answer(ffn_forward(k, ws, true, static_cast<cudaStream_t>(stream)));
}

moe_status moe_ffn_backward(const moe_ffn_config* cfg, int64_t T, const void* dy, int64_t dy_stride, const moe_ffn_weights* w,
                            const moe_ffn_kept* kept, void* dx, int64_t dx_stride, const moe_ffn_grads* grads, int32_t g_type,
                            int32_t accumulate, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace moe;
    size_t need = 0;
    const moe_status s = moe_ffn_size(cfg, T, 1, &need);
    if (s != MOE_OK) return s;
    const int64_t H = cfg->hidden, I = cfg->inter;
    const int32_t gt = g_type == MOE_G_BF16 ? MOE_T_BF16 : MOE_T_FP32;
    if (!ok_grad(g_type, accumulate) || dy_stride < H || (dx && dx_stride < H)) return MOE_ERR_INVALID_ARG;
    if (grads && (!ok_rows(grads->gate, gt, grads->gate_stride, H) || !ok_rows(grads->up, gt, grads->up_stride, H) ||
                  !ok_rows(grads->down, gt, grads->down_stride, I) || grads->gate == grads->up || grads->gate == grads->down ||
                  grads->up == grads->down))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        if (!grads) return MOE_OK;
        cudaError_t e = no_rows(grads->gate, grads->gate_stride, I, H, g_type, accumulate, st);
        if (e == cudaSuccess) e = no_rows(grads->up, grads->up_stride, I, H, g_type, accumulate, st);
        if (e == cudaSuccess) e = no_rows(grads->down, grads->down_stride, H, I, g_type, accumulate, st);
        return answer(e);
    }
    if (!ok_rows(dy, MOE_T_BF16, dy_stride, H) || (dx && !ok_rows(dx, MOE_T_BF16, dx_stride, H)) || !w || !ok_codes(&w->gate, H) ||
        !ok_codes(&w->up, H) || !ok_codes(&w->down, I) || !kept || !ok_codes(&kept->x, H) || !ok_codes(&kept->gate, I) ||
        !ok_codes(&kept->up, I) || !ok_workspace(workspace, workspace_bytes, need))
        return MOE_ERR_INVALID_ARG;
    const FfnCall k = {cfg, T, dy, dy_stride, codes_of(w->gate), codes_of(w->up), codes_of(w->down), codes_of(kept->x),
                       codes_of(kept->gate), codes_of(kept->up), dx, dx_stride, grads, g_type, accumulate};
    Arena ws(workspace);
    return answer(ffn_backward(k, ws, true, st));
}

moe_status moe_fp8_status(void* stream) {
    bool gave_up = false;
    const cudaError_t e = moe::f8_status(gave_up, static_cast<cudaStream_t>(stream));
    return gave_up ? MOE_ERR_TIMEOUT : moe::answer(e);
}

moe_status moe_fp8_selftest_timeout(void* stream) { return moe::answer(moe::launch_f8_wait_selftest(static_cast<cudaStream_t>(stream))); }

}  // extern "C"
