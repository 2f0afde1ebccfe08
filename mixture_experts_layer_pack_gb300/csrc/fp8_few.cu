// The products of the dense layers in 8-bit floating point for a few tokens: y[t,n] = sum over blocks of sx(t) sw sum qx[t,k] qw[n,k].
//
// Their time is the reading of the weights once, so those are not staged: a warp takes 16 rows of the weight and multiplies them with
// 8 tokens an mma.sync (m16n8k32; the tensor rate is not what counts), and the warps of a block share the blocks of 128
// along K, each with its share's loads under way. K is summed in any order, so a lane's 32 bytes of a row's block are the operands of four
// mma as they come from memory, 16 bytes a load. Every block quantises the activations for itself, into shared memory, while its
// weights are on their way (a launch for it, and its codes read back from L2 block by block: 1 token, 7168 to 2048, 15 us).
#include "device_common.cuh"
#include "fp8.h"
#include "fp8_device.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr size_t kFewShared = 128 << 10;  // most that the activations' codes take

__device__ __forceinline__ void mma_e4m3(float (&d)[4], const uint32_t* a0, const uint32_t* a1, const uint32_t* b) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0[0]), "r"(a1[0]), "r"(a0[1]), "r"(a1[1]), "r"(b[0]), "r"(b[1]));
}

// 32 codes of a row, of which n are its own (the others read as zeros, and their bytes not at all)
__device__ __forceinline__ void codes32(const uint8_t* p, int n, uint32_t (&w)[8]) {
#pragma unroll
    for (int z = 0; z < 2; ++z) {
        uint4 x = make_uint4(0, 0, 0, 0);
        if (n >= 16 * (z + 1)) {
            x = __ldg(reinterpret_cast<const uint4*>(p) + z);
        } else if (n > 16 * z) {
            uint32_t b[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 16; ++j)
                if (16 * z + j < n) b[j >> 2] |= uint32_t(p[16 * z + j]) << (8 * (j & 3));
            x = make_uint4(b[0], b[1], b[2], b[3]);
        }
        w[4 * z] = x.x, w[4 * z + 1] = x.y, w[4 * z + 2] = x.z, w[4 * z + 3] = x.w;
    }
}

// 32 elements of an activation's row, n of them its own
__device__ __forceinline__ void elements32(const __nv_bfloat16* p, int n, bool wide, float (&v)[32]) {
    if (wide && n >= 32) {
#pragma unroll
        for (int z = 0; z < 4; ++z) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(p) + z);
            unpack_bf16x2(w.x, v[8 * z], v[8 * z + 1]), unpack_bf16x2(w.y, v[8 * z + 2], v[8 * z + 3]);
            unpack_bf16x2(w.z, v[8 * z + 4], v[8 * z + 5]), unpack_bf16x2(w.w, v[8 * z + 6], v[8 * z + 7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = j < n ? __bfloat162float(p[j]) : 0.0f;
    }
}
__device__ __forceinline__ void elements32(const float* p, int n, bool wide, float (&v)[32]) {
    if (wide && n >= 32) {
#pragma unroll
        for (int z = 0; z < 8; ++z) {
            const float4 w = __ldg(reinterpret_cast<const float4*>(p) + z);
            v[4 * z] = w.x, v[4 * z + 1] = w.y, v[4 * z + 2] = w.z, v[4 * z + 3] = w.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = j < n ? p[j] : 0.0f;
    }
}

// X: the activations' type. TILES: of 8 tokens. GATED: h = silu(g) u of two weights, eight rows of each in the place of sixteen of one, so that a
// thread gets a column's g and u. WARPS: that share K.
template <typename X, int TILES, bool GATED, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS) f8_few_kernel(const __grid_constant__ F8Few a) {
    constexpr int AHEAD = TILES == 1 ? 4 : 2;  // blocks of 128 whose weights a warp has under way, 16 registers each; at two tiles four spill
    constexpr int ROWS = GATED ? 8 : 16;       // results of a block
    __shared__ float part[WARPS][16][9];
    extern __shared__ __align__(16) uint8_t xq[];  // codes [T][128 k_blocks], scales [T][k_blocks]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n0 = blockIdx.x * ROWS;
    const uint8_t* w0 = a.w[0] + min(n0 + g, a.N - 1) * a.ld_w[0];  // rows past the last are not stored
    const uint8_t* w1 = GATED ? a.w[1] + min(n0 + g, a.N - 1) * a.ld_w[1] : a.w[0] + min(n0 + g + 8, a.N - 1) * a.ld_w[0];
    const int k_blocks = (a.K + 127) >> 7, ld_q = k_blocks * 128;
    const float* ws0 = a.ws[0] + int64_t(n0 >> 7) * k_blocks;
    const float* ws1 = a.ws[GATED ? 1 : 0] + int64_t(n0 >> 7) * k_blocks;
    float* xs = reinterpret_cast<float*>(xq + a.T * ld_q);
    uint32_t w[AHEAD][2][8];
    float ws[AHEAD][2];
    auto load = [&](int kb, uint32_t (&v)[2][8], float (&s)[2]) {
        if (kb >= k_blocks) return;
        const int at = kb * 128 + 32 * t;
        codes32(w0 + at, a.K - at, v[0]);
        codes32(w1 + at, a.K - at, v[1]);
        s[0] = __ldg(ws0 + kb);
        s[1] = GATED ? __ldg(ws1 + kb) : s[0];
    };
    if (!a.early) pdl_wait();  // early: the kernel before us has not written the weights
#pragma unroll
    for (int z = 0; z < AHEAD; ++z) load(warp + z * WARPS, w[z], ws[z]);
    if (a.early) pdl_wait();
    pdl_trigger();

    // the activations: four lanes a block of a token
    for (int i = threadIdx.x >> 2; i < a.T * k_blocks; i += 8 * WARPS) {
        const int token = i / k_blocks, kb = i - token * k_blocks, at = kb * 128 + 32 * t;
        float v[32];
        elements32(static_cast<const X*>(a.x) + int64_t(token) * a.ld_x + at, a.K - at, a.wide, v);
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 32; ++j) m = fmaxf(m, fabsf(v[j]));
        const unsigned quad = 0xfu << (lane & 28);
        m = fmaxf(m, __shfl_xor_sync(quad, m, 1));
        m = fmaxf(m, __shfl_xor_sync(quad, m, 2));
        const float s = block_scale(m), r = __frcp_rn(s);
        uint32_t q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) q[j] = e4m3x4(v[4 * j] * r, v[4 * j + 1] * r, v[4 * j + 2] * r, v[4 * j + 3] * r);
        uint4* dst = reinterpret_cast<uint4*>(xq + token * ld_q + at);
        dst[0] = make_uint4(q[0], q[1], q[2], q[3]);
        dst[1] = make_uint4(q[4], q[5], q[6], q[7]);
        if (t == 0) xs[token * k_blocks + kb] = s;
    }
    __syncthreads();

    float acc[TILES][4] = {};
    for (int kb0 = warp; kb0 < k_blocks; kb0 += AHEAD * WARPS) {
#pragma unroll
        for (int z = 0; z < AHEAD; ++z) {
            const int kb = kb0 + z * WARPS;
            if (kb >= k_blocks) break;
#pragma unroll
            for (int j = 0; j < TILES; ++j) {
                const int token = 8 * j + g, c = 8 * j + 2 * t;
                uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                if (token < a.T) {
                    const uint4* src = reinterpret_cast<const uint4*>(xq + token * ld_q + kb * 128 + 32 * t);
                    const uint4 lo = src[0], hi = src[1];
                    x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
                }
                // the scales of this lane's columns of the product, tokens 2 t and 2 t + 1
                const float s0 = c < a.T ? xs[c * k_blocks + kb] : 0.0f, s1 = c + 1 < a.T ? xs[(c + 1) * k_blocks + kb] : 0.0f;
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int i = 0; i < 4; ++i) mma_e4m3(d, w[z][0] + 2 * i, w[z][1] + 2 * i, x + 2 * i);
                acc[j][0] = fmaf(d[0], ws[z][0] * s0, acc[j][0]), acc[j][1] = fmaf(d[1], ws[z][0] * s1, acc[j][1]);
                acc[j][2] = fmaf(d[2], ws[z][1] * s0, acc[j][2]), acc[j][3] = fmaf(d[3], ws[z][1] * s1, acc[j][3]);
            }
            load(kb + AHEAD * WARPS, w[z], ws[z]);
        }
    }
    // the warps' sums, in their order
#pragma unroll
    for (int j = 0; j < TILES; ++j) {
        if (j) __syncthreads();
        part[warp][g][2 * t] = acc[j][0], part[warp][g][2 * t + 1] = acc[j][1];
        part[warp][g + 8][2 * t] = acc[j][2], part[warp][g + 8][2 * t + 1] = acc[j][3];
        __syncthreads();
        const int r = threadIdx.x % ROWS, c = threadIdx.x / ROWS, token = 8 * j + c;
        if (c < 8 && token < a.T && n0 + r < a.N) {
            auto sum = [&](int row) {
                float s = 0.0f;
#pragma unroll
                for (int z = 0; z < WARPS; ++z) s += part[z][row][c];
                return s;
            };
            float y = sum(r);
            if (GATED) {
                float gate = y, up = sum(r + 8);
                if (a.limit > 0.0f) gate = clamp_top(gate, a.limit), up = clamp_both(up, a.limit);
                y = gate * sigmoidf_(gate) * up;
            }
            store_one(a.out, int64_t(token) * a.ld_out + n0 + r, a.bf16, false, y);
        }
    }
}

size_t few_shared(int64_t T, int64_t K) { return size_t(T) * size_t((K + 127) / 128) * (128 + 4); }

template <auto Kernel>
cudaError_t launch_kernel(const F8Few& a, int rows, int warps, cudaStream_t st) {
    const cudaError_t e = f8_allow_shared<Kernel>(kFewShared);
    if (e != cudaSuccess) return e;
    count_launch();
    return launch_pdl(Kernel, dim3(unsigned((a.N + rows - 1) / rows)), dim3(32 * warps), few_shared(a.T, a.K), st, a);
}

// Sixteen warps share K where the blocks are no more than the SMs, eight where two blocks an SM keep more loads under way than one. Measured with
// 1 token, us, sixteen and eight: 424 rows (27 blocks) 2.4, 3.1; 2048 rows of 7168 (128) 5.7, 5.9; 4096 of 2048 (256) 4.5, 3.7; 8192 of 4096
// (512) 12.1, 10.7.
template <typename X, int TILES, bool GATED>
cudaError_t launch_warps(const F8Few& a, int sms, cudaStream_t st) {
    constexpr int rows = GATED ? 8 : 16;
    if ((a.N + rows - 1) / rows > sms) return launch_kernel<f8_few_kernel<X, TILES, GATED, 8>>(a, rows, 8, st);
    return launch_kernel<f8_few_kernel<X, TILES, GATED, 16>>(a, rows, 16, st);
}

template <typename X, bool GATED>
cudaError_t launch_tiles(const F8Few& a, int sms, cudaStream_t st) {
    return a.T <= 8 ? launch_warps<X, 1, GATED>(a, sms, st) : launch_warps<X, 2, GATED>(a, sms, st);
}

}  // namespace

// Every block of 16 rows, or 8 of two weights, quantises all the activations, so this way is for few tokens and not too wide a weight: up
// to 600 blocks of 128 an SM quantises. Measured with them, us, here and through the tiles: 2048 to 4096, 16 tokens (430) 7.2, 10.1;
// 7168 to 2048, 16 tokens (754) 11.5, 11.9; 4096 to 8192, 4 tokens (431) 13.2, 16.4, 8 tokens (862) 16.6, 16.1; gated and back, 7168 and
// 2048, 4 tokens (377) 20.5, 25.6, 8 tokens (754) 27.7, 25.7; 4096 and 8192, 1 token (216) 26.2, 33.8, 4 tokens (862) 39.0, 36.5.
bool f8_few_fits(int64_t T, int64_t N, int64_t K, bool gated, int sms) {
    const int64_t rows = gated ? 8 : 16, units = T * ((K + 127) / 128);
    return T <= 16 && few_shared(T, K) <= kFewShared && (N + rows - 1) / rows * units <= 600 * int64_t(sms);
}

cudaError_t launch_f8_few(const F8Few& a, bool x_bf16, int sms, cudaStream_t st) {
    if (a.w[1]) return x_bf16 ? launch_tiles<__nv_bfloat16, true>(a, sms, st) : cudaErrorInvalidValue;
    return x_bf16 ? launch_tiles<__nv_bfloat16, false>(a, sms, st) : launch_tiles<float, false>(a, sms, st);
}

}  // namespace moe
