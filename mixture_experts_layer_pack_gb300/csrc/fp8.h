// Host-side declarations of the dense layers in 8-bit floating point (fp8.cu, fp8_gemm.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/moe.h"

namespace moe {

constexpr int kF8Block = 128;   // elements of a scale's block, rows and columns of a tile, K of a pipeline stage

// The products, all with fp32 sums:
//   F8_NT  out[M,N] = A[M,K] B[N,K]^T   A: row blocks, B: square blocks (a weight)
//   F8_NN  out[M,N] = A[M,K] B[K,N]     A: row blocks, B: square blocks; up to two such products summed (K parts)
//   F8_TN  out[M,N] = A[K,M]^T B[K,N]   both: column blocks (K = tokens); up to three such products a launch
//   F8_GU  h[M,N] = silu(A Bg^T) (A Bu^T) with the clamp, stored as row blocks; A: row blocks, Bg, Bu: square blocks
enum F8Op : int { F8_NT = 0, F8_NN = 1, F8_TN = 2, F8_GU = 3 };

struct F8Scales {               // of a part (F8_NN, F8_GU) or a product (F8_TN)
    const float *a, *b;
    int64_t ld_a, ld_b;
};

struct F8Out {
    void* out;                  // bf16 or fp32 [M, N]
    int64_t ld;
    float* partial;             // splits > 1: fp32 [splits][M][ld_partial], ld_partial a multiple of 256
    int64_t ld_partial;
    int M, N, m_tiles, n_tiles;
    int bf16;                   // type of out
    int accumulate;             // out += (bf16: out = bf16(out + bf16(sum)))
};

struct F8Args {
    F8Scales s[3];
    F8Out o[3];
    int products;               // F8_TN: 1..3, else 1
    int k_blocks, k_part;       // blocks of 128 along K, and those of the first part (F8_NN)
    int splits;                 // the K blocks of a tile are divided among this many work items
    // F8_GU (splits > 1: the partials are [splits][2][M][ld_partial], g and u)
    uint8_t *h, *g, *u;         // codes [M, N]; g, u null: not kept
    float *hs, *gs, *us;        // row-block scales [n_tiles][M]
    int64_t ld_h, ld_g, ld_u;
    float limit;
};

struct F8Maps {
    CUtensorMap a[3], b[3];
};

// bn: columns of a tile (128, 256); cg: CTAs of a tile (1; 2: a pair shares a tile of 256 rows and 256 columns)
cudaError_t launch_f8_gemm(int op, int bn, int cg, const F8Maps& maps, const F8Args& args, int sms, cudaStream_t st);
// sums the partials of every product of `args` into its output
cudaError_t launch_f8_reduce(const F8Args& args, cudaStream_t st);
// whether a wait of a product on the current device gave up since the last call; synchronises `st`
cudaError_t f8_status(bool& gave_up, cudaStream_t st);
cudaError_t launch_f8_wait_selftest(cudaStream_t st);

// The shared memory that a kernel may ask for, said once for each device
template <auto Kernel>
cudaError_t f8_allow_shared(size_t bytes) {
    static std::atomic<uint64_t> said{0};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (device & 63);
    if (device < 64 && (said.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    if (e == cudaSuccess) said.fetch_or(bit, std::memory_order_release);
    return e;
}

// A few tokens' product with a weight, or with two and the gate between them (fp8_few.cu)
struct F8Few {
    const uint8_t* w[2];   // codes [N, K]; w[1] null: one weight
    int64_t ld_w[2];
    const float* ws[2];    // scales of square blocks
    const void* x;         // [T, K], quantised on the way
    int64_t ld_x;          // elements
    void* out;             // [T, N]: the sums, or with two weights h = silu(g) u
    int64_t ld_out;
    int T, N, K;
    int bf16;              // type of out
    int wide;              // rows of x start on 16 bytes
    int early;             // the kernel before in the stream is one of the same call: it has not written the weights
    float limit;
};
bool f8_few_fits(int64_t T, int64_t N, int64_t K, bool gated, int sms);
cudaError_t launch_f8_few(const F8Few& a, bool x_bf16, int sms, cudaStream_t st);

}  // namespace moe
