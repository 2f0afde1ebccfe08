// Host-side declarations of the dense layers in 8-bit floating point (fp8.cu, fp8_gemm.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

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
    float* partial;             // splits > 1: fp32 [splits][M][ld_partial]
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
    // F8_GU
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

}  // namespace moe
