// The router's choice of experts from its logits, forward and backward, with the
// balancing losses.
//
// A warp owns a row (a token): lane l holds the logits of experts l, l + 32, ...
// With m the row's largest logit and z = sum_e exp(l_e - m): softmax scores
// exp(l_e - m) / z, log-sum-exp m + log z; sigmoid scores 1 / (1 + exp(-l_e)).
// The choice compares logits, mapped to unsigned integers of the same order, one
// warp-wide maximum and one warp-wide minimum index per slot: exact, ties to the
// lower id, whatever the scores round to.
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "../../include/moe.h"
#include "device_common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kRouterWarps = 8;
constexpr int kRouterBlocks = 304;  // most blocks of the forward, each with its own partial sums

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// order-preserving map of a float to an unsigned; 0 is kept for what cannot be chosen
// (-inf and NaN), both zeros get one key
__device__ __forceinline__ uint32_t order_key(float v) {
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float sigmoid_exact(float z) { return 1.0f / (1.0f + expf(-z)); }

struct RouterArgs {
    const void* logits;
    int64_t ld;
    int64_t T;
    int E, k;
    bool bf16, sigmoid, normalise;
    float scale, aux, z;
    const float* bias;
    // forward
    int* ids;
    float* probs;
    float* part;  // per block: [E] score sums, [E] counts (as int), [1] sum of lse^2
    int* counts;
    float* losses;
    int blocks;
    // backward
    const int* ids_in;
    const int* counts_in;
    const float* dprobs;
    float loss_grad;
    void* dlogits;
    int64_t dld;
};

__device__ __forceinline__ float load_logit(const RouterArgs& a, int64_t t, int e) {
    return a.bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(a.logits)[t * a.ld + e])
                  : static_cast<const float*>(a.logits)[t * a.ld + e];
}

// a row's scores: p[j] = softmax or sigmoid of l[j] (0 where closed); returns the
// log-sum-exp (0 for a row without an open expert); NaN anywhere makes lse NaN.
// wanted: whether the log-sum-exp is needed with sigmoid scores
template <int N>
__device__ __forceinline__ float row_scores(const float (&l)[N], float (&p)[N], bool sigmoid, bool lse_wanted) {
    float lse = 0.0f;
    if (!sigmoid || lse_wanted) {
        float m = -INFINITY;
#pragma unroll
        for (int j = 0; j < N; ++j) m = fmaxf(m, l[j]);  // fmaxf passes over NaN
        m = warp_max(m);
        const float base = m == -INFINITY ? 0.0f : m;
        float z = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            p[j] = expf(l[j] - base);
            z += p[j];
        }
        z = warp_sum(z);
        if (z != 0.0f) {
            lse = base + logf(z);
#pragma unroll
            for (int j = 0; j < N; ++j) p[j] = p[j] / z;
        }
    }
    if (sigmoid) {
#pragma unroll
        for (int j = 0; j < N; ++j) p[j] = sigmoid_exact(l[j]);
    }
    return lse;
}

template <int N>
__global__ void __launch_bounds__(32 * kRouterWarps) router_forward_kernel(RouterArgs a) {
    extern __shared__ float smem[];  // [E] score sums, [E] counts, [warps] z terms
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int* s_counts = reinterpret_cast<int*>(smem);
    float* s_sum = smem + a.E;
    const bool sums = a.counts != nullptr;
    if (sums) {
        for (int i = threadIdx.x; i < a.E; i += blockDim.x) s_counts[i] = 0;
        __syncthreads();
    }
    const bool losses = a.losses != nullptr;
    float psum[N] = {};
    float zsum = 0.0f;
    for (int64_t t = int64_t(blockIdx.x) * kRouterWarps + warp; t < a.T; t += int64_t(gridDim.x) * kRouterWarps) {
        float l[N], p[N];
        bool bad = false;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = lane + 32 * j;
            l[j] = e < a.E ? load_logit(a, t, e) : -INFINITY;
            bad |= isnan(l[j]);
        }
        bad = __any_sync(0xffffffffu, bad);
        const float lse = row_scores<N>(l, p, a.sigmoid, losses);
        if (losses) {
            float total = 1.0f;
            if (a.sigmoid) {
                total = 0.0f;
#pragma unroll
                for (int j = 0; j < N; ++j) total += p[j];
                total = warp_sum(total);
                if (total == 0.0f) total = 1.0f;
            }
#pragma unroll
            for (int j = 0; j < N; ++j) psum[j] += p[j] / total;
            zsum = fmaf(lse, lse, zsum);
        }
        uint32_t key[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const int e = lane + 32 * j;
            key[j] = order_key(l[j]);
            if (a.bias && key[j]) key[j] = order_key(p[j] + a.bias[e]);
        }
        int my_id = -1;
        float my_p = 0.0f;
        for (int s = 0; s < a.k; ++s) {
            uint32_t best = 0;
#pragma unroll
            for (int j = 0; j < N; ++j) best = max(best, key[j]);
            best = __reduce_max_sync(0xffffffffu, best);
            if (best == 0) break;
            uint32_t at = 0xffffffffu;
#pragma unroll
            for (int j = N - 1; j >= 0; --j)
                if (key[j] == best) at = lane + 32 * j;
            at = __reduce_min_sync(0xffffffffu, at);
            float v = 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (lane + 32 * j == int(at)) {
                    v = p[j];
                    key[j] = 0;
                }
            v = __shfl_sync(0xffffffffu, v, at & 31);
            if (lane == s) {
                my_id = int(at);
                my_p = v;
            }
        }
        if (a.normalise) {
            const float total = warp_sum(my_p);
            if (total != 0.0f) my_p = my_p / total;
        }
        if (lane < a.k) {
            a.ids[t * a.k + lane] = my_id;
            a.probs[t * a.k + lane] = bad ? NAN : my_p * a.scale;
            if (sums && my_id >= 0) atomicAdd(s_counts + my_id, 1);
        }
    }
    if (!sums) return;
    // the warps' score sums, added in warp order
    for (int w = 0; w < kRouterWarps && losses; ++w) {
        __syncthreads();
        if (warp == w) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const int e = lane + 32 * j;
                if (e < a.E) s_sum[e] = (w ? s_sum[e] : 0.0f) + psum[j];
            }
            if (lane == 0) s_sum[a.E] = (w ? s_sum[a.E] : 0.0f) + zsum;
        }
    }
    __syncthreads();
    float* part = a.part + int64_t(blockIdx.x) * (2 * a.E + 1);
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) {
        reinterpret_cast<int*>(part)[i] = s_counts[i];
        if (losses) part[a.E + i] = s_sum[i];
    }
    if (threadIdx.x == 0 && losses) part[2 * a.E] = s_sum[a.E];
}

// counts and losses from the blocks' partial sums, in block order
__global__ void __launch_bounds__(1024) router_finish_kernel(RouterArgs a) {
    __shared__ float s_red[32];
    const int e = threadIdx.x;
    const int64_t step = 2 * a.E + 1;
    float term = 0.0f;
    if (e < a.E) {
        int n = 0;
        float p = 0.0f;
        for (int b = 0; b < a.blocks; ++b) {
            n += reinterpret_cast<const int*>(a.part + b * step)[e];
            if (a.losses) p += a.part[b * step + a.E + e];
        }
        a.counts[e] = n;
        term = float(n) * p;
    }
    if (!a.losses) return;
    term = warp_sum(term);
    if ((e & 31) == 0) s_red[e >> 5] = term;
    __syncthreads();
    if (e == 0) {
        float total = 0.0f, z = 0.0f;
        for (int w = 0; w < 32; ++w) total += s_red[w];
        for (int b = 0; b < a.blocks; ++b) z += a.part[b * step + 2 * a.E];
        const float T = float(a.T);
        a.losses[0] = a.T ? a.aux * float(a.E) / (float(a.k) * T) * (total / T) : 0.0f;
        a.losses[1] = a.T ? a.z / T * z : 0.0f;
    }
}

template <int N>
__global__ void __launch_bounds__(32 * kRouterWarps) router_backward_kernel(RouterArgs a) {
    extern __shared__ float smem[];  // per warp: [E] gradients of the chosen scores
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = int64_t(blockIdx.x) * kRouterWarps + warp;
    if (t >= a.T) return;
    float* s_d = smem + warp * a.E;
    const bool aux = a.aux != 0.0f && a.loss_grad != 0.0f;
    const bool zl = a.z != 0.0f && a.loss_grad != 0.0f;
    float l[N], p[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = lane + 32 * j;
        l[j] = e < a.E ? load_logit(a, t, e) : -INFINITY;
        if (e < a.E) s_d[e] = 0.0f;
    }
    const float lse = row_scores<N>(l, p, a.sigmoid, zl);
    __syncwarp();
    int id = lane < a.k ? a.ids_in[t * a.k + lane] : -1;
    if (id >= a.E) id = -1;
    float d = id >= 0 ? a.dprobs[t * a.k + lane] * a.scale : 0.0f;
    float c = 0.0f;
    if (id >= 0) {
        const float v = load_logit(a, t, id);
        c = a.sigmoid ? sigmoid_exact(v) : expf(v - lse);
    }
    if (a.normalise) {
        float total = warp_sum(c);
        if (total == 0.0f) total = 1.0f;
        const float mean = warp_sum(d * (c / total));
        d = id >= 0 ? (d - mean) / total : 0.0f;
    }
    if (id >= 0) s_d[id] = d;
    __syncwarp();
    const float w_aux = aux ? a.loss_grad * a.aux * float(a.E) / (float(a.k) * float(a.T)) / float(a.T) : 0.0f;
    float total = 1.0f;
    if (a.sigmoid && aux) {
        total = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) total += p[j];
        total = warp_sum(total);
        if (total == 0.0f) total = 1.0f;
    }
    // v: gradient of the score (softmax) or of the distribution over the experts (sigmoid)
    float v[N], dot = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = lane + 32 * j;
        v[j] = 0.0f;
        if (e < a.E) {
            v[j] = aux ? w_aux * float(a.counts_in[e]) : 0.0f;
            if (!a.sigmoid) v[j] += s_d[e];
        }
        dot = fmaf(v[j], p[j] / total, dot);
    }
    dot = warp_sum(dot);
    const float w_z = zl ? a.loss_grad * 2.0f * a.z / float(a.T) * lse : 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = lane + 32 * j;
        if (e >= a.E) continue;
        float g;
        if (a.sigmoid)
            g = (s_d[e] + (v[j] - dot) / total) * p[j] * (1.0f - p[j]);
        else
            g = p[j] * (v[j] - dot);
        if (zl) g += w_z * (a.sigmoid ? expf(l[j] - lse) : p[j]);
        if (l[j] == -INFINITY) g = 0.0f;
        if (a.bf16)
            static_cast<__nv_bfloat16*>(a.dlogits)[t * a.dld + e] = __float2bfloat16_rn(g);
        else
            static_cast<float*>(a.dlogits)[t * a.dld + e] = g;
    }
}

moe_status check_router(const moe_router_config* c, int64_t T) {
    if (!c || T < 0 || c->num_experts <= 0 || c->topk <= 0 || c->topk > c->num_experts) return MOE_ERR_INVALID_ARG;
    if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
    if (c->normalise != 0 && c->normalise != 1) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(c->scale) || !std::isfinite(c->aux_coeff) || !std::isfinite(c->z_coeff))
        return MOE_ERR_INVALID_ARG;
    if (c->x_type != MOE_T_BF16 && c->x_type != MOE_T_FP32) return MOE_ERR_INVALID_ARG;
    if (c->num_experts > 1024 || c->topk > 32 || T > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

int router_blocks(int64_t T) {
    const int64_t b = (T + kRouterWarps - 1) / kRouterWarps;
    return int(b < 1 ? 1 : b > kRouterBlocks ? kRouterBlocks : b);
}

RouterArgs router_args(const moe_router_config* c, int64_t T, const void* logits, int64_t ld) {
    RouterArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.T = T;
    a.E = int(c->num_experts);
    a.k = int(c->topk);
    a.bf16 = c->x_type == MOE_T_BF16;
    a.sigmoid = c->score == MOE_SCORE_SIGMOID;
    a.normalise = c->normalise != 0;
    a.scale = c->scale;
    a.aux = c->aux_coeff;
    a.z = c->z_coeff;
    return a;
}

template <typename F>
void by_experts(int E, F f) {
    if (E <= 32) f(std::integral_constant<int, 1>());
    else if (E <= 64) f(std::integral_constant<int, 2>());
    else if (E <= 128) f(std::integral_constant<int, 4>());
    else if (E <= 256) f(std::integral_constant<int, 8>());
    else if (E <= 512) f(std::integral_constant<int, 16>());
    else f(std::integral_constant<int, 32>());
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

}  // namespace

}  // namespace moe

extern "C" {

moe_status moe_router_size(const moe_router_config* cfg, int64_t T, size_t* bytes) {
    using namespace moe;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = 0;
    const moe_status st = check_router(cfg, T);
    if (st != MOE_OK) return st;
    *bytes = size_t(router_blocks(T)) * size_t(2 * cfg->num_experts + 1) * sizeof(float);
    return MOE_OK;
}

moe_status moe_router_forward(const moe_router_config* cfg, int64_t T, const void* logits, int64_t logits_stride,
                              const float* select_bias, int32_t* ids, float* probs, int32_t* counts, float* losses,
                              void* workspace, size_t workspace_bytes, void* stream) {
    using namespace moe;
    size_t need = 0;
    const moe_status st = moe_router_size(cfg, T, &need);
    if (st != MOE_OK) return st;
    if (logits_stride < cfg->num_experts || (losses && !counts)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!logits || !ids || !probs)) return MOE_ERR_INVALID_ARG;
    if (!aligned_to(logits, cfg->x_type == MOE_T_BF16 ? 2 : 4) || !aligned_to(ids, 4) || !aligned_to(probs, 4) ||
        !aligned_to(counts, 4) || !aligned_to(losses, 4) || !aligned_to(select_bias, 4))
        return MOE_ERR_INVALID_ARG;
    if (counts && (!workspace || workspace_bytes < need || !aligned_to(workspace, 256))) return MOE_ERR_INVALID_ARG;
    RouterArgs a = router_args(cfg, T, logits, logits_stride);
    a.bias = select_bias;
    a.ids = ids;
    a.probs = probs;
    a.part = static_cast<float*>(workspace);
    a.counts = counts;
    a.losses = losses;
    a.blocks = router_blocks(T);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (T == 0) a.blocks = 0;
    if (T > 0) {
        const size_t smem = (2 * size_t(a.E) + 1) * sizeof(float);
        by_experts(a.E, [&](auto n) {
            router_forward_kernel<decltype(n)::value><<<a.blocks, 32 * kRouterWarps, smem, s>>>(a);
        });
        count_launch();
        if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    }
    if (counts) {
        router_finish_kernel<<<1, 1024, 0, s>>>(a);
        count_launch();
    }
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_router_backward(const moe_router_config* cfg, int64_t T, const void* logits, int64_t logits_stride,
                               const int32_t* ids, const float* dprobs, const int32_t* counts, float loss_grad,
                               void* dlogits, int64_t dlogits_stride, void* stream) {
    using namespace moe;
    const moe_status st = check_router(cfg, T);
    if (st != MOE_OK) return st;
    if (logits_stride < cfg->num_experts || dlogits_stride < cfg->num_experts || !std::isfinite(loss_grad))
        return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!logits || !ids || !dprobs || !dlogits) return MOE_ERR_INVALID_ARG;
    if (cfg->aux_coeff != 0.0f && loss_grad != 0.0f && !counts) return MOE_ERR_INVALID_ARG;
    const size_t es = cfg->x_type == MOE_T_BF16 ? 2 : 4;
    if (!aligned_to(logits, es) || !aligned_to(dlogits, es) || !aligned_to(ids, 4) || !aligned_to(dprobs, 4) ||
        !aligned_to(counts, 4))
        return MOE_ERR_INVALID_ARG;
    RouterArgs a = router_args(cfg, T, logits, logits_stride);
    a.ids_in = ids;
    a.counts_in = counts;
    a.dprobs = dprobs;
    a.loss_grad = loss_grad;
    a.dlogits = dlogits;
    a.dld = dlogits_stride;
    const int64_t blocks = (T + kRouterWarps - 1) / kRouterWarps;
    const size_t smem = size_t(kRouterWarps) * size_t(a.E) * sizeof(float);
    by_experts(a.E, [&](auto n) {
        router_backward_kernel<decltype(n)::value>
            <<<unsigned(blocks), 32 * kRouterWarps, smem, static_cast<cudaStream_t>(stream)>>>(a);
    });
    count_launch();
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
