// Layer norm and RMS norm of the rows in front of the expert layer, forward and
// backward, with the residual add before the norm and the residual stream's
// gradient after it.
//
// Forward: s = x + r (rounded to the stream's type, which is what later layers
// read), mean = sum(s)/H, var = sum((s - mean)^2)/H, y = (s - mean) rstd w + b.
// Backward, with g = w dy and xhat = (s - mean) rstd:
//   dx = rstd (g - sum(g)/H - xhat sum(g xhat)/H) + dsum,
//   dw = sum_t dy xhat, db = sum_t dy.
// All statistics and sums are fp32.
#include <cmath>
#include <type_traits>

#include "../../include/moe.h"
#include "device_common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kMaxHidden = 32768;
constexpr int kMaxChunks = 304;  // row chunks of the weight gradient's sums

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ float round_to(float v, const float*) { return v; }
__device__ __forceinline__ float round_to(float v, const __nv_bfloat16*) {
    return __bfloat162float(__float2bfloat16_rn(v));
}
// weight and bias come in either type; the row's sums dominate, so their type is a run-time branch
__device__ __forceinline__ float load_w(const void* p, int64_t i, bool bf16) {
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]) : static_cast<const float*>(p)[i];
}

// sum over the block's threads, in an order fixed by the block size; every thread gets it
__device__ float block_sum(float v) {
    __shared__ float part[33];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        float t = threadIdx.x < (blockDim.x >> 5) ? part[threadIdx.x] : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (threadIdx.x == 0) part[32] = t;
    }
    __syncthreads();
    return part[32];
}

struct NormFwd {
    const void *x, *r, *w, *b;
    void *s, *y;
    float *mean, *rstd;
    int64_t xs, rs, ss, ys;
    int H;
    float eps;
    bool w_bf16;
};

template <typename XT, typename YT, bool RMS>
__global__ void __launch_bounds__(256) norm_forward_kernel(NormFwd a) {
    const int64_t t = blockIdx.x;
    const XT* x = static_cast<const XT*>(a.x) + t * a.xs;
    const XT* r = a.r ? static_cast<const XT*>(a.r) + t * a.rs : nullptr;
    XT* s = static_cast<XT*>(a.s) + t * a.ss;
    YT* y = static_cast<YT*>(a.y) + t * a.ys;
    auto value = [&](int i) {
        const float v = load_f(x + i);
        return r ? round_to(v + load_f(r + i), x) : v;
    };
    float sum = 0.0f;
    if (!RMS) {
        for (int i = threadIdx.x; i < a.H; i += blockDim.x) sum += value(i);
        sum = block_sum(sum);
    }
    const float mean = RMS ? 0.0f : sum / a.H;
    float sq = 0.0f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float d = value(i) - mean;
        sq = fmaf(d, d, sq);
    }
    sq = block_sum(sq);
    const float rstd = rsqrtf(sq / a.H + a.eps);
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float v = value(i);
        float o = (v - mean) * rstd * load_w(a.w, i, a.w_bf16);
        if (a.b) o += load_w(a.b, i, a.w_bf16);
        if (r) store_f(s + i, v);
        store_f(y + i, o);
    }
    if (threadIdx.x == 0) {
        if (!RMS && a.mean) a.mean[t] = mean;
        if (a.rstd) a.rstd[t] = rstd;
    }
}

struct NormBwd {
    const void *dy, *x, *w, *ds;
    const float *mean, *rstd;
    void* dx;
    float* part;  // [chunks][2][H]: dweight, dbias of a chunk of rows
    int64_t dys, xs, dss, dxs;
    int64_t T;
    int H;
    int chunks;
    bool w_bf16, want_w, want_b;
};

template <typename XT, typename YT, bool RMS>
__global__ void __launch_bounds__(256) norm_backward_kernel(NormBwd a) {
    const int64_t t = blockIdx.x;
    const YT* dy = static_cast<const YT*>(a.dy) + t * a.dys;
    const XT* x = static_cast<const XT*>(a.x) + t * a.xs;
    const XT* ds = a.ds ? static_cast<const XT*>(a.ds) + t * a.dss : nullptr;
    XT* dx = static_cast<XT*>(a.dx) + t * a.dxs;
    const float mean = RMS ? 0.0f : a.mean[t];
    const float rstd = a.rstd[t];
    float sg = 0.0f, sgx = 0.0f;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float g = load_f(dy + i) * load_w(a.w, i, a.w_bf16);
        const float xh = (load_f(x + i) - mean) * rstd;
        sg += g;
        sgx = fmaf(g, xh, sgx);
    }
    const float mg = RMS ? 0.0f : block_sum(sg) / a.H;
    const float mgx = block_sum(sgx) / a.H;
    for (int i = threadIdx.x; i < a.H; i += blockDim.x) {
        const float g = load_f(dy + i) * load_w(a.w, i, a.w_bf16);
        const float xh = (load_f(x + i) - mean) * rstd;
        float o = rstd * (g - mg - xh * mgx);
        if (ds) o += load_f(ds + i);
        store_f(dx + i, o);
    }
}

// part[c] = sums of chunk c's rows (c, c + chunks, ...) over dy xhat and dy; a thread owns a column
template <typename XT, typename YT, bool RMS>
__global__ void __launch_bounds__(256) norm_wgrad_kernel(NormBwd a) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= a.H) return;
    float dw = 0.0f, db = 0.0f;
    for (int64_t t = blockIdx.y; t < a.T; t += a.chunks) {
        const float d = load_f(static_cast<const YT*>(a.dy) + t * a.dys + i);
        const float xh = (load_f(static_cast<const XT*>(a.x) + t * a.xs + i) - (RMS ? 0.0f : a.mean[t])) * a.rstd[t];
        dw = fmaf(d, xh, dw);
        db += d;
    }
    float* p = a.part + int64_t(blockIdx.y) * 2 * a.H;
    p[i] = dw;
    p[a.H + i] = db;
}

__device__ __forceinline__ void put_grad(void* g, int i, float v, bool bf16, bool add) {
    if (bf16) {
        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(g) + i;
        const __nv_bfloat16 d = __float2bfloat16_rn(v);
        *p = add ? __float2bfloat16_rn(__bfloat162float(*p) + __bfloat162float(d)) : d;
    } else {
        float* p = static_cast<float*>(g) + i;
        *p = add ? *p + v : v;
    }
}

// dweight, dbias from the chunks' sums, in chunk order
__global__ void __launch_bounds__(256) norm_wgrad_reduce_kernel(const float* __restrict__ part, int chunks, int H,
                                                                void* dw, void* db, bool bf16, bool add) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= H) return;
    float w = 0.0f, b = 0.0f;
    for (int c = 0; c < chunks; ++c) {
        w += part[int64_t(c) * 2 * H + i];
        b += part[int64_t(c) * 2 * H + H + i];
    }
    if (dw) put_grad(dw, i, w, bf16, add);
    if (db) put_grad(db, i, b, bf16, add);
}

int norm_chunks(int64_t T) { return int(T < kMaxChunks ? (T < 1 ? 1 : T) : kMaxChunks); }

moe_status check_norm(const moe_norm_config* c, int64_t T) {
    if (!c || T < 0 || c->hidden <= 0) return MOE_ERR_INVALID_ARG;
    if (!(c->eps >= 0.0f) || !std::isfinite(c->eps)) return MOE_ERR_INVALID_ARG;
    if (c->kind != MOE_NORM_LAYER && c->kind != MOE_NORM_RMS) return MOE_ERR_INVALID_ARG;
    for (int32_t t : {c->x_type, c->y_type, c->w_type})
        if (t != MOE_T_BF16 && t != MOE_T_FP32) return MOE_ERR_INVALID_ARG;
    if (c->hidden > kMaxHidden || T > INT32_MAX) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool elem_aligned(const void* p, int32_t type) {
    return (reinterpret_cast<uintptr_t>(p) & (type == MOE_T_BF16 ? 1 : 3)) == 0;
}

template <typename F>
cudaError_t by_type(const moe_norm_config& c, F f) {
    const bool rms = c.kind == MOE_NORM_RMS;
    using B = __nv_bfloat16;
    if (c.x_type == MOE_T_BF16)
        return c.y_type == MOE_T_BF16 ? (rms ? f(B(), B(), std::true_type()) : f(B(), B(), std::false_type()))
                                      : (rms ? f(B(), 0.0f, std::true_type()) : f(B(), 0.0f, std::false_type()));
    return c.y_type == MOE_T_BF16 ? (rms ? f(0.0f, B(), std::true_type()) : f(0.0f, B(), std::false_type()))
                                  : (rms ? f(0.0f, 0.0f, std::true_type()) : f(0.0f, 0.0f, std::false_type()));
}

}  // namespace

}  // namespace moe

extern "C" {

moe_status moe_norm_forward(const moe_norm_config* cfg, int64_t T, const void* x, int64_t x_stride,
                            const void* residual, int64_t residual_stride, const void* weight, const void* bias,
                            void* sum, int64_t sum_stride, void* y, int64_t y_stride, float* mean, float* rstd,
                            void* stream) {
    using namespace moe;
    const moe_status st = check_norm(cfg, T);
    if (st != MOE_OK) return st;
    const int64_t H = cfg->hidden;
    if (x_stride < H || y_stride < H || (residual && (residual_stride < H || sum_stride < H)))
        return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!x || !y || !weight || (residual && !sum)) return MOE_ERR_INVALID_ARG;
    if (!elem_aligned(x, cfg->x_type) || !elem_aligned(y, cfg->y_type) || !elem_aligned(weight, cfg->w_type) ||
        !elem_aligned(bias, cfg->w_type) || !elem_aligned(residual, cfg->x_type) || !elem_aligned(mean, MOE_T_FP32) ||
        !elem_aligned(rstd, MOE_T_FP32) || (residual && !elem_aligned(sum, cfg->x_type)))
        return MOE_ERR_INVALID_ARG;
    NormFwd a{x, residual, weight, bias, sum, y, mean, rstd, x_stride, residual_stride, sum_stride, y_stride,
              int(H), cfg->eps, cfg->w_type == MOE_T_BF16};
    const cudaError_t e = by_type(*cfg, [&](auto xt, auto yt, auto rms) {
        norm_forward_kernel<decltype(xt), decltype(yt), decltype(rms)::value>
            <<<unsigned(T), 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
        return cudaGetLastError();
    });
    count_launch();
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_norm_backward_size(const moe_norm_config* cfg, int64_t T, size_t* bytes) {
    using namespace moe;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = 0;
    const moe_status st = check_norm(cfg, T);
    if (st != MOE_OK) return st;
    *bytes = size_t(norm_chunks(T)) * 2 * size_t(cfg->hidden) * sizeof(float);
    return MOE_OK;
}

moe_status moe_norm_backward(const moe_norm_config* cfg, int64_t T, const void* dy, int64_t dy_stride,
                             const void* x, int64_t x_stride, const void* weight, const float* mean,
                             const float* rstd, const void* dsum, int64_t dsum_stride, void* dx, int64_t dx_stride,
                             void* dweight, void* dbias, int32_t g_type, int32_t accumulate, void* workspace,
                             size_t workspace_bytes, void* stream) {
    using namespace moe;
    size_t need = 0;
    moe_status st = moe_norm_backward_size(cfg, T, &need);
    if (st != MOE_OK) return st;
    const int64_t H = cfg->hidden;
    if (dy_stride < H || x_stride < H || dx_stride < H || (dsum && dsum_stride < H)) return MOE_ERR_INVALID_ARG;
    if ((g_type != MOE_G_FP32 && g_type != MOE_G_BF16) || (accumulate != 0 && accumulate != 1))
        return MOE_ERR_INVALID_ARG;
    const bool sums = dweight || dbias;
    if (sums && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255)))
        return MOE_ERR_INVALID_ARG;
    const int32_t gt = g_type == MOE_G_BF16 ? MOE_T_BF16 : MOE_T_FP32;
    if (!elem_aligned(dweight, gt) || !elem_aligned(dbias, gt)) return MOE_ERR_INVALID_ARG;
    if (T > 0 && (!dy || !x || !weight || !rstd || !dx || (cfg->kind == MOE_NORM_LAYER && !mean)))
        return MOE_ERR_INVALID_ARG;
    if (!elem_aligned(dy, cfg->y_type) || !elem_aligned(x, cfg->x_type) || !elem_aligned(dx, cfg->x_type) ||
        !elem_aligned(dsum, cfg->x_type) || !elem_aligned(weight, cfg->w_type) || !elem_aligned(mean, MOE_T_FP32) ||
        !elem_aligned(rstd, MOE_T_FP32))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int chunks = T == 0 ? 0 : norm_chunks(T);
    NormBwd a{dy, x, weight, dsum, mean, rstd, dx, static_cast<float*>(workspace), dy_stride, x_stride, dsum_stride,
              dx_stride, T, int(H), chunks, cfg->w_type == MOE_T_BF16, dweight != nullptr, dbias != nullptr};
    cudaError_t e = cudaSuccess;
    if (T > 0) {
        e = by_type(*cfg, [&](auto xt, auto yt, auto rms) {
            using X = decltype(xt);
            using Y = decltype(yt);
            constexpr bool R = decltype(rms)::value;
            norm_backward_kernel<X, Y, R><<<unsigned(T), 256, 0, s>>>(a);
            if (sums) norm_wgrad_kernel<X, Y, R><<<dim3(unsigned((H + 255) / 256), unsigned(chunks)), 256, 0, s>>>(a);
            return cudaGetLastError();
        });
        count_launch(sums ? 2 : 1);
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    if (sums) {
        norm_wgrad_reduce_kernel<<<unsigned((H + 255) / 256), 256, 0, s>>>(
            static_cast<const float*>(workspace), chunks, int(H), dweight, dbias, g_type == MOE_G_BF16,
            accumulate != 0);
        e = cudaGetLastError();
        count_launch();
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
