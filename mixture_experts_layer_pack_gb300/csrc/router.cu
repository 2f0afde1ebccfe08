// The router's choice of experts from its logits, forward and backward, with the
// balancing losses.
//
// A warp owns a row (a token): lane l holds the logits of experts l, l + 32, ...
// With m the row's largest logit and z = sum_e exp(l_e - m): softmax scores
// exp(l_e - m) / z, log-sum-exp m + log z; sigmoid scores 1 / (1 + exp(-l_e)).
// The choice compares logits, mapped to unsigned integers of the same order, one
// warp-wide maximum and one warp-wide minimum index per slot: exact, ties to the
// lower id, whatever the scores round to.
// Sigmoid scores come from exp(-|l|) alike: the smaller of score and 1 - score is right to its last bits, and so are both.
//
// Bound by the instructions of the choice, not by memory: 16384 x 128 fp32, k 8, 12 us, with counts 16, with the losses
// 20 us (0.5 TB/s); 16384 x 384, k 6, 23, 28 and 33 us; the backward with losses, sigmoid, at 8192 x 384 10.5 us
// (2.4 TB/s), softmax at 16384 x 128 8.2 us (2.2 TB/s).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "../../include/moe.h"
#include "device_common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kRouterWarps = 8;     // of a block of the backward
// most blocks of the forward, each with its own partial sums: two per SM (a block for every few rows instead: 16384 x 128
// k 8 without counts 12.7 us, not 12.1; 16384 x 512 40 us, not 37)
constexpr int kRouterBlocks = 304;
// warps of a block of the forward for rows of 32 n experts: as many as the registers of two blocks an SM allow
constexpr int forward_warps(int n) { return n <= 4 ? 24 : n <= 8 ? 16 : n <= 12 ? 12 : n <= 16 ? 10 : 6; }

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

// order-preserving map of a float to an unsigned, and back; 0 is kept for what cannot be chosen
// (-inf and NaN), both zeros get one key
__device__ __forceinline__ uint32_t order_key(float v) {
    if (!(v > -INFINITY)) return 0u;
    const uint32_t b = __float_as_uint(v + 0.0f);
    return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
    return __uint_as_float((key & 0x80000000u) ? key & 0x7fffffffu : ~key);
}

// quotients by the hardware reciprocal: 1 ulp, a quarter of a rounded division's time
__device__ __forceinline__ float reciprocal(float v) { return __fdividef(1.0f, v); }
// the smaller of sigmoid(z) and 1 - sigmoid(z), exp(-|z|) / (1 + exp(-|z|)): nothing overflows, and both are right to the
// last bits at either end, down to the smallest that fp32 holds
__device__ __forceinline__ float sigmoid_tail(float z) {
    const float e = expf(-fabsf(z));
    return e * reciprocal(1.0f + e);
}
__device__ __forceinline__ float sigmoid_of(float z, float tail) { return z < 0.0f ? tail : 1.0f - tail; }
__device__ __forceinline__ float sigmoid(float z) { return sigmoid_of(z, sigmoid_tail(z)); }

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
    float* part;    // per block: [E] counts (as int), [E] score sums, [1] sum of lse^2
    float* finish;  // see router_finish_kernel
    int* counts;
    float* losses;
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
template <int N>
__device__ __forceinline__ void load_row(const RouterArgs& a, int64_t t, float (&l)[N]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int j = 0; j < N; ++j) l[j] = lane + 32 * j < a.E ? load_logit(a, t, lane + 32 * j) : -INFINITY;
}

// A row's log-sum-exp parts: its largest logit m (0 for a row without an open expert), q[j] = exp(l[j] - m),
// 1 / z with z = sum q (0 for such a row), and the log-sum-exp m + log z (0). NaN anywhere makes z NaN.
struct RowSums {
    float m, rz, lse;
};
template <int N>
__device__ __forceinline__ RowSums row_exp(const float (&l)[N], float (&q)[N]) {
    RowSums r;
    r.m = -INFINITY;
#pragma unroll
    for (int j = 0; j < N; ++j) r.m = fmaxf(r.m, l[j]);  // fmaxf passes over NaN
    r.m = warp_max(r.m);
    if (r.m == -INFINITY) r.m = 0.0f;
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        q[j] = expf(l[j] - r.m);
        z += q[j];
    }
    z = warp_sum(z);
    const bool none = z == 0.0f;
    r.rz = none ? 0.0f : reciprocal(z);
    r.lse = none ? 0.0f : r.m + logf(z);
    return r;
}

// The share of a lane's chosen score in the sum of all of them (0 for a lane without one); `l`: its logit. A bias may choose
// scores whose sum has no reciprocal, or that are too small for their ratio to be right: such rows take the exponents'
// differences from the largest chosen logit, whose sum is 1 at least. (A sigmoid that small is exp(l).) Past kNoScore a
// sigmoid counts as 0, as it does with 64 bits, and there is nothing to divide by.
constexpr float kNoScore = -700.0f;
__device__ __forceinline__ float share_of(float score, float l, bool chosen, bool sigmoid) {
    float total = warp_sum(score);
    if (total < 1e-30f) {  // the same in every lane; a NaN passes
        const float top = warp_max(chosen ? l : -INFINITY);
        score = !chosen || (sigmoid && top < kNoScore) ? 0.0f : expf(l - top);
        total = warp_sum(score);
        if (total == 0.0f) return 0.0f;
    }
    return score * reciprocal(total);
}

// losses from the sums over the experts (counts times score sums) and over the tokens (log-sum-exp squared)
__device__ __forceinline__ void put_losses(const RouterArgs& a, float total, float z) {
    const float T = float(a.T);
    a.losses[0] = a.T ? a.aux * float(a.E) / (float(a.k) * T) * (total / T) : 0.0f;
    a.losses[1] = a.T ? a.z / T * z : 0.0f;
}

// A lane's keys, from which its best is taken again and again. Up to four are sorted once (stable: equal keys stay in
// the order of their experts), and the next is a shift away; more are looked through when their best goes. 16384 x 128
// with k 8 and losses: 20.4 us sorted, 23.1 looked through.
template <int N>
struct LaneKeys {
    uint32_t key[N];
    uint32_t b;
    int place;  // N <= 4: the places in order, a byte each
    __device__ __forceinline__ explicit LaneKeys(const uint32_t (&k)[N]) {
#pragma unroll
        for (int j = 0; j < N; ++j) key[j] = k[j];
        if constexpr (N <= 4) {
            uint32_t at[N];
#pragma unroll
            for (int j = 0; j < N; ++j) at[j] = j;
#pragma unroll
            for (int end = N - 1; end > 0; --end)
#pragma unroll
                for (int j = 0; j < end; ++j) {
                    const bool swap = key[j] < key[j + 1];
                    const uint32_t hi = max(key[j], key[j + 1]), lo = min(key[j], key[j + 1]);
                    const uint32_t first = swap ? at[j + 1] : at[j];
                    at[j + 1] = swap ? at[j] : at[j + 1];
                    at[j] = first;
                    key[j] = hi;
                    key[j + 1] = lo;
                }
            place = 0;
#pragma unroll
            for (int j = 0; j < N; ++j) place |= at[j] << (8 * j);
        } else {
            place = -1;
            look();
        }
    }
    __device__ __forceinline__ uint32_t best() const { return N <= 4 ? key[0] : b; }
    __device__ __forceinline__ int at() const { return N <= 4 ? place & 255 : place; }
    __device__ __forceinline__ void next() {
        if constexpr (N <= 4) {
#pragma unroll
            for (int j = 0; j + 1 < N; ++j) key[j] = key[j + 1];
            key[N - 1] = 0;
            place = int(uint32_t(place) >> 8);
        } else {
            look();
        }
    }
    // the best without the one at `place`
    __device__ __forceinline__ void look() {
        b = 0;
        int found = 0;
#pragma unroll
        for (int j = N - 1; j >= 0; --j) {
            if (j == place) key[j] = 0;
            if (key[j] >= b) {
                b = key[j];
                found = j;
            }
        }
        place = found;
    }
};

template <int N>
__global__ void __launch_bounds__(32 * forward_warps(N)) router_forward_kernel(RouterArgs a) {
    constexpr int kWarps = forward_warps(N);
    __shared__ float s_z[kWarps];
    extern __shared__ float smem[];  // [E] counts, [warps][E] score sums
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int* s_counts = reinterpret_cast<int*>(smem);
    float* s_sum = smem + a.E;
    const bool sums = a.counts != nullptr, losses = a.losses != nullptr;
    float psum[N] = {};
    float zsum = 0.0f;
    const int64_t step = int64_t(gridDim.x) * kWarps;
    // a block's rows lie gridDim apart: the last round's fall to every block, not to the first ones' warps
    int64_t t = int64_t(warp) * gridDim.x + blockIdx.x;
    float ahead[N];  // the next row, under way during this one
    if (t < a.T) load_row<N>(a, t, ahead);
    if (threadIdx.x == 0 && blockIdx.x == 0 && losses) reinterpret_cast<unsigned*>(a.finish)[0] = 0;
    if (sums) {
        for (int i = threadIdx.x; i < a.E; i += blockDim.x) s_counts[i] = 0;
        __syncthreads();
    }
    for (; t < a.T; t += step) {
        float l[N], p[N];
        bool bad = false;
#pragma unroll
        for (int j = 0; j < N; ++j) {
            l[j] = ahead[j];
            bad |= isnan(l[j]);
        }
        if (t + step < a.T) load_row<N>(a, t + step, ahead);
        bad = __any_sync(0xffffffffu, bad);
        RowSums r{0.0f, 0.0f, 0.0f};
        if (!a.sigmoid || losses) r = row_exp<N>(l, p);
        float rp = r.rz;  // a score's distribution over the experts: p * rp
        if (a.sigmoid && (losses || a.bias)) {
            float total = 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                p[j] = sigmoid(l[j]);
                total += p[j];
            }
            if (losses) {
                total = warp_sum(total);
                rp = total == 0.0f ? 0.0f : reciprocal(total);
            }
        }
        if (losses) {
#pragma unroll
            for (int j = 0; j < N; ++j) psum[j] = fmaf(p[j], rp, psum[j]);
            zsum = fmaf(r.lse, r.lse, zsum);
        }
        uint32_t key[N];
#pragma unroll
        for (int j = 0; j < N; ++j) key[j] = order_key(l[j]);
        // a NaN, or +inf, leaves no softmax score of the row a number: its order stays the logits', and the chosen experts
        // carry the NaN on in their probs
        const float rk = a.sigmoid ? 1.0f : r.rz;
        if (a.bias && !isnan(rk)) {
#pragma unroll
            for (int j = 0; j < N; ++j)
                if (key[j]) key[j] = order_key(p[j] * rk + a.bias[lane + 32 * j]);
        }
        LaneKeys<N> mine(key);
        int my_id = -1;
        uint32_t my_key = 0;
        for (int s = 0; s < a.k; ++s) {
            const uint32_t top = __reduce_max_sync(0xffffffffu, mine.best());
            if (top == 0) break;
            const uint32_t here = uint32_t(lane + 32 * mine.at());
            const uint32_t id = __reduce_min_sync(0xffffffffu, mine.best() == top ? here : 0xffffffffu);
            if (lane == s) {
                my_id = int(id);
                my_key = top;
            }
            if (here == id) mine.next();  // a lane whose best is not the top has another place
        }
        // the chosen scores, one a lane: from the logit, which the key still is (not with a bias)
        float my_l = value_of(my_key);
        if (a.bias && my_id >= 0) my_l = load_logit(a, t, my_id);
        float my_p = my_id < 0 ? 0.0f : a.sigmoid ? sigmoid(my_l) : expf(my_l - r.m) * r.rz;
        if (a.normalise) my_p = share_of(my_p, my_l, my_id >= 0, a.sigmoid);
        if (lane < a.k) {
            a.ids[t * a.k + lane] = my_id;
            a.probs[t * a.k + lane] = bad ? NAN : my_p * a.scale;
            if (sums && my_id >= 0) atomicAdd(s_counts + my_id, 1);  // integers: any order
        }
    }
    if (!sums) return;
    // the warps' score sums, added in warp order
    if (losses) {
#pragma unroll
        for (int j = 0; j < N; ++j)
            if (lane + 32 * j < a.E) s_sum[warp * a.E + lane + 32 * j] = psum[j];
        if (lane == 0) s_z[warp] = zsum;
    }
    __syncthreads();
    if (losses) {
        for (int i = threadIdx.x; i < a.E; i += blockDim.x) {
            float v = s_sum[i];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) v += s_sum[w * a.E + i];
            s_sum[i] = v;
        }
        if (warp == 0) zsum = warp_sum(lane < kWarps ? s_z[lane] : 0.0f);
    }
    __syncthreads();
    if (gridDim.x == 1) {  // nothing to add up with
        float term = 0.0f;
        for (int i = threadIdx.x; i < a.E; i += blockDim.x) {
            a.counts[i] = s_counts[i];
            if (losses) term = fmaf(float(s_counts[i]), s_sum[i], term);
        }
        if (losses) {
            term = warp_sum(term);
            if (lane == 0) s_z[warp] = term;
            __syncthreads();
            if (threadIdx.x == 0) {
                for (int w = 1; w < kWarps; ++w) term += s_z[w];
                put_losses(a, term, zsum);
            }
        }
        return;
    }
    float* part = a.part + int64_t(blockIdx.x) * (2 * a.E + 1);
    for (int i = threadIdx.x; i < a.E; i += blockDim.x) {
        reinterpret_cast<int*>(part)[i] = s_counts[i];
        if (losses) part[a.E + i] = s_sum[i];
    }
    if (threadIdx.x == 0 && losses) part[2 * a.E] = zsum;
}

// Counts and losses from the blocks' partial sums. Block g: 32 experts, warp w adding the blocks w,
// w + 32, ... in order, then the warps' sums in warp order; block 0 the z terms too. The block that
// finishes last adds up the experts' parts of the balance loss, in block order.
// a.finish: [0] blocks done (0 at the start), [1] z, [2 + g] block g's part.
constexpr int kFinishWarps = 32;
__global__ void __launch_bounds__(32 * kFinishWarps) router_finish_kernel(RouterArgs a, int blocks) {
    __shared__ int s_n[kFinishWarps][32];
    __shared__ float s_p[kFinishWarps][32];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e = blockIdx.x * 32 + lane;
    const int64_t step = 2 * a.E + 1;
    int n = 0;
    float p = 0.0f;
    if (e < a.E) {
        const float* from = a.part + e;
#pragma unroll 10
        for (int b = warp; b < blocks; b += kFinishWarps) {
            n += reinterpret_cast<const int*>(from)[b * step];
            if (a.losses) p += from[b * step + a.E];
        }
    }
    s_n[warp][lane] = n;
    s_p[warp][lane] = p;
    __syncthreads();
    if (blockIdx.x == 0 && a.losses && warp == 1) {  // lane l: blocks l, l + 32, ...
        float z = 0.0f;
#pragma unroll 10
        for (int b = lane; b < blocks; b += 32) z += a.part[b * step + 2 * a.E];
        z = warp_sum(z);
        if (lane == 0) {
            a.finish[1] = z;
            __threadfence();
        }
    }
    __syncthreads();
    if (warp) return;
#pragma unroll
    for (int w = 1; w < kFinishWarps; ++w) {
        n += s_n[w][lane];
        p += s_p[w][lane];
    }
    if (e < a.E) a.counts[e] = n;
    if (!a.losses) return;
    const float term = warp_sum(e < a.E ? float(n) * p : 0.0f);
    if (lane) return;
    a.finish[2 + blockIdx.x] = term;
    __threadfence();
    if (atomicAdd(reinterpret_cast<unsigned*>(a.finish), 1u) != gridDim.x - 1) return;
    __threadfence();
    float total = 0.0f;
    for (unsigned g = 0; g < gridDim.x; ++g) total += __ldcg(a.finish + 2 + g);
    put_losses(a, total, __ldcg(a.finish + 1));
}

template <int N>
__global__ void __launch_bounds__(32 * kRouterWarps) router_backward_kernel(RouterArgs a) {
    extern __shared__ float smem[];  // per warp: [E] gradients of the chosen scores, or with shares of the chosen logits
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = int64_t(blockIdx.x) * kRouterWarps + warp;
    if (t >= a.T) return;
    float* s_d = smem + warp * a.E;
    const bool aux = a.aux != 0.0f && a.loss_grad != 0.0f;
    const bool zl = a.z != 0.0f && a.loss_grad != 0.0f;
    float l[N], q[N];
    load_row<N>(a, t, l);
    int id = lane < a.k ? a.ids_in[t * a.k + lane] : -1;
    if (id >= a.E) id = -1;
    float d = id >= 0 ? a.dprobs[t * a.k + lane] * a.scale : 0.0f;
    const float my_l = id >= 0 ? load_logit(a, t, id) : 0.0f;
#pragma unroll
    for (int j = 0; j < N; ++j)
        if (lane + 32 * j < a.E) s_d[lane + 32 * j] = 0.0f;
    RowSums r{0.0f, 0.0f, 0.0f};
    if (!a.sigmoid || zl) r = row_exp<N>(l, q);
    __syncwarp();
    const float tail = a.sigmoid ? sigmoid_tail(my_l) : 0.0f;
    const float c = id < 0 ? 0.0f : a.sigmoid ? sigmoid_of(my_l, tail) : expf(my_l - r.m) * r.rz;
    if (a.normalise) {  // of shares: softmax share (d - mean), sigmoid the same times 1 - score; nothing to divide by
        const float share = share_of(c, my_l, id >= 0, a.sigmoid);
        const float mean = warp_sum(d * share);
        d = share * (d - mean) * (a.sigmoid ? sigmoid_of(-my_l, tail) : 1.0f);
    }
    if (id >= 0) s_d[id] = d;
    __syncwarp();
    const float w_aux = aux ? a.loss_grad * a.aux * float(a.E) / (float(a.k) * float(a.T)) / float(a.T) : 0.0f;
    const float w_z = zl ? a.loss_grad * 2.0f * a.z / float(a.T) * r.lse * r.rz : 0.0f;  // times exp(l - m)
    float g[N];
    if (a.sigmoid) {
        float tails[N], rp = 0.0f, dot = 0.0f;
#pragma unroll
        for (int j = 0; j < N; ++j) tails[j] = sigmoid_tail(l[j]);
        if (aux) {
            // with P = p / sum(p): gradient (w - sum(w P)) / sum(p) of the balance loss at each score
            float total = 0.0f, wp = 0.0f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                g[j] = lane + 32 * j < a.E ? w_aux * float(a.counts_in[lane + 32 * j]) : 0.0f;
                const float p = sigmoid_of(l[j], tails[j]);
                total += p;
                wp = fmaf(g[j], p, wp);
            }
            total = warp_sum(total);
            rp = total == 0.0f ? 1.0f : reciprocal(total);
            dot = warp_sum(wp) * rp;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            if (lane + 32 * j >= a.E) continue;
            const float own = s_d[lane + 32 * j];
            const float v = (a.normalise ? 0.0f : own) + (aux ? (g[j] - dot) * rp : 0.0f);
            g[j] = fmaf(v, tails[j] * (1.0f - tails[j]), a.normalise ? own : 0.0f);
            if (zl) g[j] = fmaf(w_z, q[j], g[j]);
        }
    } else {
        auto softmax = [&](auto shares) {  // s_d: gradients of the chosen logits, not of their scores
            const bool scores = !shares || aux;
            float dot = 0.0f;
            if (scores) {
#pragma unroll
                for (int j = 0; j < N; ++j) {
                    g[j] = 0.0f;
                    if (lane + 32 * j >= a.E) continue;
                    if (!shares) g[j] = s_d[lane + 32 * j];
                    if (aux) g[j] = fmaf(w_aux, float(a.counts_in[lane + 32 * j]), g[j]);
                    dot = fmaf(g[j], q[j], dot);
                }
                dot = warp_sum(dot) * r.rz;
            }
#pragma unroll
            for (int j = 0; j < N; ++j) {
                float v = shares && lane + 32 * j < a.E ? s_d[lane + 32 * j] : 0.0f;
                if (scores) v = fmaf(q[j] * r.rz, g[j] - dot, v);
                g[j] = zl ? fmaf(w_z, q[j], v) : v;
            }
        };
        if (a.normalise)
            softmax(std::true_type{});
        else
            softmax(std::false_type{});
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const int e = lane + 32 * j;
        if (e >= a.E) continue;
        const float v = l[j] == -INFINITY ? 0.0f : g[j];
        if (a.bf16)
            static_cast<__nv_bfloat16*>(a.dlogits)[t * a.dld + e] = __float2bfloat16_rn(v);
        else
            static_cast<float*>(a.dlogits)[t * a.dld + e] = v;
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

int router_blocks(int64_t T, int E) {
    const int warps = forward_warps((E + 31) / 32);
    return int(std::min<int64_t>(kRouterBlocks, std::max<int64_t>(1, (T + warps - 1) / warps)));
}
constexpr int kFinish = 64;  // words of a.finish

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

// the build for E experts, 32 N of them at most
template <typename F>
cudaError_t by_experts(int E, F f) {
    const int n = (E + 31) / 32;
    if (n <= 1) return f(std::integral_constant<int, 1>());
    if (n <= 2) return f(std::integral_constant<int, 2>());
    if (n <= 3) return f(std::integral_constant<int, 3>());
    if (n <= 4) return f(std::integral_constant<int, 4>());
    if (n <= 8) return f(std::integral_constant<int, 8>());
    if (n <= 12) return f(std::integral_constant<int, 12>());
    if (n <= 16) return f(std::integral_constant<int, 16>());
    return f(std::integral_constant<int, 32>());
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
    *bytes = (size_t(router_blocks(T, int(cfg->num_experts))) * size_t(2 * cfg->num_experts + 1) + kFinish) * sizeof(float);
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
    a.finish = static_cast<float*>(workspace);
    a.part = counts ? a.finish + kFinish : nullptr;
    a.counts = counts;
    a.losses = losses;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const int blocks = T == 0 ? 0 : router_blocks(T, a.E);
    cudaError_t e = cudaSuccess;
    if (T > 0) {
        e = by_experts(a.E, [&](auto n) {
            constexpr int N = decltype(n)::value, W = forward_warps(N);
            const size_t smem = size_t(a.E) * (1 + (losses ? W : 0)) * sizeof(float);
            return launch_pdl(router_forward_kernel<N>, dim3(unsigned(blocks)), dim3(32 * W), smem, s, a);
        });
        count_launch();
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    if (counts && blocks != 1) {
        // without tokens nothing has set the counter of finished blocks
        if (T == 0 && losses && cudaMemsetAsync(a.finish, 0, sizeof(float), s) != cudaSuccess) return MOE_ERR_CUDA;
        e = launch_pdl(router_finish_kernel, dim3(unsigned((a.E + 31) / 32)), dim3(32 * kFinishWarps), 0, s, a, blocks);
        count_launch();
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
    const cudaError_t e = by_experts(a.E, [&](auto n) {
        return launch_pdl(router_backward_kernel<decltype(n)::value>, dim3(unsigned(blocks)), dim3(32 * kRouterWarps), smem,
                          static_cast<cudaStream_t>(stream), a);
    });
    count_launch();
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
