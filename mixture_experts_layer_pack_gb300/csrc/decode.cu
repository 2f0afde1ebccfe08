// The layer for a few tokens: out = gate * SharedSwiGLU(x) + sum_s p_s RoutedSwiGLU_s(x).
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "../../include/moe.h"
#include "device_common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr size_t kDecodeAlign = 256;

// one weight matrix of every expert: expert e at base + e * expert_bytes, or at table[e]
struct DecodeWeight {
    const uint8_t* base;
    int64_t expert_bytes;
    int64_t row_bytes;
    const void* const* table;        // device array of E pointers, or null
    const uint8_t* scale;            // MXFP8: E8M0 codes, row stride row_bytes / 32
    const void* const* scale_table;
    __device__ __forceinline__ const uint8_t* expert(int e) const {
        return table ? static_cast<const uint8_t*>(table[e]) : base + e * expert_bytes;
    }
    __device__ __forceinline__ const uint8_t* scales(int e) const {
        return scale_table ? static_cast<const uint8_t*>(scale_table[e]) : scale + e * (expert_bytes / 32);
    }
};

enum : int { W_SHARED_GATE = 0, W_SHARED_UP, W_SHARED_DOWN, W_GATE, W_UP, W_DOWN, W_COUNT };

struct DecodeArgs {
    int T, H, I, E, k;
    bool mx, shared;
    float limit;
    const __nv_bfloat16* x;
    int64_t xs;
    const int* ids;
    const float* probs;
    const __nv_bfloat16* gate_w;
    __nv_bfloat16* out;
    int64_t os;
    DecodeWeight w[W_COUNT];
    float* a;  // [T][k + 1][I]: the activations of each slot, the shared expert's last
    int* status;
};

// whether the k ids of a token are in [-1, E) and distinct
__device__ __forceinline__ bool row_valid(const int* ids, int k, int E) {
    for (int i = 0; i < k; ++i) {
        if (ids[i] < -1 || ids[i] >= E) return false;
        for (int j = 0; j < i; ++j)
            if (ids[i] >= 0 && ids[i] == ids[j]) return false;
    }
    return true;
}

// dot product of row n of an expert's matrix with v (fp32 or bf16), by one warp
template <typename V>
__device__ float warp_dot(const uint8_t* w, const uint8_t* sc, int64_t row_bytes, bool mx, int64_t n, const V* v,
                          int K) {
    float acc = 0.0f;
    for (int i = threadIdx.x & 31; i < K; i += 32) {
        float x;
        if constexpr (sizeof(V) == 2)
            x = __bfloat162float(v[i]);
        else
            x = v[i];
        float wv;
        if (mx)
            wv = e4m3_value(w[n * row_bytes + i]) * e8m0_scale(sc[n * (row_bytes / 32) + i / 32]);
        else
            wv = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(w + n * row_bytes)[i]);
        acc = fmaf(wv, x, acc);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
    return acc;
}

// one warp per (token, slot, i)
__global__ void __launch_bounds__(256) decode_up_kernel(DecodeArgs a) {
    const int64_t n = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int slots = a.k + 1;
    if (n >= int64_t(a.T) * slots * a.I) return;
    const int i = int(n % a.I);
    const int s = int(n / a.I % slots);
    const int t = int(n / a.I / slots);
    const bool routed = s < a.k;
    if (routed && !row_valid(a.ids + int64_t(t) * a.k, a.k, a.E)) {
        if ((threadIdx.x & 31) == 0) atomicOr(a.status, kStatusRouting);
        return;
    }
    const int e = routed ? a.ids[int64_t(t) * a.k + s] : 0;
    if (e < 0 || (!routed && !a.shared)) return;
    const DecodeWeight& wg = a.w[routed ? W_GATE : W_SHARED_GATE];
    const DecodeWeight& wu = a.w[routed ? W_UP : W_SHARED_UP];
    const bool mx = routed && a.mx;
    const __nv_bfloat16* x = a.x + t * a.xs;
    float g = warp_dot(wg.expert(e), mx ? wg.scales(e) : nullptr, wg.row_bytes, mx, i, x, a.H);
    float u = warp_dot(wu.expert(e), mx ? wu.scales(e) : nullptr, wu.row_bytes, mx, i, x, a.H);
    if (a.limit > 0.0f) {
        g = fminf(g, a.limit);
        u = fminf(fmaxf(u, -a.limit), a.limit);
    }
    if ((threadIdx.x & 31) == 0) a.a[(int64_t(t) * slots + s) * a.I + i] = g * sigmoidf_(g) * u;
}

// one warp per (token, h)
__global__ void __launch_bounds__(256) decode_down_kernel(DecodeArgs a) {
    const int64_t n = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    if (n >= int64_t(a.T) * a.H) return;
    const int h = int(n % a.H);
    const int t = int(n / a.H);
    const int slots = a.k + 1;
    const float* act = a.a + int64_t(t) * slots * a.I;
    float out = 0.0f;
    if (a.shared) {
        const DecodeWeight& w = a.w[W_SHARED_DOWN];
        out = warp_dot(w.base, nullptr, w.row_bytes, false, h, act + int64_t(a.k) * a.I, a.I);
        if (a.gate_w)
            out *= sigmoidf_(warp_dot(reinterpret_cast<const uint8_t*>(a.gate_w), nullptr, 0, false, 0, a.x + t * a.xs,
                                      a.H));
    }
    if (row_valid(a.ids + int64_t(t) * a.k, a.k, a.E)) {
        const DecodeWeight& w = a.w[W_DOWN];
        for (int s = 0; s < a.k; ++s) {
            const int e = a.ids[int64_t(t) * a.k + s];
            if (e < 0) continue;
            const float y = warp_dot(w.expert(e), a.mx ? w.scales(e) : nullptr, w.row_bytes, a.mx, h,
                                     act + int64_t(s) * a.I, a.I);
            out = fmaf(a.probs[int64_t(t) * a.k + s], y, out);
        }
    }
    if ((threadIdx.x & 31) == 0) a.out[t * a.os + h] = __float2bfloat16_rn(out);
}

struct DecodeShape {
    int64_t Tmax, H, E, k, I;
    bool mx, shared;
    float limit;
};

moe_status check_decode(const moe_config* c, DecodeShape* s) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (c->max_tokens < 0 || c->hidden <= 0 || c->num_experts <= 0 || c->topk <= 0 || c->inter <= 0)
        return MOE_ERR_INVALID_ARG;
    if (!(c->swiglu_limit >= 0.0f) || !std::isfinite(c->swiglu_limit)) return MOE_ERR_INVALID_ARG;
    if (c->act_precision != MOE_ACT_FP32 && c->act_precision != MOE_ACT_BF16) return MOE_ERR_INVALID_ARG;
    if (c->no_shared_expert != 0 && c->no_shared_expert != 1) return MOE_ERR_INVALID_ARG;
    if (c->recompute_dispatch != 0) return MOE_ERR_INVALID_ARG;
    if (c->routed_wtype != MOE_W_BF16 && c->routed_wtype != MOE_W_MXFP8) return MOE_ERR_UNSUPPORTED;
    const bool mx = c->routed_wtype == MOE_W_MXFP8;
    if (c->max_tokens > MOE_DECODE_MAX_TOKENS) return MOE_ERR_UNSUPPORTED;
    if (c->num_experts > 1024 || c->topk > 32 || c->topk > c->num_experts) return MOE_ERR_UNSUPPORTED;
    const int64_t step = mx ? 32 : 8;
    if (c->hidden % step || c->inter % step || c->hidden > 65536 || c->inter > 65536) return MOE_ERR_UNSUPPORTED;
    *s = DecodeShape{c->max_tokens, c->hidden, c->num_experts, c->topk, c->inter, mx, c->no_shared_expert == 0,
                     c->swiglu_limit};
    return MOE_OK;
}

struct DecodeSpace {
    int* status;
    const void** tables;  // [6][E]: gate, up, down payloads, then their scales
    float* a;
};

size_t carve_decode(const DecodeShape& s, uint8_t* base, DecodeSpace* w) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        uint8_t* p = base ? base + off : nullptr;
        off += (bytes + kDecodeAlign - 1) / kDecodeAlign * kDecodeAlign;
        return p;
    };
    w->status = reinterpret_cast<int*>(take(sizeof(int)));
    w->tables = reinterpret_cast<const void**>(take(6 * size_t(s.E) * sizeof(void*)));
    w->a = reinterpret_cast<float*>(take(size_t(s.Tmax) * size_t(s.k + 1) * size_t(s.I) * sizeof(float)));
    return off;
}

bool is16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

}  // namespace moe

struct moe_decoder {
    moe::DecodeShape s;
    moe::DecodeSpace ws;
    std::vector<const void*> host[3];  // the per-expert pointers last uploaded: gate, up, down
};

namespace moe {

namespace {

// a shared or strided routed view, or a per-expert table, as the kernels take it
moe_status decode_weight(moe_decoder* d, const moe_wview& v, int64_t N, int64_t K, bool routed, int slot,
                         cudaStream_t st, DecodeWeight* out) {
    const bool mx = routed && d->s.mx;
    const int64_t es = mx ? 1 : 2;
    if (v.row_stride < K || (v.row_stride * es) % (mx ? 32 : 16)) return MOE_ERR_INVALID_ARG;
    *out = DecodeWeight{};
    out->row_bytes = v.row_stride * es;
    if (routed && v.expert_ptrs) {
        const int64_t E = d->s.E;
        std::vector<const void*> want(size_t(2 * E), nullptr);
        for (int64_t e = 0; e < E; ++e) {
            want[size_t(e)] = v.expert_ptrs[e];
            if (!want[size_t(e)] || !is16(want[size_t(e)])) return MOE_ERR_INVALID_ARG;
            if (mx && !(want[size_t(E + e)] = v.expert_ptrs[2 * E + e])) return MOE_ERR_INVALID_ARG;
        }
        const void** dev = d->ws.tables + size_t(2 * slot) * size_t(E);
        if (want != d->host[slot]) {
            d->host[slot].clear();
            // pageable source: staged before the call returns
            if (cudaMemcpyAsync(dev, want.data(), want.size() * sizeof(void*), cudaMemcpyHostToDevice, st) !=
                cudaSuccess)
                return MOE_ERR_CUDA;
            d->host[slot] = std::move(want);
        }
        out->table = dev;
        if (mx) out->scale_table = dev + E;
        return MOE_OK;
    }
    if (!v.data || !is16(v.data)) return MOE_ERR_INVALID_ARG;
    if (routed) {
        if (d->s.E > 1 && (v.expert_stride < 0 || (v.expert_stride * es) % (mx ? 32 : 16))) return MOE_ERR_INVALID_ARG;
        out->expert_bytes = v.expert_stride * es;
        if (mx && !v.scale) return MOE_ERR_INVALID_ARG;
        out->scale = v.scale;
    }
    out->base = static_cast<const uint8_t*>(v.data);
    return MOE_OK;
}

}  // namespace

}  // namespace moe

extern "C" {

moe_status moe_decode_size(const moe_config* cfg, size_t* bytes) {
    using namespace moe;
    if (!bytes) return MOE_ERR_INVALID_ARG;
    *bytes = 0;
    DecodeShape s;
    const moe_status st = check_decode(cfg, &s);
    if (st != MOE_OK) return st;
    DecodeSpace w;
    *bytes = carve_decode(s, nullptr, &w);
    return MOE_OK;
}

moe_status moe_decode_create(const moe_config* cfg, void* workspace, size_t workspace_bytes, moe_decoder** out) {
    using namespace moe;
    if (!out) return MOE_ERR_INVALID_ARG;
    *out = nullptr;
    DecodeShape s;
    const moe_status st = check_decode(cfg, &s);
    if (st != MOE_OK) return st;
    DecodeSpace w;
    if (!workspace || workspace_bytes < carve_decode(s, nullptr, &w) ||
        (reinterpret_cast<uintptr_t>(workspace) % kDecodeAlign))
        return MOE_ERR_INVALID_ARG;
    moe_decoder* d = new (std::nothrow) moe_decoder;
    if (!d) return MOE_ERR_INVALID_ARG;
    d->s = s;
    carve_decode(s, static_cast<uint8_t*>(workspace), &d->ws);
    if (cudaMemset(d->ws.status, 0, sizeof(int)) != cudaSuccess) {
        delete d;
        return MOE_ERR_CUDA;
    }
    *out = d;
    return MOE_OK;
}

void moe_decode_destroy(moe_decoder* d) { delete d; }

moe_status moe_decode(moe_decoder* d, int64_t T, const void* hidden, int64_t hidden_stride, const int32_t* topk_ids,
                      const float* topk_probs, const moe_weights* w, void* out, int64_t out_stride, void* stream) {
    using namespace moe;
    if (!d || !w || T < 0 || T > d->s.Tmax) return MOE_ERR_INVALID_ARG;
    const DecodeShape& s = d->s;
    if (hidden_stride < s.H || hidden_stride % 8 || out_stride < s.H) return MOE_ERR_INVALID_ARG;
    if (T == 0) return MOE_OK;
    if (!hidden || !topk_ids || !topk_probs || !out || !is16(hidden)) return MOE_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(topk_ids) & 3) || (reinterpret_cast<uintptr_t>(topk_probs) & 3) ||
        (reinterpret_cast<uintptr_t>(out) & 1))
        return MOE_ERR_INVALID_ARG;
    if (w->shared_output_gate && (!s.shared || !is16(w->shared_output_gate))) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    DecodeArgs a{};
    a.T = int(T);
    a.H = int(s.H);
    a.I = int(s.I);
    a.E = int(s.E);
    a.k = int(s.k);
    a.mx = s.mx;
    a.shared = s.shared;
    a.limit = s.limit;
    a.x = static_cast<const __nv_bfloat16*>(hidden);
    a.xs = hidden_stride;
    a.ids = topk_ids;
    a.probs = topk_probs;
    a.gate_w = static_cast<const __nv_bfloat16*>(w->shared_output_gate);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.os = out_stride;
    a.a = d->ws.a;
    a.status = d->ws.status;
    const moe_wview* views[W_COUNT] = {&w->shared_gate, &w->shared_up,   &w->shared_down,
                                       &w->routed_gate, &w->routed_up, &w->routed_down};
    for (int i = s.shared ? 0 : 3; i < W_COUNT; ++i) {
        const bool down = i % 3 == 2;
        const moe_status r = decode_weight(d, *views[i], down ? s.H : s.I, down ? s.I : s.H, i >= 3, i % 3, st, &a.w[i]);
        if (r != MOE_OK) return r;
    }
    const int64_t up = int64_t(a.T) * (a.k + 1) * a.I, down = int64_t(a.T) * a.H;
    decode_up_kernel<<<unsigned((up + 7) / 8), 256, 0, st>>>(a);
    decode_down_kernel<<<unsigned((down + 7) / 8), 256, 0, st>>>(a);
    count_launch(2);
    return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_decode_status(moe_decoder* d, void* stream) {
    using namespace moe;
    if (!d) return MOE_ERR_INVALID_ARG;
    int v = 0;
    if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess ||
        cudaMemcpy(&v, d->ws.status, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess ||
        cudaMemset(d->ws.status, 0, sizeof(int)) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (v & kStatusTimeout) return MOE_ERR_TIMEOUT;
    if (v & kStatusRouting) return MOE_ERR_ROUTING;
    return MOE_OK;
}

}  // extern "C"
