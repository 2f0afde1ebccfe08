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
//
// Bound by memory where rows are many: 16384 x 4096 bf16 with a residual, forward 85 us (6.3 TB/s), backward with the
// joining gradient and the weights' 87 us (6.2 TB/s); 16384 x 2051, rows that start anywhere, 55 and 57 us (4.8 TB/s). One
// row of 2048: 2.1 us. s and y are rounded once each, to the types that the next reader takes.
#include <algorithm>
#include <atomic>
#include <climits>
#include <cmath>
#include <type_traits>

#include "../../include/moe.h"
#include "device_common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kMaxHidden = 32768;
constexpr int kMaxChunks = 608;     // blocks of the backward that sum weight gradients: four per SM at most
constexpr int kRowThreads = 512;    // most threads of a row: 128 registers each
constexpr int kColumns = 16;        // columns of a thread where rows are streamed

// V consecutive elements as fp32: one 16-byte access (two for 8 fp32, one of 8 bytes for 4 bf16), or with V 1 a scalar
template <int V>
__device__ __forceinline__ void load_v(const __nv_bfloat16* p, float (&f)[V]) {
    if constexpr (V == 8) {
        const uint4 w = *reinterpret_cast<const uint4*>(p);
        unpack_bf16x2(w.x, f[0], f[1]);
        unpack_bf16x2(w.y, f[2], f[3]);
        unpack_bf16x2(w.z, f[4], f[5]);
        unpack_bf16x2(w.w, f[6], f[7]);
    } else if constexpr (V == 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(p);
        unpack_bf16x2(w.x, f[0], f[1]);
        unpack_bf16x2(w.y, f[2], f[3]);
    } else {
        f[0] = __bfloat162float(*p);
    }
}
template <int V>
__device__ __forceinline__ void load_v(const float* p, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = *p;
    } else {
#pragma unroll
        for (int q = 0; q < V; q += 4) {
            const float4 w = *reinterpret_cast<const float4*>(p + q);
            f[q] = w.x, f[q + 1] = w.y, f[q + 2] = w.z, f[q + 3] = w.w;
        }
    }
}
template <int V>
__device__ __forceinline__ void store_v(__nv_bfloat16* p, const float (&f)[V]) {
    if constexpr (V == 8)
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                  pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    else if constexpr (V == 4)
        *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    else
        *p = __float2bfloat16_rn(f[0]);
}
template <int V>
__device__ __forceinline__ void store_v(float* p, const float (&f)[V]) {
    if constexpr (V == 1) {
        *p = f[0];
    } else {
#pragma unroll
        for (int q = 0; q < V; q += 4) *reinterpret_cast<float4*>(p + q) = make_float4(f[q], f[q + 1], f[q + 2], f[q + 3]);
    }
}
// weight and bias come in either type, a run-time branch: they are read from cache
template <int V>
__device__ __forceinline__ void load_w(const void* p, int i, bool bf16, float (&f)[V]) {
    if (bf16)
        load_v<V>(static_cast<const __nv_bfloat16*>(p) + i, f);
    else
        load_v<V>(static_cast<const float*>(p) + i, f);
}
__device__ __forceinline__ float round_to(float v, const float*) { return v; }
__device__ __forceinline__ float round_to(float v, const __nv_bfloat16*) {
    return __bfloat162float(__float2bfloat16_rn(v));
}

constexpr int kWidest = 768;   // most threads of a row
constexpr int kSumWarps = 32;  // places of a sum

// Sums over the `warps` warps of a row (warps first, first + 1, ... of the block); every thread of
// the row gets them, in an order fixed by the number of warps. part: kSumWarps values for each sum, zeros
// where there is no warp, of which the callers alternate two, so that one barrier a sum is enough.
template <int N>
__device__ __forceinline__ void row_sum(float (&v)[N], int warps, int first, float* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(0xffffffffu, v[n], o);
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int n = 0; n < N; ++n) part[n * kSumWarps + (threadIdx.x >> 5)] = v[n];
    __syncthreads();
    if (warps <= 4) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            float p[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) p[w] = w < warps ? part[n * kSumWarps + first + w] : 0.0f;
            v[n] = (p[0] + p[1]) + (p[2] + p[3]);
        }
    } else if (warps <= 8) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
            const float4 p = reinterpret_cast<const float4*>(part + n * kSumWarps)[0];
            const float4 q = reinterpret_cast<const float4*>(part + n * kSumWarps)[1];
            v[n] = ((p.x + p.y) + (p.z + p.w)) + ((q.x + q.y) + (q.z + q.w));
        }
    } else {
        auto eight = [&](int n, int q) {
            const float4 x = reinterpret_cast<const float4*>(part + n * kSumWarps)[q];
            const float4 y = reinterpret_cast<const float4*>(part + n * kSumWarps)[q + 1];
            return ((x.x + x.y) + (x.z + x.w)) + ((y.x + y.y) + (y.z + y.w));
        };
#pragma unroll
        for (int n = 0; n < N; ++n) v[n] = eight(n, 0) + eight(n, 2);
        if (warps > 16)
#pragma unroll
            for (int n = 0; n < N; ++n) v[n] += eight(n, 4);
        static_assert(kWidest <= 24 * 32, "24 warps a row");
    }
}

// Two fp32 operations an instruction, each rounded as by itself: the streamed rows are bound by the
// instructions that their warps issue (16384 x 4096 bf16 without a residual: 58.5 -> 57 us, backward 80 -> 78)
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void un2(uint64_t v, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ float sum2(uint64_t v) {
    float a, b;
    un2(v, a, b);
    return a + b;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

struct NormFwd {
    const void *x, *r, *w, *b;
    void *s, *y;
    float *mean, *rstd;
    int64_t xs, rs, ss, ys;
    int64_t T;
    int H, tpr;
    float eps;
    bool w_bf16;
};

// ---- bf16 rows of more than kStreamed columns, up to 16384, in whole 16-byte pieces: a block a row
// The row stays in the registers of its threads, NV pieces of V elements each: read once,
// written once, and the variance is of differences from the mean, not of squares.
template <typename XT, typename YT, bool RMS, int V, int NV>
__global__ void __launch_bounds__(kRowThreads) norm_forward_kernel(NormFwd a) {
    __shared__ __align__(16) float part[2][kSumWarps];
    if (threadIdx.x < 32) part[0][threadIdx.x] = part[1][threadIdx.x] = 0.0f;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int tpr = blockDim.x, col = threadIdx.x, warps = tpr >> 5;
    const int64_t t = blockIdx.x;
    const XT* x = static_cast<const XT*>(a.x) + t * a.xs;
    float v[NV][V];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = (col + j * tpr) * V;
        if (i < a.H) load_v<V>(x + i, v[j]);
    }
    if (a.r) {
        const XT* r = static_cast<const XT*>(a.r) + t * a.rs;
        XT* s = static_cast<XT*>(a.s) + t * a.ss;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = (col + j * tpr) * V;
            if (i >= a.H) continue;
            float f[V];
            load_v<V>(r + i, f);
#pragma unroll
            for (int q = 0; q < V; ++q) v[j][q] = round_to(v[j][q] + f[q], x);
            store_v<V>(s + i, v[j]);
        }
    }
    const float inv = 1.0f / a.H;
    float mean = 0.0f;
    if (!RMS) {
        float sum[1] = {0.0f};
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if ((col + j * tpr) * V < a.H)
#pragma unroll
                for (int q = 0; q < V; ++q) sum[0] += v[j][q];
        row_sum<1>(sum, warps, 0, part[0]);
        mean = sum[0] * inv;
    }
    float sq[1] = {0.0f};
#pragma unroll
    for (int j = 0; j < NV; ++j)
        if ((col + j * tpr) * V < a.H)
#pragma unroll
            for (int q = 0; q < V; ++q) {
                v[j][q] -= mean;
                sq[0] = fmaf(v[j][q], v[j][q], sq[0]);
            }
    row_sum<1>(sq, warps, 0, part[1]);
    const float rstd = rsqrtf(sq[0] * inv + a.eps);
    YT* y = static_cast<YT*>(a.y) + t * a.ys;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = (col + j * tpr) * V;
        if (i >= a.H) continue;
        float w[V], b[V], o[V];
        load_w<V>(a.w, i, a.w_bf16, w);
        if (a.b) load_w<V>(a.b, i, a.w_bf16, b);
#pragma unroll
        for (int q = 0; q < V; ++q) {
            o[q] = v[j][q] * rstd * w[q];
            if (a.b) o[q] += b[q];
        }
        store_v<V>(y + i, o);
    }
    if (col == 0) {
        if (!RMS && a.mean) a.mean[t] = mean;
        if (a.rstd) a.rstd[t] = rstd;
    }
}

// ---- Rows of up to kStreamed columns: streamed through shared memory (one row of 2048 2.5 us, as without it)
// A stage holds one row of each input for each row group of the block, brought by bulk copies;
// `stages` of them are under way while one is worked on. A copy takes the 16-byte words that cover
// its row, so rows may start anywhere; rows that start on 16 bytes are then read in pieces of V
// elements, others one by one. The barrier of a row's sums also says that nobody reads the rows
// before any more: one warp, each in its turn, then asks for the rows that take their place. (A warp of its own for
// that leaves 96 registers a thread where there are 128 now, and the sums of the weights' gradients
// no longer fit: 16384 x 4096 backward 153 us against 100.)
constexpr int kMaxStages = 8;
// threads of a block: several row groups or one of up to 256 threads, two blocks an SM; or one of up to 512, or of 768
// (80 registers a thread: the backward spills some 130 bytes)
constexpr int kNarrow = 256, kWide = 512;  // and kWidest
constexpr int kStreamed = kColumns * kWidest;  // the widest row that is streamed
constexpr size_t kMostShared = 225 << 10;      // and the most shared memory for it beside what the kernels declare
struct Stream {
    int stages, arrays;
    int row_bytes[3], at[3];  // of each input: bytes of a row, and its place in a row group's part of a stage
    const char* from[3];
    int64_t step[3];          // bytes from row to row
    int group_bytes;          // a row group's part of a stage
};

// where a lane asks: the same input and row of a step every time (in shared memory: it is looked at once a row)
struct Ask {
    const char* from;
    int64_t step;
    int row_bytes, to;
};

struct StreamRing {
    const Stream& st;
    uint64_t* full;
    Ask* asks;
    uint8_t* mem;
    int groups;
    int s = 0;
    uint32_t parity = 0;  // bit 0: of the current round; bit 1: a wait gave up (no register of its own: there is none to spare)
    __device__ __forceinline__ bool late() const { return parity > 1; }
    __device__ __forceinline__ void init() const {
        if (threadIdx.x < st.stages) mbar_init(full + threadIdx.x, 1);
        if (threadIdx.x < 32) {
            const int g = threadIdx.x / st.arrays, i = threadIdx.x - g * st.arrays;
            asks[threadIdx.x] = g < groups ? Ask{st.from[i] + g * st.step[i], st.step[i], st.row_bytes[i], g * st.group_bytes + st.at[i]}
                                           : Ask{nullptr, 0, 0, 0};
        }
        fence_mbar_init();
        __syncthreads();
    }
    // one warp: asks for the rows t0 ... t0 + groups - 1 (those below T) into stage `at`, a lane per row and input
    __device__ __forceinline__ void ask(int at, unsigned t0, unsigned T) const {
        const int lane = threadIdx.x & 31;
        const Ask q = asks[lane];
        const bool mine = q.row_bytes != 0 && !late() && unsigned(lane / st.arrays) < T - t0;
        const char* src = q.from + t0 * q.step;
        const uint32_t off = uint32_t(reinterpret_cast<uintptr_t>(src)) & 15u;
        const uint32_t bytes = mine ? (off + uint32_t(q.row_bytes) + 15u) & ~15u : 0u;
        const uint32_t total = __reduce_add_sync(0xffffffffu, bytes);
        if (lane == 0 && !late()) mbar_arrive_expect_tx(full + at, total);
        __syncwarp();
        if (mine)
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             smem_u32(mem + at * groups * st.group_bytes + q.to)),
                         "l"(src - off), "r"(bytes), "r"(smem_u32(full + at))
                         : "memory");
    }
    // The next rows are there; bounded: after a wait that gave up the thread waits and asks for nothing more, and makes its
    // results NaN (there is no status word to say it in).
    __device__ __forceinline__ void wait() {
        if (mbar_try_wait(full + s, parity & 1)) return;
        const uint64_t t0 = globaltimer_ns();
        while (!mbar_try_wait(full + s, parity & 1))
            if (globaltimer_ns() - t0 > (late() ? 0 : kWaitLimitNs)) {
                parity |= 2;
                return;
            }
    }
    // before the block gives back its shared memory: the copies that were not waited for land in it
    __device__ __forceinline__ void end() const {
        if (!late()) return;
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 1000000) __nanosleep(1000);
    }
    // input i's row t, of row group g in the current stage; whole: rows are known to begin on 16 bytes
    template <typename E, bool Whole>
    __device__ __forceinline__ const E* row(int i, int g, unsigned t) const {
        const uint32_t off = Whole ? 0u : (uint32_t(reinterpret_cast<uintptr_t>(st.from[i])) + t * uint32_t(st.step[i])) & 15u;
        return reinterpret_cast<const E*>(mem + (s * groups + g) * st.group_bytes + st.at[i] + off);
    }
    __device__ __forceinline__ void next() {
        if (++s == st.stages) {
            s = 0;
            parity ^= 1;
        }
    }
};

// A thread's columns of a row: NV pieces of V, a piece of each lane beside the next, so that a warp has
// kColumns * 32 columns on end. The pieces' places are then constants beside one pointer, and a warp that has all its
// columns (most do) looks at no bounds: f(true) runs there, f(false) in a warp where the row ends.
template <int V, int NV>
struct Columns {
    static constexpr int kStep = 32 * V;  // from piece to piece
    int base, limit;                      // the first column, and how many columns of the row come from there on
    bool all;
    __device__ __forceinline__ Columns(int col, int H) {
        const int first = (col >> 5) * NV * kStep;
        base = first + (threadIdx.x & 31) * V;
        limit = H - base;
        all = first + NV * kStep <= H;
    }
    template <typename F>
    __device__ __forceinline__ void run(F f) const {
        if (all)
            f(std::true_type{});
        else
            f(std::false_type{});
    }
};
// element e of a thread's columns
template <int V, int NV>
__device__ __forceinline__ float& at(float (&v)[NV][V], int e) { return v[e / V][e % V]; }
template <int V, int NV>
__device__ __forceinline__ uint64_t two(float (&v)[NV][V], int e) { return f2(at<V, NV>(v, e), at<V, NV>(v, e + 1)); }
template <int V, int NV>
__device__ __forceinline__ void put2(float (&v)[NV][V], int e, uint64_t x) { un2(x, at<V, NV>(v, e), at<V, NV>(v, e + 1)); }

template <typename XT, typename YT, bool RMS, int V, int NV, int NT>
__global__ void __launch_bounds__(NT, NT == kNarrow ? 2 : 1) norm_forward_stream_kernel(NormFwd a, const __grid_constant__ Stream st) {
    __shared__ __align__(16) float part[2][2][kSumWarps];
    __shared__ uint64_t full[kMaxStages];
    __shared__ Ask asks[32];
    extern __shared__ __align__(128) uint8_t mem[];
    constexpr bool kWhole = V > 1;
    constexpr int N = NV * V, kStep = Columns<V, NV>::kStep;
    if (threadIdx.x < 32)
        part[0][0][threadIdx.x] = part[0][1][threadIdx.x] = part[1][0][threadIdx.x] = part[1][1][threadIdx.x] = 0.0f;
    const int tpr = a.tpr, groups = blockDim.x / tpr, group = threadIdx.x / tpr, col = threadIdx.x - group * tpr;
    const unsigned T = unsigned(a.T), first = blockIdx.x * groups, step = gridDim.x * groups;  // T < 2^31
    const int warps = tpr >> 5;
    const Columns<V, NV> cols(col, a.H);
    const int limit = cols.limit;
    const float inv = 1.0f / a.H;
    StreamRing ring{st, full, asks, mem, groups};
    ring.init();
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5;
    if (warp == 0)
        for (int s = 0; s < st.stages && first + s * step < T; ++s) ring.ask(s, first + s * step, T);
    float w[NV][V], b[NV][V];  // a thread has the same columns in every row: their weights stay in registers
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
        for (int q = 0; q < V; ++q) w[j][q] = b[j][q] = 0.0f;
        if (j * kStep >= limit) continue;
        load_w<V>(a.w, cols.base + j * kStep, a.w_bf16, w[j]);
        if (a.b) load_w<V>(a.b, cols.base + j * kStep, a.w_bf16, b[j]);
    }
    int turn = 0, asker = 0;
    for (unsigned t0 = first; t0 < T; t0 += step, turn ^= 1) {
        const unsigned t = t0 + group;
        const bool live = t < T;  // the last rows may not exist: their threads join the sums
        ring.wait();
        const XT* x = ring.row<XT, kWhole>(0, group, t) + cols.base;
        float v[NV][V], sum[1] = {0.0f}, sq[1] = {0.0f};
        if (!live) {
#pragma unroll
            for (int e = 0; e < N; ++e) at<V, NV>(v, e) = 0.0f;
        } else if (!a.r) {
            cols.run([&](auto all) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if (all || j * kStep < limit)
                        load_v<V>(x + j * kStep, v[j]);
                    else
#pragma unroll
                        for (int q = 0; q < V; ++q) v[j][q] = 0.0f;
                }
            });
        } else {
            const XT* r = ring.row<XT, kWhole>(1, group, t) + cols.base;
            XT* total = static_cast<XT*>(a.s) + t * a.ss + cols.base;
            cols.run([&](auto all) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
#pragma unroll
                    for (int q = 0; q < V; ++q) v[j][q] = 0.0f;
                    if (!all && j * kStep >= limit) continue;
                    float f[V];
                    load_v<V>(x + j * kStep, v[j]);
                    load_v<V>(r + j * kStep, f);
#pragma unroll
                    for (int q = 0; q < V; ++q) v[j][q] = round_to(v[j][q] + f[q], x);
                    store_v<V>(total + j * kStep, v[j]);
                }
            });
        }
        float mean = 0.0f;
        if (!RMS) {
            uint64_t s2 = 0;
#pragma unroll
            for (int e = 0; e < N; e += 2) s2 = add2(s2, two<V, NV>(v, e));
            sum[0] = sum2(s2);
            row_sum<1>(sum, warps, group * warps, part[turn][0]);
            mean = sum[0] * inv;
        }
        cols.run([&](auto all) {
            const uint64_t m2 = f2(-mean, -mean);
            uint64_t q2 = 0;
#pragma unroll
            for (int e = 0; e < N; e += 2) {
                if (!RMS) put2<V, NV>(v, e, add2(two<V, NV>(v, e), m2));
                if (!all) {
                    if (e / V * kStep >= limit) at<V, NV>(v, e) = 0.0f;
                    if ((e + 1) / V * kStep >= limit) at<V, NV>(v, e + 1) = 0.0f;
                }
                q2 = fma2(two<V, NV>(v, e), two<V, NV>(v, e), q2);
            }
            sq[0] = sum2(q2);
        });
        row_sum<1>(sq, warps, group * warps, part[turn][1]);
        if (warps == 1) __syncthreads();  // the sums had no barrier
        // the rows are in everybody's registers
        if (warp == asker && t0 + st.stages * step < T) ring.ask(ring.s, t0 + st.stages * step, T);
        asker = asker + 1 == int(blockDim.x >> 5) ? 0 : asker + 1;
        ring.next();
        if (!live) continue;
        const float rstd = rsqrtf(sq[0] * inv + (ring.late() ? NAN : a.eps));
        YT* y = static_cast<YT*>(a.y) + t * a.ys + cols.base;
        cols.run([&](auto all) {
            const uint64_t r2 = f2(rstd, rstd);
#pragma unroll
            for (int e = 0; e < N; e += 2)
                put2<V, NV>(v, e, fma2(mul2(two<V, NV>(v, e), r2), two<V, NV>(w, e), two<V, NV>(b, e)));
#pragma unroll
            for (int j = 0; j < NV; ++j)
                if (all || j * kStep < limit) store_v<V>(y + j * kStep, v[j]);
        });
        if (col == 0) {
            if (!RMS && a.mean) a.mean[t] = mean;
            if (a.rstd) a.rstd[t] = rstd;
        }
    }
    ring.end();
}

// Rows too wide for that: row blockIdx.x read three times (the second and third from cache)
template <typename XT, typename YT, bool RMS, int V>
__global__ void __launch_bounds__(kRowThreads) norm_forward_wide_kernel(NormFwd a) {
    __shared__ __align__(16) float part[2][kSumWarps];
    if (threadIdx.x < 32) part[0][threadIdx.x] = part[1][threadIdx.x] = 0.0f;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const XT* x = static_cast<const XT*>(a.x) + t * a.xs;
    const XT* r = a.r ? static_cast<const XT*>(a.r) + t * a.rs : nullptr;
    YT* y = static_cast<YT*>(a.y) + t * a.ys;
    // sum may be x or residual itself: the rounded sum is written in the last pass, where it is last needed
    auto value = [&](int i, float (&v)[V]) {
        load_v<V>(x + i, v);
        if (!r) return;
        float f[V];
        load_v<V>(r + i, f);
#pragma unroll
        for (int q = 0; q < V; ++q) v[q] = round_to(v[q] + f[q], x);
    };
    float mean = 0.0f, sum[1] = {0.0f};
    if (!RMS) {
#pragma unroll 4
        for (int i = threadIdx.x * V; i < a.H; i += blockDim.x * V) {
            float v[V];
            value(i, v);
#pragma unroll
            for (int q = 0; q < V; ++q) sum[0] += v[q];
        }
        row_sum<1>(sum, blockDim.x >> 5, 0, part[0]);
        mean = sum[0] / a.H;
    }
    float sq[1] = {0.0f};
#pragma unroll 4
    for (int i = threadIdx.x * V; i < a.H; i += blockDim.x * V) {
        float v[V];
        value(i, v);
#pragma unroll
        for (int q = 0; q < V; ++q) sq[0] = fmaf(v[q] - mean, v[q] - mean, sq[0]);
    }
    row_sum<1>(sq, blockDim.x >> 5, 0, part[1]);
    const float rstd = rsqrtf(sq[0] / a.H + a.eps);
#pragma unroll 4
    for (int i = threadIdx.x * V; i < a.H; i += blockDim.x * V) {
        float v[V], w[V], b[V], o[V];
        value(i, v);
        load_w<V>(a.w, i, a.w_bf16, w);
        if (a.b) load_w<V>(a.b, i, a.w_bf16, b);
#pragma unroll
        for (int q = 0; q < V; ++q) {
            o[q] = (v[q] - mean) * rstd * w[q];
            if (a.b) o[q] += b[q];
        }
        if (r) store_v<V>(static_cast<XT*>(a.s) + t * a.ss + i, v);
        store_v<V>(y + i, o);
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
    float* part;  // [blocks][2][H]: a block's sums over its rows of dy xhat and of dy
    int64_t dys, xs, dss, dxs;
    int64_t T;
    int H, tpr;
    bool w_bf16;
};

// dx of a block's rows, streamed like the forward's, and the block's part of the weight
// gradients: a thread has the same columns in every row and keeps their sums in registers, so
// x and dy are read once for all three gradients. The weights lie in shared memory as fp32: the registers go to the sums.
template <typename XT, typename YT, bool RMS, int V, int NV, int NT>
__global__ void __launch_bounds__(NT, NT == kNarrow ? 2 : 1) norm_backward_kernel(NormBwd a, const __grid_constant__ Stream st) {
    __shared__ __align__(16) float part[2][2][kSumWarps];
    __shared__ uint64_t full[kMaxStages];
    __shared__ Ask asks[32];
    extern __shared__ __align__(128) uint8_t mem[];
    constexpr bool kWhole = V > 1;
    constexpr int N = NV * V, kStep = Columns<V, NV>::kStep;
    if (threadIdx.x < 32)
        part[0][0][threadIdx.x] = part[0][1][threadIdx.x] = part[1][0][threadIdx.x] = part[1][1][threadIdx.x] = 0.0f;
    const int tpr = a.tpr, groups = blockDim.x / tpr, group = threadIdx.x / tpr, col = threadIdx.x - group * tpr;
    const unsigned T = unsigned(a.T), first = blockIdx.x * groups, step = gridDim.x * groups;  // T < 2^31
    const int warps = tpr >> 5;
    const Columns<V, NV> cols(col, a.H);
    const int limit = cols.limit;
    const float inv = 1.0f / a.H;
    float* weight = reinterpret_cast<float*>(mem);  // of all kColumns * tpr columns, zeros past the row
    StreamRing ring{st, full, asks, mem + kColumns * tpr * sizeof(float), groups};
    ring.init();
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5;
    if (warp == 0)
        for (int s = 0; s < st.stages && first + s * step < T; ++s) ring.ask(s, first + s * step, T);
    weight += cols.base;
    if (group == 0) {
        float f[NV][V] = {};
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (j * kStep < limit) load_w<V>(a.w, cols.base + j * kStep, a.w_bf16, f[j]);
#pragma unroll
        for (int j = 0; j < NV; ++j) store_v<V>(weight + j * kStep, f[j]);
    }
    if (groups > 1) __syncthreads();  // else a thread reads its own only
    float dw[NV][V] = {}, db[NV][V] = {};
    float mean = 0.0f, rstd = 0.0f;
    if (first + group < T) {
        if (!RMS) mean = a.mean[first + group];
        rstd = a.rstd[first + group];
    }
    int turn = 0, asker = 0, before = -1;  // before: the stage of the rows before
    for (unsigned t0 = first; t0 < T; t0 += step, turn ^= 1) {
        const unsigned t = t0 + group;
        const bool live = t < T;  // the last rows may not exist: their threads join the sums
        float mean_after = 0.0f, rstd_after = 0.0f;  // under way during these rows
        if (t + step < T) {
            if (!RMS) mean_after = a.mean[t + step];
            rstd_after = a.rstd[t + step];
        }
        ring.wait();
        if (ring.late()) rstd = NAN;
        const XT* x = ring.row<XT, kWhole>(0, group, t) + cols.base;
        const YT* dy = ring.row<YT, (V > 1 && V * sizeof(YT) >= 16)>(1, group, t) + cols.base;
        float xh[NV][V], g[NV][V], sum[2];  // of g xhat, g
        if (!live) {
#pragma unroll
            for (int e = 0; e < N; ++e) at<V, NV>(xh, e) = at<V, NV>(g, e) = 0.0f;
        } else {
            cols.run([&](auto all) {
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if (all || j * kStep < limit) {
                        load_v<V>(x + j * kStep, xh[j]);
                        load_v<V>(dy + j * kStep, g[j]);
                    } else {
#pragma unroll
                        for (int q = 0; q < V; ++q) xh[j][q] = g[j][q] = 0.0f;
                    }
                }
            });
        }
        {
            const uint64_t m2 = f2(-mean, -mean), r2 = f2(rstd, rstd);
            uint64_t sa = 0, sb = 0;
#pragma unroll
            for (int j = 0; j < (V > 1 ? NV : NV / 2); ++j) {
                constexpr int P = V > 1 ? V : 2;
                float w[P];
                if constexpr (V > 1) {
                    load_v<V>(weight + j * kStep, w);
                } else {
                    w[0] = weight[2 * j * kStep];
                    w[1] = weight[(2 * j + 1) * kStep];
                }
#pragma unroll
                for (int q = 0; q < P; q += 2) {
                    const int e = j * P + q;
                    const uint64_t h = mul2(RMS ? two<V, NV>(xh, e) : add2(two<V, NV>(xh, e), m2), r2);
                    uint64_t d = two<V, NV>(g, e);
                    put2<V, NV>(dw, e, fma2(d, h, two<V, NV>(dw, e)));
                    put2<V, NV>(db, e, add2(d, two<V, NV>(db, e)));
                    d = mul2(d, f2(w[q], w[q + 1]));
                    sa = fma2(d, h, sa);
                    sb = add2(sb, d);
                    put2<V, NV>(xh, e, h);
                    put2<V, NV>(g, e, d);
                }
            }
            sum[0] = sum2(sa);
            sum[1] = sum2(sb);
        }
        row_sum<2>(sum, warps, group * warps, part[turn][0]);
        if (warps == 1) __syncthreads();  // the sums had no barrier
        // nobody reads the rows before any more
        if (warp == asker && before >= 0 && t0 + (st.stages - 1) * step < T) ring.ask(before, t0 + (st.stages - 1) * step, T);
        const float cx = sum[0] * inv * rstd, c = RMS ? 0.0f : sum[1] * inv * rstd;
        if (live) {
            const XT* ds = ring.row<XT, kWhole>(2, group, t) + cols.base;
            XT* dx = static_cast<XT*>(a.dx) + t * a.dxs + cols.base;
            cols.run([&](auto all) {
                const uint64_t r2 = f2(rstd, rstd), cx2 = f2(-cx, -cx), c2 = f2(-c, -c);
#pragma unroll
                for (int e = 0; e < N; e += 2)
                    put2<V, NV>(g, e, fma2(two<V, NV>(g, e), r2, fma2(two<V, NV>(xh, e), cx2, c2)));
#pragma unroll
                for (int j = 0; j < NV; ++j) {
                    if (!all && j * kStep >= limit) continue;
                    if (a.ds) {
                        float d[V];
                        load_v<V>(ds + j * kStep, d);
#pragma unroll
                        for (int q = 0; q < V; ++q) g[j][q] += d[q];
                    }
                    store_v<V>(dx + j * kStep, g[j]);
                }
            });
        }
        mean = mean_after;
        rstd = rstd_after;
        asker = asker + 1 == int(blockDim.x >> 5) ? 0 : asker + 1;
        before = ring.s;
        ring.next();
    }
    ring.end();
    if (a.part == nullptr) return;
    float* out = a.part + int64_t(blockIdx.x) * 2 * a.H;
    if (groups == 1) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (j * kStep >= limit) continue;
            store_v<V>(out + cols.base + j * kStep, dw[j]);  // V > 1: H is a multiple of V
            store_v<V>(out + a.H + cols.base + j * kStep, db[j]);
        }
        return;
    }
    float* rows = reinterpret_cast<float*>(mem);  // the row groups' sums, added in group order
    for (int r = 0; r < groups; ++r) {
        __syncthreads();
        if (r != group) continue;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (j * kStep >= limit) continue;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const int i = cols.base + j * kStep + q;
                rows[i] = (r ? rows[i] : 0.0f) + dw[j][q];
                rows[a.H + i] = (r ? rows[a.H + i] : 0.0f) + db[j][q];
            }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.H; i += blockDim.x) out[i] = rows[i];
}

// Rows too wide for that: dx of row blockIdx.x, read twice (the second time from cache)
template <typename XT, typename YT, bool RMS, int V>
__global__ void __launch_bounds__(kRowThreads) norm_backward_wide_kernel(NormBwd a) {
    __shared__ __align__(16) float part[2][kSumWarps];
    if (threadIdx.x < 32) part[0][threadIdx.x] = part[1][threadIdx.x] = 0.0f;
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    const XT* x = static_cast<const XT*>(a.x) + t * a.xs;
    const YT* dy = static_cast<const YT*>(a.dy) + t * a.dys;
    const XT* ds = a.ds ? static_cast<const XT*>(a.ds) + t * a.dss : nullptr;
    XT* dx = static_cast<XT*>(a.dx) + t * a.dxs;
    const float mean = RMS ? 0.0f : a.mean[t], rstd = a.rstd[t];
    float sum[2] = {0.0f, 0.0f};  // of g xhat, g
#pragma unroll 4
    for (int i = threadIdx.x * V; i < a.H; i += blockDim.x * V) {
        float xv[V], g[V], w[V];
        load_v<V>(x + i, xv);
        load_v<V>(dy + i, g);
        load_w<V>(a.w, i, a.w_bf16, w);
#pragma unroll
        for (int q = 0; q < V; ++q) {
            const float gq = g[q] * w[q];
            sum[0] = fmaf(gq, (xv[q] - mean) * rstd, sum[0]);
            sum[1] += gq;
        }
    }
    row_sum<2>(sum, blockDim.x >> 5, 0, part[0]);
    const float mgx = sum[0] / a.H, mg = RMS ? 0.0f : sum[1] / a.H;
#pragma unroll 4
    for (int i = threadIdx.x * V; i < a.H; i += blockDim.x * V) {
        float xv[V], g[V], w[V], d[V], o[V];
        load_v<V>(x + i, xv);
        load_v<V>(dy + i, g);
        load_w<V>(a.w, i, a.w_bf16, w);
        if (ds) load_v<V>(ds + i, d);
#pragma unroll
        for (int q = 0; q < V; ++q) {
            o[q] = rstd * (g[q] * w[q] - mg - (xv[q] - mean) * rstd * mgx);
            if (ds) o[q] += d[q];
        }
        store_v<V>(dx + i, o);
    }
}

// and their weight gradients: part[c] = sums of rows c, c + chunks, ...; a thread owns a column
template <typename XT, typename YT, bool RMS>
__global__ void __launch_bounds__(256) norm_wgrad_kernel(NormBwd a) {
    pdl_wait();
    pdl_trigger();
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= a.H) return;
    float dw = 0.0f, db = 0.0f;
#pragma unroll 8
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        float d[1], x[1];
        load_v<1>(static_cast<const YT*>(a.dy) + t * a.dys + i, d);
        load_v<1>(static_cast<const XT*>(a.x) + t * a.xs + i, x);
        dw = fmaf(d[0], (x[0] - (RMS ? 0.0f : a.mean[t])) * a.rstd[t], dw);
        db += d[0];
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

// dweight (blockIdx.y 0) or dbias of 32 columns from the blocks' sums: warp w adds the blocks
// w, w + 32, ... in order, then the warps' sums are added in warp order
constexpr int kReduceWarps = 32;
__global__ void __launch_bounds__(32 * kReduceWarps) norm_wgrad_reduce_kernel(const float* __restrict__ part, int chunks,
                                                                              int H, void* dw, void* db, bool bf16,
                                                                              bool add) {
    __shared__ float s_sum[kReduceWarps][33];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.x * 32 + lane;
    void* out = blockIdx.y == 0 ? dw : db;
    if (out == nullptr) return;
    float v = 0.0f;
    if (i < H) {
        const float* p = part + int64_t(blockIdx.y) * H + i;
#pragma unroll 10
        for (int c = warp; c < chunks; c += kReduceWarps) v += p[int64_t(c) * 2 * H];
    }
    s_sum[warp][lane] = v;
    __syncthreads();
    if (warp || i >= H) return;
#pragma unroll
    for (int w = 1; w < kReduceWarps; ++w) v += s_sum[w][lane];
    put_grad(out, i, v, bf16, add);
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

bool rows_aligned(const void* p, int64_t stride, int32_t type, size_t bytes) {
    const size_t es = type == MOE_T_BF16 ? 2 : 4;
    return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | (size_t(stride) * es)) & (bytes - 1)) == 0;
}

template <int N>
using Int = std::integral_constant<int, N>;

// Threads of a row of H columns, and of the block: rows of up to 128 threads share a block of 256.
struct RowShape {
    int tpr, threads;
};
RowShape row_shape(int64_t H) {
    const int tpr = (int((H + kColumns - 1) / kColumns) + 31) / 32 * 32;
    if (tpr <= 128) {
        int p = 32;
        while (p < tpr) p *= 2;
        return {p, 256};
    }
    return {tpr, tpr};
}

// The streamed kernels' shape, 16 columns a thread: row groups to a block of 256 threads (or one
// of more), and two such blocks an SM where shared memory holds two stages of each.
// Stages: `least`, and more up to `aim` bytes an SM. Reads that run far ahead of the writes cost memory rate once the
// rows do not stay in L2: the forward with a residual at 16384 x 4096 bf16 takes 84 us with two stages (64 KB), 92
// with three, 96 with five; at 16384 x 1024 24.3 with two and 22.9 with three. Without a residual more is better:
// 4000 x 8192 fp32 45 us with 96 KB, 41 with 176. The backward: 16384 x 4096 75 us with 128 KB, 70 with 176;
// 8192 x 7168 with a joining gradient 86 and 78; but 1500 x 4096 15.2 and 16.2, 3000 x 9001 75 and 85.
// 32 columns a thread: 52 against 57 us at 16384 x 4096 bf16, but 46 against 41 at 4000 x 8192 fp32 and 21.6 against
// 17.3 at 32768 x 512 bf16; 8 columns: 86 us.
constexpr int64_t kLargeBytes = int64_t(256) << 20;  // read and written: twice what L2 holds
constexpr int kStreamBytes = 176 << 10;  // most of an SM's shared memory that is asked for
struct StreamShape {
    int tpr, threads, blocks;
    size_t smem;
};
void add_input(Stream& st, const void* p, int64_t stride, int32_t type, int64_t H) {
    const int es = type == MOE_T_BF16 ? 2 : 4, i = st.arrays++;
    st.from[i] = static_cast<const char*>(p);
    st.step[i] = stride * es;
    st.row_bytes[i] = int(H) * es;
    st.at[i] = st.group_bytes;
    st.group_bytes += (int(H) * es + 15 + 15) / 16 * 16;
}
StreamShape stream_shape(int64_t H, int most, int64_t T, int least, int aim, bool weights, Stream& st) {
    int sms = 152, device = 0;
    if (cudaGetDevice(&device) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, device);
    const RowShape r = row_shape(H);
    const int groups = r.threads / r.tpr, stage = groups * st.group_bytes;
    int per = std::max(1, 512 / r.threads);  // 128 registers a thread
    if (2 * stage * per > kStreamBytes) per = 1;
    const size_t fixed = weights ? kColumns * r.tpr * sizeof(float) : 0;
    const int most_stages = std::min(kMaxStages, std::max(2, kStreamBytes / per / stage));
    st.stages = std::min(most_stages, std::max(least, aim / per / stage));
    // No more blocks than have rows. The backward's write partial sums, which have to stay small beside the rows: two rows
    // a group once there is a block for every SM (608 x 2048 bf16 8.7 us, 10.9 with one; 64 x 2048 7.5, 6.5 with one)
    const int64_t single = (T + groups - 1) / groups;
    const int64_t blocks = std::min<int64_t>(std::min(per * sms, most), weights && single > sms ? (single + 1) / 2 : single);
    const size_t sums = groups > 1 ? 2 * size_t(H) * sizeof(float) : 0;
    return {r.tpr, r.threads, int(blocks), fixed + std::max(size_t(st.stages) * size_t(stage), sums)};
}

// the shared memory that a kernel may ask for, said once for each device
template <auto Kernel>
cudaError_t allow_shared() {
    static std::atomic<uint64_t> said{0};
    int device = 0;
    cudaError_t e = cudaGetDevice(&device);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (device & 63);
    if (device < 64 && (said.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMostShared));
    if (e == cudaSuccess) said.fetch_or(bit, std::memory_order_release);
    return e;
}

template <auto Kernel, typename A>
cudaError_t launch_stream(const StreamShape& sh, A& a, Stream& st, cudaStream_t cs) {
    const cudaError_t e = allow_shared<Kernel>();
    if (e != cudaSuccess) return e;
    a.tpr = sh.tpr;
    count_launch();
    return launch_pdl(Kernel, dim3(unsigned(sh.blocks)), dim3(unsigned(sh.threads)), sh.smem, cs, a, st);
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
    NormFwd a{x, residual, weight, bias, sum, y, mean, rstd, x_stride, residual_stride, sum_stride, y_stride, T,
              int(H), 0, cfg->eps, cfg->w_type == MOE_T_BF16};
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const cudaError_t e = by_type(*cfg, [&](auto xt, auto yt, auto rms) {
        using X = decltype(xt);
        using Y = decltype(yt);
        constexpr bool R = decltype(rms)::value;
        constexpr int V = 16 / sizeof(X);
        constexpr size_t YB = V * sizeof(Y) < 16 ? V * sizeof(Y) : 16;
        const size_t wb = std::min<size_t>(16, V * (cfg->w_type == MOE_T_BF16 ? 2 : 4));
        const bool wide = H % V == 0 && rows_aligned(x, x_stride, cfg->x_type, 16) &&
                          rows_aligned(residual, residual_stride, cfg->x_type, 16) &&
                          (!residual || rows_aligned(sum, sum_stride, cfg->x_type, 16)) &&
                          rows_aligned(y, y_stride, cfg->y_type, YB) && rows_aligned(weight, 0, cfg->w_type, wb) &&
                          rows_aligned(bias, 0, cfg->w_type, wb);
        if (H <= kStreamed) {
            Stream st{};
            add_input(st, x, x_stride, cfg->x_type, H);
            if (residual) add_input(st, residual, residual_stride, cfg->x_type, H);
            const bool large = 4 * T * H * int64_t(sizeof(X)) > kLargeBytes;
            const StreamShape sh = !residual ? stream_shape(H, INT_MAX, T, 3, kStreamBytes, false, st)
                                   : large   ? stream_shape(H, INT_MAX, T, 2, 96 << 10, false, st)
                                             : stream_shape(H, INT_MAX, T, 3, 128 << 10, false, st);
            auto go = [&](auto nt) {
                constexpr int NT = decltype(nt)::value;
                return wide ? launch_stream<norm_forward_stream_kernel<X, Y, R, V, kColumns / V, NT>>(sh, a, st, cs)
                            : launch_stream<norm_forward_stream_kernel<X, Y, R, 1, kColumns, NT>>(sh, a, st, cs);
            };
            if (sh.smem <= kMostShared)
                return sh.threads <= kNarrow ? go(Int<kNarrow>{}) : sh.threads <= kWide ? go(Int<kWide>{}) : go(Int<kWidest>{});
        }
        count_launch();
        if constexpr (V * 4 * kRowThreads > kStreamed) {  // bf16: up to 16384 columns (fp32 rows of 8192 are streamed)
            if (wide && H / V <= 4 * kRowThreads)
                return launch_pdl(norm_forward_kernel<X, Y, R, V, 4>, dim3(unsigned(T)), dim3(unsigned((H / V + 127) / 128 * 32)), 0,
                                  cs, a);
        }
        return wide ? launch_pdl(norm_forward_wide_kernel<X, Y, R, V>, dim3(unsigned(T)), dim3(kRowThreads), 0, cs, a)
                    : launch_pdl(norm_forward_wide_kernel<X, Y, R, 1>, dim3(unsigned(T)), dim3(kRowThreads), 0, cs, a);
    });
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
    NormBwd a{dy, x, weight, dsum, mean, rstd, dx, static_cast<float*>(workspace), dy_stride, x_stride, dsum_stride,
              dx_stride, T, int(H), 0, cfg->w_type == MOE_T_BF16};
    int chunks = 0;
    cudaError_t e = cudaSuccess;
    if (T > 0) {
        e = by_type(*cfg, [&](auto xt, auto yt, auto rms) {
            using X = decltype(xt);
            using Y = decltype(yt);
            constexpr bool R = decltype(rms)::value;
            constexpr int V = 16 / sizeof(X), NV = kColumns / V;
            constexpr size_t YB = V * sizeof(Y) < 16 ? V * sizeof(Y) : 16;
            const size_t wb = std::min<size_t>(16, V * (cfg->w_type == MOE_T_BF16 ? 2 : 4));
            const bool wide = H % V == 0 && rows_aligned(x, x_stride, cfg->x_type, 16) &&
                              rows_aligned(dsum, dsum_stride, cfg->x_type, 16) &&
                              rows_aligned(dx, dx_stride, cfg->x_type, 16) &&
                              rows_aligned(dy, dy_stride, cfg->y_type, YB) && rows_aligned(weight, 0, cfg->w_type, wb);
            if (H <= kStreamed) {
                Stream st{};
                add_input(st, x, x_stride, cfg->x_type, H);
                add_input(st, dy, dy_stride, cfg->y_type, H);
                if (dsum) add_input(st, dsum, dsum_stride, cfg->x_type, H);
                // dy is read from shared memory in pieces too: its rows start on 16 bytes as well, or none is
                const bool w16 = wide && rows_aligned(dy, dy_stride, cfg->y_type, 16);
                const bool large = (dsum ? 4 : 3) * T * H * int64_t(sizeof(X)) > kLargeBytes;
                const StreamShape sh = stream_shape(H, kMaxChunks, T, 3, large ? kStreamBytes : 128 << 10, true, st);
                NormBwd b = a;
                if (!sums) b.part = nullptr;
                auto go = [&](auto nt) {
                    constexpr int NT = decltype(nt)::value;
                    chunks = sh.blocks;
                    return w16 ? launch_stream<norm_backward_kernel<X, Y, R, V, NV, NT>>(sh, b, st, s)
                               : launch_stream<norm_backward_kernel<X, Y, R, 1, kColumns, NT>>(sh, b, st, s);
                };
                if (sh.smem <= kMostShared)
                    return sh.threads <= kNarrow ? go(Int<kNarrow>{}) : sh.threads <= kWide ? go(Int<kWide>{}) : go(Int<kWidest>{});
            }
            count_launch();
            const dim3 grid{unsigned(T)}, block{kRowThreads};
            const cudaError_t r = wide ? launch_pdl(norm_backward_wide_kernel<X, Y, R, V>, grid, block, 0, s, a)
                                       : launch_pdl(norm_backward_wide_kernel<X, Y, R, 1>, grid, block, 0, s, a);
            if (r != cudaSuccess || !sums) return r;
            chunks = norm_chunks(T / 8);
            count_launch();
            return launch_pdl(norm_wgrad_kernel<X, Y, R>, dim3(unsigned((H + 255) / 256), unsigned(chunks)), dim3(256), 0,
                              s, a);
        });
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    if (sums) {
        e = launch_pdl(norm_wgrad_reduce_kernel, dim3(unsigned((H + 31) / 32), 2u), dim3(32 * kReduceWarps), 0, s,
                       static_cast<const float*>(workspace), chunks, int(H), dweight, dbias, g_type == MOE_G_BF16,
                       accumulate != 0);
        count_launch();
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
