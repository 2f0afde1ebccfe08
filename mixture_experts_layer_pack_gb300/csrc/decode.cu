// The layer for a few tokens in one launch:
//   out[t] = gate[t] SharedSwiGLU(x_t) + sum_s p[t,s] RoutedSwiGLU_{id[t,s]}(x_t).
//
// What bounds it is the reading of the chosen experts' weights, once: 3 H I values
// per expert for 6 H I operations per token that chose it. So the kernel is one
// stream of weights: a persistent cooperative launch of one block per SM, in which
// eight producer warps keep a ring of bulk copies (cp.async.bulk into shared memory,
// one mbarrier per slot) full from their first instruction to their last, and eight
// consumer warps each multiply the slots of their own row tile.
//
//  * A group is up to 8 NT tokens of one expert (the shared expert is one more
//    expert, with every token). Every block sorts the routes into groups for itself.
//  * A slot is 16 weight rows by KC columns, the weights as the 16-row operand of
//    mma.m16n8k16, and one warp's. Up to eight tiles of one group form a set; the warps
//    of a set share the columns' slice of the group's tokens, in a ring of its own.
//  * First product: a tile holds 8 gate rows and the 8 up rows of the same i, which
//    leaves g and u of a token in one thread: a = silu(g) u needs no exchange.
//    Second product: a warp keeps its 16 rows of H for a set of tiles and adds up
//    p y over the groups in shared memory. No warp waits for another's sums.
//  * Each block takes an equal, contiguous share of the first product's tiles, and of the
//    second product's slots. Row tiles that blocks share are summed by the block that
//    finishes last, from partial sums in global memory, in block order.
//  * Between the products the blocks wait for one another. The weights' producers do not:
//    they fill the ring with the second product's weights meanwhile.
//
// A thread loads 8 consecutive elements of a weight row and the same 8 of a token's
// row, which are the operands of two instructions if the sum's index is taken in that
// order. Tensor rate is not what limits it (most often a weight meets one token, and rarely more than 8).
// The activations a = silu(g) u go to the second product as two bf16 terms, hi + lo: off by at most 2^-16 of themselves,
// which the rounding of `out` to bf16 (2^-8) hides but for one value in some hundreds, next to a rounding boundary (64
// tokens: 344 of 131072 outputs are not the exact value's nearest, 115 of an fp32 evaluation's). A third term would cost
// half as many instructions and token bytes again in the second product.
// MXFP8 weights become f16 in registers (exact, one instruction a pair; bf16 takes
// four) and their block scales multiply the fp32 sums of 32 columns. Their tokens are
// f16 too: a slice of a token's row is scaled by the power of two that brings its
// largest value under 2^15, and the scale is taken back per slot. x (8 significant bits) is one f16 term then, off by
// at most 2^-39 of the slice's largest value (what lies under f16's smallest), and a, which is fp32, two, off by at
// most 2^-23 of it (a low term of up to 8 beside a high one of 2^14 and more).
//
// Measured (graph replays): H 2048, I 1024, E 96 top-6 in BF16 with 1, 8, 64 tokens 24 us (3.7 TB/s), 83 us (6.0),
// 205 us (5.8); H 7168, I 2048, E 128 top-6 in MXFP8 with 4 tokens 204 us (5.4).
#include <algorithm>
#include <cmath>
#include <memory>
#include <new>
#include <utility>

#include <cuda_fp16.h>

#include "../../include/moe.h"
#include "device_common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr size_t kDecodeAlign = 256;
constexpr int kConsumers = 8;        // consumer warps: tiles of a set
constexpr int kProducers = 8;        // producer warps
constexpr int kDecodeThreads = 32 * (kConsumers + kProducers);
constexpr int kSlots = 24;           // most slots of the weights' ring
constexpr int kTokenSlots = 8;       // most slots of the tokens' ring
constexpr int kSmemMax = 232448;     // shared memory a block can have (227 KB)

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
    bool shared;
    float limit;
    const __nv_bfloat16* x;
    int64_t xs;
    const int* ids;
    const float* probs;
    const __nv_bfloat16* gate_w;
    __nv_bfloat16* out;
    int64_t os;
    DecodeWeight w[W_COUNT];
    // the activations by position (below): bf16 routed weights: [chunks of I][2][chunk], their two bf16
    // terms; MXFP8 ones: [I] fp32
    void* acts;
    int act_row;              // 4-byte words of a position
    float* gate;              // [T]
    float* part;              // [blocks][2][8][T][16]: partial sums of shared sets of row tiles
    unsigned* counters;       // per row tile: blocks done with it; 0 between launches
    unsigned* barrier;        // top bit flips when every block has arrived
    int* status;
    // chunks of H and of I by weight type (the shared expert's, routed), tiles of I and H, and
    // what a slot of the shared expert costs beside one of a routed one
    int c1_shared, c1, c2_shared, c2, it, ht, shared_cost, routed_cost;
    // shared memory plan
    int max_groups;
    int slots, token_slots, token_slot_bytes;
    int tokens_off, ring_off;
};

// A build of the kernel: up to 8 NT tokens a group, slots of KC columns (with MXFP8 routed
// weights: of E4M3 weights; the shared expert's bf16 rows take half the columns in the
// same bytes). Row pitches are chosen so that the rows that one shared-memory pass of
// a warp touches (two of 64 bytes, or four of 32) lie in different banks.
template <int NT_, int KC_, bool MX_>
struct Build {
    static constexpr int NT = NT_, KC = KC_;
    static constexpr bool MX = MX_;
    static constexpr int CAP = 8 * NT;          // tokens of a group
    static constexpr int CH = NT == 1 ? 8 : 2;  // sets of sums: an instruction's result is late, its successor another's
    static constexpr int KB = MX ? KC / 2 : KC; // columns of a slot of bf16 weights
    static constexpr int P16 = 2 * KB + 64;     // pitch of a weight row of bf16
    static constexpr int P8 = KC + 32;          // pitch of a weight row of E4M3
    static constexpr int PS = KC / 8 + 16;      // pitch of a row's block scales, in fp32
    static constexpr int SCALES = 16 * P8;      // offset of the scales in a slot
    static constexpr int SLOT = MX ? 16 * (P8 + PS) : 16 * P16;
    static_assert(SLOT % 64 == 0 && SLOT >= 16 * P16, "slots start on 16 bytes and hold either type");
    static __host__ __device__ constexpr int columns(bool mx) { return MX && mx ? KC : KB; }
    // pitch of a token row of `terms` terms of kc columns
    static __host__ __device__ constexpr int token_pitch(int kc, int terms) { return 2 * kc * terms + 64; }
    static constexpr int ZEROS = 4 * KC;        // a token row of zeros, two terms
    static constexpr int TS = MX ? 128 : 0;     // a token slot starts with its tokens' scales
    static_assert(4 * CAP <= 128, "the scales fit");
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, int bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// d = a b + c on 16 x 16 weights and 16 x 8 tokens
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
    if (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, "
            "%12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, "
            "%11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// 2^(code - 127) of an E8M0 code; 255 is NaN
__device__ __forceinline__ float e8m0_value(uint32_t code) {
    return code == 255u ? __uint_as_float(0x7fffffffu) : e8m0_scale(code);
}

// four E4M3 codes -> two f16 pairs (exact; NaN stays NaN)
__device__ __forceinline__ void e4m3_to_f16(uint32_t q, uint32_t& lo, uint32_t& hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(q));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
// a value as two bf16 terms, hi + lo. A value that rounds past bf16's range keeps its highest bits as they are, and an
// infinity has no second term (inf - inf is NaN, which the sum would be then)
__device__ __forceinline__ __nv_bfloat16 high_bf16(float v) {
    const __nv_bfloat16 hi = __float2bfloat16_rn(v);
    return __hisinf(hi) ? __float2bfloat16_rz(v) : hi;
}
__device__ __forceinline__ float low_part(float v, float hi) { return isinf(v) ? 0.0f : v - hi; }
__device__ __forceinline__ float2 unpack_f16x2(uint32_t w) { return __half22float2(*reinterpret_cast<const __half2*>(&w)); }

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kConsumers) : "memory"); }

__device__ __forceinline__ unsigned load_acquire(const unsigned* p) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void add_release(unsigned* p, unsigned v) {
    asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
__device__ __forceinline__ unsigned add_acq_rel(unsigned* p, unsigned v) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}

// waits until the grid barrier's top bit differs from `before`; bounded: past the limit it
// records the timeout and goes on (every address that follows is valid either way)
__device__ __forceinline__ void grid_wait(const unsigned* bar, unsigned before, int* status) {
    const uint64_t t0 = globaltimer_ns();
    while (((load_acquire(bar) ^ before) & 0x80000000u) == 0) {
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            atomicOr(status, kStatusTimeout);
            return;
        }
    }
}

// An equal share: the first n mod blocks blocks have one item more than the others. Where
// block c's items of n begin, and the block that owns item u.
__device__ __forceinline__ int share(int n, int c, int blocks) {
    const int each = n / blocks;
    return each * c + min(c, n - each * blocks);
}
__device__ __forceinline__ int owner(int n, int u, int blocks) {
    const int each = n / blocks, more = n - each * blocks, wide = more * (each + 1);
    return u < wide ? u / (each + 1) : more + (u - wide) / each;
}


// The routes sorted by expert. Position p < T: token p of the shared expert (if any);
// the routed positions follow, by (expert, token). Group g: `count` positions from `start`.
struct Group {
    int expert;  // E: the shared expert
    int start;
    int count;
};

struct Tables {
    Group* groups;
    int* tok;       // token of a position
    float* coef;    // its weight in the sum: prob, or the output gate
    int n_shared;   // groups of the shared expert, which come first
    int n_groups;
};

// Sorts the routes, by the whole block. A token chooses an expert once, so an expert's
// tokens are a 64-bit mask, whatever order its bits are set in; counts and ranks are
// population counts. A row with a bad id keeps none of its routes.
// scratch: E masks, E starts, T k ids, 40 ints; id, prob: of route tid, already under way.
template <int CAP>
__device__ __forceinline__ void sort_routes(const DecodeArgs& a, Tables& tb, uint8_t* scratch, int id, float prob) {
    const int R = a.T * a.k, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kWarps = kDecodeThreads / 32;
    auto* s_mask = reinterpret_cast<unsigned long long*>(scratch);
    auto* s_bad = s_mask + a.E;
    int* s_start = reinterpret_cast<int*>(s_bad + 1);
    int* s_id = s_start + a.E;
    int* s_warp = s_id + R;
    for (int i = tid; i <= a.E; i += kDecodeThreads) s_mask[i] = 0;
    for (int r = tid; r < R; r += kDecodeThreads) s_id[r] = r == tid ? id : a.ids[r];
    __syncthreads();
    for (int r = tid; r < R; r += kDecodeThreads) {
        const int t = r / a.k, v = s_id[r];
        bool ok = v >= -1 && v < a.E;
        for (int i = t * a.k; i < r; ++i) ok &= v < 0 || s_id[i] != v;
        if (!ok) {
            atomicOr(s_bad, 1ull << t);
            if (blockIdx.x == 0) atomicOr(a.status, kStatusRouting);
        }
    }
    __syncthreads();
    const unsigned long long bad = *s_bad;
    for (int r = tid; r < R; r += kDecodeThreads) {
        const int t = r / a.k, v = s_id[r];
        if (v >= 0 && !((bad >> t) & 1)) atomicOr(s_mask + v, 1ull << t);
    }
    __syncthreads();
    // exclusive sums over the experts of (routes << 16 | groups); a thread has two experts
    int cnt[2], mine = 0;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int e = 2 * tid + q;
        cnt[q] = e < a.E ? __popcll(s_mask[e]) : 0;
        mine += cnt[q] << 16 | (cnt[q] + CAP - 1) / CAP;
    }
    static_assert(2 * kDecodeThreads >= 1024, "two experts a thread");
    int sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += x;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int before = sum - mine, total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        const int x = s_warp[w];
        if (w < warp) before += x;
        total += x;
    }
    tb.n_shared = a.shared ? (a.T + CAP - 1) / CAP : 0;
    tb.n_groups = tb.n_shared + (total & 0xffff);
    const int base = a.shared ? a.T : 0;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int e = 2 * tid + q, start = base + (before >> 16), g = tb.n_shared + (before & 0xffff);
        if (e < a.E) s_start[e] = start;
        const int ng = (cnt[q] + CAP - 1) / CAP;
        for (int i = 0; i < ng; ++i) tb.groups[g + i] = Group{e, start + i * CAP, min(CAP, cnt[q] - i * CAP)};
        before += cnt[q] << 16 | ng;
    }
    if (tid < tb.n_shared) tb.groups[tid] = Group{a.E, tid * CAP, min(CAP, a.T - tid * CAP)};
    __syncthreads();
    for (int r = tid; r < R; r += kDecodeThreads) {
        const int t = r / a.k, v = s_id[r];
        if (v < 0 || ((bad >> t) & 1)) continue;
        const int pos = s_start[v] + __popcll(s_mask[v] & ((1ull << t) - 1));
        tb.tok[pos] = t;
        tb.coef[pos] = r == tid ? prob : a.probs[r];
    }
    if (a.shared && tid < a.T) {
        tb.tok[tid] = tid;
        tb.coef[tid] = 1.0f;
    }
}

// The same for up to 32 routes, by one warp with a route a lane: no barrier of the block between its steps (a call for one
// token 1.5 us shorter). The number of routed groups goes to *n_routed.
template <int CAP>
__device__ __forceinline__ void sort_few(const DecodeArgs& a, const Tables& tb, int id, float prob, int* n_routed) {
    const int R = a.T * a.k, r = threadIdx.x & 31, t = r / a.k;
    const unsigned row = (a.k == 32 ? 0xffffffffu : (1u << a.k) - 1) << (t * a.k & 31), lower = (1u << r) - 1;
    const unsigned like = __match_any_sync(0xffffffffu, id);  // a lane past the routes has id -1
    const bool ok = id == -1 || (id >= 0 && id < a.E && !(like & row & lower));
    const unsigned bad = __ballot_sync(0xffffffffu, !ok);
    if (bad && r == 0 && blockIdx.x == 0) atomicOr(a.status, kStatusRouting);
    const bool live = r < R && id >= 0 && !(bad & row);
    const unsigned alive = __ballot_sync(0xffffffffu, live);
    const int same = __popc(like & alive), before = __popc(like & alive & lower);  // of this expert; and of a lower token
    const bool lead = live && before % CAP == 0;                                   // a group's first route
    const unsigned leads = __ballot_sync(0xffffffffu, lead);
    const int mine = live ? id : 0x7fffffff;
    int sum = 0;  // routes of lower experts, and << 16 their groups
    for (int j0 = 0; j0 < R; j0 += 8)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int v = __shfl_sync(0xffffffffu, mine, j0 + j);
            sum += v < mine ? 1 + (leads >> (j0 + j) << 16 & 0x10000) : 0;
        }
    const int less = sum & 0xffff, groups = sum >> 16;
    const int base = a.shared ? a.T : 0, pos = base + less + before;
    if (live) {
        tb.tok[pos] = t;
        tb.coef[pos] = prob;
    }
    if (lead) tb.groups[tb.n_shared + groups + before / CAP] = Group{id, pos, min(CAP, same - before)};
    if (r < tb.n_shared) tb.groups[r] = Group{a.E, r * CAP, min(CAP, a.T - r * CAP)};
    if (a.shared && r < a.T) {
        tb.tok[r] = r;
        tb.coef[r] = 1.0f;
    }
    if (r == 0) *n_routed = __popc(leads);
}

// A block's share. First product: tiles u = group * it + tile of I, from u_begin to u_end.
// Second product: slots of (set of 8 tiles of H, group, chunk, tile), the tile fastest. Shares
// are equal in cost: a slot of a routed group counts routed_cost, one of the shared expert shared_cost.
struct Plan {
    int n_shared;
    int c2_shared, c2, it, ht;
    int u_begin, u_end;
    int shared_cost, routed_cost;
    int q_shared, q;           // chunks of I over the shared groups, over all groups
    int tile_cost;             // of one tile of H: all its chunks
    int n2, cost2, blocks2;    // second product: slots, their cost, and the blocks that have any
    int s_begin, s_end;
    // the cost of the slots before s, and the first slot before which the cost is at least x
    __device__ __forceinline__ int cost_before(int s) const {
        const int set = s / (kConsumers * q), in = s - set * kConsumers * q;
        const int heavy = min(kConsumers, ht - set * kConsumers) * q_shared;
        return set * kConsumers * tile_cost + min(in, heavy) * shared_cost + max(in - heavy, 0) * routed_cost;
    }
    __device__ __forceinline__ int slot_at(int x) const {
        const int set = x / (kConsumers * tile_cost), in = x - set * kConsumers * tile_cost;
        const int heavy = min(kConsumers, ht - set * kConsumers) * q_shared, hc = heavy * shared_cost;
        return set * kConsumers * q + (in <= hc ? (in + shared_cost - 1) / shared_cost : heavy + (in - hc + routed_cost - 1) / routed_cost);
    }
    __device__ __forceinline__ int begin(int block) const { return slot_at(share(cost2, block, blocks2)); }
    // the second product's part: worked out when the first product's copies are under way
    __device__ __forceinline__ void second(const DecodeArgs& a, const Tables& tb) {
        const int c = blockIdx.x, n = gridDim.x;
        q_shared = tb.n_shared * a.c2_shared;
        q = q_shared + (tb.n_groups - tb.n_shared) * a.c2;
        tile_cost = q_shared * a.shared_cost + (q - q_shared) * routed_cost;
        n2 = q * a.ht;
        cost2 = tile_cost * a.ht;
        blocks2 = max(1, min(cost2 / max(a.shared_cost, a.routed_cost), n));  // no share is smaller than a slot: none is empty
        s_begin = c < blocks2 ? begin(c) : n2;
        s_end = c + 1 < blocks2 ? begin(c + 1) : n2;
    }
};

__device__ __forceinline__ Plan make_plan(const DecodeArgs& a, const Tables& tb) {
    Plan p;
    const int c = blockIdx.x, n = gridDim.x, routed = tb.n_groups - tb.n_shared;
    p.n_shared = tb.n_shared;
    p.c2_shared = a.c2_shared;
    p.c2 = a.c2;
    p.it = a.it;
    p.ht = a.ht;
    p.shared_cost = a.shared_cost;
    p.routed_cost = a.routed_cost;
    const int per_shared = a.c1_shared * a.shared_cost, per = a.c1 * a.routed_cost;  // of a tile of I
    const int cost_shared = a.it * tb.n_shared * per_shared, cost = cost_shared + a.it * routed * per;
    auto tile = [&](int x) {
        return x <= cost_shared ? (x + per_shared - 1) / per_shared
                                : a.it * tb.n_shared + (x - cost_shared + per - 1) / per;
    };
    p.u_begin = tile(share(cost, c, n));
    p.u_end = tile(share(cost, c + 1, n));
    return p;
}

// The first product's walk: sets of up to eight tiles of one group.
struct Tiles {
    int u, g, tile, size;
    __device__ __forceinline__ Tiles(const Plan& p) : u(p.u_begin), g(p.u_begin / p.it), tile(p.u_begin % p.it) { fit(p); }
    __device__ __forceinline__ void fit(const Plan& p) { size = min(kConsumers, min(p.u_end - u, p.it - tile)); }
    __device__ __forceinline__ bool more(const Plan& p) const { return u < p.u_end; }
    __device__ __forceinline__ void next(const Plan& p) {
        u += size;
        if ((tile += size) == p.it) {
            tile = 0;
            ++g;
        }
        fit(p);
    }
};

// The second product's walk: steps of (set, group, chunk), tiles [lo, hi) of the set.
struct Steps {
    int set, g, c, lo, hi, s;
    __device__ __forceinline__ static int width(const Plan& p, int set) { return min(kConsumers, p.ht - set * kConsumers); }
    __device__ __forceinline__ Steps(const Plan& p) : s(p.s_begin) {
        const int per = kConsumers * p.q;
        set = s / per;
        const int r = s - set * per, wd = width(p, set), q = r / max(wd, 1);
        lo = r - q * wd;
        const bool routed = q >= p.q_shared;
        const int in = routed ? q - p.q_shared : q, n = routed ? p.c2 : p.c2_shared;
        g = in / n;
        c = in - g * n;
        if (routed) g += p.n_shared;
        fit(p);
    }
    __device__ __forceinline__ void fit(const Plan& p) { hi = min(width(p, set), lo + p.s_end - s); }
    __device__ __forceinline__ bool more(const Plan& p) const { return s < p.s_end; }
    __device__ __forceinline__ void next(const Plan& p, int n_groups) {
        s += hi - lo;
        lo = 0;
        if (++c == (g >= p.n_shared ? p.c2 : p.c2_shared)) {
            c = 0;
            if (++g == n_groups) {
                g = 0;
                ++set;
            }
        }
        fit(p);
    }
};

// One k-step: the 16 x 32 weights (wa: row r, wb: row r + 8, 8 elements each) times 8 N tokens,
// whose elements start at px[t]. Two sets of sums keep two chains of instructions going: of
// the two halves of the step, or with TERMS 2 of the two terms of a token's row, which lie
// `gap` bytes apart. ZERO: the sums start from zero here.
template <bool F16, bool ZERO, int N, int TERMS>
__device__ __forceinline__ void k_step(float (*acc0)[4], float (*acc1)[4], const uint4& wa, const uint4& wb,
                                       const uint8_t* const (&px)[N], int k2, int gap) {
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
        for (int term = 0; term < TERMS; ++term) {
            const uint4 x = *reinterpret_cast<const uint4*>(px[t] + k2 + term * gap);
            float(&d0)[4] = term == 0 ? acc0[t] : acc1[t];
            float(&d1)[4] = term == 0 && TERMS == 2 ? acc0[t] : acc1[t];
            if (ZERO)
                mma_16816<F16>(d0, wa.x, wb.x, wa.y, wb.y, x.x, x.y, 0.0f, 0.0f, 0.0f, 0.0f);
            else
                mma_16816<F16>(d0, wa.x, wb.x, wa.y, wb.y, x.x, x.y, d0[0], d0[1], d0[2], d0[3]);
            if (ZERO && TERMS == 1)
                mma_16816<F16>(d1, wa.z, wb.z, wa.w, wb.w, x.z, x.w, 0.0f, 0.0f, 0.0f, 0.0f);
            else
                mma_16816<F16>(d1, wa.z, wb.z, wa.w, wb.w, x.z, x.w, d1[0], d1[1], d1[2], d1[3]);
        }
}

// acc += (16 weight rows at A) x (N tiles of 8 tokens at X), over n columns of a slot; `none`
// holds a row of zeros, for the tokens that a tile lacks
template <class B, int N, int TERMS>
__device__ __forceinline__ void multiply_tiles(float (&acc)[B::CH][B::NT][4], const uint8_t* A, const uint8_t* X,
                                               const uint8_t* none, int pitch, int count, int n, bool mx, int lane) {
    const int r = lane >> 2, c8 = (lane & 3) * 8;
    const uint8_t* px[N];
#pragma unroll
    for (int t = 0; t < N; ++t) px[t] = (8 * t + r < count ? X + (8 * t + r) * pitch : none) + 2 * c8;
    if (B::MX && mx) {
        const uint8_t *pa = A + r * B::P8 + c8, *S = A + B::SCALES + r * B::PS;
        float sum[2][N][4] = {};  // of this slot, in the tokens' scales
        auto step = [&](int k, float sa, float sb) {
            const uint2 qa = *reinterpret_cast<const uint2*>(pa + k);
            const uint2 qb = *reinterpret_cast<const uint2*>(pa + 8 * B::P8 + k);
            uint4 wa, wb;
            e4m3_to_f16(qa.x, wa.x, wa.y);
            e4m3_to_f16(qa.y, wa.z, wa.w);
            e4m3_to_f16(qb.x, wb.x, wb.y);
            e4m3_to_f16(qb.y, wb.z, wb.w);
            float d[2][N][4];
            k_step<true, true, N, TERMS>(d[0], d[1], wa, wb, px, 2 * k, 2 * B::KC);
#pragma unroll
            for (int t = 0; t < N; ++t)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    sum[h][t][0] = fmaf(sa, d[h][t][0], sum[h][t][0]);
                    sum[h][t][1] = fmaf(sa, d[h][t][1], sum[h][t][1]);
                    sum[h][t][2] = fmaf(sb, d[h][t][2], sum[h][t][2]);
                    sum[h][t][3] = fmaf(sb, d[h][t][3], sum[h][t][3]);
                }
        };
        int k = 0;
        for (; k + 128 <= n; k += 128) {  // four steps without a branch: with two warps a scheduler the loads have to overlap
            const float4 sa = *reinterpret_cast<const float4*>(S + k / 8);
            const float4 sb = *reinterpret_cast<const float4*>(S + 8 * B::PS + k / 8);
            step(k, sa.x, sb.x);
            step(k + 32, sa.y, sb.y);
            step(k + 64, sa.z, sb.z);
            step(k + 96, sa.w, sb.w);
        }
        for (; k < n; k += 32)  // n is a multiple of 32
            step(k, *reinterpret_cast<const float*>(S + k / 8), *reinterpret_cast<const float*>(S + 8 * B::PS + k / 8));
        const float* scale = reinterpret_cast<const float*>(X - B::TS) + 2 * (lane & 3);  // of this thread's tokens
#pragma unroll
        for (int t = 0; t < N; ++t) {
            const float2 f = *reinterpret_cast<const float2*>(scale + 8 * t);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[0][t][i] = fmaf(i & 1 ? f.y : f.x, sum[0][t][i] + sum[1][t][i], acc[0][t][i]);
        }
        return;
    }
    const uint8_t* pa = A + r * B::P16 + 2 * c8;
    const int whole = n & ~31;
    int k = 0;
    for (; k + 128 <= n; k += 128)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            k_step<false, false, N, TERMS>(acc[2 * j % B::CH], acc[(2 * j + 1) % B::CH],
                                           *reinterpret_cast<const uint4*>(pa + 2 * (k + 32 * j)),
                                           *reinterpret_cast<const uint4*>(pa + 8 * B::P16 + 2 * (k + 32 * j)), px,
                                           2 * (k + 32 * j), 2 * B::KB);
    for (; k < whole; k += 32)
        k_step<false, false, N, TERMS>(acc[0], acc[1], *reinterpret_cast<const uint4*>(pa + 2 * k),
                                       *reinterpret_cast<const uint4*>(pa + 8 * B::P16 + 2 * k), px, 2 * k, 2 * B::KB);
    if (whole < n) {  // some threads' columns lie past the end: zeros on both sides
        const bool in = whole + c8 < n;
        const int k2 = in ? 2 * whole : 0;
        uint4 wa = *reinterpret_cast<const uint4*>(pa + k2), wb = *reinterpret_cast<const uint4*>(pa + 8 * B::P16 + k2);
        if (!in) wa = wb = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int t = 0; t < N; ++t)
            if (!in) px[t] = none;
        k_step<false, false, N, TERMS>(acc[0], acc[1], wa, wb, px, k2, 2 * B::KB);
    }
}

template <class B, int TERMS>
__device__ __forceinline__ void multiply(float (&acc)[B::CH][B::NT][4], const uint8_t* A, const uint8_t* X,
                                         const uint8_t* none, int pitch, int count, int n, bool mx, int lane) {
    if (B::NT == 1 || count <= 8)
        multiply_tiles<B, 1, TERMS>(acc, A, X, none, pitch, count, n, mx, lane);
    else
        multiply_tiles<B, B::NT, TERMS>(acc, A, X, none, pitch, count, n, mx, lane);
}

// the sets of sums as one, in acc[0]
template <class B>
__device__ __forceinline__ void join(float (&acc)[B::CH][B::NT][4]) {
#pragma unroll
    for (int t = 0; t < B::NT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int c = 1; c < B::CH; ++c) acc[0][t][i] += acc[c][t][i];
}

// The rings' barriers, and the round (use) that each slot was last filled for. A barrier's
// parity tells a round from its neighbours only, and a warp does not take every use of a
// slot: so a warp looks for the round first, and then waits for the round's phase.
struct Bars {
    uint64_t full[kSlots], empty[kSlots], tfull[kTokenSlots], tempty[kTokenSlots];
    int filled[kSlots], tfilled[kTokenSlots];
    int met;  // 1 once the blocks have met: one thread of a block asks global memory
};

__device__ __forceinline__ int round_of(const int* p) {
    int v;
    asm volatile("ld.acquire.cta.shared.u32 %0, [%1];" : "=r"(v) : "r"(smem_u32(p)) : "memory");
    return v;
}
__device__ __forceinline__ void set_round(int* p, int v) {
    asm volatile("st.release.cta.shared.u32 [%0], %1;" ::"r"(smem_u32(p)), "r"(v) : "memory");
}
// waits for phase `round` of bar (if any), whose slot was or will be filled for that round; bounded like mbar_wait
__device__ __forceinline__ void wait_round(const int* filled, uint64_t* bar, int round, volatile int* abort, int* status) {
    if (round_of(filled) != round) {
        const uint64_t t0 = globaltimer_ns();
        while (round_of(filled) != round) {
            if (*abort) return;
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
                *abort = 1;
                atomicOr(status, kStatusTimeout);
                return;
            }
        }
    }
    if (bar) mbar_wait(bar, uint32_t(round) & 1, abort, status);
}

// the word of scale codes at c (any alignment), of which those below `end` are wanted
__device__ __forceinline__ uint32_t load_codes(const uint8_t* c, const uint8_t* end) {
    const unsigned shift = unsigned(reinterpret_cast<uintptr_t>(c) & 3);
    const uint32_t* w = reinterpret_cast<const uint32_t*>(c - shift);
    const uint32_t lo = __ldg(w);
    const uint32_t hi = shift && reinterpret_cast<const uint8_t*>(w + 1) < end ? __ldg(w + 1) : 0u;
    return __funnelshift_r(lo, hi, 8 * shift);
}

// One producer warp. Items (a set's token slice, then its weight slots) go round the warps:
// one warp issues a copy in about a hundred cycles, so it takes several to keep the memory
// busy (152 blocks of 1, 2, 4, 8 warps with 1 KB copies and 192 KB in flight: 1.7, 3.3,
// 6.6, 6.8 TB/s).
template <class B>
struct Producer {
    const DecodeArgs& a;
    const Tables& tb;
    Plan& p;
    uint8_t *ring, *tokens;
    Bars* bars;
    volatile int* abort;
    int pw, lane;
    int turn = 0, slot = 0, round = 0, tslot = 0, tround = 0;
    bool met = false;

    __device__ __forceinline__ bool mine() {
        const bool m = turn == pw;
        turn = turn + 1 == kProducers ? 0 : turn + 1;
        return m;
    }
    __device__ __forceinline__ void next_slot() {
        if (++slot == a.slots) {
            slot = 0;
            ++round;
        }
    }
    __device__ __forceinline__ void next_token_slot() {
        if (++tslot == a.token_slots) {
            tslot = 0;
            ++tround;
        }
    }
    // 16 rows (live: this lane has one, at src) of n columns into the next slot; with mx also
    // their scale codes: codes(r), row r's first (of rows past the end: any row's)
    template <typename F>
    __device__ __forceinline__ void weights(bool mx, bool live, int rows, const uint8_t* src, int n, F codes) {
        constexpr int W = B::KC / 256;  // words of codes of a lane: two lanes a row
        const uint8_t* first = nullptr;
        const int left = n / 32 - (lane & 1) * 4 * W;  // codes that are this lane's
        uint32_t code[W] = {};
        if (B::MX && mx) {
            first = codes(lane >> 1) + (lane & 1) * 4 * W;
            if ((reinterpret_cast<uintptr_t>(first) & (4 * W - 1)) == 0 && left >= 4 * W) {
                if (W == 4) {
                    const uint4 v = __ldg(reinterpret_cast<const uint4*>(first));
                    code[0] = v.x;
                    code[W > 1 ? 1 : 0] = v.y;
                    code[W > 2 ? 2 : 0] = v.z;
                    code[W > 3 ? 3 : 0] = v.w;
                } else {
                    const uint2 v = __ldg(reinterpret_cast<const uint2*>(first));
                    code[0] = v.x;
                    code[W > 1 ? 1 : 0] = v.y;
                }
            } else {
#pragma unroll
                for (int q = 0; q < W; ++q)
                    if (4 * q < left) code[q] = load_codes(first + 4 * q, first + left);
            }
        }
        if (round) wait_round(bars->filled + slot, bars->empty + slot, round - 1, abort, a.status);
        if (*abort) return;  // a wait gave up: nothing more is asked for
        __syncwarp();
        if (lane == 0) set_round(bars->filled + slot, round);
        uint8_t* A = ring + slot * B::SLOT;
        uint64_t* bar = bars->full + slot;
        const int bytes = B::MX && mx ? n : 2 * n;
        if (B::MX) fence_proxy_async_smem();  // copies may land where scales were written
        if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(rows * bytes));
        __syncwarp();
        if (live) bulk_load(A + lane * (B::MX && mx ? B::P8 : B::P16), src, bytes, bar);
        if (B::MX) {
            if (mx) {
                float4* to = reinterpret_cast<float4*>(A + B::SCALES + (lane >> 1) * B::PS) + (lane & 1) * W;
#pragma unroll
                for (int q = 0; q < W; ++q)
                    to[q] = make_float4(e8m0_value(code[q] & 255u), e8m0_value(code[q] >> 8 & 255u),
                                        e8m0_value(code[q] >> 16 & 255u), e8m0_value(code[q] >> 24));
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(bar);  // the scales are there
        }
    }
    // the next token slot, free; null after a wait that gave up
    __device__ __forceinline__ uint8_t* token_slot() {
        if (tround) wait_round(bars->tfilled + tslot, bars->tempty + tslot, tround - 1, abort, a.status);
        if (*abort) return nullptr;
        __syncwarp();
        if (lane == 0) set_round(bars->tfilled + tslot, tround);
        return tokens + tslot * a.token_slot_bytes;
    }
    // this lane's token row (if it has one) into the next token slot, as it is
    __device__ __forceinline__ void token_rows(int count, const void* src, int pitch, int bytes) {
        uint8_t* to = token_slot();
        if (to == nullptr) return;
        uint64_t* bar = bars->tfull + tslot;
        if (B::MX) fence_proxy_async_smem();  // copies may land where converted rows were written
        if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(count * bytes));
        __syncwarp();
        if (lane < count) bulk_load(to + B::TS + lane * pitch, src, bytes, bar);
    }
    // MXFP8: n columns of `count` rows into the next token slot as TERMS terms of f16 under a scale,
    // or (not F16) of bf16; load(r, c, v): 8 values of row r from column c
    template <bool F16, int TERMS, typename F>
    __device__ __forceinline__ void token_values(int count, int kc, int n, F load) {
        uint8_t* to = token_slot();
        if (to == nullptr) return;
        constexpr int V = B::KC / 256;  // 8-column pieces of a lane
        const int pitch = B::token_pitch(kc, TERMS);
        for (int r = 0; r < count; ++r) {
            float v[V][8], top = 0.0f;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const int c = (q * 32 + lane) * 8;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[q][i] = 0.0f;
                if (c < n) load(r, c, v[q]);
#pragma unroll
                for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[q][i]));  // fmaxf passes over NaN
            }
            float mul = 1.0f;
            if (F16) {
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int e = max(-113, min(126, 141 - int(__float_as_uint(top) >> 23)));  // top 2^e < 2^15
                mul = __uint_as_float(uint32_t(127 + e) << 23);
                if (lane == 0) reinterpret_cast<float*>(to)[r] = __uint_as_float(uint32_t(127 - e) << 23);
            }
            uint8_t* row = to + B::TS + r * pitch;
#pragma unroll
            for (int q = 0; q < V; ++q) {
                const int c = (q * 32 + lane) * 8;
                if (c >= n) continue;
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float x0 = v[q][2 * i] * mul, x1 = v[q][2 * i + 1] * mul;
                    if (F16) {
                        hi[i] = pack_f16x2(x0, x1);
                        const float2 h = unpack_f16x2(hi[i]);
                        lo[i] = TERMS == 2 ? pack_f16x2(low_part(x0, h.x), low_part(x1, h.y)) : 0u;
                    } else {
                        const float h0 = __bfloat162float(high_bf16(x0)), h1 = __bfloat162float(high_bf16(x1));
                        hi[i] = pack_bf16x2(h0, h1);
                        lo[i] = pack_bf16x2(low_part(x0, h0), low_part(x1, h1));
                    }
                }
                *reinterpret_cast<uint4*>(row + 2 * c) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                if (TERMS == 2) *reinterpret_cast<uint4*>(row + 2 * (kc + c)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bars->tfull + tslot);
    }

    __device__ __forceinline__ void run() {
        static_assert(B::CAP <= 32, "a lane copies a row");
        for (Tiles w(p); w.more(p); w.next(p)) {
            const Group gr = tb.groups[w.g];
            const bool routed = gr.expert < a.E, mx = B::MX && routed;
            const DecodeWeight& wg = a.w[routed ? W_GATE : W_SHARED_GATE];
            const DecodeWeight& wu = a.w[routed ? W_UP : W_SHARED_UP];
            const int e = routed ? gr.expert : 0, es = mx ? 1 : 2, kc = B::columns(mx);
            const uint8_t *bg = wg.expert(e), *bu = wu.expert(e);
            const __nv_bfloat16* x = a.x + (lane < gr.count ? tb.tok[gr.start + lane] : 0) * a.xs;
            for (int k0 = 0; k0 < a.H; k0 += kc) {
                const int n = min(kc, a.H - k0);
                if (mine()) {
                    if (mx)
                        token_values<true, 1>(gr.count, kc, n, [&](int r, int c, float (&v)[8]) {
                            const uint4 q = __ldg(reinterpret_cast<const uint4*>(a.x + tb.tok[gr.start + r] * a.xs + k0 + c));
                            unpack_bf16x2(q.x, v[0], v[1]);
                            unpack_bf16x2(q.y, v[2], v[3]);
                            unpack_bf16x2(q.z, v[4], v[5]);
                            unpack_bf16x2(q.w, v[6], v[7]);
                        });
                    else
                        token_rows(gr.count, x + k0, B::token_pitch(kc, 1), 2 * n);
                }
                next_token_slot();
                for (int q = 0; q < w.size; ++q, next_slot()) {
                    if (!mine()) continue;
                    const int i0 = (w.tile + q) * 8, rows = min(8, a.I - i0), i = i0 + (lane & 7);
                    const uint8_t* src = ((lane & 8) ? bu + i * wu.row_bytes : bg + i * wg.row_bytes) + int64_t(k0) * es;
                    weights(mx, lane < 16 && (lane & 7) < rows, 2 * rows, src, n, [&](int r) -> const uint8_t* {
                        const int64_t ir = i0 + min(r & 7, rows - 1);
                        return ((r & 8) ? wu.scales(e) + ir * (wu.row_bytes / 32) : wg.scales(e) + ir * (wg.row_bytes / 32)) + k0 / 32;
                    });
                }
            }
        }
        if (B::NT == 1) p.second(a, tb);
        for (Steps w(p); w.more(p); w.next(p, tb.n_groups)) {
            const Group gr = tb.groups[w.g];
            const bool routed = gr.expert < a.E, mx = B::MX && routed;
            const DecodeWeight& wd = a.w[routed ? W_DOWN : W_SHARED_DOWN];
            const int e = routed ? gr.expert : 0, es = mx ? 1 : 2, kc = B::columns(mx);
            const int k0 = w.c * kc, n = min(kc, a.I - k0);
            if (mine()) {
                if (!met) {  // the activations are there once the blocks have met
                    wait_round(&bars->met, nullptr, 1, abort, a.status);
                    __syncwarp();
                    asm volatile("fence.proxy.async;" ::: "memory");
                    met = true;
                }
                const float* act = static_cast<const float*>(a.acts) + int64_t(gr.start) * a.act_row + k0;
                auto load = [&](int r, int c, float (&v)[8]) {
                    const float4* f = reinterpret_cast<const float4*>(act + int64_t(r) * a.act_row + c);
                    const float4 lo = __ldcg(f), hi = __ldcg(f + 1);
                    v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
                    v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
                };
                if (!B::MX)  // two bf16 terms of a chunk take the chunk's words
                    token_rows(gr.count, act + int64_t(lane) * a.act_row, B::token_pitch(kc, 2), 2 * (kc + n));
                else if (mx)
                    token_values<true, 2>(gr.count, kc, n, load);
                else
                    token_values<false, 2>(gr.count, kc, n, load);
            }
            next_token_slot();
            const uint8_t* base = wd.expert(e);
            for (int q = w.lo; q < w.hi; ++q, next_slot()) {
                if (!mine()) continue;
                const int h0 = (w.set * kConsumers + q) * 16, rows = min(16, a.H - h0);
                weights(mx, lane < rows, rows, base + (h0 + lane) * wd.row_bytes + int64_t(k0) * es, n,
                        [&](int r) -> const uint8_t* {
                            return wd.scales(e) + (h0 + min(r, rows - 1)) * (wd.row_bytes / 32) + k0 / 32;
                        });
            }
        }
        if (*abort) {  // copies in flight land while the block still has its memory
            const uint64_t t0 = globaltimer_ns();
            while (globaltimer_ns() - t0 < 1000000) __nanosleep(1000);
        }
    }
};

// One consumer warp: tile `warp` of every set.
template <class B>
struct Consumer {
    const DecodeArgs& a;
    const Tables& tb;
    Plan& p;
    const uint8_t *ring, *tokens;
    Bars* bars;
    volatile int* abort;
    float* s_out;  // [T][16]: this warp's row tile of the second product
    const uint8_t* none;
    int warp, lane;
    int slot = 0, round = 0, tslot = 0, tround = 0;

    // the step of a set's chunk: `n` columns; f(A, X): multiply the warp's slot, if `at` (its number in the step) is one of `size`
    template <typename F>
    __device__ __forceinline__ void step(int at, int size, F f) {
        mbar_wait(bars->tfull + tslot, tround & 1, abort, a.status);
        if (at >= 0 && at < size) {
            int s = slot + at, r = round;
            while (s >= a.slots) {
                s -= a.slots;
                ++r;
            }
            wait_round(bars->filled + s, bars->full + s, r, abort, a.status);
            f(ring + s * B::SLOT, tokens + tslot * a.token_slot_bytes + B::TS);
            __syncwarp();
            if (lane == 0) mbar_arrive(bars->empty + s);
        } else {
            __syncwarp();  // every lane has seen this use of the token slot before it is given back
        }
        if (lane == 0) mbar_arrive(bars->tempty + tslot);
        slot += size;
        while (slot >= a.slots) {  // a ring of many tokens' block may have fewer slots than a set has tiles
            slot -= a.slots;
            ++round;
        }
        if (++tslot == a.token_slots) {
            tslot = 0;
            ++tround;
        }
    }

    __device__ __forceinline__ void gates() {  // the shared expert's output gates, one warp a token
        for (int t = blockIdx.x * kConsumers + warp; t < a.T; t += gridDim.x * kConsumers) {
            float v = 0.0f;
            for (int i = lane * 8; i < a.H; i += 256) {
                const uint4 x = *reinterpret_cast<const uint4*>(a.x + t * a.xs + i);
                const uint4 w = *reinterpret_cast<const uint4*>(a.gate_w + i);
                const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    float x0, x1, w0, w1;
                    unpack_bf16x2(xs[q], x0, x1);
                    unpack_bf16x2(ws[q], w0, w1);
                    v = fmaf(x0, w0, fmaf(x1, w1, v));
                }
            }
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) a.gate[t] = sigmoidf_(v);
        }
    }

    __device__ __forceinline__ void first() {
        for (Tiles w(p); w.more(p); w.next(p)) {
            const Group gr = tb.groups[w.g];
            const bool mx = B::MX && gr.expert < a.E;
            const int kc = B::columns(mx), pitch = B::token_pitch(kc, 1);
            float acc[B::CH][B::NT][4] = {};
            for (int k0 = 0; k0 < a.H; k0 += kc)
                step(warp, w.size, [&](const uint8_t* A, const uint8_t* X) {
                    multiply<B, 1>(acc, A, X, none, pitch, gr.count, min(kc, a.H - k0), mx, lane);
                });
            if (warp >= w.size) continue;
            join<B>(acc);
            const int i = (w.tile + warp) * 8 + (lane >> 2);
            if (i >= a.I) continue;
            // this thread has g and u of row i for tokens 8 t + 2 (lane & 3), and the next
#pragma unroll
            for (int t = 0; t < B::NT; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int n = 8 * t + 2 * (lane & 3) + j;
                    if (n >= gr.count) continue;
                    float g = acc[0][t][j], u = acc[0][t][2 + j];
                    if (a.limit > 0.0f) {  // comparisons, so that NaN passes through
                        g = g > a.limit ? a.limit : g;
                        u = u > a.limit ? a.limit : u < -a.limit ? -a.limit : u;
                    }
                    const float v = g * sigmoidf_(g) * u;
                    float* row = static_cast<float*>(a.acts) + int64_t(gr.start + n) * a.act_row;
                    if (B::MX) {
                        row[i] = v;
                    } else {
                        const __nv_bfloat16 hi = high_bf16(v);
                        __nv_bfloat16* d = reinterpret_cast<__nv_bfloat16*>(row + i / kc * kc) + i % kc;
                        d[0] = hi;
                        d[kc] = __float2bfloat16_rn(low_part(v, __bfloat162float(hi)));
                    }
                }
        }
    }

    __device__ __forceinline__ void put_out(int h0, int n_out) const {
        const int h = h0 + (lane & 15);
        if (h < a.H)
            for (int i = lane; i < n_out; i += 32) a.out[i / 16 * a.os + h] = __float2bfloat16_rn(s_out[i]);
    }

    // the blocks that share a set, and whether the first of them begins where the set does (the others begin inside it)
    struct Sharing {
        int first, last;
        bool whole;
    };
    __device__ __forceinline__ Sharing sharing(int set) const {
        const int s0 = set * kConsumers * p.q, first = owner(p.cost2, p.cost_before(s0), p.blocks2);
        return {first, owner(p.cost2, p.cost_before(s0 + p.q * Steps::width(p, set) - 1), p.blocks2), p.begin(first) == s0};
    }
    // out = bf16(sum) of this warp's row tile; a set that other blocks share goes through global memory
    __device__ __forceinline__ void flush(int set, const Sharing& sh) {
        const int tile = set * kConsumers + warp, n_out = a.T * 16;
        __syncwarp();
        if (tile < p.ht) {
            const int h0 = tile * 16;
            if (sh.first == sh.last) {
                put_out(h0, n_out);
            } else {
                // block b's partial sums of this set: in its first place if the set is where it begins
                auto part = [&](int b) {
                    return reinterpret_cast<float4*>(a.part + ((int64_t(b) * 2 + (b > sh.first || sh.whole ? 0 : 1)) * kConsumers + warp) * n_out);
                };
                float4* to = part(blockIdx.x);
                for (int i = lane; i < n_out / 4; i += 32) to[i] = reinterpret_cast<const float4*>(s_out)[i];
                __syncwarp();
                unsigned seen = 0;
                if (lane == 0) seen = add_acq_rel(a.counters + tile, 1u);
                if (__shfl_sync(0xffffffffu, seen, 0) == unsigned(sh.last - sh.first)) {
                    __syncwarp();  // what lane 0 acquired, every lane may read
                    float4* to_sum = reinterpret_cast<float4*>(s_out);
                    if (B::NT > 1) {  // many values: four of a block's at a time
                        for (int i = lane; i < n_out / 4; i += 32) to_sum[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        for (int b = sh.first; b <= sh.last; ++b) {
                            const float4* from = part(b);
#pragma unroll 4
                            for (int i = lane; i < n_out / 4; i += 32) {
                                const float4 v = __ldcg(from + i), d = to_sum[i];
                                to_sum[i] = make_float4(d.x + v.x, d.y + v.y, d.z + v.z, d.w + v.w);
                            }
                        }
                    }
                    for (int i = lane; B::NT == 1 && i < n_out / 4; i += 32) {  // few: of four blocks at a time
                        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        for (int b = sh.first; b <= sh.last; b += 4) {
                            float4 v[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) v[j] = __ldcg(part(min(b + j, sh.last)) + i);
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (b + j <= sh.last)
                                    sum = make_float4(sum.x + v[j].x, sum.y + v[j].y, sum.z + v[j].z, sum.w + v[j].w);
                        }
                        to_sum[i] = sum;
                    }
                    __syncwarp();
                    put_out(h0, n_out);
                    if (lane == 0) a.counters[tile] = 0;
                }
            }
        }
        __syncwarp();
        for (int i = lane; i < n_out; i += 32) s_out[i] = 0.0f;
        __syncwarp();
    }

    // w: at the block's first step; sh: of its set, worked out before it is needed where registers allow
    __device__ __forceinline__ void second(Steps w, Sharing sh) {
        while (w.more(p)) {
            const int g = w.g, set = w.set;
            const Group gr = tb.groups[g];
            const bool mx = B::MX && gr.expert < a.E;
            const int kc = B::columns(mx), pitch = B::token_pitch(kc, 2);
            float acc[B::CH][B::NT][4] = {};
            do {
                step(warp - w.lo, w.hi - w.lo, [&](const uint8_t* A, const uint8_t* X) {
                    multiply<B, 2>(acc, A, X, none, pitch, gr.count, min(kc, a.I - w.c * kc), mx, lane);
                });
                w.next(p, tb.n_groups);
            } while (w.more(p) && w.g == g && w.set == set);
            join<B>(acc);
#pragma unroll
            for (int t = 0; t < B::NT; ++t)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int n = 8 * t + 2 * (lane & 3) + j;
                    if (n >= gr.count) continue;
                    const float c = tb.coef[gr.start + n];
                    float* d = s_out + tb.tok[gr.start + n] * 16 + (lane >> 2);
                    d[0] = fmaf(c, acc[0][t][j], d[0]);
                    d[8] = fmaf(c, acc[0][t][2 + j], d[8]);
                }
            __syncwarp();
            if (!w.more(p) || w.set != set) {
                if (B::NT > 1) sh = sharing(set);
                flush(set, sh);
                if (B::NT == 1 && w.more(p)) sh = sharing(w.set);
            }
        }
    }
};

template <class B>
__global__ void __launch_bounds__(kDecodeThreads, 1) decode_kernel(const __grid_constant__ DecodeArgs a) {
    extern __shared__ __align__(128) uint8_t smem[];
    Bars* bars = reinterpret_cast<Bars*>(smem);
    int* s_abort = reinterpret_cast<int*>(bars + 1);
    Tables tb;
    tb.groups = reinterpret_cast<Group*>(s_abort + 4);
    tb.tok = reinterpret_cast<int*>(tb.groups + a.max_groups);
    tb.coef = reinterpret_cast<float*>(tb.tok + a.T * a.k + a.T);
    uint8_t *tokens = smem + a.tokens_off, *ring = smem + a.ring_off;
    uint8_t* none = tokens - B::ZEROS;
    float* s_out = reinterpret_cast<float*>(none - kConsumers * a.T * 16 * sizeof(float));  // [8][T][16]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int id = tid < a.T * a.k ? __ldg(a.ids + tid) : -1;
    const float prob = tid < a.T * a.k ? __ldg(a.probs + tid) : 0.0f;
    const unsigned before = __ldcg(a.barrier);  // no block can have passed: this one has not arrived
    if (tid < kSlots) {
        mbar_init(bars->full + tid, B::MX ? 2 : 1);  // the byte count's arrival, and the scales'
        mbar_init(bars->empty + tid, 1);
        bars->filled[tid] = -1;
        if (tid < kTokenSlots) {
            mbar_init(bars->tfull + tid, 1);
            mbar_init(bars->tempty + tid, kConsumers);
            bars->tfilled[tid] = -1;
        }
        fence_mbar_init();
    }
    if (tid == 0) {
        *s_abort = 0;
        bars->met = 0;
    }
    for (int i = tid; i < kConsumers * a.T * 16 + B::ZEROS / 4; i += kDecodeThreads) s_out[i] = 0.0f;
    const bool few = a.T * a.k <= 32;
    if (!few) {
        sort_routes<B::CAP>(a, tb, tokens, id, prob);  // its scratch: the rings' space
        fence_proxy_async_smem();
    } else {
        tb.n_shared = a.shared ? (a.T + B::CAP - 1) / B::CAP : 0;
        if (warp == 0) sort_few<B::CAP>(a, tb, id, prob, s_abort + 1);
    }
    __syncthreads();
    if (few) tb.n_groups = tb.n_shared + s_abort[1];
    if (tb.n_groups == 0) {  // nothing chosen and nothing shared, for every block alike
        for (int i = blockIdx.x * kDecodeThreads + tid; i < a.T * a.H; i += gridDim.x * kDecodeThreads)
            a.out[i / a.H * a.os + i % a.H] = __float2bfloat16_rn(0.0f);
        return;
    }
    Plan p = make_plan(a, tb);
    if (B::NT > 1) p.second(a, tb);  // no later: the code in the loops' middle costs 3 us at T = 64
    if (warp >= kConsumers) {
        Producer<B>{a, tb, p, ring, tokens, bars, s_abort, warp - kConsumers, lane}.run();
        return;
    }
    Consumer<B> c{a, tb, p, ring, tokens, bars, s_abort, s_out + warp * a.T * 16, none, warp, lane};
    if (a.gate_w) c.gates();
    c.first();
    // the blocks meet: every activation and gate is written
    asm volatile("fence.proxy.async.global;" ::: "memory");  // the activations are read by bulk copies
    consumer_sync();
    if (tid == 0) add_release(a.barrier, blockIdx.x == 0 ? 0x80000000u - (gridDim.x - 1) : 1u);
    if (B::NT == 1) p.second(a, tb);  // while the blocks arrive
    Steps w(p);
    typename Consumer<B>::Sharing sh{};
    if (B::NT == 1 && w.more(p)) sh = c.sharing(w.set);
    if (tid == 0) {
        grid_wait(a.barrier, before, a.status);
        set_round(&bars->met, 1);
    }
    if (a.gate_w) {
        consumer_sync();
        for (int t = tid; t < a.T; t += 32 * kConsumers) tb.coef[t] = __ldcg(a.gate + t);
        consumer_sync();
    }
    c.second(w, sh);
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
    if (c->hidden % step || c->inter % step || c->hidden > 32768 || c->inter > 32768) return MOE_ERR_UNSUPPORTED;
    *s = DecodeShape{c->max_tokens, c->hidden, c->num_experts, c->topk, c->inter, mx, c->no_shared_expert == 0,
                     c->swiglu_limit};
    return MOE_OK;
}

constexpr int kMaxBlocks = 256;
constexpr int kTableSets = MOE_DECODE_TABLE_SETS;

struct DecodeSpace {
    unsigned* state;      // [0] status, [1] barrier, then the row tiles' counters
    const void** tables;  // [3][kTableSets][2][E]: gate, up, down: payloads, scales
    float* gate;
    void* acts;
    float* part;
};

size_t state_words(const DecodeShape& s) { return 2 + size_t((s.H + 15) / 16); }

size_t carve_decode(const DecodeShape& s, uint8_t* base, DecodeSpace* w) {
    size_t off = 0;
    auto take = [&](size_t bytes) {
        uint8_t* p = base ? base + off : nullptr;
        off += (bytes + kDecodeAlign - 1) / kDecodeAlign * kDecodeAlign;
        return p;
    };
    const size_t T = size_t(s.Tmax), chunks = size_t((s.I + 1023) / 1024);
    w->state = reinterpret_cast<unsigned*>(take(state_words(s) * sizeof(unsigned)));
    w->tables = reinterpret_cast<const void**>(take(6 * size_t(kTableSets) * size_t(s.E) * sizeof(void*)));
    w->gate = reinterpret_cast<float*>(take(T * sizeof(float)));
    w->acts = take(T * size_t(s.k + 1) * chunks * 1024 * sizeof(float));
    w->part = reinterpret_cast<float*>(take(size_t(kMaxBlocks) * 2 * kConsumers * T * 16 * sizeof(float)));
    return off;
}

bool is16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

}  // namespace moe

struct moe_decoder {
    moe::DecodeShape s;
    moe::DecodeSpace ws;
    int device, blocks;
    // The sets of per-expert pointers that lie in the workspace, by matrix (gate, up, down), and the one being compared.
    // A set has one place as long as it is kept: a captured graph reads its table there with every replay, so a set that
    // was used under capture stays, and the others make room, the one used longest ago first.
    struct TableSet {
        std::unique_ptr<const void*[]> host;  // payloads, scales; null: the place is free
        uint64_t used = 0;
        bool captured = false;
    } sets[3][moe::kTableSets];
    std::unique_ptr<const void*[]> fresh;
    int last[3] = {0, 0, 0};  // the set of the call before
    uint64_t calls = 0;
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
        const size_t n = size_t(mx ? 2 * E : E);
        const void** want = d->fresh.get();
        for (int64_t e = 0; e < E; ++e) {
            want[e] = v.expert_ptrs[e];
            if (!want[e] || !is16(want[e])) return MOE_ERR_INVALID_ARG;
            if (mx && !(want[E + e] = v.expert_ptrs[2 * E + e])) return MOE_ERR_INVALID_ARG;
        }
        cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
        if (cudaStreamIsCapturing(st, &cap) != cudaSuccess) return MOE_ERR_CUDA;
        const bool capturing = cap != cudaStreamCaptureStatusNone;
        auto& sets = d->sets[slot];
        auto same = [&](int i) { return sets[i].host && std::equal(want, want + n, sets[i].host.get()); };
        int at = d->last[slot];
        if (!same(at))
            for (at = 0; at < kTableSets && !same(at);) ++at;
        auto place = [&](int i) { return d->ws.tables + (size_t(slot) * kTableSets + size_t(i)) * 2 * size_t(E); };
        if (at == kTableSets) {
            if (capturing) return MOE_ERR_STATE;
            for (int i = 0; i < kTableSets; ++i) {
                if (sets[i].captured) continue;
                if (!sets[i].host) {
                    at = i;
                    break;
                }
                if (at == kTableSets || sets[i].used < sets[at].used) at = i;
            }
            if (at == kTableSets) return MOE_ERR_STATE;
            auto& set = sets[at];
            std::unique_ptr<const void*[]> host = std::move(set.host);
            if (!host) host.reset(new (std::nothrow) const void*[n]);
            if (!host) return MOE_ERR_STATE;
            std::copy(want, want + n, host.get());
            // pageable source: staged before the call returns
            if (cudaMemcpyAsync(place(at), host.get(), n * sizeof(void*), cudaMemcpyHostToDevice, st) != cudaSuccess)
                return MOE_ERR_CUDA;
            set.host = std::move(host);
        }
        sets[at].used = ++d->calls;
        sets[at].captured |= capturing;
        d->last[slot] = at;
        const void* const* dev = place(at);
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

// Groups of up to 8 tokens: an expert that more tokens chose is read again for every 8 of them, from L2. With bf16
// weights groups of 32 (slots of half the columns, for the room that their tokens take) win once experts have more than
// some 16 tokens each. us, groups of 8 against 32: T 64, H 2048, I 1024: E 128 k 4 235 / 248, E 8 k 2 62 / 63,
// E 4 k 4 80 / 71; T 64, H 4096, I 2048, E 8 k 4 298 / 198; T 12, H 4096, I 1536, E 64 k 6 274 / 299. With MXFP8 weights
// groups of 16 lost to 8 everywhere (T 64, H 4096, I 2048, E 8 k 4: 470 against 336).
using Few16 = Build<1, 512, false>;
using More16 = Build<4, 256, false>;
using Few8 = Build<1, 1024, true>;

template <typename F>
cudaError_t by_build(bool mx, int64_t T, int64_t k, int64_t E, F f) {
    if (mx) return f(Few8());
    return T * k <= 16 * E ? f(Few16()) : f(More16());
}

template <class B>
cudaError_t launch_decode(DecodeArgs& a, int blocks, cudaStream_t st) {
    const int R = a.T * a.k, cap = std::min(B::CAP, a.T);
    auto up = [](int v) { return (v + 127) / 128 * 128; };
    a.max_groups = std::min(a.E, R) + R / B::CAP + (a.T + B::CAP - 1) / B::CAP;
    a.tokens_off = up(int(sizeof(Bars)) + 16 + a.max_groups * int(sizeof(Group)) + (R + a.T) * 8 +
                      kConsumers * a.T * 16 * int(sizeof(float)) + B::ZEROS);
    // the tokens' ring: about 48 KB, two slots at least
    a.token_slot_bytes = up(B::TS + cap * B::token_pitch(B::KC, 2));
    a.token_slots = std::min(kTokenSlots, std::max(2, 49152 / a.token_slot_bytes));
    a.ring_off = a.tokens_off + a.token_slots * a.token_slot_bytes;
    a.slots = std::min(kSlots, (kSmemMax - a.ring_off) / B::SLOT);
    const int scratch = 12 * a.E + 8 + 4 * R + 160;
    if (a.slots < 4 || a.tokens_off + scratch > kSmemMax) return cudaErrorInvalidConfiguration;
    a.act_row = (a.I + 1023) / 1024 * 1024;
    auto chunks = [](int n, bool mx) { return (n + B::columns(mx) - 1) / B::columns(mx); };
    a.c1_shared = chunks(a.H, false);
    a.c2_shared = chunks(a.I, false);
    a.c1 = chunks(a.H, true);
    a.c2 = chunks(a.I, true);
    a.it = (a.I + 7) / 8;
    a.ht = (a.H + 15) / 16;
    // E4M3 weights take more work a slot than the shared expert's bf16 ones. us at 4 : 4, 3 : 4, 2 : 4 of T, H, I, E, k:
    // 4, 7168, 2048, 128, 6 210 / 203 / 251; 64, 4096, 2048, 8, 2 264 / 239 / 255; 2, 1024, 512, 32, 4 18.3 / 17.6 / 18.9;
    // 1, 4096, 2048, 16, 2 34.9 / 34.0 / 34.0; 1, 2048, 1024, 64, 6 23.5 / 23.3 / 24.0; but 16, 4096, 1408, 64, 6
    // 232 / 239 / 272 and 64, 2048, 768, 128, 8 207 / 211 / 248. In groups of 32 the shared expert's are the full ones.
    a.shared_cost = B::MX || B::NT > 1 ? 3 : 2;
    a.routed_cost = B::MX ? 4 : 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(kDecodeThreads);
    cfg.dynamicSmemBytes = size_t(kSmemMax);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, decode_kernel<B>, a);
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
    std::unique_ptr<moe_decoder> d(new (std::nothrow) moe_decoder());
    if (!d) return MOE_ERR_INVALID_ARG;
    d->s = s;
    d->fresh.reset(new (std::nothrow) const void*[2 * size_t(s.E)]());
    if (!d->fresh) return MOE_ERR_INVALID_ARG;
    carve_decode(s, static_cast<uint8_t*>(workspace), &d->ws);
    int sms = 0;
    // A memset returns before it has run, and streams that do not wait for the default one would run a first call before
    // or during it: so it is waited for here.
    const cudaStream_t own = cudaStreamPerThread;
    if (cudaGetDevice(&d->device) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, d->device) != cudaSuccess ||
        cudaMemsetAsync(d->ws.state, 0, state_words(s) * sizeof(unsigned), own) != cudaSuccess ||
        cudaStreamSynchronize(own) != cudaSuccess)
        return MOE_ERR_CUDA;
    d->blocks = std::min(sms, kMaxBlocks);
    for (const int64_t T : {int64_t(1), int64_t(MOE_DECODE_MAX_TOKENS)})  // few tokens an expert, and many: both builds
        if (by_build(s.mx, T, 1, 1, [](auto b) {
                return cudaFuncSetAttribute(decode_kernel<decltype(b)>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                            kSmemMax);
            }) != cudaSuccess)
            return MOE_ERR_CUDA;
    *out = d.release();
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
    int device = 0;  // a launch goes to the current device, and the workspace and the number of blocks are of the decoder's
    if (cudaGetDevice(&device) != cudaSuccess) return MOE_ERR_CUDA;
    if (device != d->device) return MOE_ERR_INVALID_ARG;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    DecodeArgs a{};
    a.T = int(T);
    a.H = int(s.H);
    a.I = int(s.I);
    a.E = int(s.E);
    a.k = int(s.k);
    a.shared = s.shared;
    a.limit = s.limit;
    a.x = static_cast<const __nv_bfloat16*>(hidden);
    a.xs = hidden_stride;
    a.ids = topk_ids;
    a.probs = topk_probs;
    a.gate_w = static_cast<const __nv_bfloat16*>(w->shared_output_gate);
    a.out = static_cast<__nv_bfloat16*>(out);
    a.os = out_stride;
    a.acts = d->ws.acts;
    a.gate = d->ws.gate;
    a.part = d->ws.part;
    a.status = reinterpret_cast<int*>(d->ws.state);
    a.barrier = d->ws.state + 1;
    a.counters = d->ws.state + 2;
    const moe_wview* views[W_COUNT] = {&w->shared_gate, &w->shared_up,   &w->shared_down,
                                       &w->routed_gate, &w->routed_up, &w->routed_down};
    for (int i = s.shared ? 0 : 3; i < W_COUNT; ++i) {
        const bool down = i % 3 == 2;
        const moe_status r = decode_weight(d, *views[i], down ? s.H : s.I, down ? s.I : s.H, i >= 3, i % 3, st, &a.w[i]);
        if (r != MOE_OK) return r;
    }
    const cudaError_t e = by_build(s.mx, T, s.k, s.E, [&](auto b) { return launch_decode<decltype(b)>(a, d->blocks, st); });
    if (e == cudaErrorInvalidConfiguration) return MOE_ERR_UNSUPPORTED;
    count_launch();
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_decode_status(moe_decoder* d, void* stream) {
    using namespace moe;
    if (!d) return MOE_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    int v = 0;
    if (cudaMemcpyAsync(&v, d->ws.state, sizeof(int), cudaMemcpyDeviceToHost, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return MOE_ERR_CUDA;
    // After a wait that gave up the barrier and the counters start anew as well. Between this stream's calls, and done
    // when this returns: the next call may be on another stream.
    const size_t words = (v & kStatusTimeout) ? state_words(d->s) : 1;
    if (cudaMemsetAsync(d->ws.state, 0, words * sizeof(unsigned), st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
        return MOE_ERR_CUDA;
    if (v & kStatusTimeout) return MOE_ERR_TIMEOUT;
    if (v & kStatusRouting) return MOE_ERR_ROUTING;
    return MOE_OK;
}

}  // extern "C"
