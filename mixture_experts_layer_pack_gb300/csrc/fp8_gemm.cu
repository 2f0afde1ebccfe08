// Products of E4M3 matrices with one fp32 scale for a block of 128 (sm_103a).
//
//   out[m,n] = sum over blocks kb of 128 of  sa(m,kb) sb(n,kb) sum over k in kb of qa[m,k] qb[n,k]
//
// The inner sums are tcgen05.mma products of one K block (four K = 32 steps) into one of two TMEM buffers; the
// scales are arbitrary fp32 numbers, so the outer sum is the CUDA cores': the epilogue warps read each
// block's sums from TMEM and add them, scaled, to fp32 accumulators in registers, while the tensor
// cores fill the other buffer. For a block of a 128 x 256 tile the tensor cores take 512 cycles (8192 E4M3
// multiply-adds a cycle and SM), and the epilogue, if it is alone, 300: paired multiply-adds, as single ones leave the
// thread that issues the products too few issue slots (a block 737 cycles instead of 512, measured with nothing else).
//
// Warp 0 loads operands (TMA, 128-byte swizzle), warp 1 issues the products, warps 4..11 hold the accumulators: two warps a
// quarter of the 128 TMEM lanes, half of the columns each, and read their scales. A weight is stored once: the product with it
// and the one with its transpose read the same codes, K-major and MN-major (8-bit operands may be
// either), and so do the two operands of a weight's gradient, whose K are the tokens. A pair of CTAs shares a tile
// of 256 x 256 where there are tiles enough: each loads half of it, half of what two tiles of 128 x 256 would.
//
// Every wait is bounded; after one that gave up the results are NaN, and the device's status word says so.
#include "device_common.cuh"
#include "fp8.h"
#include "fp8_device.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kF8EpiWarps = 8;
constexpr int kF8Threads = 128 + 32 * kF8EpiWarps;
// Three warps share a quarter of the register file, 168 registers a thread at launch. An epilogue thread wants 128 accumulators and
// two sets of 16 sums, so the first warpgroup (loads and products) gives up what the two others take: 56 + 2 * 224 = 3 * 168. The compiler spills 8 bytes
// in the kernels of 128 columns and 20 in the pairs' weight's gradient, none in the others.
constexpr int kFewRegs = 56, kManyRegs = 224;
constexpr uint32_t kTileBytes = 128 * 128;   // 128 rows of 128 codes

__device__ int f8_gave_up;  // a wait on this device gave up since the status was last asked for

template <int OP, int BN, int CG>
struct F8Cfg {
    static constexpr uint32_t A_BYTES = kTileBytes;
    static constexpr uint32_t B_BYTES = BN / CG * 128;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = int(196608 / STAGE_BYTES);
    static constexpr int BUFS = 512 / BN;
    static constexpr size_t SMEM = size_t(STAGES) * STAGE_BYTES + (OP == F8_GU ? 3 * 2 * 128 * 4 : 0) + 1024 + 512;
    static_assert(SMEM <= 227 * 1024, "shared memory per CTA");
};

// ---------------------------------------------------------------- PTX
// Shared-memory descriptor, 128-byte swizzle, 8-row groups 1024 bytes apart: the low word's lowest 14 bits are the address / 16, so an
// offset is added to it; the high word is a constant
__device__ __forceinline__ uint32_t f8_desc_lo(uint32_t addr, uint32_t lbo) { return (addr >> 4) | (lbo >> 4) << 16; }
constexpr uint32_t kDescHi = (1024 >> 4) | 1u << 14 | 2u << 29;

// one lane of a warp, so that the compiler knows that its instructions are the warp's (a condition on the lane costs 3 % more)
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}
__device__ __forceinline__ uint32_t cta_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// shared::cluster address of the same place in the pair's first CTA
__device__ __forceinline__ uint32_t in_leader(const void* p) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}

template <int CG>
__device__ __forceinline__ void f8_load(void* dst, const void* map, uint32_t bar, int x, int y) {
    if (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
                smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], "
            "[%4];" ::"r"(smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
}

template <int CG>
__device__ __forceinline__ void f8_mma(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, uint32_t accumulate) {
    if (CG == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(kDescHi), "r"(accumulate)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b64 a, {%1, %4};\n\tmov.b64 b, {%2, %4};\n\t"
            "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], a, b, %3, p;\n\t}" ::"r"(d),
            "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(kDescHi), "r"(accumulate)
            : "memory");
}

// arrives on `bar` (CG 2: at the same place in both CTAs) once the products issued so far are complete
template <int CG>
__device__ __forceinline__ void f8_commit(uint64_t* bar) {
    if (CG == 1)
        mma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"(uint16_t(3))
            : "memory");
}

template <int CG>
__device__ __forceinline__ void f8_tmem_alloc(uint32_t* slot, uint32_t cols) {
    if (CG == 1) {
        tmem_alloc(slot, cols);
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}

template <int CG>
__device__ __forceinline__ void f8_tmem_free(uint32_t addr, uint32_t cols) {
    if (CG == 1)
        tmem_dealloc(addr, cols);
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}

// An arrival at a barrier of this CTA or of the pair's first (its shared::cluster address). What it orders are reads of TMEM, whose fence
// is tcgen05's own: release and acquire of the cluster's scope beside it made every block wait for a memory barrier
// (8192 x 7168 x 4096 forward: 519 us with them).
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// whether the phase of the given parity is complete; asks for up to 100 us before it says no (1 to 2 % less time than with the default)
__device__ __forceinline__ bool f8_ready(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 100000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// bounded wait; gives up when another role of the CTA did, or after kWaitLimitNs
__device__ __forceinline__ bool f8_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (f8_ready(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    while (true) {
        for (int i = 0; i < 16; ++i)
            if (f8_ready(bar, parity)) return true;
        if (*abort) return false;
        if (globaltimer_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            return false;
        }
    }
}

// The same for a warp. All lanes ask: one that asks for the others, and their vote, lengthens the way round of a buffer (8192 x 7168 x 4096
// forward 219 us, 204 like this).
__device__ __forceinline__ bool f8_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
    return __all_sync(0xffffffffu, f8_wait(bar, parity, abort));
}

// the same while winding down: whatever the others did
__device__ __forceinline__ void f8_drain(uint64_t* bar, uint32_t parity) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity) && globaltimer_ns() - t0 <= kWaitLimitNs) {
    }
}

// 32 lanes x 16 columns; the registers are valid after tmem_wait
__device__ __forceinline__ void tmem_ask16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
}

// 16 lanes x 16 columns, of which a thread gets rows lane / 4 (registers 0, 1, 4, 5) and lane / 4 + 8 (2, 3, 6, 7), columns 2 (lane % 4), + 1
// of the first eight and of the second
__device__ __forceinline__ void tmem_ask_pairs(uint32_t taddr, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// y += a b, both numbers of a pair
__device__ __forceinline__ void fma2(uint64_t& y, uint64_t a, uint64_t b) { asm volatile("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(y) : "l"(a), "l"(b)); }

// ---------------------------------------------------------------- work items
struct Item {
    int p;          // product (F8_TN)
    int m0, n0;     // first row of this CTA's 128 (its own of a pair), first column of the tile
    int ks;         // which part of the K blocks, [k_lo, k_hi)
    int k_lo, k_hi;
};

// Tiles go down the rows within a band of eight row tiles before they move to the next columns, so that the operands
// of the tiles that run at one time stay in L2.
template <int OP, int BN, int CG>
__device__ __forceinline__ Item f8_item(int i, const F8Args& a, uint32_t rank) {
    constexpr int TN = OP == F8_GU ? 128 : BN;
    constexpr int kBand = 8;
    Item t;
    t.ks = i % a.splits;
    int tile = i / a.splits;
    t.p = 0;
    if (OP == F8_TN)
        while (t.p + 1 < a.products && tile >= a.o[t.p].m_tiles * a.o[t.p].n_tiles) {
            tile -= a.o[t.p].m_tiles * a.o[t.p].n_tiles;
            ++t.p;
        }
    const int mt = a.o[t.p].m_tiles, nt = a.o[t.p].n_tiles;
    const int band = tile / (kBand * nt), in = tile - band * kBand * nt;
    const int rows = min(kBand, mt - band * kBand);
    t.m0 = ((band * kBand + in % rows) * CG + int(rank)) * 128;
    t.n0 = in / rows * TN;
    const int per = a.k_blocks / a.splits, more = a.k_blocks % a.splits;
    t.k_lo = t.ks * per + min(t.ks, more);
    t.k_hi = t.k_lo + per + (t.ks < more ? 1 : 0);
    return t;
}

// ---------------------------------------------------------------- results
// Where a product's results go
struct Sink {
    void* out;
    int64_t ld;
    bool bf16, add;
};
__device__ __forceinline__ Sink f8_sink(const F8Args& a, const Item& t, int part = 0, int parts = 1) {
    const F8Out& o = a.o[t.p];
    const bool split = a.splits > 1;
    Sink s;
    s.out = split ? static_cast<void*>(o.partial + int64_t(t.ks * parts + part) * o.M * o.ld_partial) : o.out;
    s.ld = split ? o.ld_partial : o.ld;
    s.bf16 = !split && o.bf16;
    s.add = !split && o.accumulate;
    return s;
}

// 32 bytes, a whole sector, at once
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                 "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// A thread's N columns of its row, by whole sectors
template <int N>
__device__ __forceinline__ void row_store(const F8Out& o, const Sink& s, int row, int col, const float* v) {
    if (row >= o.M) return;
    const int64_t at = int64_t(row) * s.ld + col;
    if (s.bf16) {
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(s.out) + at;
#pragma unroll
        for (int c = 0; c < N / 16; ++c) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = pack_bf16x2(v[16 * c + 2 * j], v[16 * c + 2 * j + 1]);
            store32(dst + 16 * c, w);
        }
    } else {
        float* dst = static_cast<float*>(s.out) + at;
#pragma unroll
        for (int c = 0; c < N / 8; ++c) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * c + j]);
            store32(dst + 8 * c, w);
        }
    }
}

// The same, `left` of the columns the matrix's, of a row that starts anywhere: the words move up by the row's offset in its first piece
// of 32 bytes (bf16: 16, fewer results are single ones then), in steps of selections, and go out by whole pieces but for the ends. (Through shared memory, 16
// columns at a time: 8192 x 2048 to 2050 81 us, so 53.)
template <int N, typename Y>
__device__ __forceinline__ void row_ragged(Y* to, int left, const float* v) {
    constexpr int BYTES = sizeof(Y) == 4 ? 32 : 16;
    constexpr int W = BYTES / 4, PER = BYTES / int(sizeof(Y)), WORDS = N * int(sizeof(Y)) / 4;  // words and results of a piece
    const int o = int(reinterpret_cast<uintptr_t>(to) & (BYTES - 1)) / int(sizeof(Y));
    to -= o;
    const int end = min(left, N) + o;  // results [o, end) from there
    const int s = sizeof(Y) == 2 ? o >> 1 : o;
    auto word = [&](int i) -> uint32_t {
        if (i >= WORDS) return 0u;
        if constexpr (sizeof(Y) == 4)
            return __float_as_uint(v[i]);
        else
            return pack_bf16x2(v[2 * i], v[2 * i + 1]);
    };
    uint32_t last[W], before = 0;
#pragma unroll
    for (int j = 0; j < W; ++j) last[j] = 0;
#pragma unroll
    for (int k = 0; k <= N / PER; ++k) {
        uint32_t w[2 * W];
#pragma unroll
        for (int j = 0; j < W; ++j) {
            w[j] = last[j];
            uint32_t x = word(W * k + j);
            if constexpr (sizeof(Y) == 2) {
                const uint32_t y = x;
                x = o & 1 ? __funnelshift_l(before, x, 16) : x;
                before = y;
            }
            last[j] = w[W + j] = x;
        }
#pragma unroll
        for (int bit = W / 2; bit >= 1; bit /= 2)
#pragma unroll
            for (int j = 2 * W - 1; j >= W - bit + 1; --j) w[j] = s & bit ? w[j - bit] : w[j];
        const int from = k == 0 ? o : 0, to_end = end - k * PER;  // of this piece
        Y* p = to + k * PER;
        if (from == 0 && to_end >= PER) {
            if constexpr (W == 8) {
                const uint32_t x[8] = {w[8], w[9], w[10], w[11], w[12], w[13], w[14], w[15]};
                store32(p, x);
            } else {
                *reinterpret_cast<uint4*>(p) = make_uint4(w[4], w[5], w[6], w[7]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j)
                if (j >= from && j < to_end) {
                    if constexpr (sizeof(Y) == 4)
                        p[j] = __uint_as_float(w[W + j]);
                    else
                        reinterpret_cast<unsigned short*>(p)[j] = static_cast<unsigned short>(w[W + (j >> 1)] >> (16 * (j & 1)));
                }
        }
    }
}

// 16 codes of one row; the row's bytes past N are not the product's to write
__device__ __forceinline__ void put_codes(uint8_t* row, int col, int N, const float* v, float r) {
    uint4 w;
    w.x = e4m3x4(v[0] * r, v[1] * r, v[2] * r, v[3] * r);
    w.y = e4m3x4(v[4] * r, v[5] * r, v[6] * r, v[7] * r);
    w.z = e4m3x4(v[8] * r, v[9] * r, v[10] * r, v[11] * r);
    w.w = e4m3x4(v[12] * r, v[13] * r, v[14] * r, v[15] * r);
    if (col + 16 <= N) {
        *reinterpret_cast<uint4*>(row + col) = w;
    } else {
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int z = 0; z < 16; ++z)
            if (col + z < N) row[col + z] = uint8_t(x[z >> 2] >> (8 * (z & 3)));
    }
}

// h = silu(g) u of a row's 64 columns (g in acc[0, 64), u in acc[64, 128)), stored as codes with the scale of the row's 128:
// the other 64 are the partner warp's, and the two exchange their largest magnitudes through `most`. g and u are stored
// first where they are kept, so that h can take g's registers: the logistic function's two slow instructions (16 a cycle and SM)
// run once an element.
__device__ __forceinline__ void gated_results(const F8Args& a, const Item& t, float (&acc)[128], int q, int half, float* most) {
    const int lane = threadIdx.x & 31;
    const int row = t.m0 + q * 32 + lane, col = t.n0 + 64 * half, N = a.o[0].N;
    const bool store = row < a.o[0].M;
    const int64_t sat = int64_t(t.n0 >> 7) * a.o[0].M + row;
    float* mine = most + (half * 128 + q * 32 + lane);
    const float* other = most + ((half ^ 1) * 128 + q * 32 + lane);
    auto meet = [&] { asm volatile("bar.sync %0, 64;" ::"r"(1 + q) : "memory"); };
    if (a.g) {
        float mg = 0.0f, mu = 0.0f;
#pragma unroll
        for (int j = 0; j < 64; ++j) mg = fmaxf(mg, fabsf(acc[j])), mu = fmaxf(mu, fabsf(acc[64 + j]));
        mine[0] = mg;
        mine[256] = mu;
        meet();
        const float sg = block_scale(fmaxf(mg, other[0])), su = block_scale(fmaxf(mu, other[256]));
        if (store) {
            if (half == 0) a.gs[sat] = sg, a.us[sat] = su;
            const float rg = __frcp_rn(sg), ru = __frcp_rn(su);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                put_codes(a.g + int64_t(row) * a.ld_g, col + 16 * c, N, acc + 16 * c, rg);
                put_codes(a.u + int64_t(row) * a.ld_u, col + 16 * c, N, acc + 64 + 16 * c, ru);
            }
        }
    }
    float mh = 0.0f;
    const bool clamp = a.limit > 0.0f;
#pragma unroll
    for (int j = 0; j < 64; ++j) {
        float g = acc[j], u = acc[64 + j];
        if (clamp) g = clamp_top(g, a.limit), u = clamp_both(u, a.limit);
        acc[j] = g * sigmoidf_(g) * u;
        mh = fmaxf(mh, fabsf(acc[j]));
    }
    mine[512] = mh;
    meet();
    const float sh = block_scale(fmaxf(mh, other[512]));
    if (store) {
        if (half == 0) a.hs[sat] = sh;
        const float rh = __frcp_rn(sh);
#pragma unroll
        for (int c = 0; c < 4; ++c) put_codes(a.h + int64_t(row) * a.ld_h, col + 16 * c, N, acc + 16 * c, rh);
    }
    meet();  // both have read before the next tile's are written
}

// ---------------------------------------------------------------- a weight's gradient
// Its columns have scales of their own, a vector for each block of tokens. A thread therefore takes four rows (lane / 4 + 8 i) and
// HALF / 4 columns, in adjacent pairs, instead of a row: HALF / 4 scales from global memory a block, not HALF from shared memory (which
// the products keep busy: 1950 cycles a block). acc[4 g + i]: row i, columns 8 g + 2 (lane % 4), + 1.
template <int BN, int CG>
__device__ __forceinline__ bool column_sums(const F8Scales& s, const F8Out& o, const Item& t, uint64_t (&acc)[BN / 4], uint32_t lanes, int q,
                                            int half, uint64_t* tfull, uint32_t given, int& buf, uint32_t& bphase, bool ok, volatile int* abort) {
    constexpr int HALF = BN / 2, BUFS = 512 / BN;
    const int lane = threadIdx.x & 31;
    const int col = t.n0 + HALF * half + 2 * (lane & 3);
    const float* pc = s.b + t.k_lo * s.ld_b + col;
    const float* pr[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) pr[i] = s.a + t.k_lo * s.ld_a + min(t.m0 + q * 32 + (lane >> 2) + 8 * i, o.M - 1);
    const bool paired = ((reinterpret_cast<uintptr_t>(s.b) & 7) | (s.ld_b & 1)) == 0 && t.n0 + BN <= o.N;
    uint64_t cs[HALF / 8];
    float r[4];
    auto fetch = [&] {
        if (paired) {
#pragma unroll
            for (int g = 0; g < HALF / 8; ++g) cs[g] = __ldg(reinterpret_cast<const unsigned long long*>(pc + 8 * g));
        } else {
#pragma unroll
            for (int g = 0; g < HALF / 8; ++g)
                cs[g] = pair(col + 8 * g < o.N ? __ldg(pc + 8 * g) : 0.0f, col + 8 * g + 1 < o.N ? __ldg(pc + 8 * g + 1) : 0.0f);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = __ldg(pr[i]);
    };
    if (t.k_lo < t.k_hi) fetch();
    for (int kb = t.k_lo; kb < t.k_hi; ++kb) {
        if (ok) ok = f8_wait_warp(&tfull[buf], bphase, abort);
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = lanes + uint32_t(buf * BN + HALF * half);
        uint64_t r2[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r2[i] = pair(r[i], r[i]);
#pragma unroll
        for (int c = 0; c < HALF / 16; ++c) {
            uint32_t v[16];
            tmem_ask_pairs(at + 16 * c, v);
            tmem_ask_pairs(at + 16 * c + (16u << 16), v + 8);
            tmem_wait();
            if (c == HALF / 16 - 1) {  // the buffer is read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(given + 8 * buf);
            }
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t* x = v + 8 * (i >> 1) + 4 * z + 2 * (i & 1);
                    fma2(acc[4 * (2 * c + z) + i], pair(x[0], x[1]), mul2(r2[i], cs[2 * c + z]));
                }
        }
        if (kb + 1 < t.k_hi) {
            pc += s.ld_b;
#pragma unroll
            for (int i = 0; i < 4; ++i) pr[i] += s.ld_a;
            fetch();
        }
        if (++buf == BUFS) buf = 0, bphase ^= 1;
    }
    return ok;
}

// The sums of column_sums to their place, or added to it; four lanes write 8 adjacent columns of a row. What is added to is read B pairs at a time:
// one after the other, each behind the store before it, 4096 x 4096 took 80 us more in bf16 and 16 in fp32 than the results alone.
template <int HALF, bool ADD, typename Y>
__device__ __forceinline__ void column_whole(const F8Out& o, const Item& t, Y* out, int64_t ld, const uint64_t (&acc)[HALF / 2], int q, int half) {
    constexpr int G = HALF / 8, B = 8;
    const int lane = threadIdx.x & 31;
    const int col = t.n0 + HALF * half + 2 * (lane & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = t.m0 + q * 32 + (lane >> 2) + 8 * i;
        if (row >= o.M) continue;
        Y* p = out + int64_t(row) * ld + col;
#pragma unroll
        for (int g0 = 0; g0 < G; g0 += B) {
            Two<Y> old[B];
#pragma unroll
            for (int g = 0; g < B; ++g)
                if (ADD) old[g] = load_two(p + 8 * (g0 + g));
#pragma unroll
            for (int g = 0; g < B; ++g) {
                float a, b;
                unpair(acc[4 * (g0 + g) + i], a, b);
                save_two<ADD>(p + 8 * (g0 + g), a, b, old[g]);
            }
        }
    }
}

// The same of a tile past the last column or of rows whose pairs are not aligned, which takes pairs (b, a') of a lane and the next
// one then: written element by element a tile of 128 x 256 took 9 us in fp32 and 12 in bf16, this way 5, whole ones 3. Without `add` the
// results are added to zero: a way of its own for each made every tile of the others half a microsecond longer.
template <int HALF, typename Y>
__device__ __forceinline__ void column_ragged(const F8Out& o, const Item& t, Y* out, int64_t ld, bool add, const uint64_t (&acc)[HALF / 2], int q, int half) {
    constexpr int G = HALF / 8, B = 2;
    const int lane = threadIdx.x & 31, quad = lane & 3, next = (lane & 28) | ((lane + 1) & 3);
    const int col = t.n0 + HALF * half + 2 * quad;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = t.m0 + q * 32 + (lane >> 2) + 8 * i;
        Y* p = out + int64_t(row) * ld + col;
        const int odd = int(reinterpret_cast<uintptr_t>(p) / sizeof(Y)) & 1;
        const int left = row < o.M ? o.N - col - odd : 0;                        // columns from p + odd on
        const int most = odd && quad == 3 ? min(left, 8 * G - 7) : left;        // (the last lane's second of the last pair is another tile's)
        float a, b, c, d;
        unpair(acc[i], a, b);
        if (odd && quad == 0 && row < o.M && col < o.N) save_one<true>(p, a, add ? load_one(p) : 0.0f);
        p += odd;
#pragma unroll
        for (int g0 = 0; g0 < G; g0 += B) {
            float lo[B], hi[B];
            Two<Y> old[B];
#pragma unroll
            for (int z = 0; z < B; ++z) {
                const int g = g0 + z;
                unpair(acc[4 * (g + 1 < G ? g + 1 : g) + i], c, d);
                const float after = __shfl_sync(0xffffffffu, quad == 0 ? c : a, next);
                lo[z] = odd ? b : a, hi[z] = odd ? after : b;
                a = c, b = d;
                old[z] = Two<Y>();
                if (add) {
                    if (8 * g + 1 < most)
                        old[z] = load_two(p + 8 * g);
                    else if (8 * g < left)
                        old[z] = load_first(p + 8 * g);
                }
            }
#pragma unroll
            for (int z = 0; z < B; ++z) {
                const int g = g0 + z;
                if (8 * g + 1 < most)
                    save_two<true>(p + 8 * g, lo[z], hi[z], old[z]);
                else if (8 * g < left)
                    save_one<true>(p + 8 * g, lo[z], first_of(old[z]));
            }
        }
    }
}

// (One of the ways is taken as a whole: with the choice at each element the code is as long as all of them, and fetching it, once a tile,
// took several times the writing.)
template <int HALF, typename Y>
__device__ __forceinline__ void column_store(const F8Out& o, const Item& t, Y* out, int64_t ld, bool add, const uint64_t (&acc)[HALF / 2], int q, int half) {
    // partial sums have room for whole tiles
    const bool whole = (static_cast<void*>(out) != o.out || t.n0 + 2 * HALF <= o.N) &&
                       ((reinterpret_cast<uintptr_t>(out) | uintptr_t(ld) * sizeof(Y)) & (2 * sizeof(Y) - 1)) == 0;
    if (whole && add)
        column_whole<HALF, true>(o, t, out, ld, acc, q, half);
    else if (whole)
        column_whole<HALF, false>(o, t, out, ld, acc, q, half);
    else
        column_ragged<HALF>(o, t, out, ld, add, acc, q, half);
}

// ---------------------------------------------------------------- the kernel
template <int OP, int BN, int CG>
__global__ void __launch_bounds__(kF8Threads, 1) f8_gemm_kernel(const __grid_constant__ F8Maps maps, const __grid_constant__ F8Args a) {
    using C = F8Cfg<OP, BN, CG>;
    constexpr bool A_MN = OP == F8_TN, B_MN = OP == F8_TN || OP == F8_NN;
    constexpr uint32_t IDESC = (1u << 4) | ((A_MN ? 1u : 0u) << 15) | ((B_MN ? 1u : 0u) << 16) | (uint32_t(BN >> 3) << 17) |
                               (uint32_t(128 * CG >> 4) << 24);  // E4M3 operands, fp32 sums
    constexpr int HALF = BN / 2;

    extern __shared__ uint8_t raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    float* most = reinterpret_cast<float*>(smem + C::STAGES * C::STAGE_BYTES);  // F8_GU: [3][2][128]
    uint64_t* full = reinterpret_cast<uint64_t*>(most + (OP == F8_GU ? 3 * 256 : 0));
    uint64_t* empty = full + C::STAGES;
    uint64_t* tfull = empty + C::STAGES;
    uint64_t* tempty = tfull + C::BUFS;
    uint64_t* drain = tempty + C::BUFS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CG == 1 ? 0 : cta_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], 1);
        for (int b = 0; b < C::BUFS; ++b) mbar_init(&tfull[b], 1), mbar_init(&tempty[b], CG * kF8EpiWarps);
        mbar_init(drain, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_map(&maps.a[0]);
        tma_prefetch_map(&maps.b[0]);
    }
    if (warp == 1) f8_tmem_alloc<CG>(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    if (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_trigger();

    int items = a.o[0].m_tiles * a.o[0].n_tiles;
    if (OP == F8_TN)
        for (int p = 1; p < a.products; ++p) items += a.o[p].m_tiles * a.o[p].n_tiles;
    items *= a.splits;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;

    if (warp == 0) {
        // ---------------- operands
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, filled = 0, fill_parity = 0;
            bool ok = true;
            const uint32_t bars = CG == 1 ? smem_u32(full) : in_leader(full);
            for (int i = first; ok && i < items; i += step) {
                const Item t = f8_item<OP, BN, CG>(i, a, rank);
                const int b0 = OP == F8_GU ? t.n0 + 64 * int(rank) * (CG - 1) : t.n0 + 128 * int(rank);  // first of this CTA's part of B
                for (int kb = t.k_lo; kb < t.k_hi; ++kb) {
                    ok = f8_wait(&empty[stage], phase ^ 1, abort_flag);
                    if (!ok) break;
                    const int part = OP == F8_TN ? t.p : (OP == F8_NN && kb >= a.k_part ? 1 : 0);
                    const int k0 = (OP == F8_NN && part ? kb - a.k_part : kb) * 128;
                    uint8_t* sa = smem + stage * C::STAGE_BYTES;
                    uint8_t* sb = sa + C::A_BYTES;
                    const uint32_t bar = bars + 8 * stage;
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], CG * C::STAGE_BYTES);
                    f8_load<CG>(sa, &maps.a[part], bar, A_MN ? t.m0 : k0, A_MN ? k0 : t.m0);
#pragma unroll
                    for (int c = 0; c < BN / 128 / CG; ++c) {
                        uint8_t* dst = sb + c * kTileBytes;
                        if (OP == F8_GU) {  // 64 columns of the gate beside the same 64 of the up weight, so that a warp gets both
                            f8_load<CG>(dst, &maps.b[0], bar, k0, b0 + 64 * c);
                            f8_load<CG>(dst + 8192, &maps.b[1], bar, k0, b0 + 64 * c);
                        } else {
                            f8_load<CG>(dst, &maps.b[part], bar, B_MN ? b0 + 128 * c : k0, B_MN ? k0 : b0 + 128 * c);
                        }
                    }
                    filled |= 1u << stage;
                    fill_parity = (fill_parity & ~(1u << stage)) | (phase << stage);
                    if (++stage == C::STAGES) stage = 0, phase ^= 1;
                }
            }
            if (!ok && rank == 0)  // every copy lands before the memory is given back (the first CTA's barriers count both CTAs')
                for (int s = 0; s < C::STAGES; ++s)
                    if (filled & (1u << s)) f8_drain(&full[s], (fill_parity >> s) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------- products
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
        if (rank == 0) {
            int stage = 0, buf = 0;
            uint32_t phase = 0, bphase = 0;
            bool ok = true;
            const uint32_t a_base = f8_desc_lo(smem_u32(smem), A_MN ? kTileBytes : 16);
            const uint32_t b_base = f8_desc_lo(smem_u32(smem) + C::A_BYTES, B_MN ? kTileBytes : 16);
            for (int i = first; ok && i < items; i += step) {
                const Item t = f8_item<OP, BN, CG>(i, a, rank);
                for (int kb = t.k_lo; kb < t.k_hi; ++kb) {
                    ok = f8_wait_warp(&full[stage], phase, abort_flag) && f8_wait_warp(&tempty[buf], bphase ^ 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    const uint32_t d = tmem + buf * BN, al = a_base + stage * (C::STAGE_BYTES >> 4), bl = b_base + stage * (C::STAGE_BYTES >> 4);
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            f8_mma<CG>(d, al + kk * (A_MN ? 4096 >> 4 : 32 >> 4), bl + kk * (B_MN ? 4096 >> 4 : 32 >> 4), IDESC, kk != 0 ? 1u : 0u);
                        f8_commit<CG>(&tfull[buf]);
                        f8_commit<CG>(&empty[stage]);
                    }
                    __syncwarp();
                    if (++buf == C::BUFS) buf = 0, bphase ^= 1;
                    if (++stage == C::STAGES) stage = 0, phase ^= 1;
                }
            }
            if (elect_one()) {
                if (CG == 1)
                    mma_commit(drain);
                else
                    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(drain))
                                 : "memory");
            }
            __syncwarp();
            f8_drain(drain, 0);  // every product is complete before TMEM is released
        }
        __syncwarp();
    } else if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kFewRegs));
    } else {
        // ---------------- sums over the blocks, and results
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kManyRegs));
        const int q = warp & 3, half = (warp - 4) >> 2;
        const uint32_t lanes = tmem + (uint32_t(q * 32) << 16);
        int buf = 0;
        uint32_t bphase = 0;
        bool ok = true;
        const uint32_t given = CG == 1 ? smem_u32(tempty) : in_leader(tempty);
        for (int i = first; i < items; i += step) {
            __syncwarp();
            const Item t = f8_item<OP, BN, CG>(i, a, rank);
            uint64_t acc[HALF / 2];
#pragma unroll
            for (int j = 0; j < HALF / 2; ++j) acc[j] = 0;
            const F8Out& o = a.o[t.p];
            if constexpr (OP == F8_TN) {
                ok = column_sums<BN, CG>(a.s[t.p], o, t, acc, lanes, q, half, tfull, given, buf, bphase, ok, abort_flag);
#pragma unroll
                for (int j = 0; j < HALF / 2; ++j)
                    if (!ok) acc[j] = 0x7fffffff7fffffffull;
                const Sink s = f8_sink(a, t);
                if (s.bf16)
                    column_store<HALF>(o, t, static_cast<__nv_bfloat16*>(s.out), s.ld, s.add, acc, q, half);
                else
                    column_store<HALF>(o, t, static_cast<float*>(s.out), s.ld, s.add, acc, q, half);
                continue;
            }
            // The scales of this row and of the columns: read two blocks ahead, into registers (beside the products'
            // reads of their operands a read of shared memory takes some hundred cycles).
            const int row = min(t.m0 + q * 32 + lane, o.M - 1);  // rows past the last are not stored
            const int nb = min((t.n0 + (OP == F8_GU ? 0 : HALF * half)) >> 7, (o.N - 1) >> 7);
            auto fetch = [&](int kb, float& r, float& c0, float& c1) {  // (addresses from the parameters: pointers kept would be spilled)
                const bool second = OP == F8_NN && kb >= a.k_part;
                const F8Scales& s = a.s[second ? 1 : 0];
                const int64_t kl = second ? kb - a.k_part : kb;
                r = __ldg(s.a + kl * s.ld_a + row);
                c0 = __ldg(OP == F8_NN ? s.b + kl * s.ld_b + nb : s.b + nb * s.ld_b + kl);
                if (OP == F8_GU) c1 = __ldg(a.s[1].b + nb * a.s[1].ld_b + kl);
            };
            float r0 = 0.0f, r1, c00 = 0.0f, c01, c10 = 0.0f, c11 = 0.0f;
            if (t.k_lo < t.k_hi) fetch(t.k_lo, r0, c00, c10);
            r1 = r0, c01 = c00, c11 = c10;
            if (t.k_lo + 1 < t.k_hi) fetch(t.k_lo + 1, r1, c01, c11);
            for (int kb = t.k_lo; kb < t.k_hi; ++kb) {
                const float f0 = r0 * c00, f1 = OP == F8_GU ? r0 * c10 : f0;
                const uint64_t g0 = pair(f0, f0), g1 = OP == F8_GU ? pair(f1, f1) : g0;
                r0 = r1, c00 = c01, c10 = c11;
                if (kb + 2 < t.k_hi) fetch(kb + 2, r1, c01, c11);
                if (ok) ok = f8_wait_warp(&tfull[buf], bphase, abort_flag);
                if (!ok) break;
                tc_fence_after();
                uint32_t v[2][16];
                const uint32_t at = lanes + uint32_t(buf * BN + HALF * half);
                tmem_ask16(at, v[0]);
#pragma unroll
                for (int c = 0; c < HALF / 16; ++c) {
                    tmem_wait();
                    if (c + 1 < HALF / 16) {
                        tmem_ask16(at + 16 * (c + 1), v[(c + 1) & 1]);
                    } else {  // the buffer is read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) arrive_cluster(given + 8 * buf);
                    }
                    const uint32_t(&x)[16] = v[c & 1];
#pragma unroll
                    for (int j = 0; j < 8; ++j) fma2(acc[8 * c + j], pair(x[2 * j], x[2 * j + 1]), c < HALF / 32 ? g0 : g1);
                }
                if (++buf == C::BUFS) buf = 0, bphase ^= 1;
            }
            float sum[HALF];
#pragma unroll
            for (int j = 0; j < HALF / 2; ++j) {
                if (!ok) acc[j] = 0x7fffffff7fffffffull;
                unpair(acc[j], sum[2 * j], sum[2 * j + 1]);
            }
            if constexpr (OP == F8_GU) {
                if (CG == 2 || a.splits == 1) {
                    gated_results(a, t, sum, q, half, most);
                    continue;
                }
            }
            if (CG == 1 && a.splits > 1) {  // whole tiles: the partial sums' rows have room for them (a pair's tiles are not split)
                constexpr int WIDTH = OP == F8_GU ? 64 : HALF;  // F8_GU: the first half is g's, the second u's
#pragma unroll
                for (int z = 0; z < HALF / WIDTH; ++z)
                    row_store<WIDTH>(o, f8_sink(a, t, z, HALF / WIDTH), t.m0 + q * 32 + lane, t.n0 + WIDTH * half, sum + WIDTH * z);
                continue;
            }
            const Sink sink = f8_sink(a, t);
            if (t.n0 + HALF * (half + 1) <= o.N &&
                ((reinterpret_cast<uintptr_t>(sink.out) | uintptr_t(sink.ld) * (sink.bf16 ? 2 : 4)) & 31) == 0) {
                row_store<HALF>(o, sink, t.m0 + q * 32 + lane, t.n0 + HALF * half, sum);
                continue;
            }
            const int col = t.n0 + HALF * half;
            if (t.m0 + q * 32 + lane < o.M && col < o.N) {
                const int64_t at = int64_t(row) * sink.ld + col;
                if (sink.bf16)
                    row_ragged<HALF>(static_cast<__nv_bfloat16*>(sink.out) + at, o.N - col, sum);
                else
                    row_ragged<HALF>(static_cast<float*>(sink.out) + at, o.N - col, sum);
            }
        }
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag) f8_gave_up = 1;
    if (CG == 2) cluster_sync();
    if (warp == 1) {
        tc_fence_after();
        f8_tmem_free<CG>(tmem, 512);
    }
}

// a warp that waits as the kernel's do, on a barrier that nothing arrives at
__global__ void __launch_bounds__(32) f8_wait_selftest_kernel() {
    __shared__ uint64_t bar;
    __shared__ int abort_flag;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    __syncwarp();
    (void)f8_wait_warp(&bar, 0, &abort_flag);
    __syncwarp();
    if (threadIdx.x == 0 && abort_flag) f8_gave_up = 1;
}

// ---------------------------------------------------------------- sums of the parts
// out = the partials' sum in their order (plus out); blockIdx.y: the product
__global__ void __launch_bounds__(256) f8_reduce_kernel(const __grid_constant__ F8Args a) {
    pdl_wait();
    pdl_trigger();
    const F8Out& o = a.o[blockIdx.y];
    const int quads = (o.N + 3) / 4;
    const int64_t total = int64_t(o.M) * quads, plane = int64_t(o.M) * o.ld_partial;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += int64_t(gridDim.x) * blockDim.x) {
        const int64_t m = i / quads;
        const int n = int(i - m * quads) * 4;
        float4 sum = make_float4(0, 0, 0, 0);
        const float* src = o.partial + m * o.ld_partial + n;
        for (int s = 0; s < a.splits; ++s) {
            const float4 x = __ldcs(reinterpret_cast<const float4*>(src + s * plane));
            sum = make_float4(sum.x + x.x, sum.y + x.y, sum.z + x.z, sum.w + x.w);
        }
        const float v[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
        for (int z = 0; z < 4; ++z)
            if (n + z < o.N) store_one(o.out, m * o.ld + n + z, o.bf16, o.accumulate, v[z]);
    }
}

template <int OP, int BN, int CG>
cudaError_t launch_one(const F8Maps& maps, const F8Args& a, int sms, cudaStream_t st) {
    using C = F8Cfg<OP, BN, CG>;
    constexpr auto kernel = f8_gemm_kernel<OP, BN, CG>;
    const cudaError_t e = f8_allow_shared<kernel>(C::SMEM);
    if (e != cudaSuccess) return e;
    int64_t items = 0;
    for (int p = 0; p < (OP == F8_TN ? a.products : 1); ++p) items += int64_t(a.o[p].m_tiles) * a.o[p].n_tiles;
    items *= a.splits;
    const int grid = int(items < sms / CG ? items : sms / CG) * CG;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(grid));
    cfg.blockDim = dim3(kF8Threads);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 1 ? 1 : 2;
    count_launch();
    return cudaLaunchKernelEx(&cfg, kernel, maps, a);
}

template <int OP>
cudaError_t launch_op(int bn, int cg, const F8Maps& maps, const F8Args& a, int sms, cudaStream_t st) {
    if (cg == 2) return launch_one<OP, 256, 2>(maps, a, sms, st);
    if constexpr (OP != F8_GU)
        if (bn == 128) return launch_one<OP, 128, 1>(maps, a, sms, st);
    return launch_one<OP, 256, 1>(maps, a, sms, st);
}

}  // namespace

cudaError_t launch_f8_gemm(int op, int bn, int cg, const F8Maps& maps, const F8Args& a, int sms, cudaStream_t st) {
    switch (op) {
        case F8_NT: return launch_op<F8_NT>(bn, cg, maps, a, sms, st);
        case F8_NN: return launch_op<F8_NN>(bn, cg, maps, a, sms, st);
        case F8_TN: return launch_op<F8_TN>(bn, cg, maps, a, sms, st);
        default: return launch_op<F8_GU>(bn, cg, maps, a, sms, st);
    }
}

cudaError_t f8_status(bool& gave_up, cudaStream_t st) {
    int v = 0;
    void* word = nullptr;
    cudaError_t e = cudaGetSymbolAddress(&word, f8_gave_up);
    if (e == cudaSuccess) e = cudaMemcpyAsync(&v, word, sizeof v, cudaMemcpyDeviceToHost, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
    gave_up = v != 0;
    if (e != cudaSuccess || !gave_up) return e;
    e = cudaMemsetAsync(word, 0, sizeof v, st);
    return e == cudaSuccess ? cudaStreamSynchronize(st) : e;  // the next call may be on another stream
}

cudaError_t launch_f8_wait_selftest(cudaStream_t st) {
    f8_wait_selftest_kernel<<<1, 32, 0, st>>>();
    count_launch();
    return cudaGetLastError();
}

cudaError_t launch_f8_reduce(const F8Args& a, cudaStream_t st) {
    int64_t most = 0;
    for (int p = 0; p < a.products; ++p) {
        const int64_t n = int64_t(a.o[p].M) * ((a.o[p].N + 3) / 4);
        most = n > most ? n : most;
    }
    const int64_t blocks = (most + 255) / 256;
    count_launch();
    return launch_pdl(f8_reduce_kernel, dim3(unsigned(blocks < 4096 ? blocks : 4096), unsigned(a.products)), dim3(256), 0, st, a);
}

}  // namespace moe
