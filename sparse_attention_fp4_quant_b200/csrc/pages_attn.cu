// pages_attn.cu -- attention over the paged FP8 cache on tcgen05: the sliding-window form
// with first tokens that stay visible, and the form for a batch behind a shared prefix.
//
// Keys are the M axis.  A CTA takes NQ queries (R = 16 NQ rows: query x head) and a range of
// 128-key tiles.  With K the tile's E4M3 rows and P the weights,
//     S^T [128 keys x 2R]  = K Q^T             16 steps of 32 channels,
//     O^T [512 channels x R] += K^T P            4 blocks of 128 channels, steps of 32 keys,
// both kind::f8f6f4, so cache bytes go from HBM through one TMA copy to the tensor cores
// unconverted: the same shared-memory tile is read K-major for S and channel-major for O.
// What the other operand loses is bounded:
//   Q   a bf16 has 8 significant bits, an E4M3 pair hi + lo holds 4 + 4: exact, apart from
//       elements below 2^-9 of the row's largest (each row scaled by its own power of two),
//       which are held to 2^-17 of it.  hi and lo are separate columns of S, added in fp32.
//   P   each weight times its token scale, as f16 with 2^12 of headroom below the maximum,
//       split in three E5M2 terms (f16's exponent range): 9 of the f16's 11 significant bits, so
//       within 2^-11 + 2^-9 of itself, or 2^-29 of the row's largest where that is more (below
//       about 2^-20 of it: half of E5M2's smallest step, 2^-16, against 2^12).
// Softmax: fp32, one thread per key, one pass with a running reference m per row.  The
// reference is the maximum of z + log2(token scale), the size of what enters P, and it moves
// only when a tile exceeds it by 2^3 (P keeps that much room), so the accumulators are
// rescaled rarely.  l = sum 2^(z - m) stays in fp32 registers.
// A slot may hold NaN bytes, and a weight of 0 times NaN is NaN: a query that does not see the key would
// get it.  Such a key's S is NaN in every column, so its threads find out for nothing, and zero the row
// before P K.  A query that does see it has a NaN weight there, and gets NaN by that.
//
// What bounds it (B200, calls in a graph; the join included):
//   many queries over long lists  64 rows x 128 keys are 16 products of 64 cycles for S and 48 of 48 cycles for O, 3,340
//       of the 5,100 that a tile takes: two tiles fit beside the queries, and a tile's turn (fetch 900 cycles after the
//       last product of the one before, S 2,200, softmax 2,600, O 3,100, waits) is 10,200 for every second one.  32
//       queries behind 131,072 tokens 174 us, 0.48 of the time of the products at the measured bf16 rate (192 and 0.43
//       in a long loop of calls, at the power limit's clocks); 3 x 1,017 of a 1,024-token window 149 us, 0.37 (156 and
//       0.35).
//   one query, long lists         the stream: 61 queries of 4,096 tokens in pages of 16 37.5 us, 5.6 TB/s while it runs,
//       by 122 of the 148 SMs.
//   many queries, short windows   a chain of 17,200 cycles an item (queries in, two tiles, output): 4,096 queries of a
//       128-token window 75 us.
//   one token                     the same chain after the launch: 7.6 us for one sequence, 7.9 for 32.
#include <cuda.h>

#include <algorithm>

#include "attn_common.cuh"
#include "tc.cuh"

namespace csa2 {

namespace {

using namespace tc;

constexpr int kTileKeys = 128;
constexpr int kGroup = 8;                              // keys of one swizzle atom
constexpr int kBlocks = kD / 128;                      // channel blocks of 128 channels: 128 bytes, a swizzle row
constexpr int kTileBytes = kTileKeys * kD;             // 64 KB
constexpr int kAux = 96;                               // producer, S issuer, O issuer
constexpr int kWg = 128;                               // threads of a softmax warpgroup: one query, a thread per key
constexpr float kHeadroom = 3.0f;                      // log2 of how far a weight may exceed the reference
constexpr float kPScale = 4096.0f;                     // weight 1 at 2^12, 2^15 with the headroom: in range of f16, E5M2
constexpr float kMinLogScale = -100.0f;                // token scales below 2^-100 count as 2^-100 in the reference
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr int kMaxSplits = 2 * kSplitSMs;

// One list of keys of a CTA, for its queries [qa, qa + nq): units of `unit` slots of one table row (a unit is
// one TMA box, inside one page), `sink` first units and then the window's (virtual unit v is unit v, or
// v + delta from `sink` on).
struct Seg {
    int tile0;      // first tile of the list in the CTA's order
    int units, sink, delta;
    int own;        // 0 = the shared prefix, 1 = a sequence's own pages
    int qa, nq;
    int pos0, end;  // position of slot 0, and of the first slot behind the stored tokens
    int imin, lmax;  // every query of the list sees the stored tokens in [lmax, imin]
    int page_size, n_pages;
    const int32_t* table;   // the sequence's row
    const float* scales;

    __device__ __forceinline__ int unit(int v) const { return v < sink ? v : v + delta; }
};

__device__ __forceinline__ Seg make_seg(const csa2_pages& pg, int own, int b, int tile0, int units, int sink, int delta,
                                        int qa, int nq, int end, int imin, int lmax) {
    return {tile0, units, sink, delta, own, qa, nq, pg.pos0, end, imin, lmax, pg.page_size, (int)pg.n_pages,
            pg.table + (int64_t)b * pg.max_pages, pg.kv_sc};
}

// What the roles need of a tile, written by the producer with its copies.
struct __align__(16) Tile {
    int qa, nq;     // queries
    int steps;      // steps of 32 keys
    int interior;   // every key is stored and seen by all of them
    int end, sink;  // first position behind the stored tokens; positions below sink stay visible
    int own;        // 0 = tokens of the shared prefix
    int n_pages;    // the producer's own
};

// A tile lies in shared memory as 8-key x 128-byte swizzle atoms, [16 key groups][4 channel blocks], and moves and is
// freed in four parts of 32 keys.  One copy moves all channels of a unit: with pages of 16 tokens a tile takes 1,060
// cycles to fetch.  (The other order, [4 channel blocks][16 key groups], lets S begin with a quarter of the tile, but
// moves a unit by four copies: 2,340 cycles, and with pages of 64 tokens no faster: 32 queries behind 131,072 tokens 174
// us either way.)
constexpr int kParts = 4;
constexpr uint32_t kGroupStep = 4096, kBlockStep = 1024, kPartStep = 4 * kGroupStep;   // bytes from one to the next

// A CTA's item (queries and a split of their keys): what the producer tells the other roles.
template <int NQ>
struct Item {
    int tiles;
    int64_t part;   // block * splits + split
    int qi[NQ], qlow[NQ];   // each query's token, and the first that its window holds
};

template <int NQ, int ST, int W>
struct Smem {
    static constexpr int RQ = kH * NQ, R = kH * W;       // rows: of the queries, and of the accumulators
    alignas(1024) uint8_t K[ST][kTileBytes];
    alignas(1024) uint8_t Qs[kBlocks][2 * RQ][128];      // [channel block][query][hi 16 | lo 16][128 B], 128-byte swizzle
    alignas(1024) uint8_t P[3 * W][kTileKeys][16];       // [term][query] or [warpgroup][term]: 16 rows of each key, no swizzle
    alignas(16) float sc[ST][kTileKeys];                 // the keys' token scales
    int upos[ST][kTileKeys / kGroup];                    // position of each unit's first key; -1 without a page
    Tile tile[ST];
    alignas(16) float wmax[4][R];
    alignas(16) float mref[R];
    alignas(16) float fac[R];
    alignas(16) float rowf[2][RQ];   // by item
    float lsum[4][R];
    Seg seg[NQ + 1];   // the producer's own
    Item<NQ> item[2];
    int dead;
    uint32_t tmem;
    uint64_t full[ST][kParts], empty[ST][kParts], s_full[2], s_free[2], p_full[2], pv_done[2], wind_down[2];
    uint64_t item_full[2], item_empty[2], q_full[2];
};

// The issuing warp runs its loop converged and one elected lane (lead != 0) issues: descriptors then stay in
// uniform registers.  Issued from a divergent branch, each MMA cost about 110 cycles of descriptor moves.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

__device__ __forceinline__ void mma_f8(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead)
        : "memory");
}

__device__ __forceinline__ void commit(uint32_t lead, uint64_t* bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
        "r"(lead)
        : "memory");
}

// Instruction descriptors, M = 128, K = 32, fp32 accumulation: E4M3 x E4M3, both K-major; and
// E4M3 (channel-major) x E5M2 (row-major, "MN-major").
__device__ __forceinline__ uint32_t idesc_qk(int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24); }
__device__ __forceinline__ uint32_t idesc_pv(int N) {
    return (1u << 4) | (1u << 10) | (1u << 15) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
constexpr uint32_t kSw128 = 2;

// All channels of one unit's 8-key groups.
__device__ __forceinline__ void tma_unit(void* dst, const CUtensorMap* map, int group, uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %2, %2, %3}], "
        "[%4];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(0), "r"(group), "r"(smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// The largest |bf16| of eight, by bits (the order of their integers puts infinity and NaN on top), one per half.
__device__ __forceinline__ uint32_t bf16x8_topbits(uint4 v) {
    const uint32_t m = 0x7FFF7FFFu;
    return __vmaxu2(__vmaxu2(v.x & m, v.y & m), __vmaxu2(v.z & m, v.w & m));
}

__device__ __forceinline__ float redux_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float ex2(float v) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Barrier of one softmax warpgroup, alone or with the OR of a condition over its threads.
__device__ __forceinline__ void wg_bar(int wg) { asm volatile("bar.sync %0, %1;" ::"r"(1 + wg), "n"(kWg) : "memory"); }
__device__ __forceinline__ bool wg_any(int wg, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)v), "r"(1 + wg), "n"(kWg)
        : "memory");
    return r != 0;
}

// Two weights (f16x2) -> three terms of E5M2 in the high bytes of each half.  An E5M2 value is an
// f16 whose low byte is zero: hi and mid truncate (each leaves a remainder of the next bits,
// exact in f16), lo rounds to nearest by adding half of its last place.
__device__ __forceinline__ void split_e5m2(uint32_t p, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = p & 0xFF00FF00u;
    __half2 r = __hsub2(*reinterpret_cast<__half2*>(&p), *reinterpret_cast<__half2*>(&hi));
    const uint32_t rb = *reinterpret_cast<uint32_t*>(&r);
    mid = rb & 0xFF00FF00u;
    r = __hsub2(r, *reinterpret_cast<const __half2*>(&mid));
    lo = *reinterpret_cast<uint32_t*>(&r) + 0x00800080u;   // the low bytes are not used
}

// A load that stays where it is written, ahead of the waits of the tile before.
__device__ __forceinline__ int ldg_now(const int32_t* p) {
    int v;
    asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

// A copy of 16 bytes, and an arrival on a barrier once this thread's copies so far have landed.
__device__ __forceinline__ void cp_async16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ int stored_end(const csa2_pages& pg, int b) {
    const int64_t cap = (int64_t)pg.max_pages * pg.page_size;
    int64_t n = pg.n_tokens[b];
    n = n < 0 ? 0 : n > cap ? cap : n;
    return (int)(pg.pos0 + n);
}

// Division of n < 2^32 by d >= 1: n floor((2^32 - 1) / d) / 2^32 is at most 1 below the quotient.  A division
// instruction sequence takes some 150 cycles, and an item's first copies wait for four of them.
struct Div {
    uint32_t d, m;

    __device__ __forceinline__ int operator()(int n) const {
        const uint32_t q = __umulhi((uint32_t)n, m);
        return (int)(q + ((uint32_t)n - q * d >= d ? 1u : 0u));
    }
};
Div div_by(int64_t d) { return {(uint32_t)d, 0xFFFFFFFFu / (uint32_t)d}; }

struct KernelArgs {
    PagesAttnParams p;
    int items;        // blocks x splits; CTA i takes items i, i + gridDim.x, ...
    int unit_log2;    // keys of a TMA box: 8, 16 or 32, divides every page
    int splits;
    int test_starve;  // test hook (csa2_test_starve_copies): the producer issues no copies
    Div by_splits, by_q, by_per;          // by splits, Q, a sequence's blocks
    Div by_page_own, by_page_prefix;      // by a page's units
    float* part_o;    // [block][split][R][512]
    float* part_ml;   // [block][split][R][2]
};

// NQ queries, ST tiles in flight, whether the three terms of P have accumulator columns of their own (one product for
// all three, 3 RQ columns, where TMEM has room), CTAs on an SM.  kPair: one query whose tiles two warpgroups take in turn,
// each with its own references, P and accumulators: two splits that share the tiles in flight.
template <int NQ, int ST, bool kConcat, int kCtas, bool kPair = false>
__global__ void __launch_bounds__(kWg * (kPair ? 2 : NQ) + kAux, kCtas)
    pages_attn_kernel(const __grid_constant__ CUtensorMap map_own, const __grid_constant__ CUtensorMap map_prefix,
                      const __grid_constant__ KernelArgs args) {
    static_assert(!kPair || (NQ == 1 && kConcat), "a pair takes one query");
    constexpr int W = kPair ? 2 : NQ;                  // softmax warpgroups
    using Sm = Smem<NQ, ST, W>;
    constexpr int RQ = Sm::RQ, R = Sm::R;
    constexpr int kOCols = (kConcat ? 3 : 1) * RQ;     // accumulator columns of one channel block
    constexpr int kOSet = kPair ? 4 * kOCols : 0;      // from one warpgroup's accumulators to the next's
    constexpr uint32_t kTmemCols = 512 / kCtas;
    constexpr uint32_t kS0 = kOSet + 4 * kOCols;       // S^T buffers behind the accumulators
    static_assert(kS0 + 2 * 2 * RQ <= kTmemCols, "TMEM budget");
    // Barrier and parity of tile n's P and of its products: a pair's warpgroups have one each.
    auto pbar = [](int n) { return kPair ? n & 1 : 0; };
    auto ppar = [](int n) { return (uint32_t)((kPair ? n >> 1 : n) & 1); };
    constexpr int kTurn = kPair ? 2 : 1;               // tiles from one of a warpgroup to its next
    extern __shared__ uint8_t smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const PagesAttnParams& p = args.p;
    constexpr int kProducer = 4 * W, kIssuer = kProducer + 1;   // behind the softmax warpgroups
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ul = args.unit_log2, unit = 1 << ul, upt = kTileKeys >> ul;   // keys of a unit, units of a tile

    if (tid == 32 * kProducer) {
        for (int s = 0; s < ST; ++s)
            for (int c = 0; c < kParts; ++c) {
                mbar_init(&sm.full[s][c], c == 0 ? 33 : 1);   // with the first part come the scales, by every lane
                mbar_init(&sm.empty[s][c], 1);
            }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_free[i], 4 * NQ);
            mbar_init(&sm.p_full[i], kWg * NQ);
            mbar_init(&sm.pv_done[i], 1);
            mbar_init(&sm.wind_down[i], 1);
            mbar_init(&sm.item_full[i], 1);
            mbar_init(&sm.item_empty[i], 4 * W + 2);
            mbar_init(&sm.q_full[i], 4 * W);
        }
        fence_mbar_init();
        sm.dead = 0;
    }
    if (tid < R) sm.mref[tid] = -INFINITY;
    __syncthreads();
    pdl_enter();
    // TMEM is taken behind the wait.  Held through it, the columns could be those that a CTA of the kernel before waits for
    // on this SM, without a limit: the kernels let the next one start before they allocate.
    if (warp == kIssuer) tmem_alloc(&sm.tmem, kTmemCols);
    // Its address, for all but the producer, which goes ahead meanwhile.
    auto tmem_base = [&]() -> uint32_t {
        tc_fence_before();
        asm volatile("bar.sync %0, %1;" ::"n"(1 + W), "n"(kWg * W + 64) : "memory");
        tc_fence_after();
        return sm.tmem;
    };

    // A bounded wait; the first to run out of time tells every other.  From then on producer and issuers stop, and softmax
    // threads pass their waits but arrive for nothing any more: a stage that never filled must not be freed and armed
    // again (its barrier's count would run below zero).
    auto wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        if (mbar_try_wait(bar, parity)) return true;
        const uint64_t start = globaltimer_ns();
        for (uint32_t it = 1;; ++it) {
            if (mbar_try_wait(bar, parity)) return true;
            if ((it & 63u) == 0u) {
                if (*(volatile int*)&sm.dead) return false;
                if (globaltimer_ns() - start > kTimeoutNs) {
                    *(volatile int*)&sm.dead = 1;
                    if (p.flag) *p.flag = 1;
                    return false;
                }
            }
        }
    };
    const bool shared_prefix = p.prefix.B != 0;
    auto queries_of = [&](int block, int& f0, int& nq) {
        if (shared_prefix) {
            f0 = block * NQ;
            nq = min(NQ, p.B * p.Q - f0);
        } else {
            const int b = args.by_per(block), q0 = (block - b * (int)args.by_per.d) * NQ;
            f0 = b * p.Q + q0;
            nq = min(NQ, p.Q - q0);
        }
    };
    int nseg = 0;
    auto seg_of = [&](int tile) -> int {
        int s = 0;
        while (s + 1 < nseg && tile >= sm.seg[s + 1].tile0) ++s;
        return s;
    };
    // Producer.  A tile is prepared in steps, each a tile ahead of the next, so that no load's latency falls on the
    // copies: the page of the lane's unit (one lane per unit), the unit's row, the copies.
    struct Ahead {
        int page, at;          // the unit's page (not waited for before rows_of), and its first slot in there; -1: no unit
        int row, first;        // its row in the pool (-1: none), its first key's position
        uint32_t live;         // units that have a row
        bool inside;           // every query sees all of its keys
        Tile info;
        const float* scales;   // of keys 4 lane .. 4 lane + 3, or null
    };
    Seg sg;          // the list of the next tile to be read
    int sg_at = -1;
    auto page_of = [&](int t) -> Ahead {
        const int s = seg_of(t);
        if (s != sg_at) {
            sg = sm.seg[s];
            sg_at = s;
        }
        Ahead a;
        const int v0 = (t - sg.tile0) * upt, v = v0 + lane, u = sg.unit(min(v, sg.units - 1));
        const int d = sg.page_size >> ul;   // units of a page
        const int i = (sg.own ? args.by_page_own : args.by_page_prefix)(u), r = u - i * d;
        a.page = ldg_now(sg.table + i);   // a load in every lane, so that nothing here depends on it
        const bool have = lane < upt && v < sg.units;
        a.at = have ? r << ul : -1;
        a.first = sg.pos0 + (u << ul);
        const int last = a.first + unit - 1;
        a.inside = have && last < sg.end && last <= sg.imin && (a.first >= sg.lmax || (sg.own && last < p.n_sink));
        const int keys = min(kTileKeys, (sg.units - v0) << ul);
        a.info = {sg.qa, sg.nq, (keys + 31) / 32, 0, sg.end, sg.own ? p.n_sink : 0, sg.own, sg.n_pages};
        a.row = sg.page_size;
        a.scales = sg.scales;
        return a;
    };
    auto rows_of = [&](Ahead& a) {
        a.row = a.at >= 0 && a.page >= 0 && a.page < a.info.n_pages ? a.page * a.row + a.at : -1;
        if (a.row < 0) a.first = -1;
        const int row4 = __shfl_sync(0xFFFFFFFFu, a.row, (4 * lane) >> ul);
        a.scales = row4 >= 0 ? a.scales + row4 + ((4 * lane) & (unit - 1)) : nullptr;
        a.live = __ballot_sync(0xFFFFFFFFu, a.row >= 0);
        a.info.interior = __popc(__ballot_sync(0xFFFFFFFFu, a.inside && a.row >= 0)) == upt;
    };
    // The copies of the CTA's n-th tile, part by part, the keys' scales with the first.
    auto load_tile = [&](const Ahead& a, int n) -> bool {
        const int st = n % ST;
        const CUtensorMap* map = a.info.own ? &map_own : &map_prefix;
#pragma unroll
        for (int c = 0; c < kParts; ++c) {
            bool ok = true;
            if (n >= ST) ok = wait(&sm.empty[st][c], (uint32_t)((n / ST - 1) & 1));
            if (!__all_sync(0xFFFFFFFFu, ok)) return false;
            if (c == 0) {
                if (lane < upt) sm.upos[st][lane] = a.first;
                if (lane == 0) sm.tile[st] = a.info;
                if (a.scales) cp_async16(&sm.sc[st][4 * lane], a.scales);
                cp_async_arrive(&sm.full[st][0]);
            }
            const int upp = 32 >> ul;   // units of a part
            const uint32_t bytes = __popc(a.live & (((1u << upp) - 1u) << (c * upp))) * unit * kD;
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&sm.full[st][c], bytes);
            __syncwarp();
            if (a.row >= 0 && lane >> (5 - ul) == c && !args.test_starve)
                tma_unit(sm.K[st] + lane * unit * kD, map, a.row / kGroup, &sm.full[st][c]);
        }
        return true;
    };

    if (warp == kProducer) {
        // ---- producer: an item's key lists and its tiles' copies.  It runs ahead of the others, so that an item's
        // chain of loads (positions, page table, rows) passes under the item before.
        auto units_of = [&](int n) { return ((n - 1) >> ul) + 1; };   // n >= 1 keys; n + unit - 1 might not fit
        auto tiles_of = [&](int u) { return ((u - 1) >> (7 - ul)) + 1; };
        int tile_no = 0;
        bool ok = true;
        for (int k = 0, it = blockIdx.x; ok && it < args.items; ++k, it += gridDim.x) {
            if (k >= 2) ok = __all_sync(0xFFFFFFFFu, wait(&sm.item_empty[k & 1], (uint32_t)((k / 2 - 1) & 1)));
            if (!ok) break;
            const int block = args.by_splits(it), split = it - block * args.splits;
            int f0, nq;
            queries_of(block, f0, nq);
            // lanes 0 .. NQ-1: a query each
            int i = -1, low = 0, end = 0, pend = 0;
            const int b = args.by_q(f0 + min(lane, nq - 1));
            if (lane < nq) i = p.q_pos[f0 + lane];
            if (lane < NQ) end = stored_end(p.own, b);
            if (shared_prefix && lane == 0) pend = stored_end(p.prefix, 0);
            if (i < 0) i = -1;
            int64_t lw = p.window == 0x7FFFFFFF ? 0 : (int64_t)i - p.window + 1;
            if (p.replay_start && lane < nq) lw = max(lw, (int64_t)p.replay_start[b]);
            low = (int)max(lw, (int64_t)0);
            Item<NQ>& item = sm.item[k & 1];
            if (lane < NQ) {
                item.qi[lane] = i;
                item.qlow[lane] = low;
            }
            // Each lane's run of queries of one sequence: its extent and what its keys range over (every lane < nq alike).
            const bool mine = lane < nq;
            const int seq = mine ? b : -1;
            int count = 0, head = 1, hi = 0, lo = 0x7FFFFFFF, rmin = 0x7FFFFFFF, rlow = 0, imax = -1, imin = 0x7FFFFFFF;
#pragma unroll
            for (int c = 0; c < NQ; ++c) {
                const int oi = __shfl_sync(0xFFFFFFFFu, i, c), ol = __shfl_sync(0xFFFFFFFFu, low, c);
                const bool same = __shfl_sync(0xFFFFFFFFu, seq, c) == seq;
                if (c < nq) {
                    imax = max(imax, oi);
                    imin = min(imin, oi);
                }
                if (c < nq && same) {
                    ++count;
                    if (c < lane) head = 0;
                    rmin = min(rmin, oi);
                    rlow = max(rlow, ol);
                    if (oi >= 0) {
                        hi = max(hi, oi < end ? oi + 1 : end);
                        lo = min(lo, ol);
                    }
                }
            }
            int n = 0, tiles = 0;
            if (shared_prefix) {
                pend = __shfl_sync(0xFFFFFFFFu, pend, 0);
                const int e = (imax < pend ? imax + 1 : pend) - p.prefix.pos0;
                if (e > 0) {
                    const int u = units_of(e);
                    if (lane == 0) sm.seg[0] = make_seg(p.prefix, 0, 0, 0, u, 0, 0, 0, nq, pend, imin, 0);
                    n = 1;
                    tiles = tiles_of(u);
                }
            }
            {
                // the sinks' units, then the window's from the first that holds no sink
                const int base = p.own.pos0, ns = min(p.n_sink, hi) - base;
                const int us = ns > 0 ? units_of(ns) : 0;
                const int ue = hi > base ? units_of(hi - base) : 0;
                const int uw = max(us, lo > base ? (lo - base) >> ul : 0);
                const int u = mine && head && hi > base ? us + max(0, ue - uw) : 0;
                const int mytiles = u > 0 ? tiles_of(u) : 0;
                int at = n, tile0 = tiles;   // lists and tiles of the runs before this one
#pragma unroll
                for (int c = 0; c < NQ; ++c) {
                    const int ot = __shfl_sync(0xFFFFFFFFu, mytiles, c);
                    if (c < lane) {
                        at += ot > 0;
                        tile0 += ot;
                    }
                    n += ot > 0;
                    tiles += ot;
                }
                if (u > 0) sm.seg[at] = make_seg(p.own, 1, b, tile0, u, us, uw - us, lane, count, end, rmin, rlow);
            }
            nseg = n;
            const int each = tiles / args.splits, extra = tiles - each * args.splits;   // the first splits take one tile more
            const int t0 = split * each + min(split, extra), nt = each + (split < extra);
            if (lane == 0) {
                item.tiles = nt;
                item.part = it;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&sm.item_full[k & 1]);
                if (it + gridDim.x < args.items) {   // the next item's queries on their way to L2
                    int g0, gn;
                    queries_of(args.by_splits(it + gridDim.x), g0, gn);
                    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p.q + (int64_t)g0 * kH * kD),
                                 "r"(gn * kH * kD * 2)
                                 : "memory");
                }
            }
            if (nt > 0) {
                sg_at = -1;
                Ahead a = page_of(t0), next = page_of(t0 + min(1, nt - 1));
                rows_of(a);
                for (int t = 0;;) {
                    ok = load_tile(a, tile_no);
                    if (!ok) break;
                    ++tile_no;
                    if (++t == nt) break;
                    a = next;
                    if (t + 1 < nt) next = page_of(t0 + t + 1);
                    rows_of(a);
                }
            }
        }
        if (!ok) {   // wind down: the copies in flight land before the CTA ends
            for (int n = max(0, tile_no - ST); n <= tile_no; ++n)
                for (int c = 0; c < kParts; ++c) mbar_wait(&sm.full[n % ST][c], (uint32_t)((n / ST) & 1), kTimeoutNs / 16);
        }
    } else if (warp == kIssuer) {
        // ---- S issuer.  S and O have a warp each: one thread issues a product in about 50 cycles, more than most of
        // these take, and each stream's waits then leave the other alone.  A tile's products are unrolled.
        const uint32_t lead = elect_one();
        const uint32_t td = __shfl_sync(0xFFFFFFFFu, tmem_base(), 0);
        const uint32_t k0 = smem_u32(sm.K[0]);
        const uint64_t qd = smem_desc(smem_u32(sm.Qs), 16, 1024, kSw128);
        bool ok = true;
        int n = 0;
        for (int k = 0, it = blockIdx.x; ok && it < args.items; ++k, it += gridDim.x) {
            ok = wait(&sm.item_full[k & 1], (uint32_t)((k >> 1) & 1)) && wait(&sm.q_full[k & 1], (uint32_t)((k >> 1) & 1));
            ok = __all_sync(0xFFFFFFFFu, ok);
            const int last = n + __shfl_sync(0xFFFFFFFFu, sm.item[k & 1].tiles, 0);
            for (; n < last && ok; ++n) {
                const int st = n % ST;
                if (n >= 2) ok = wait(&sm.s_free[n & 1], (uint32_t)((n / 2 - 1) & 1));
#pragma unroll
                for (int c = 0; c < kParts; ++c) ok = ok && wait(&sm.full[st][c], (uint32_t)((n / ST) & 1));
                ok = __all_sync(0xFFFFFFFFu, ok);
                if (!ok) break;
                const int qa = __shfl_sync(0xFFFFFFFFu, sm.tile[st].qa, 0), qn = __shfl_sync(0xFFFFFFFFu, sm.tile[st].nq, 0);
                const uint64_t a = smem_desc(k0 + st * kTileBytes, 16, kGroupStep, kSw128), b = qd + qa * (4096 / 16);
                const uint32_t d = td + kS0 + (n & 1) * 2 * RQ + 32 * qa, id = idesc_qk(32 * qn);
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kBlocks; ++c) {
#pragma unroll
                    for (int s = 0; s < 4; ++s)
                        mma_f8(lead, d, a + (c * kBlockStep + s * 32) / 16, b + (c * (2 * RQ * 128) + s * 32) / 16, id, c + s > 0);
                }
                commit(lead, &sm.s_full[n & 1]);
            }
            if (lane == 0) mbar_arrive(&sm.item_empty[k & 1]);
        }
        if (!ok) {   // wind down: no product in flight when TMEM is freed
            commit(lead, &sm.wind_down[0]);
            mbar_wait(&sm.wind_down[0], 0);
        }
        __syncwarp();
    } else if (warp == kIssuer + 1) {
        // ---- O issuer ----
        const uint32_t lead = elect_one();
        const uint32_t td = __shfl_sync(0xFFFFFFFFu, tmem_base(), 0);
        const uint32_t k0 = smem_u32(sm.K[0]);
        const uint64_t pd = smem_desc(smem_u32(sm.P), 128, 2048, kLayoutNone);
        bool ok = true;
        int n = 0;
        for (int k = 0, it = blockIdx.x; ok && it < args.items; ++k, it += gridDim.x) {
            ok = __all_sync(0xFFFFFFFFu, wait(&sm.item_full[k & 1], (uint32_t)((k >> 1) & 1)));
            const int last = n + __shfl_sync(0xFFFFFFFFu, sm.item[k & 1].tiles, 0);
            for (; n < last && ok; ++n) {
                const int st = n % ST;
                ok = __all_sync(0xFFFFFFFFu, wait(&sm.p_full[pbar(n)], ppar(n)));
                if (!ok) break;
                const int qa = __shfl_sync(0xFFFFFFFFu, sm.tile[st].qa, 0), qn = __shfl_sync(0xFFFFFFFFu, sm.tile[st].nq, 0);
                const int steps = __shfl_sync(0xFFFFFFFFu, sm.tile[st].steps, 0);
                const uint64_t a = smem_desc(k0 + st * kTileBytes, 16, kGroupStep, kSw128);
                tc_fence_after();
                const uint64_t b = pd + (qa + 3 * pbar(n)) * (2048 / 16);
                const uint32_t d = td + kH * qa + pbar(n) * kOSet;
                // Part i of the tile; its memory is free for a coming tile when its products are done.
                auto parts = [&](auto product) {
#pragma unroll
                    for (int s = 0; s < kParts; ++s) {
#pragma unroll
                        for (int c = 0; c < kBlocks; ++c)
                            if (s < steps) product(c, a + (c * kBlockStep + s * kPartStep) / 16, b + s * (512 / 16));
                        commit(lead, &sm.empty[st][s]);
                    }
                };
                if (kConcat && qn == NQ) {   // the three terms as one product
                    parts([&](int c, uint64_t as, uint64_t bs) { mma_f8(lead, d + c * kOCols, as, bs, idesc_pv(3 * RQ), 1); });
                } else {
                    const uint32_t id = idesc_pv(kH * qn);
                    parts([&](int c, uint64_t as, uint64_t bs) {
#pragma unroll
                        for (int x = 0; x < 3; ++x)
                            mma_f8(lead, d + c * kOCols + (kConcat ? x * RQ : 0), as, bs + x * NQ * (2048 / 16), id, 1);
                    });
                }
                commit(lead, &sm.pv_done[pbar(n)]);
            }
            if (lane == 0) mbar_arrive(&sm.item_empty[k & 1]);
        }
        if (!ok) {
            commit(lead, &sm.wind_down[1]);
            mbar_wait(&sm.wind_down[1], 0);
        }
        __syncwarp();
    } else {
        // ---- softmax: warpgroup = query (or every other tile of one), thread = key ----
        const int wg = warp >> 2, query = kPair ? 0 : wg, key = tid & (kWg - 1), quarter = warp & 3;
        uint32_t tq = 0;   // this warp's lanes of TMEM
        // this warpgroup's accumulator columns: 16 of each channel block (and of each term)
        auto ocol = [&](int b, int x) -> uint32_t { return tq + wg * kOSet + b * kOCols + x * RQ + kH * query; };
        constexpr int kTerms = kConcat ? 3 : 1;
        auto row4 = [&](const float (&a)[R], int j) { return *reinterpret_cast<const float4*>(&a[kH * wg + 4 * j]); };
        const bool split = kPair || args.splits > 1;   // partial sums go to the workspace
        const int ku = key >> ul, ko = key & (unit - 1);
        int n = 0;
        // Item by item: its queries are converted as soon as the item before has seen its last S, so that the first S
        // of the next is made while the output of the last is written.
        int f0 = 0, nq = 0, nt = 0, prev_f0 = 0, prev_nq = 0;
        int64_t part = 0;
        int last = -1;   // a pair: this warpgroup's last tile in the item
        for (int k_item = 0, it = blockIdx.x;; ++k_item, it += gridDim.x) {
            const bool have = it < args.items;
            float(&rowf)[RQ] = sm.rowf[k_item & 1];
            auto rowf4 = [&](int j) { return *reinterpret_cast<const float4*>(&rowf[kH * query + 4 * j]); };
            prev_f0 = f0;
            prev_nq = nq;
            if (have) {
                // Q: four rows (heads; of a pair two) in each warp, 16 channels per lane -> E4M3 hi and lo, each row scaled
                // so that its largest is in [2^7, 2^8)
                queries_of(args.by_splits(it), f0, nq);
                constexpr int kRows = 4 * NQ / W;
                auto head = [&](int k) { return kPair ? warp + 8 * k : quarter + 4 * k; };
                uint4 v[kRows][2];
#pragma unroll
                for (int k = 0; k < kRows; ++k) {
                    v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
                    if (query < nq) {
                        const int64_t row = (int64_t)(f0 + query) * kH + head(k);
                        const uint4* src = reinterpret_cast<const uint4*>(p.q + row * kD) + 2 * lane;
                        v[k][0] = __ldg(src);
                        v[k][1] = __ldg(src + 1);
                    }
                }
                if (k_item == 0) tq = tmem_base() + ((uint32_t)(quarter * 32) << 16);   // no CTA is without an item
                bool told = wait(&sm.item_full[k_item & 1], (uint32_t)((k_item >> 1) & 1));
                // the other warpgroup's last S of the item before still reads Q
                if (kPair && n > 0) told = wait(&sm.s_full[(n - 1) & 1], (uint32_t)(((n - 1) >> 1) & 1)) && told;
                if (wg_any(wg, !told)) break;   // a wait ran out: no item to work on
                uint32_t top[kRows];   // bits of the row's largest |bf16|; from 0x7F80 on the row holds an infinity or NaN
#pragma unroll
                for (int k = 0; k < kRows; ++k) {
                    const uint32_t t = __vmaxu2(bf16x8_topbits(v[k][0]), bf16x8_topbits(v[k][1]));
                    top[k] = __reduce_max_sync(0xFFFFFFFFu, max(t & 0xFFFFu, t >> 16));
                    // such a row enters the products as zeros and gets its NaN by rowf: S is NaN only where K is
                    if (top[k] >= 0x7F80u) v[k][0] = v[k][1] = make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int k = 0; k < kRows; ++k) {
                    const int h = head(k), r = kH * query + h;
                    const int e = max((int)(top[k] >> 7) - 127 - 7, -120);
                    const float mul = __uint_as_float((uint32_t)(127 - e) << 23);
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint4& vv = v[k][j >> 1];
                        const uint32_t w0 = (j & 1) ? vv.z : vv.x, w1 = (j & 1) ? vv.w : vv.y;
                        const float x[4] = {__uint_as_float(w0 << 16) * mul, __uint_as_float(w0 & 0xFFFF0000u) * mul,
                                            __uint_as_float(w1 << 16) * mul, __uint_as_float(w1 & 0xFFFF0000u) * mul};
                        uint16_t a, b2;
                        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(x[1]), "f"(x[0]));
                        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b2) : "f"(x[3]), "f"(x[2]));
                        hi[j] = (uint32_t)a | ((uint32_t)b2 << 16);
                        float y[4];
                        e4m3x4_to_f32(hi[j], y);
                        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(x[1] - y[1]), "f"(x[0] - y[0]));
                        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b2) : "f"(x[3] - y[3]), "f"(x[2] - y[2]));
                        lo[j] = (uint32_t)a | ((uint32_t)b2 << 16);
                    }
                    const int rh = 32 * query + h, rl = rh + 16, at = ((lane & 7) ^ (rh & 7)) << 4;   // rl & 7 is the same
                    *reinterpret_cast<uint4*>(&sm.Qs[lane >> 3][rh][at]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(&sm.Qs[lane >> 3][rl][at]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    const float scale = __uint_as_float((uint32_t)(127 + e) << 23) * (p.sm_scale * 1.4426950408889634f);
                    if (lane == 0) rowf[r] = top[k] < 0x7F80u ? scale : __uint_as_float(0x7FC00000u);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.q_full[k_item & 1]);
            }
            if (k_item > 0) {
                // ---- the output of the item before ----
                wg_bar(wg);
                if (key < kH) {
                    const int r = kH * wg + key;
                    const float sum = (sm.lsum[0][r] + sm.lsum[1][r]) + (sm.lsum[2][r] + sm.lsum[3][r]), ref = sm.mref[r];
                    if (split) {
                        float* ml = args.part_ml + (part * R + r) * 2;
                        *reinterpret_cast<float2*>(ml) = make_float2(ref, sum);
                    } else if (p.lse && query < prev_nq) {
                        p.lse[(int64_t)(prev_f0 + query) * kH + key] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
                    }
                    sm.mref[r] = -INFINITY;   // for the next item
                    sm.fac[r] = (split ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum) * (1.0f / kPScale);
                }
                wg_bar(wg);
                const int done = kPair ? last : nt > 0 ? n - 1 : -1;
                if (done >= 0) wait(&sm.pv_done[pbar(done)], ppar(done));
                tc_fence_after();
                float fac[kH];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 f = row4(sm.fac, j);
                    fac[4 * j] = f.x, fac[4 * j + 1] = f.y, fac[4 * j + 2] = f.z, fac[4 * j + 3] = f.w;
                }
                float* po = args.part_o + (part * R + kH * wg) * kD;
                // bf16 out: lanes 2 i and 2 i + 1 trade rows, so that each stores two channels of eight rows
                uint16_t* out = p.out + ((int64_t)(prev_f0 + query) * kH + 8 * (lane & 1)) * kD + (key & ~1);
#pragma unroll
                for (int b = 0; b < kBlocks; ++b) {
                    uint32_t o[kTerms][16];
#pragma unroll
                    for (int y = 0; y < kTerms; ++y) tmem_ld_32x32b_x16(ocol(b, y), o[y]);
                    tmem_ld_wait();
                    float y[kH];
#pragma unroll
                    for (int h = 0; h < kH; ++h) {
                        y[h] = __uint_as_float(o[0][h]);
#pragma unroll
                        for (int x = 1; x < kTerms; ++x) y[h] += __uint_as_float(o[x][h]);
                        y[h] *= fac[h];
                    }
                    if (split) {
#pragma unroll
                        for (int h = 0; h < kH; ++h) po[h * kD + 128 * b + key] = y[h];
                    } else if (query < prev_nq) {
#pragma unroll
                        for (int h = 0; h < 8; ++h) {
                            const uint32_t own = pack_bf16(y[h], y[h + 8]), other = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
                            *reinterpret_cast<uint32_t*>(out + h * kD + 128 * b) =
                                (lane & 1) ? __byte_perm(other, own, 0x7632) : __byte_perm(own, other, 0x5410);
                        }
                    }
                }
                tc_fence_before();
                wg_bar(wg);   // fac and mref are free
            }
            if (!have) break;

            const Item<NQ>& item = sm.item[k_item & 1];
            const int qi = item.qi[query], qlow = item.qlow[query];
            nt = item.tiles;
            part = item.part;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.item_empty[k_item & 1]);
            {
                uint32_t zero[16] = {};
#pragma unroll
                for (int b = 0; b < kBlocks; ++b)
#pragma unroll
                    for (int x = 0; x < kTerms; ++x) tmem_st_x16(ocol(b, x), zero);
                tmem_st_wait();
            }
            if (kPair)   // rowf of the whole query
                wait(&sm.q_full[k_item & 1], (uint32_t)((k_item >> 1) & 1));
            else
                wg_bar(wg);
            last = -1;
            float l[kH];
#pragma unroll
            for (int h = 0; h < kH; ++h) l[h] = 0.0f;

            // After a wait that ran out the loop goes on with what is there: every thread passes every named barrier.
            for (int i = 0; i < nt; ++i, ++n) {
                if (kPair && (n & 1) != wg) continue;
                const int st = n % ST;
                bool ok = wait(&sm.full[st][0], (uint32_t)((n / ST) & 1));   // the scales and what the producer says of the tile
                const Tile tile = sm.tile[st];
                const bool active = kPair || (wg >= tile.qa && wg < tile.qa + tile.nq);   // this tile's products cover this query
                bool seen = active;
                if (!tile.interior) {
                    const int first_pos = sm.upos[st][ku], pos = first_pos + ko;
                    seen = active && first_pos >= 0 && pos < tile.end && pos <= qi && (pos >= qlow || pos < tile.sink);
                }
                const float ts = seen ? sm.sc[st][key] : 0.0f;
                bool dirty = false;
                ok = wait(&sm.s_full[n & 1], (uint32_t)((n >> 1) & 1)) && ok;
                tc_fence_after();
                if (active) {
                    const float lsc = fmaxf(__log2f(ts), kMinLogScale);
                    float x[kH];   // logits in log2 units less the rows' references
                    auto sums = [&](uint32_t (&u)[32]) {   // hi in u[0 .. 15], lo in u[16 .. 31]
                        tmem_ld_32x32b_x32(tq + kS0 + (n & 1) * 2 * RQ + 32 * query, u);
                        tmem_ld_wait();
                        dirty = isnan(__uint_as_float(u[0]));   // in every query of the tile alike, or they would not share the zeroing
                    };
                    const bool first = i < kTurn;
                    bool move = first;
                    if (!first) {
                        uint32_t u[32];
                        sums(u);
                        float top = -INFINITY;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 f4 = rowf4(j), m4 = row4(sm.mref, j);
                            const float f[4] = {f4.x, f4.y, f4.z, f4.w}, m[4] = {m4.x, m4.y, m4.z, m4.w};
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                const int h = 4 * j + c;
                                x[h] = fmaf(__uint_as_float(u[h]) + __uint_as_float(u[16 + h]), ts * f[c], -m[c]);
                                top = fmaxf(top, x[h]);
                            }
                        }
                        move = wg_any(wg, seen && top + lsc > kHeadroom);
                    }
                    // A weight beyond the headroom (or a row's first keys, against a reference of -inf): move the references.
                    if (__builtin_expect(move, 0)) {
                        // here each product is rounded for itself, in the maximum as below: huge logits meet it exactly
                        float mx[kH];
                        {
                            uint32_t u[32];
                            sums(u);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float4 f4 = rowf4(j);
                                const float f[4] = {f4.x, f4.y, f4.z, f4.w};
#pragma unroll
                                for (int c = 0; c < 4; ++c) {
                                    const int h = 4 * j + c;
                                    x[h] = __fmul_rn(__fmul_rn(__uint_as_float(u[h]) + __uint_as_float(u[16 + h]), ts), f[c]);
                                }
                            }
                        }
#pragma unroll
                        for (int h = 0; h < kH; ++h) mx[h] = redux_max(seen ? x[h] + lsc : -INFINITY);
                        if (lane == 0) {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                *reinterpret_cast<float4*>(&sm.wmax[quarter][kH * wg + 4 * j]) =
                                    make_float4(mx[4 * j], mx[4 * j + 1], mx[4 * j + 2], mx[4 * j + 3]);
                        }
                        wg_bar(wg);
                        if (key < kH) {
                            const int r = kH * wg + key;
                            const float m = fmaxf(fmaxf(sm.wmax[0][r], sm.wmax[1][r]), fmaxf(sm.wmax[2][r], sm.wmax[3][r]));
                            const float old = sm.mref[r];
                            sm.fac[r] = m > old ? (old == -INFINITY ? 0.0f : ex2(old - m)) : 1.0f;
                            sm.mref[r] = fmaxf(m, old);
                        }
                        wg_bar(wg);
                        if (!first) {
                            wait(&sm.pv_done[pbar(n)], ppar(n - kTurn));
                            tc_fence_after();
#pragma unroll 1
                            for (int b = 0; b < kBlocks; ++b)
#pragma unroll 1
                                for (int y = 0; y < kTerms; ++y) {
                                uint32_t o[16];
                                tmem_ld_32x32b_x16(ocol(b, y), o);
                                tmem_ld_wait();
#pragma unroll
                                for (int h = 0; h < kH; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * sm.fac[kH * wg + h]);
                                tmem_st_x16(ocol(b, y), o);
                            }
                            tmem_st_wait();
                        }
                        if (!first) {
#pragma unroll
                            for (int h = 0; h < kH; ++h) l[h] *= sm.fac[kH * wg + h];
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 m = row4(sm.mref, j);
                            x[4 * j] -= m.x, x[4 * j + 1] -= m.y, x[4 * j + 2] -= m.z, x[4 * j + 3] -= m.w;
                        }
                    }
                    if (!tile.interior) {
#pragma unroll
                        for (int h = 0; h < kH; ++h) x[h] = seen ? x[h] : -INFINITY;
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0 && ok) mbar_arrive(&sm.s_free[n & 1]);
                    if (quarter < tile.steps) {   // else P K stops before this warp's keys
                        const float tp = ts * kPScale;
                        uint32_t w[3][4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float e[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                e[i] = ex2(x[4 * j + i]);
                                l[4 * j + i] += e[i];
                            }
                            uint32_t h0, m0, l0, h1, m1, l1;
                            split_e5m2(pack_f16(e[0] * tp, e[1] * tp), h0, m0, l0);
                            split_e5m2(pack_f16(e[2] * tp, e[3] * tp), h1, m1, l1);
                            w[0][j] = __byte_perm(h0, h1, 0x7531);
                            w[1][j] = __byte_perm(m0, m1, 0x7531);
                            w[2][j] = __byte_perm(l0, l1, 0x7531);
                        }
                        // P is free when the products of the warpgroup's last tile are done
                        if (n >= kTurn) ok = wait(&sm.pv_done[pbar(n)], ppar(n - kTurn)) && ok;
#pragma unroll
                        for (int y = 0; y < 3; ++y)
                            *reinterpret_cast<uint4*>(&sm.P[kPair ? 3 * wg + y : y * NQ + wg][key][0]) =
                                make_uint4(w[y][0], w[y][1], w[y][2], w[y][3]);
                    } else if (n >= kTurn) {
                        ok = wait(&sm.pv_done[pbar(n)], ppar(n - kTurn)) && ok;
                    }
                } else if (n > 0) {
                    // a warpgroup that sits a tile out must not arrive for it before the last tile's arrivals are complete
                    ok = wait(&sm.pv_done[0], ppar(n - 1)) && ok;
                }
                if (!active && lane == 0 && ok) mbar_arrive(&sm.s_free[n & 1]);
                if (dirty && ok) {   // S of this tile is done: only P K still reads the row, of which each query zeroes a part
                    for (int b = query - tile.qa; b < kBlocks; b += tile.nq)
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                        {
                            const uint32_t at = (key >> 3) * kGroupStep + b * kBlockStep + (key & 7) * 128 + 16 * ((j + key) & 7);
                            *reinterpret_cast<uint4*>(&sm.K[st][at]) = make_uint4(0, 0, 0, 0);
                        }
                }
                fence_proxy_async_smem();
                tc_fence_before();
                if (ok) mbar_arrive(&sm.p_full[pbar(n)]);
                if (kPair) last = n;
            }
            // ---- row sums over the 128 threads ----
            {
                // halving exchange: after step o a lane holds the sums over lane pairs of half as many rows
                float v[kH];
#pragma unroll
                for (int h = 0; h < kH; ++h) v[h] = l[h];
#pragma unroll
                for (int o = 8; o > 0; o >>= 1) {
                    const bool up = (lane & o) != 0;
#pragma unroll
                    for (int h = 0; h < o; ++h) {
                        const float keep = up ? v[h + o] : v[h], give = up ? v[h] : v[h + o];
                        v[h] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, o);
                    }
                }
                v[0] += __shfl_xor_sync(0xFFFFFFFFu, v[0], 16);   // lane i: row i & 15
                if (lane < kH) sm.lsum[quarter][kH * wg + lane] = v[0];
            }
        }
    }
    __syncthreads();
    if (warp == kIssuer) tmem_dealloc(sm.tmem, kTmemCols);
}

// Joins the splits of a block, weight 2^(m_s - M) / L with L = sum_s l_s 2^(m_s - M).  The weights come first, a thread
// per split, so that the loads of the partial rows do not wait on one another.  Few splits: a CTA of 128 threads per
// row.  Twelve and more: four groups of 128 threads that take every fourth split (12 queries in 49 splits 36 us in all
// against 44 with one group; 61 queries in 4 splits 47.6 against 45.5).  64 and more, which leave few rows: four CTAs per
// row, 128 channels each, whose 16 warps take every sixteenth split (one query, 131,072 keys, 296 parts: 26.0 us in all
// against 38.3 with four groups; four queries of 74 parts 55.0 against 57.9; four of 49 parts 17.7 against 17.0).
constexpr int kMergeMany = 12, kMergeSlice = 64;
template <int kGroups, int kLanes>
__global__ void __launch_bounds__(kGroups * kLanes) pages_merge_kernel(const __grid_constant__ KernelArgs args, int NQ) {
    pdl_enter();
    constexpr int kWarps = kGroups * kLanes / 32;
    __shared__ float w[kMaxSplits], red[kWarps], red2[kWarps];
    __shared__ float4 part[kGroups][kLanes];
    static_assert(kMaxSplits <= 512 && kMergeMany <= 128, "a thread per split");
    const PagesAttnParams& p = args.p;
    const int S = args.splits, R = kH * NQ, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int group = tid / kLanes, at = tid % kLanes, col = blockIdx.y * kLanes + at;
    const int f = blockIdx.x / kH, h = blockIdx.x % kH;
    int blk, c;
    if (p.prefix.B) {
        blk = f / NQ;
        c = f % NQ;
    } else {
        const int per = (p.Q + NQ - 1) / NQ, b = f / p.Q, q = f % p.Q;
        blk = b * per + q / NQ;
        c = q % NQ;
    }
    const int64_t r0 = ((int64_t)blk * S) * R + 16 * c + h;   // row of split s: r0 + s R
    const float2 v = tid < S ? __ldcg(reinterpret_cast<const float2*>(args.part_ml) + r0 + (int64_t)tid * R)
                             : make_float2(-INFINITY, 0.0f);
    const float wm = redux_max(v.x);
    if (lane == 0) red[warp] = wm;
    __syncthreads();
    float M = red[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) M = fmaxf(M, red[i]);
    const float Mu = M == -INFINITY ? 0.0f : M;
    const float e = exp2f(v.x - Mu);
    if (tid < S) w[tid] = e;
    float L = v.y * e;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xFFFFFFFFu, L, o);
    if (lane == 0) red2[warp] = L;
    __syncthreads();
    const float4* po = reinterpret_cast<const float4*>(args.part_o + r0 * kD) + col;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int s = group; s < S; s += kGroups) {
        const float4 y = __ldcg(po + (int64_t)s * R * (kD / 4));
        const float ws = w[s];
        o.x = fmaf(y.x, ws, o.x);
        o.y = fmaf(y.y, ws, o.y);
        o.z = fmaf(y.z, ws, o.z);
        o.w = fmaf(y.w, ws, o.w);
    }
    L = red2[0];
#pragma unroll
    for (int i = 1; i < kWarps; ++i) L += red2[i];
    if (kGroups > 1) {
        if (group > 0) part[group][at] = o;
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g = 1; g < kGroups; ++g) {
            const float4 y = part[g][at];
            o = make_float4(o.x + y.x, o.y + y.y, o.z + y.z, o.w + y.w);
        }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    *reinterpret_cast<uint2*>(p.out + (int64_t)blockIdx.x * kD + 4 * col) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (p.lse && tid == 0 && blockIdx.y == 0) p.lse[blockIdx.x] = L == 0.0f ? -INFINITY : (Mu + log2f(L)) * 0.6931471805599453f;
}

// ---- host ----------------------------------------------------------------------------------

struct Plan {
    int nq, blocks, splits;
    bool two;   // two CTAs on an SM, one tile in flight each
    bool pair;  // one query by two warpgroups, each of which leaves a part of its own
    int parts;  // partial results of a block
    size_t o_bytes, bytes;
};

// Queries of a CTA, and how its keys are split.  Sizes alone decide, so that a workspace can be sized without a device.
Plan plan(bool prefix, int B, int Q, int64_t keys) {
    Plan pl{};
    const int64_t n = (int64_t)B * Q;
    const int64_t together = prefix ? n : Q;   // queries that share keys
    int64_t tiles = (keys + kTileKeys - 1) / kTileKeys + (prefix ? 1 : 0);
    if (tiles < 1) tiles = 1;
    // Four queries share a tile's copies and products where there is much work: 100 x 4 queries of 640 keys 24 us against 42
    // with a query in each CTA, 4 x 128 of a 128-token window 13.7 against 21.5.  While it fits the GPU about once, single
    // queries have the shorter chain: 4 queries of a 128-token window 7.8 us against 12.5, 4 behind 4,096 tokens 13.2
    // against 17.6, 16 behind 4,096 16.8 against 20.4; the two meet at about 1,000 tiles (32 behind 4,096 23.5 and 22.6).
    pl.nq = together == 1 || (n <= 2 * kSplitSMs && n * tiles <= 1024) ? 1 : 4;
    pl.blocks = (int)(pl.nq == 1 ? n : prefix ? (n + 3) / 4 : (int64_t)B * ((Q + 3) / 4));
    // Up to three tiles cost a CTA no more than the join does (one query of 384 keys 8.8 us whole, 9.6 split; of 512 12.0
    // and 9.8; four queries of 384 15.9 and 14.8, of 512 18.2 and 15.1; a caller's workspace not counted).
    const int64_t most = tiles < 4 ? 1 : tiles;
    auto splits = [&](int64_t ctas) { return std::max<int64_t>(1, std::min(ctas / pl.blocks, most)); };
    int64_t s = splits(pl.nq == 1 ? 2 * kSplitSMs : kSplitSMs);
    // One query.  With few tiles and CTAs, all of them in flight in one CTA (8 queries of 1,000 keys 9.9 us against 11.8 by
    // a pair, one of 132 keys 8.4 against 9.6 by two CTAs).  Else a pair, whose two warpgroups share three tiles in flight,
    // where a CTA has one item or long ones (148 queries of 640 keys 19.6 us against 24.6 by two CTAs, 300 of 4,096 150
    // against 195); two CTAs of one tile each where items are many and short, so that one works while the other changes
    // its item (250 of 500 keys 23.3 us against 31.2 by a pair, 600 of 1,024 92.7 against 96.8).
    if (pl.nq == 1) {
        const bool few = tiles <= 3 * s && pl.blocks * s <= kSplitSMs;
        pl.pair = !few && (pl.blocks <= kSplitSMs || tiles >= 16);
        pl.two = !few && !pl.pair;
        if (pl.pair) s = splits(kSplitSMs);
    }
    pl.splits = (int)s;
    pl.parts = pl.splits * (pl.pair ? 2 : 1);
    pl.bytes = 256;
    if (pl.parts > 1) {
        const size_t rows = (size_t)pl.blocks * pl.parts * kH * pl.nq;
        pl.o_bytes = rows * kD * 4;
        pl.bytes += pl.o_bytes + rows * 8;
    }
    return pl;
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor map encoder, found at run time: the library does not link libcuda.
EncodeFn encoder() {
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
            r != cudaDriverEntryPointSuccess)
            f = nullptr;
        return (EncodeFn)f;
    }();
    return fn;
}

// The pool as a tensor [groups of 8 rows][4 channel blocks][8 rows][128 B], a box being a unit's groups: they land in the
// tile's order.
cudaError_t pool_map(const csa2_pages& pg, int unit, CUtensorMap* map) {
    const EncodeFn fn = encoder();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t rows = (cuuint64_t)(pg.n_pages * pg.page_size);
    const cuuint64_t dims[4] = {128, kGroup, kBlocks, rows / kGroup}, strides[3] = {kD, 128, (cuuint64_t)kGroup * kD};
    const cuuint32_t es[4] = {1, 1, 1, 1}, box[4] = {128, kGroup, kBlocks, (cuuint32_t)(unit / kGroup)};
    const auto encode = [&] {
        return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, pg.kv, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    };
    if (encode() == CUDA_SUCCESS) return cudaSuccess;
    // The encoder is the driver's and needs a context.  A host thread has none before its first call of the runtime that
    // works on the device, and in such a thread this is the first: bind the current device's.
    const cudaError_t e = cudaSetDevice(current_device());
    if (e != cudaSuccess) return e;
    return encode() == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int NQ, int ST, bool kConcat, int kCtas, bool kPair = false>
cudaError_t launch(const KernelArgs& a, const CUtensorMap& own, const CUtensorMap& prefix, cudaStream_t st) {
    static DeviceOnce attr;
    const auto kernel = pages_attn_kernel<NQ, ST, kConcat, kCtas, kPair>;
    constexpr int W = kPair ? 2 : NQ;
    const int smem = (int)sizeof(Smem<NQ, ST, W>) + 1024, most = device_sm_count() * kCtas;
    cudaError_t e = attr.run([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    return launch_ex(kernel, dim3(most > 0 && a.items > most ? most : a.items), dim3(kWg * W + kAux), smem, st, 0, own, prefix, a);
}

}  // namespace

size_t pages_attn_ws_bytes(bool prefix, int B, int Q, int64_t keys) { return plan(prefix, B, Q, keys).bytes; }

cudaError_t launch_pages_attn(const PagesAttnParams& p, int64_t keys, void* ws, cudaStream_t st) {
    const bool prefix = p.prefix.B != 0;
    const Plan pl = plan(prefix, p.B, p.Q, keys);
    KernelArgs a{};
    a.p = p;
    a.splits = pl.splits;
    a.items = pl.blocks * pl.splits;
    a.test_starve = test_starve_copies();
    a.part_o = (float*)ws;
    a.part_ml = (float*)((char*)ws + pl.o_bytes);
    // A unit lies in one page.  Units of 32 keys cost half as many copies as 16 (300 queries of 4,096 keys 148.5 us against
    // 153.5); a short window takes 16, as its first unit reaches back over up to unit - 1 keys that no query sees.
    int unit = prefix || p.window >= 512 ? 32 : 16;
    while (p.own.page_size % unit || (prefix && p.prefix.page_size % unit)) unit /= 2;
    while ((1 << a.unit_log2) < unit) ++a.unit_log2;
    a.by_splits = div_by(pl.splits);
    a.by_q = div_by(p.Q);
    a.by_per = div_by((p.Q + pl.nq - 1) / pl.nq);
    a.by_page_own = div_by(p.own.page_size / unit);
    a.by_page_prefix = div_by(prefix ? p.prefix.page_size / unit : 1);
    CUtensorMap mo, mp;
    cudaError_t e = pool_map(p.own, unit, &mo);
    if (e != cudaSuccess) return e;
    mp = mo;
    if (prefix && (p.prefix.kv != p.own.kv || p.prefix.n_pages * p.prefix.page_size != p.own.n_pages * p.own.page_size)) {
        e = pool_map(p.prefix, unit, &mp);
        if (e != cudaSuccess) return e;
    }
    e = pl.nq == 4 ? launch<4, 2, false, 1>(a, mo, mp, st)
        : pl.pair  ? launch<1, 3, true, 1, true>(a, mo, mp, st)
        : pl.two   ? launch<1, 1, true, 2>(a, mo, mp, st)
                   : launch<1, 3, true, 1>(a, mo, mp, st);
    if (e != cudaSuccess || pl.parts == 1) return e;
    a.splits = pl.parts;
    const unsigned rows = (unsigned)(p.B * p.Q * kH);
    return pl.parts < kMergeMany   ? launch_ex(pages_merge_kernel<1, 128>, dim3(rows), dim3(128), 0, st, 0, a, pl.nq)
           : pl.parts < kMergeSlice ? launch_ex(pages_merge_kernel<4, 128>, dim3(rows), dim3(512), 0, st, 0, a, pl.nq)
                                    : launch_ex(pages_merge_kernel<16, 32>, dim3(rows, 4), dim3(512), 0, st, 0, a, pl.nq);
}

}  // namespace csa2
