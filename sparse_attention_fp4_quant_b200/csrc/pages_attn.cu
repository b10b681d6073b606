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
//       elements 2^-10 below the row's largest (each row scaled by its own power of two),
//       which are held to 2^-18 of it.  hi and lo are separate columns of S, added in fp32.
//   P   each weight times its token scale, as f16 with 2^12 of headroom below the maximum,
//       split in three E5M2 terms (f16's exponent range): at least 9 significant bits and
//       nothing lost down to 2^-36 of the largest weight.
// Softmax: fp32, one thread per key, one pass with a running reference m per row.  The
// reference is the maximum of z + log2(token scale), the size of what enters P, and it moves
// only when a tile exceeds it by 2^3 (P keeps that much room), so the accumulators are
// rescaled rarely.  l = sum 2^(z - m) stays in fp32 registers.
// Keys that no query of the CTA sees have their rows zeroed in shared memory before P K:
// a slot may hold NaN bytes, and 0 times NaN is NaN.
#include <cuda.h>

#include "attn_common.cuh"
#include "tc.cuh"

namespace csa2 {

namespace {

using namespace tc;

constexpr int kTileKeys = 128;
constexpr int kGroup = 8;                              // keys per TMA box: rows of one swizzle atom
constexpr int kTileGroups = kTileKeys / kGroup;
constexpr int kTileBytes = kTileKeys * kD;             // 64 KB
constexpr int kSoftmaxThreads = 128;
constexpr int kThreads = kSoftmaxThreads + 64;         // + producer warp + MMA warp
constexpr float kHeadroom = 3.0f;                      // log2 of how far a weight may exceed the reference
constexpr float kPScale = 4096.0f;                     // weight 1 at 2^12, 2^15 with the headroom: below f16's and E5M2's largest
constexpr float kMinLogScale = -100.0f;                // token scales below 2^-100 count as 2^-100 in the reference
constexpr uint64_t kTimeoutNs = 2000000000ull;

// One list of keys of a CTA: groups of 8 slots of one table row, `sink` first groups and then the
// window's (virtual group v is group v, or v + delta from `sink` on), for queries [qa, qa + nq).
struct Seg {
    int tile0;      // first tile of the list in the CTA's order
    int groups, sink, delta;
    int which, b;   // 0 = prefix, 1 = own; table row
    int qa, nq;
    int end;        // first position behind the stored tokens
};

template <int NQ, int ST>
struct Smem {
    static constexpr int R = kH * NQ;
    alignas(1024) uint8_t K[ST][kTileBytes];     // [16 groups][4 channel blocks][8 keys][128 B], 128-byte swizzle
    alignas(1024) uint8_t Qs[4][2 * R][128];     // [channel block][query][hi 16 | lo 16][128 B], 128-byte swizzle
    alignas(1024) uint8_t P[3 * NQ][kTileKeys][16];   // [term][query]: 16 rows of each key, no swizzle
    float wmax[4][R];
    alignas(16) float mref[R];
    alignas(16) float fac[R];
    alignas(16) float rowf[R];
    float lsum[R];
    Seg seg[NQ + 1];
    int nseg, ntiles;
    int qi[NQ], qlow[NQ];
    int rescale[2];
    int dead;
    uint32_t tmem;
    uint64_t full[ST], empty[ST], s_full[2], p_full, pv_done, wind_down;
};

__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Instruction descriptors, M = 128, K = 32, fp32 accumulation: E4M3 x E4M3, both K-major; and
// E4M3 (channel-major) x E5M2 (row-major, "MN-major").
__device__ __forceinline__ uint32_t idesc_qk(int N) { return (1u << 4) | ((uint32_t)(N >> 3) << 17) | (8u << 24); }
__device__ __forceinline__ uint32_t idesc_pv(int N) {
    return (1u << 4) | (1u << 10) | (1u << 15) | (1u << 16) | ((uint32_t)(N >> 3) << 17) | (8u << 24);
}
constexpr uint32_t kSw128 = 2;

__device__ __forceinline__ void tma_group(void* dst, const CUtensorMap* map, int group, uint64_t* bar) {
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

__device__ __forceinline__ void softmax_bar() { asm volatile("bar.sync 1, %0;" ::"n"(kSoftmaxThreads) : "memory"); }

// Two weights (f16x2) -> three terms of E5M2 in the high bytes of each half.  An E5M2 value is an
// f16 whose low byte is zero: hi and mid truncate (each leaves a remainder of the next bits,
// exact in f16), lo rounds to nearest by adding half of its last place.
__device__ __forceinline__ void split_e5m2(uint32_t p, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
    hi = p & 0xFF00FF00u;
    __half2 r = __hsub2(*reinterpret_cast<__half2*>(&p), *reinterpret_cast<__half2*>(&hi));
    const uint32_t rb = *reinterpret_cast<uint32_t*>(&r);
    mid = rb & 0xFF00FF00u;
    r = __hsub2(r, *reinterpret_cast<const __half2*>(&mid));
    lo = (*reinterpret_cast<uint32_t*>(&r) + 0x00800080u) & 0xFF00FF00u;
}

__device__ __forceinline__ int stored_end(const csa2_pages& pg, int b) {
    const int64_t cap = (int64_t)pg.max_pages * pg.page_size;
    int64_t n = pg.n_tokens[b];
    n = n < 0 ? 0 : n > cap ? cap : n;
    return (int)(pg.pos0 + n);
}

struct KernelArgs {
    PagesAttnParams p;
    int splits;
    int test_starve;  // test hook (csa2_test_starve_copies): the producer issues no copies
    float* part_o;    // [block][split][R][512]
    float* part_ml;   // [block][split][R][2]
};

template <int NQ, int ST>
__global__ void __launch_bounds__(kThreads, (NQ == 1 && ST == 1) ? 2 : 1)
    pages_attn_kernel(const __grid_constant__ CUtensorMap map_own, const __grid_constant__ CUtensorMap map_prefix,
                      const __grid_constant__ KernelArgs args) {
    using Sm = Smem<NQ, ST>;
    constexpr int R = Sm::R;
    constexpr bool kConcat = NQ <= 2;                  // the three terms of P in columns of their own (TMEM has room)
    constexpr int kOCols = (kConcat ? 3 : 1) * R;      // accumulator columns of one channel block
    constexpr uint32_t kTmemCols = NQ == 1 ? 256 : 512;
    constexpr uint32_t kS0 = 4 * kOCols;               // S^T buffers behind the accumulators
    static_assert(kS0 + 2 * 2 * R <= kTmemCols, "TMEM budget");
    extern __shared__ uint8_t smem_raw[];
    Sm& sm = *reinterpret_cast<Sm*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    const PagesAttnParams& p = args.p;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == 5) tmem_alloc(&sm.tmem, kTmemCols);
    if (tid == kSoftmaxThreads) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        mbar_init(&sm.s_full[0], 1);
        mbar_init(&sm.s_full[1], 1);
        mbar_init(&sm.p_full, kSoftmaxThreads);
        mbar_init(&sm.pv_done, 1);
        mbar_init(&sm.wind_down, 1);
        fence_mbar_init();
        sm.dead = 0;
        sm.rescale[0] = sm.rescale[1] = 0;
    }
    pdl_enter();

    // ---- this CTA's queries and key lists ----
    const bool shared_prefix = p.prefix.B != 0;
    int f0, nq;   // first query (b Q + q) and count
    if (shared_prefix) {
        f0 = blockIdx.y * NQ;
        nq = min(NQ, p.B * p.Q - f0);
    } else {
        const int per = (p.Q + NQ - 1) / NQ, b = blockIdx.y / per, q0 = (blockIdx.y % per) * NQ;
        f0 = b * p.Q + q0;
        nq = min(NQ, p.Q - q0);
    }
    if (warp == 4) {
        // lanes 0 .. NQ-1: a query each; its sequence's stored end; then lane 0 builds the lists
        int i = -1, low = 0, end = 0;
        const int b = (f0 + min(lane, nq - 1)) / p.Q;
        int pend = 0;
        if (lane < nq) i = p.q_pos[f0 + lane];
        if (lane < NQ) end = stored_end(p.own, b);
        if (shared_prefix && lane == 0) pend = stored_end(p.prefix, 0);
        if (i < 0) i = -1;
        int64_t lw = p.window == 0x7FFFFFFF ? 0 : (int64_t)i - p.window + 1;
        if (p.replay_start && lane < nq) lw = max(lw, (int64_t)p.replay_start[b]);
        low = (int)max(lw, (int64_t)0);
        if (lane < NQ) {
            sm.qi[lane] = i;
            sm.qlow[lane] = low;
        }
        int n = 0, tiles = 0, imax = -1;
#pragma unroll
        for (int c = 0; c < NQ; ++c) imax = max(imax, __shfl_sync(0xFFFFFFFFu, i, c));
        if (shared_prefix && lane == 0) {
            const int e = (imax < pend ? imax + 1 : pend) - p.prefix.pos0;
            if (e > 0) {
                const int g = (e + kGroup - 1) / kGroup;
                sm.seg[n++] = {0, g, 0, 0, 0, 0, 0, nq, pend};
                tiles = (g + kTileGroups - 1) / kTileGroups;
            }
        }
        int qa = 0;
        while (qa < nq) {   // runs of queries of one sequence (uniform over the warp)
            const int rb = __shfl_sync(0xFFFFFFFFu, b, qa), rend = __shfl_sync(0xFFFFFFFFu, end, qa);
            int c = qa, hi = 0, lo = 0x7FFFFFFF;
            while (c < nq && __shfl_sync(0xFFFFFFFFu, b, c) == rb) {
                const int ic = __shfl_sync(0xFFFFFFFFu, i, c), lc = __shfl_sync(0xFFFFFFFFu, low, c);
                if (ic >= 0) {
                    hi = max(hi, ic < rend ? ic + 1 : rend);
                    lo = min(lo, lc);
                }
                ++c;
            }
            if (lane == 0 && hi > p.own.pos0) {
                // sink groups, then the window's groups from the first that is not a sink group
                const int base = p.own.pos0;
                const int ns = min(p.n_sink, hi) - base;
                const int gs = ns > 0 ? (ns + kGroup - 1) / kGroup : 0;
                const int ge = (hi - base + kGroup - 1) / kGroup;
                const int gw = max(gs, lo > base ? (lo - base) / kGroup : 0);
                const int g = gs + max(0, ge - gw);
                if (g > 0) {
                    sm.seg[n++] = {tiles, g, gs, gw - gs, 1, rb, qa, c - qa, rend};
                    tiles += (g + kTileGroups - 1) / kTileGroups;
                }
            }
            qa = c;
        }
        if (lane == 0) {
            sm.nseg = n;
            sm.ntiles = tiles;
        }
    } else if (warp < 4) {
        // Q: a warp per row; 16 channels per lane -> E4M3 hi and lo, scaled so that the row's largest is in [2^7, 2^8)
        for (int r = warp; r < R; r += 4) {
            const int c = r >> 4, h = r & 15;
            uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
            if (c < nq) {
                const uint4* src = reinterpret_cast<const uint4*>(p.q + ((int64_t)(f0 + c) * kH + h) * kD) + 2 * lane;
                v[0] = __ldg(src);
                v[1] = __ldg(src + 1);
            }
            const float mx = redux_max(fmaxf(bf16x8_maxabs(v[0]), bf16x8_maxabs(v[1])));
            const int e = max((int)((__float_as_uint(mx) >> 23) & 0xFFu) - 127 - 7, -120);
            const float mul = __uint_as_float((uint32_t)(127 - e) << 23);
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4& vv = v[j >> 1];
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
            const int rh = 32 * c + h, rl = rh + 16, chunk = lane & 7;
            *reinterpret_cast<uint4*>(&sm.Qs[lane >> 3][rh][(chunk ^ (rh & 7)) << 4]) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4*>(&sm.Qs[lane >> 3][rl][(chunk ^ (rl & 7)) << 4]) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            if (lane == 0) {
                sm.rowf[r] = __uint_as_float((uint32_t)(127 + e) << 23) * (p.sm_scale * 1.4426950408889634f);
                sm.mref[r] = -INFINITY;
            }
        }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.tmem;
    const int ntiles = sm.ntiles;
    const int t0 = (int)((int64_t)ntiles * blockIdx.x / args.splits), t1 = (int)((int64_t)ntiles * (blockIdx.x + 1) / args.splits);

    // A bounded wait; the first to run out of time tells every other.
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
    auto seg_of = [&](int tile) -> int {
        int s = 0;
        while (s + 1 < sm.nseg && tile >= sm.seg[s + 1].tile0) ++s;
        return s;
    };

    if (warp == 4) {
        // ---- producer: one lane per 8-key group ----
        int issued = 0;
        bool ok = true;
        for (int t = t0; t < t1; ++t) {
            const int n = t - t0, st = n % ST;
            const Seg& sg = sm.seg[seg_of(t)];
            const csa2_pages& pg = sg.which ? p.own : p.prefix;
            const int v = (t - sg.tile0) * kTileGroups + lane;
            int row = -1;
            if (lane < kTileGroups && v < sg.groups) {
                const int slot = (v < sg.sink ? v : v + sg.delta) * kGroup;
                const int page = pg.table[(int64_t)sg.b * pg.max_pages + slot / pg.page_size];
                if (page >= 0 && page < pg.n_pages) row = page * pg.page_size + slot % pg.page_size;
            }
            const uint32_t live = __popc(__ballot_sync(0xFFFFFFFFu, row >= 0));
            if (n >= ST) ok = wait(&sm.empty[st], (uint32_t)((n / ST - 1) & 1));
            if (!__all_sync(0xFFFFFFFFu, ok)) break;
            if (lane == 0) mbar_arrive_expect_tx(&sm.full[st], live * kGroup * kD);
            __syncwarp();
            if (row >= 0 && !args.test_starve)
                tma_group(sm.K[st] + lane * kGroup * kD, sg.which ? &map_own : &map_prefix, row / kGroup, &sm.full[st]);
            ++issued;
        }
        if (*(volatile int*)&sm.dead) {   // wind down: the copies in flight land before the CTA ends
            for (int n = max(0, issued - ST); n < issued; ++n) mbar_wait(&sm.full[n % ST], (uint32_t)((n / ST) & 1));
        }
    } else if (warp == 5) {
        // ---- MMA issuer (one lane): S of the next tile or O of the last, whichever is ready ----
        if (lane == 0) {
            const uint32_t sQ = smem_u32(sm.Qs), sP = smem_u32(sm.P);
            const int n = t1 - t0;
            int iq = 0, ip = 0;
            uint64_t start = globaltimer_ns();
            uint32_t idle = 0;
            while (ip < n) {
                bool moved = false;
                if (iq < n && iq <= ip + 1 && mbar_try_wait(&sm.full[iq % ST], (uint32_t)((iq / ST) & 1))) {
                    const Seg& sg = sm.seg[seg_of(t0 + iq)];
                    const uint32_t k = smem_u32(sm.K[iq % ST]), d = tmem + kS0 + (iq & 1) * 2 * R + 32 * sg.qa;
                    const uint32_t id = idesc_qk(32 * sg.nq);
                    tc_fence_after();
#pragma unroll
                    for (int s = 0; s < kD / 32; ++s)
                        mma_f8(d, smem_desc(k + (s >> 2) * 1024 + (s & 3) * 32, 16, 4096, kSw128),
                               smem_desc(sQ + (s >> 2) * (2 * R * 128) + sg.qa * 4096 + (s & 3) * 32, 16, 1024, kSw128), id, s > 0);
                    tc_commit(&sm.s_full[iq & 1]);
                    ++iq;
                    moved = true;
                }
                if (ip < iq && mbar_try_wait(&sm.p_full, (uint32_t)(ip & 1))) {
                    const int t = t0 + ip;
                    const Seg& sg = sm.seg[seg_of(t)];
                    const uint32_t k = smem_u32(sm.K[ip % ST]);
                    const int keys = min(kTileGroups, sg.groups - (t - sg.tile0) * kTileGroups) * kGroup;
                    const int steps = (keys + 31) / 32;
                    tc_fence_after();
                    for (int s = 0; s < steps; ++s) {
#pragma unroll
                        for (int b = 0; b < 4; ++b) {
                            const uint64_t a = smem_desc(k + s * 16384 + b * 1024, 1024, 4096, kSw128);
                            const uint32_t d = tmem + b * kOCols + kH * sg.qa;
                            if (kConcat && sg.nq == NQ) {
                                mma_f8(d, a, smem_desc(sP + s * 512, 128, 2048, kLayoutNone), idesc_pv(3 * R), 1);
                            } else {
#pragma unroll
                                for (int x = 0; x < 3; ++x)
                                    mma_f8(d + (kConcat ? x * R : 0), a,
                                           smem_desc(sP + (x * NQ + sg.qa) * 2048 + s * 512, 128, 2048, kLayoutNone),
                                           idesc_pv(kH * sg.nq), 1);
                            }
                        }
                    }
                    tc_commit(&sm.empty[ip % ST]);
                    tc_commit(&sm.pv_done);
                    ++ip;
                    moved = true;
                }
                if (moved) {
                    idle = 0;
                } else if ((++idle & 63u) == 0u) {
                    if (idle == 64u) start = globaltimer_ns();
                    if (*(volatile int*)&sm.dead) break;
                    if (globaltimer_ns() - start > kTimeoutNs) {
                        *(volatile int*)&sm.dead = 1;
                        if (p.flag) *p.flag = 1;
                        break;
                    }
                }
            }
            if (*(volatile int*)&sm.dead) {   // wind down: no MMA in flight when TMEM is freed
                tc_commit(&sm.wind_down);
                mbar_wait(&sm.wind_down, 0);
            }
        }
        __syncwarp();
    } else {
        // ---- softmax: thread = key ----
        const uint32_t lanes = (uint32_t)(warp * 32) << 16;
        {
            uint32_t z[16] = {};
            for (uint32_t c = 0; c < kS0; c += 16) tmem_st_x16(tmem + lanes + c, z);
            tmem_st_wait();
        }
        float l[R];
#pragma unroll
        for (int r = 0; r < R; ++r) l[r] = 0.0f;

        // the thread's key of a tile: its row in the pool, or -1, and which queries see it
        auto key_of = [&](int t, int& row, uint32_t& vis, const float*& scales) {
            const Seg& sg = sm.seg[seg_of(t)];
            const csa2_pages& pg = sg.which ? p.own : p.prefix;
            scales = pg.kv_sc;
            row = -1;
            vis = 0;
            const int v = (t - sg.tile0) * kTileGroups + (tid >> 3);
            if (v >= sg.groups) return;
            const int slot = (v < sg.sink ? v : v + sg.delta) * kGroup + (tid & 7), pos = pg.pos0 + slot;
            if (pos >= sg.end) return;
            const int page = pg.table[(int64_t)sg.b * pg.max_pages + slot / pg.page_size];
            if (page < 0 || page >= pg.n_pages) return;
            row = page * pg.page_size + slot % pg.page_size;
#pragma unroll
            for (int c = 0; c < NQ; ++c)
                if (c >= sg.qa && c < sg.qa + sg.nq && pos <= sm.qi[c] && (pos >= sm.qlow[c] || (sg.which && pos < p.n_sink)))
                    vis |= 1u << c;
        };
        int row = -1;
        uint32_t vis = 0;
        float ts = 0.0f;
        const float* scales = nullptr;
        if (t0 < t1) {
            key_of(t0, row, vis, scales);
            if (vis) ts = __ldg(scales + row);
        }
        // After a wait that ran out the loop goes on with what is there: every thread passes every barrier.
        for (int t = t0; t < t1; ++t) {
            const int n = t - t0;
            int nrow = -1;
            uint32_t nvis = 0;
            const float* nscales = nullptr;
            if (t + 1 < t1) key_of(t + 1, nrow, nvis, nscales);
            const Seg& sg = sm.seg[seg_of(t)];
            const int keys = min(kTileGroups, sg.groups - (t - sg.tile0) * kTileGroups) * kGroup;
            const float lsc = fmaxf(__log2f(ts), kMinLogScale);
            wait(&sm.s_full[n & 1], (uint32_t)((n >> 1) & 1));
            tc_fence_after();
            float z[R];
            const uint32_t sbase = tmem + lanes + kS0 + (n & 1) * 2 * R;
#pragma unroll
            for (int c = 0; c < NQ; ++c) {
                uint32_t v[32];
                tmem_ld_32x32b_x32(sbase + 32 * c, v);
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < kH; ++h) z[16 * c + h] = __uint_as_float(v[h]) + __uint_as_float(v[16 + h]);
            }
            tc_fence_before();
            // logits (log2 units), and each row's maximum of z + log2(scale) over the warp's keys
#pragma unroll
            for (int c = 0; c < NQ; ++c) {
                const bool seen = (vis >> c) & 1u;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 f = *reinterpret_cast<const float4*>(&sm.rowf[16 * c + 4 * j]);
                    const float ff[4] = {f.x, f.y, f.z, f.w};
                    float mx[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 16 * c + 4 * j + i;
                        z[r] = seen ? z[r] * ts * ff[i] : -INFINITY;
                        mx[i] = redux_max(z[r] + lsc);
                    }
                    if (lane == 0) *reinterpret_cast<float4*>(&sm.wmax[warp][16 * c + 4 * j]) = make_float4(mx[0], mx[1], mx[2], mx[3]);
                }
            }
            softmax_bar();
            if (tid < R) {
                const float m = fmaxf(fmaxf(sm.wmax[0][tid], sm.wmax[1][tid]), fmaxf(sm.wmax[2][tid], sm.wmax[3][tid]));
                const float old = sm.mref[tid];
                float f = 1.0f;
                if (m > old + kHeadroom) {   // -inf + 3 is -inf: a row's first keys always set it
                    f = old == -INFINITY ? 0.0f : ex2(old - m);
                    sm.mref[tid] = m;
                    sm.rescale[n & 1] = 1;
                }
                sm.fac[tid] = f;
            }
            if (tid == 0) sm.rescale[(n + 1) & 1] = 0;
            softmax_bar();
            if (nvis) nscales += nrow;
            const float nts = nvis ? __ldg(nscales) : 0.0f;
            if (sm.rescale[n & 1]) {
                if (n > 0) {
                    wait(&sm.pv_done, (uint32_t)((n - 1) & 1));
                    tc_fence_after();
#pragma unroll 1
                    for (int col = 0; col < (int)kS0; col += 16) {
                        uint32_t o[16];
                        tmem_ld_32x32b_x16(tmem + lanes + col, o);
                        tmem_ld_wait();
                        const float* fc = &sm.fac[col % R];
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fc[i]);
                        tmem_st_x16(tmem + lanes + col, o);
                    }
                    tmem_st_wait();
                }
#pragma unroll
                for (int r = 0; r < R; ++r) l[r] *= sm.fac[r];
            }
            const float tp = ts * kPScale;
#pragma unroll
            for (int j = 0; j < R / 4; ++j) {
                const float4 m = *reinterpret_cast<const float4*>(&sm.mref[4 * j]);
                const float mm[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int r = 4 * j + i;
                    // a row that has seen nothing has z and m at -inf: its weight is 0
                    z[r] = z[r] == -INFINITY ? 0.0f : ex2(z[r] - mm[i]);
                    l[r] += z[r];
                }
            }
            if (n > 0) wait(&sm.pv_done, (uint32_t)((n - 1) & 1));   // P is free when the last tile's products are done
#pragma unroll
            for (int c = 0; c < NQ; ++c) {
                uint32_t w[3][4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t h0, m0, l0, h1, m1, l1;
                    split_e5m2(pack_f16(z[16 * c + 4 * j] * tp, z[16 * c + 4 * j + 1] * tp), h0, m0, l0);
                    split_e5m2(pack_f16(z[16 * c + 4 * j + 2] * tp, z[16 * c + 4 * j + 3] * tp), h1, m1, l1);
                    w[0][j] = __byte_perm(h0, h1, 0x7531);
                    w[1][j] = __byte_perm(m0, m1, 0x7531);
                    w[2][j] = __byte_perm(l0, l1, 0x7531);
                }
#pragma unroll
                for (int x = 0; x < 3; ++x)
                    *reinterpret_cast<uint4*>(&sm.P[x * NQ + c][tid][0]) = make_uint4(w[x][0], w[x][1], w[x][2], w[x][3]);
            }
            if (!vis && tid < ((keys + 31) & ~31)) {   // S of this tile is done: its rows are read only by P K from here
                uint8_t* krow = sm.K[n % ST] + (tid >> 3) * (kGroup * kD) + (tid & 7) * 128;
#pragma unroll
                for (int b = 0; b < 4; ++b)
#pragma unroll
                    for (int j = 0; j < 8; ++j) *reinterpret_cast<uint4*>(krow + b * 1024 + 16 * ((j + tid) & 7)) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            mbar_arrive(&sm.p_full);
            row = nrow;
            vis = nvis;
            ts = nts;
        }
        // ---- row sums over the 128 threads, then the output ----
        if (t1 > t0) wait(&sm.pv_done, (uint32_t)((t1 - t0 - 1) & 1));
        tc_fence_after();
        float* stage = reinterpret_cast<float*>(sm.K[0]);   // every copy and product is done: the tile is free
#pragma unroll
        for (int r = 0; r < R; ++r) stage[r * (kSoftmaxThreads + 1) + tid] = l[r];
        softmax_bar();
        if (tid < R) {
            float a[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
            for (int k = 0; k < kSoftmaxThreads; k += 4)
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] += stage[tid * (kSoftmaxThreads + 1) + k + i];
            sm.lsum[tid] = (a[0] + a[1]) + (a[2] + a[3]);
        }
        softmax_bar();
        if (tid < R) {
            const float sum = sm.lsum[tid], m = sm.mref[tid];
            const int c = tid >> 4;
            if (args.splits > 1) {
                float* ml = args.part_ml + (((int64_t)blockIdx.y * args.splits + blockIdx.x) * R + tid) * 2;
                ml[0] = m;
                ml[1] = sum;
            } else if (p.lse && c < nq) {
                p.lse[(int64_t)(f0 + c) * kH + (tid & 15)] = sum > 0.0f ? (m + log2f(sum)) * 0.6931471805599453f : -INFINITY;
            }
            sm.fac[tid] = (sum > 0.0f ? 1.0f / sum : 0.0f) * (1.0f / kPScale);
        }
        softmax_bar();
        uint16_t* ostage = reinterpret_cast<uint16_t*>(sm.K[0]);   // [R][512] bf16
        float* po = args.part_o + ((int64_t)blockIdx.y * args.splits + blockIdx.x) * R * kD;
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
            const int dim = 128 * b + tid;
#pragma unroll
            for (int c = 0; c < NQ; ++c) {
                float o[16];
                uint32_t v[16];
                tmem_ld_32x32b_x16(tmem + lanes + b * kOCols + 16 * c, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __uint_as_float(v[i]);
                if (kConcat) {
#pragma unroll
                    for (int x = 1; x < 3; ++x) {
                        tmem_ld_32x32b_x16(tmem + lanes + b * kOCols + x * R + 16 * c, v);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] += __uint_as_float(v[i]);
                    }
                }
                if (args.splits > 1) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) po[(int64_t)(16 * c + i) * kD + dim] = o[i] * (1.0f / kPScale);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const __nv_bfloat16 h = __float2bfloat16_rn(o[i] * sm.fac[16 * c + i]);
                        ostage[(16 * c + i) * kD + dim] = *reinterpret_cast<const uint16_t*>(&h);
                    }
                }
            }
        }
        if (args.splits == 1) {
            softmax_bar();
            const uint4* src = reinterpret_cast<const uint4*>(ostage);
            uint4* dst = reinterpret_cast<uint4*>(p.out + (int64_t)f0 * kH * kD);
            for (int j = tid; j < nq * kH * kD / 8; j += kSoftmaxThreads) dst[j] = src[j];
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 5) tmem_dealloc(tmem, kTmemCols);
}

// Joins the splits of a block: one CTA per row, weight 2^(m_s - M) / L with L = sum_s l_s 2^(m_s - M).
__global__ void __launch_bounds__(128) pages_merge_kernel(const __grid_constant__ KernelArgs args, int NQ) {
    pdl_enter();
    const PagesAttnParams& p = args.p;
    const int S = args.splits, R = kH * NQ, tid = threadIdx.x;
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
    float M = -INFINITY;
    for (int s = 0; s < S; ++s) M = fmaxf(M, __ldcg(args.part_ml + (r0 + (int64_t)s * R) * 2));
    const float Mu = M == -INFINITY ? 0.0f : M;
    float L = 0.0f;
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int s = 0; s < S; ++s) {
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(args.part_ml) + r0 + (int64_t)s * R);
        if (!(ml.y > 0.0f)) continue;
        const float w = exp2f(ml.x - Mu);
        const float4 v = __ldcg(reinterpret_cast<const float4*>(args.part_o + (r0 + (int64_t)s * R) * kD) + tid);
        L = fmaf(ml.y, w, L);
        o.x = fmaf(v.x, w, o.x);
        o.y = fmaf(v.y, w, o.y);
        o.z = fmaf(v.z, w, o.z);
        o.w = fmaf(v.w, w, o.w);
    }
    const float inv = L > 0.0f ? 1.0f / L : 0.0f;
    *reinterpret_cast<uint2*>(p.out + (int64_t)blockIdx.x * kD + 4 * tid) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
    if (p.lse && tid == 0) p.lse[blockIdx.x] = L > 0.0f ? (Mu + log2f(L)) * 0.6931471805599453f : -INFINITY;
}

// ---- host ----------------------------------------------------------------------------------

struct Plan {
    int nq, blocks, splits;
    size_t o_bytes, bytes;
};

Plan plan(bool prefix, int B, int Q, int64_t keys) {
    Plan pl{};
    const int64_t n = (int64_t)B * Q;
    const int64_t together = prefix ? n : Q;
    pl.nq = together >= 3 ? 4 : (int)together;
    pl.blocks = (int)(prefix ? (n + pl.nq - 1) / pl.nq : (int64_t)B * ((Q + pl.nq - 1) / pl.nq));
    int64_t tiles = (keys + kTileKeys - 1) / kTileKeys + (prefix ? 1 : 0);
    if (tiles < 1) tiles = 1;
    const int64_t ctas = pl.nq == 1 ? 2 * kSplitSMs : kSplitSMs;
    int64_t s = ctas / pl.blocks;
    if (s > tiles) s = tiles;
    if (s < 1) s = 1;
    pl.splits = (int)s;
    pl.bytes = 256;
    if (s > 1) {
        const size_t rows = (size_t)pl.blocks * s * kH * pl.nq;
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

// The pool as [group of 8 rows][4 blocks of 128 channels][8 rows][128 B]: a box is one group, in the
// order in which the tile keeps it.
cudaError_t pool_map(const csa2_pages& pg, CUtensorMap* map) {
    const EncodeFn fn = encoder();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[4] = {128, kGroup, kD / 128, (cuuint64_t)(pg.n_pages * pg.page_size / kGroup)};
    const cuuint64_t strides[3] = {kD, 128, (cuuint64_t)kGroup * kD};
    const cuuint32_t box[4] = {128, kGroup, kD / 128, 1}, es[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, pg.kv, dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

template <int NQ, int ST>
cudaError_t launch(const KernelArgs& a, int blocks, const CUtensorMap& own, const CUtensorMap& prefix, cudaStream_t st) {
    static DeviceOnce attr;
    const int smem = (int)sizeof(Smem<NQ, ST>) + 1024;
    cudaError_t e = attr.run([&] {
        return cudaFuncSetAttribute(pages_attn_kernel<NQ, ST>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    });
    if (e != cudaSuccess) return e;
    return launch_ex(pages_attn_kernel<NQ, ST>, dim3(a.splits, blocks), dim3(kThreads), smem, st, 0, own, prefix, a);
}

}  // namespace

size_t pages_attn_ws_bytes(bool prefix, int B, int Q, int64_t keys) { return plan(prefix, B, Q, keys).bytes; }

cudaError_t launch_pages_attn(const PagesAttnParams& p, int64_t keys, void* ws, cudaStream_t st) {
    const Plan pl = plan(p.prefix.B != 0, p.B, p.Q, keys);
    KernelArgs a{};
    a.p = p;
    a.splits = pl.splits;
    a.test_starve = test_starve_copies();
    a.part_o = (float*)ws;
    a.part_ml = (float*)((char*)ws + pl.o_bytes);
    CUtensorMap own, prefix;
    cudaError_t e = pool_map(p.own, &own);
    if (e != cudaSuccess) return e;
    if (p.prefix.B) {
        e = pool_map(p.prefix, &prefix);
        if (e != cudaSuccess) return e;
    } else {
        prefix = own;
    }
    e = pl.nq == 1   ? launch<1, 1>(a, pl.blocks, own, prefix, st)
        : pl.nq == 2 ? launch<2, 2>(a, pl.blocks, own, prefix, st)
                     : launch<4, 2>(a, pl.blocks, own, prefix, st);
    if (e != cudaSuccess || pl.splits == 1) return e;
    return launch_ex(pages_merge_kernel, dim3((unsigned)(p.B * p.Q * kH)), dim3(128), 0, st, 0, a, pl.nq);
}

}  // namespace csa2
