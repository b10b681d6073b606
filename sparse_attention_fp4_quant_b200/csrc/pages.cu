// pages.cu -- append of new latent rows to the paged FP8 cache: RMSNorm, RoPE by
// position, and the E4M3 row with its token scale, in one pass over the row.
//
// A warp takes a row at a time and fetches the next one meanwhile.  Lane l holds channels
// 8 l .. 8 l + 7, for l < 24 also 256 + 8 l .., and the pair 448 + 2 l, 449 + 2 l: one rotated
// pair in every lane, each with its own angle.  The time goes with the instructions (430 a row
// in its first form, 20.8 us for 32,768 rows; now 262 and 12.4 us, 4.1 TB/s in and out with the issue
// slots 66 % busy), and of the splits tried this takes the fewest.  The angle
// pos * inv_freq is formed in fp64 and reduced to a fraction of a turn before the fp32 sine: at
// position 10^6 an fp32 product would be off by up to 0.03 radian.
// The norm's factor 1 / rms is common to a row, so the codes do not depend on it: it is applied
// to the scale alone.  With a = amax |x w| (rotated), code = E4M3(x w * (448 / a)) and
// scale = a / 448 / rms; the quotient is within 2^-22 of the definition's, so a code differs
// only where that lies this close to a rounding border.  Sums and the maximum stay in fp32.
#include "common.cuh"
#include "kernels.h"

namespace csa2 {

namespace {

constexpr int kPW = 4;      // warps of a CTA, a row each at a time
constexpr int kPCtas = 7;   // CTAs on an SM

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rcp(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// Four floats -> four E4M3 bytes (nearest, ties to even, saturating).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

// A row on its way in: its bytes and where it goes.
struct Row {
    uint4 raw[2];
    uint32_t pair;
    int seq, pos;
};

__global__ void __launch_bounds__(32 * kPW, kPCtas) pages_append_kernel(const uint16_t* x, int64_t x_stride, int64_t rows,
                                                                        const int32_t* seq, const int32_t* pos,
                                                                        const float* inv_freq, const float* norm_w, float eps,
                                                                        bool normalise, int page_shift, csa2_pages pg) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t)gridDim.x * kPW;
    int64_t r = (int64_t)blockIdx.x * kPW + (threadIdx.x >> 5);
    if (r >= rows) return;
    auto fetch = [&](int64_t i, Row& d) {
        const uint4* src = reinterpret_cast<const uint4*>(x + i * x_stride);
        d.raw[0] = __ldg(src + lane);
        d.raw[1] = lane < 24 ? __ldg(src + 32 + lane) : make_uint4(0, 0, 0, 0);
        d.pair = __ldg(reinterpret_cast<const uint32_t*>(src) + 224 + lane);
        d.seq = __ldg(seq + i);
        d.pos = __ldg(pos + i);
    };
    // Slot of a row in its sequence, or -1; then the page that the table gives.
    const uint32_t slots = (uint32_t)pg.max_pages * (uint32_t)pg.page_size;   // below 2^31
    auto slot_of = [&](const Row& d) -> int {
        const uint32_t t = (uint32_t)d.pos - (uint32_t)pg.pos0;
        return d.seq >= 0 && d.seq < pg.B && d.pos >= pg.pos0 && t < slots ? (int)t : -1;
    };
    auto split = [&](int slot, int& i, int& at) {   // page of a sequence and place in it
        if (page_shift >= 0) {
            i = slot >> page_shift;
            at = slot & (pg.page_size - 1);
        } else {
            i = slot / pg.page_size;
            at = slot - i * pg.page_size;
        }
    };
    auto page_of = [&](const Row& d, int slot) {
        int i, at;
        split(slot, i, at);
        return slot >= 0 ? __ldg(pg.table + (int64_t)d.seq * pg.max_pages + i) : -1;
    };
    Row cur, next;
    fetch(r, cur);
    float w[18];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool have = norm_w && (j < 2 || lane < 24);
        const float4 v = have ? __ldg(reinterpret_cast<const float4*>(norm_w) + 64 * (j >> 1) + 2 * lane + (j & 1))
                              : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
        w[4 * j] = v.x, w[4 * j + 1] = v.y, w[4 * j + 2] = v.z, w[4 * j + 3] = v.w;
    }
    w[16] = norm_w ? __ldg(norm_w + 448 + 2 * lane) : 1.0f;
    w[17] = norm_w ? __ldg(norm_w + 449 + 2 * lane) : 1.0f;
    const double freq = inv_freq ? (double)__ldg(inv_freq + lane) * 0.15915494309189533577 : 0.0;   // turns per position
    int slot = slot_of(cur);
    int page = page_of(cur, slot);
    for (;;) {
        const bool more = r + step < rows;
        if (more) fetch(r + step, next);
        int64_t row = -1;
        if (page >= 0 && page < pg.n_pages) {
            int i, at;
            split(slot, i, at);
            row = (int64_t)page * pg.page_size + at;
        }
        if (row >= 0) {
            float v[18];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t u[4] = {cur.raw[j].x, cur.raw[j].y, cur.raw[j].z, cur.raw[j].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    v[8 * j + 2 * i] = __uint_as_float(u[i] << 16);
                    v[8 * j + 2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
                }
            }
            v[16] = __uint_as_float(cur.pair << 16);
            v[17] = __uint_as_float(cur.pair & 0xFFFF0000u);
            float rn = 1.0f;
            if (normalise) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < 18; ++i) ss = fmaf(v[i], v[i], ss);
                rn = rsqrtf(warp_sum(ss) * (1.0f / kD) + eps);
            }
#pragma unroll
            for (int i = 0; i < 18; ++i) v[i] *= w[i];
            if (inv_freq) {
                const double turns = (double)cur.pos * freq;
                float sn, cs;   // of at most half a turn: the fast functions are within 2^-20 there
                __sincosf((float)((turns - rint(turns)) * 6.283185307179586477), &sn, &cs);
                const float a = v[16], b = v[17];
                v[16] = a * cs - b * sn;
                v[17] = a * sn + b * cs;
            }
            float mx = 0.0f;
#pragma unroll
            for (int i = 0; i < 18; ++i) mx = fmaxf(mx, fabsf(v[i]));
            mx = warp_max(mx);
            float down = 1.0f;
            if (mx < 1e-30f) {   // 448 / mx would overflow: work on 2^80 times the row
                mx *= 1.2089258196146292e24f;
                down = 8.271806125530277e-25f;
#pragma unroll
                for (int i = 0; i < 18; ++i) v[i] *= 1.2089258196146292e24f;
            }
            const float a448 = mx * (1.0f / 448.0f);   // in [2^-108, 2^120]: its approximate reciprocal is within 1 ulp
            const float inv = mx > 0.0f ? rcp(a448) : 0.0f;
            uint8_t* dst = pg.kv + row * kD;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float y[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = v[8 * j + i] * inv;
                if (j == 0 || lane < 24)
                    *reinterpret_cast<uint2*>(dst + 256 * j + 8 * lane) =
                        make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
            }
            *reinterpret_cast<uint16_t*>(dst + 448 + 2 * lane) = (uint16_t)e4m3x4(v[16] * inv, v[17] * inv, 0.0f, 0.0f);
            if (lane == 0) pg.kv_sc[row] = mx > 0.0f ? a448 * rn * down : 0.0f;   // without an epsilon a zero row's rn is infinite
        }
        if (!more) break;
        r += step;
        cur = next;
        slot = slot_of(cur);
        page = page_of(cur, slot);
    }
}

}  // namespace

cudaError_t launch_pages_append(const void* x, int64_t x_stride, int64_t rows, const int32_t* seq, const int32_t* pos,
                                const float* inv_freq, const float* norm_w, float eps, bool normalise,
                                const csa2_pages& pages, cudaStream_t st) {
    const int64_t all = (rows + kPW - 1) / kPW, most = (int64_t)device_sm_count() * kPCtas;
    int page_shift = 0;
    while ((1 << page_shift) < pages.page_size) ++page_shift;
    if ((1 << page_shift) != pages.page_size) page_shift = -1;
    const dim3 grid((unsigned)(most > 0 && all > most ? most : all));
    return launch_ex(pages_append_kernel, grid, dim3(32 * kPW), 0, st, 0, (const uint16_t*)x, x_stride, rows, seq, pos,
                     inv_freq, norm_w, eps, normalise, page_shift, pages);
}

}  // namespace csa2
