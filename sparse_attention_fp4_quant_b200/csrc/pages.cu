// pages.cu -- append of new latent rows to the paged FP8 cache: RMSNorm, RoPE by
// position, and the E4M3 row with its token scale, in one pass over the row.
//
// A warp takes a row.  Lane l holds channels 8 l .. 8 l + 7 and 256 + 8 l .. (two 16-byte
// loads, two 8-byte code stores), so the rotated channels 448 .. 511 lie in lanes 24 .. 31;
// lane k computes the angle of pair k (one each), and the eight lanes fetch the four pairs
// they rotate by shuffles.  The angle pos * inv_freq is formed in fp64 and reduced to a
// fraction of a turn before the fp32 sine: at position 10^6 an fp32 product would be off by
// up to 0.03 radian.  Sums and the maximum stay in fp32 registers; the only rounding to
// fewer bits is the code itself.  The quotient n / scale is taken as n * (1 / scale),
// within 2^-23 of it: a code differs only where the quotient lies that close to a border.
#include "common.cuh"
#include "kernels.h"

namespace csa2 {

namespace {

constexpr int kPW = 4;   // rows (warps) per CTA

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}

// Four floats -> four E4M3 bytes (nearest, ties to even, saturating).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return (uint32_t)lo | ((uint32_t)hi << 16);
}

__global__ void __launch_bounds__(32 * kPW) pages_append_kernel(const uint16_t* x, int64_t x_stride, int64_t rows,
                                                                const int32_t* seq, const int32_t* pos,
                                                                const float* inv_freq, const float* norm_w, float eps,
                                                                bool normalise, csa2_pages pg) {
    pdl_enter();
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kPW + (threadIdx.x >> 5);
    if (r >= rows) return;
    const uint4* src = reinterpret_cast<const uint4*>(x + r * x_stride);
    const uint4 raw[2] = {__ldg(src + lane), __ldg(src + 32 + lane)};
    const int s = seq[r], p = pos[r];
    if (s < 0 || s >= pg.B) return;
    const int64_t t = (int64_t)p - pg.pos0;
    if (t < 0 || t >= (int64_t)pg.max_pages * pg.page_size) return;
    const int page = pg.table[(int64_t)s * pg.max_pages + t / pg.page_size];
    if (page < 0 || page >= pg.n_pages) return;
    const int64_t row = (int64_t)page * pg.page_size + t % pg.page_size;

    float v[16];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[8 * j + 2 * i] = __uint_as_float(w[i] << 16);
            v[8 * j + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
    }
    if (normalise) {
        float ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) ss = fmaf(v[i], v[i], ss);
        const float rn = 1.0f / sqrtf(warp_sum(ss) * (1.0f / kD) + eps);
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] *= rn;
    }
    if (norm_w) {
        const float4* nw = reinterpret_cast<const float4*>(norm_w);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 w = __ldg(nw + 64 * j + 2 * lane + i);
                v[8 * j + 4 * i] *= w.x;
                v[8 * j + 4 * i + 1] *= w.y;
                v[8 * j + 4 * i + 2] *= w.z;
                v[8 * j + 4 * i + 3] *= w.w;
            }
    }
    if (inv_freq) {
        const double turns = (double)p * (double)__ldg(inv_freq + lane) * 0.15915494309189533577;   // 1 / (2 pi)
        float sn, cs;
        sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cs);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int k = (4 * (lane - 24) + i) & 31;
            const float c = __shfl_sync(0xFFFFFFFFu, cs, k), sv = __shfl_sync(0xFFFFFFFFu, sn, k);
            if (lane >= 24) {
                const float a = v[8 + 2 * i], b = v[9 + 2 * i];
                v[8 + 2 * i] = a * c - b * sv;
                v[9 + 2 * i] = a * sv + b * c;
            }
        }
    }
    float mx = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) mx = fmaxf(mx, fabsf(v[i]));
    const float scale = warp_max(mx) / 448.0f;
    const bool tiny = scale < 1.17549435e-38f;   // 1 / scale may overflow: divide instead (0 stays 0)
    const float inv = tiny ? 0.0f : 1.0f / scale;
    uint8_t* dst = pg.kv + row * kD;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = tiny ? (scale > 0.0f ? v[8 * j + i] / scale : 0.0f) : v[8 * j + i] * inv;
        *reinterpret_cast<uint2*>(dst + 256 * j + 8 * lane) =
            make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
    }
    if (lane == 0) pg.kv_sc[row] = scale;
}

}  // namespace

cudaError_t launch_pages_append(const void* x, int64_t x_stride, int64_t rows, const int32_t* seq, const int32_t* pos,
                                const float* inv_freq, const float* norm_w, float eps, bool normalise,
                                const csa2_pages& pages, cudaStream_t st) {
    const dim3 grid((unsigned)((rows + kPW - 1) / kPW));
    return launch_ex(pages_append_kernel, grid, dim3(32 * kPW), 0, st, 0, (const uint16_t*)x, x_stride, rows, seq, pos,
                     inv_freq, norm_w, eps, normalise, pages);
}

}  // namespace csa2
