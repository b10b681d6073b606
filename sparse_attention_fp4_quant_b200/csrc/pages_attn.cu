// pages_attn.cu -- attention over the paged FP8 cache: the sliding-window form with first
// tokens that stay visible, and the form for a batch behind a shared prefix.
//
// A CTA takes one query (its 16 heads are the M dimension of warp-level MMAs) and streams
// the keys it sees in tiles of 64, with an online softmax; the keys' E4M3 values are exact
// in f16 and the token scale multiplies the logit and the probability.
#include "attn_common.cuh"

namespace csa2 {

namespace {

constexpr int kPT = 256;      // threads per CTA
constexpr int kPK = 64;       // keys per tile

struct PagesSmem {
    uint8_t K[kPK * kRowB];
    uint8_t Qs[kH * kRowB];
    uint8_t P[kH * kPK * 2];
    float kf[kPK];
    int kvalid[kPK];
    float red_max[8][kH];
    float red_sum[8][kH];
    float m_run[kH], l_run[kH], alpha[kH];
    float qmax[kH][2];   // each head's largest |q|, by halves
};

// Tokens [lo, hi) of a table's row.
struct Seg {
    const csa2_pages* pg;
    int64_t b, lo, hi;
};

__device__ __forceinline__ int64_t stored_end(const csa2_pages& pg, int64_t b) {
    const int64_t cap = (int64_t)pg.max_pages * pg.page_size;
    int64_t n = pg.n_tokens[b];
    n = n < 0 ? 0 : n > cap ? cap : n;
    return pg.pos0 + n;
}

__device__ __forceinline__ int64_t token_row(const csa2_pages& pg, int64_t b, int64_t pos) {
    const int64_t t = pos - pg.pos0;
    const int page = pg.table[b * pg.max_pages + t / pg.page_size];
    return page >= 0 && page < pg.n_pages ? (int64_t)page * pg.page_size + t % pg.page_size : -1;
}

__global__ void __launch_bounds__(kPT) pages_attn_kernel(PagesAttnParams p) {
    pdl_enter();
    extern __shared__ __align__(128) uint8_t smem_raw[];
    PagesSmem& sm = *reinterpret_cast<PagesSmem*>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, qd = lane & 3;
    const int bq = blockIdx.x, b = bq / p.Q;
    const int64_t i = p.q_pos[bq];
    const float scale_log2 = p.sm_scale * 1.4426950408889634f;

    Seg seg[3];
    {
        const int64_t end = min(stored_end(p.own, b), i + 1);
        int64_t lo = i - p.window + 1;
        if (p.replay_start) lo = max(lo, (int64_t)p.replay_start[b]);
        lo = min(max(lo, (int64_t)p.own.pos0), max(end, (int64_t)p.own.pos0));
        seg[1] = {&p.own, b, p.own.pos0, min(min((int64_t)p.n_sink, lo), end)};
        seg[2] = {&p.own, b, lo, end};
        seg[0] = p.prefix.B ? Seg{&p.prefix, 0, p.prefix.pos0, min(stored_end(p.prefix, 0), i + 1)} : Seg{&p.own, b, 0, 0};
    }
    int64_t n[3], total = 0;
    for (int s = 0; s < 3; ++s) total += n[s] = max(seg[s].hi - seg[s].lo, (int64_t)0);

    const uint32_t sK = (uint32_t)__cvta_generic_to_shared(sm.K);
    const uint32_t sQ = (uint32_t)__cvta_generic_to_shared(sm.Qs);
    const uint32_t sP = (uint32_t)__cvta_generic_to_shared(sm.P);
    {
        const uint4* qsrc = reinterpret_cast<const uint4*>(p.q + (int64_t)bq * kH * kD);
        uint4 qv[(kH * kD / 8) / kPT];
#pragma unroll
        for (int it = 0; it < (kH * kD / 8) / kPT; ++it) {   // chunk it * 256 + tid: two warps for each head
            qv[it] = __ldg(qsrc + it * kPT + tid);
            float qm = bf16x8_maxabs(qv[it]);
#pragma unroll
            for (int o2 = 16; o2 > 0; o2 >>= 1) qm = fmaxf(qm, __shfl_xor_sync(0xFFFFFFFFu, qm, o2));
            if (lane == 0) sm.qmax[4 * it + (warp >> 1)][warp & 1] = qm;
        }
        __syncthreads();
#pragma unroll
        for (int it = 0; it < (kH * kD / 8) / kPT; ++it) {
            const int c = it * kPT + tid, h = c >> 6;
            const int qe = q_prescale_exp(fmaxf(sm.qmax[h][0], sm.qmax[h][1]));
            *reinterpret_cast<uint4*>(sm.Qs + swz(h, c & 63)) =
                bf16x8_to_f16(qv[it], __uint_as_float((uint32_t)(127 - qe) << 23));
        }
    }
    const int qe0 = q_prescale_exp(fmaxf(sm.qmax[g][0], sm.qmax[g][1]));
    const int qe1 = q_prescale_exp(fmaxf(sm.qmax[g + 8][0], sm.qmax[g + 8][1]));
    const float sc0 = scale_log2 * __uint_as_float((uint32_t)(127 + qe0) << 23);
    const float sc1 = scale_log2 * __uint_as_float((uint32_t)(127 + qe1) << 23);
    if (tid < kH) {
        sm.m_run[tid] = -INFINITY;
        sm.l_run[tid] = 0.0f;
    }
    float o[8][4];
#pragma unroll
    for (int c = 0; c < 8; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[c][j] = 0.0f;

    const int gr = tid & (kPK - 1), gq = tid >> 6;
    for (int64_t s0 = 0; s0 < total; s0 += kPK) {
        {
            RowQuarter rq;
            rq.kind = 0;
            int64_t k = s0 + gr, row = -1;
            const csa2_pages* pg = &p.own;
            for (int s = 0; s < 3; ++s) {
                if (k >= 0 && k < n[s]) {
                    pg = seg[s].pg;
                    row = token_row(*pg, seg[s].b, seg[s].lo + k);
                }
                k -= n[s];
            }
            if (row >= 0) {
                rq.kind = 2;
                rq.fac = pg->kv_sc[row];
                const uint4* cs = reinterpret_cast<const uint4*>(pg->kv + row * kD + 128 * gq);
#pragma unroll
                for (int v = 0; v < 8; ++v) rq.raw[v] = cs[v];
            }
            store_quarter(sm.K, sm.kf, sm.kvalid, gr, gq, rq);
        }
        __syncthreads();
        float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int ks = 0; ks < kD / 16; ++ks) {
            uint32_t a0, a1, a2, a3, b0, b1;
            ldsm_x4(sQ + swz(lane & 15, 2 * ks + (lane >> 4)), a0, a1, a2, a3);
            ldsm_x2(sK + swz(8 * warp + (lane & 7), 2 * ks + ((lane >> 3) & 1)), b0, b1);
            mma_f16(s4, a0, a1, a2, a3, b0, b1);
        }
        const int key0 = 8 * warp + 2 * qd;
        const float f0 = sm.kf[key0], f1 = sm.kf[key0 + 1];
        const bool v0 = sm.kvalid[key0] != 0, v1 = sm.kvalid[key0 + 1] != 0;
        const float z[4] = {v0 ? s4[0] * f0 * sc0 : -INFINITY, v1 ? s4[1] * f1 * sc0 : -INFINITY,
                            v0 ? s4[2] * f0 * sc1 : -INFINITY, v1 ? s4[3] * f1 * sc1 : -INFINITY};
        float mx0 = fmaxf(z[0], z[1]), mx1 = fmaxf(z[2], z[3]);
#pragma unroll
        for (int o2 = 1; o2 < 4; o2 <<= 1) {
            mx0 = fmaxf(mx0, __shfl_xor_sync(0xFFFFFFFFu, mx0, o2));
            mx1 = fmaxf(mx1, __shfl_xor_sync(0xFFFFFFFFu, mx1, o2));
        }
        if (qd == 0) {
            sm.red_max[warp][g] = mx0;
            sm.red_max[warp][g + 8] = mx1;
        }
        __syncthreads();
        float mn0 = sm.m_run[g], mn1 = sm.m_run[g + 8];
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            mn0 = fmaxf(mn0, sm.red_max[w][g]);
            mn1 = fmaxf(mn1, sm.red_max[w][g + 8]);
        }
        const float mu0 = (mn0 == -INFINITY) ? 0.0f : mn0, mu1 = (mn1 == -INFINITY) ? 0.0f : mn1;
        const float p00 = exp2f(z[0] - mu0), p01 = exp2f(z[1] - mu0), p10 = exp2f(z[2] - mu1), p11 = exp2f(z[3] - mu1);
        {
            const int chunk = key0 >> 3, within = (key0 & 7) * 2;
            *reinterpret_cast<__half2*>(sm.P + g * 128 + ((chunk ^ (g & 7)) << 4) + within) =
                __floats2half2_rn(p00 * f0, p01 * f1);
            *reinterpret_cast<__half2*>(sm.P + (g + 8) * 128 + ((chunk ^ (g & 7)) << 4) + within) =
                __floats2half2_rn(p10 * f0, p11 * f1);
        }
        float sum0 = p00 + p01, sum1 = p10 + p11;
#pragma unroll
        for (int o2 = 1; o2 < 4; o2 <<= 1) {
            sum0 += __shfl_xor_sync(0xFFFFFFFFu, sum0, o2);
            sum1 += __shfl_xor_sync(0xFFFFFFFFu, sum1, o2);
        }
        if (qd == 0) {
            sm.red_sum[warp][g] = sum0;
            sm.red_sum[warp][g + 8] = sum1;
        }
        __syncthreads();
        if (tid < kH) {
            float mn = sm.m_run[tid], ssum = 0.0f;
            for (int w = 0; w < 8; ++w) {
                mn = fmaxf(mn, sm.red_max[w][tid]);
                ssum += sm.red_sum[w][tid];
            }
            const float al = (sm.m_run[tid] == -INFINITY) ? 0.0f : exp2f(sm.m_run[tid] - mn);
            sm.alpha[tid] = al;
            sm.l_run[tid] = sm.l_run[tid] * al + ssum;
            sm.m_run[tid] = mn;
        }
        __syncthreads();
        const float al0 = sm.alpha[g], al1 = sm.alpha[g + 8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
            o[c][0] *= al0;
            o[c][1] *= al0;
            o[c][2] *= al1;
            o[c][3] *= al1;
        }
#pragma unroll
        for (int kk = 0; kk < kPK / 16; ++kk) {
            uint32_t a0, a1, a2, a3;
            const int row = lane & 15, chunk = 2 * kk + (lane >> 4);
            ldsm_x4(sP + (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4)), a0, a1, a2, a3);
            const int mi = lane >> 3, key = 16 * kk + (mi & 1) * 8 + (lane & 7);
#pragma unroll
            for (int np = 0; np < 4; ++np) {
                uint32_t b0, b1, b2, b3;
                ldsm_x4_t(sK + swz(key, 8 * warp + 2 * np + (mi >> 1)), b0, b1, b2, b3);
                mma_f16(o[2 * np], a0, a1, a2, a3, b0, b1);
                mma_f16(o[2 * np + 1], a0, a1, a2, a3, b2, b3);
            }
        }
        __syncthreads();
    }
    const float l0 = sm.l_run[g], l1 = sm.l_run[g + 8];
    const float inv0 = l0 > 0.0f ? 1.0f / l0 : 0.0f, inv1 = l1 > 0.0f ? 1.0f / l1 : 0.0f;
    uint16_t* out = p.out + (int64_t)bq * kH * kD;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const int d = 64 * warp + 8 * c + 2 * qd;
        *reinterpret_cast<uint32_t*>(out + g * kD + d) = pack_bf16(o[c][0] * inv0, o[c][1] * inv0);
        *reinterpret_cast<uint32_t*>(out + (g + 8) * kD + d) = pack_bf16(o[c][2] * inv1, o[c][3] * inv1);
    }
    if (p.lse && tid < kH) {
        const float l = sm.l_run[tid];
        p.lse[(int64_t)bq * kH + tid] = l > 0.0f ? (sm.m_run[tid] + log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
}

}  // namespace

size_t pages_attn_ws_bytes(bool prefix, int B, int Q, int64_t keys) { return 256; }

cudaError_t launch_pages_attn(const PagesAttnParams& p, int64_t keys, void* ws, cudaStream_t st) {
    static DeviceOnce attr;
    const int smem = (int)sizeof(PagesSmem);
    cudaError_t e = attr.run([&] { return cudaFuncSetAttribute(pages_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
    if (e != cudaSuccess) return e;
    return launch_ex(pages_attn_kernel, dim3(p.B * p.Q), dim3(kPT), smem, st, 0, p);
}

}  // namespace csa2
