// gattn.cuh -- K12: group attention over the paged FP4 cache. Every query
// token of group g attends to the first kv_lens[g] entries of the group's
// pages (keys = values), and the result is joined with the token's own part.
//
// One CTA per query token: blocks of 32 keys are dequantised to shared memory
// once for the 16 heads, the scores go through a softmax with a running
// maximum and sum per head, and each thread keeps 36 outputs in registers.
#pragma once

#include "attn.cuh"
#include "common.cuh"

namespace csa2 {

constexpr int kGaMaxTokens = 1 << 20, kGaMaxGroups = 65535;
constexpr int kGaThreads = 256;
constexpr int kGaKeys = 32;
constexpr int kGaPer = kHeads * kDim / kGaThreads;                // 36 outputs per thread

struct GaArgs {
    const __nv_bfloat16 *q;            // [N][16][576]
    const uint8_t *kv_fp4, *kv_scale;
    int64_t num_pages;
    const int32_t *page_table;         // [G][max_pages]
    int max_pages;
    const int32_t *kv_lens;            // [G]
    const int32_t *q_offsets;          // [G + 1]
    int N, G;
    float scale_log2;
    const float *o_own, *lse_own;      // [N][16][576], [N][16], or null
    __nv_bfloat16 *out;                // [N][16][576]
    float *lse;                        // [N][16]
};

struct GaSmem {
    float q[kHeads][kDim + 1];
    float k[kGaKeys][kDim + 1];
    float s[kHeads][kGaKeys + 1];
    float m[kHeads], l[kHeads], f[kHeads];
};

__global__ void __launch_bounds__(kGaThreads)
group_attn_kernel(const GaArgs A) {
    extern __shared__ uint8_t ga_raw[];
    GaSmem &sm = *reinterpret_cast<GaSmem *>(ga_raw);
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, tok = blockIdx.x;
    int g = -1;
    for (int i = 0; i < A.G; ++i) {
        const int a = A.q_offsets[i], b = A.q_offsets[i + 1];
        if (a < 0 || b > A.N || b < a) {
            if (tid == 0) flag_status(kStatusBounds);
            continue;
        }
        if (tok >= a && tok < b) g = i;
    }
    if (g < 0) return;
    int T = A.kv_lens[g];
    if (T < 0 || T > A.max_pages * kPage) {
        if (tid == 0) flag_status(kStatusBounds);
        T = 0;
    }
    for (int i = tid; i < kHeads * kDim; i += kGaThreads)
        sm.q[i / kDim][i % kDim] = __bfloat162float(A.q[static_cast<int64_t>(tok) * kHeads * kDim + i]);
    if (tid < kHeads) {
        sm.m[tid] = -INFINITY;
        sm.l[tid] = 0.0f;
    }
    float acc[kGaPer];
#pragma unroll
    for (int i = 0; i < kGaPer; ++i) acc[i] = 0.0f;
    for (int t0 = 0; t0 < T; t0 += kGaKeys) {
        const int page = A.page_table[static_cast<int64_t>(g) * A.max_pages + t0 / kPage];
        const bool page_ok = page >= 0 && page < A.num_pages;
        if (!page_ok && tid == 0) flag_status(kStatusBounds);
        const int n = page_ok ? min(kGaKeys, T - t0) : 0;
        __syncthreads();
        for (int i = tid; i < kGaKeys * (kDim / 2); i += kGaThreads) {
            const int r = i / (kDim / 2), c = i % (kDim / 2);
            float2 v = make_float2(0.0f, 0.0f);
            if (r < n) {
                const int64_t slot = static_cast<int64_t>(page) * kPage + (t0 + r) % kPage;
                const uint32_t h = hmul2_u32(e2m1x2_to_f16x2(A.kv_fp4[slot * kFp4Bytes + c]),
                                             e4m3x2_to_f16x2(A.kv_scale[slot * kScaleBytes + c / 8] * 0x101u));
                v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            }
            sm.k[r][2 * c] = v.x;
            sm.k[r][2 * c + 1] = v.y;
        }
        __syncthreads();
        for (int i = tid; i < kHeads * kGaKeys; i += kGaThreads) {
            const int h = i / kGaKeys, r = i % kGaKeys;
            float d = 0.0f;
            for (int c = 0; c < kDim; ++c) d = fmaf(sm.q[h][c], sm.k[r][c], d);
            sm.s[h][r] = r < n ? d * A.scale_log2 : -INFINITY;
        }
        __syncthreads();
        if (tid < kHeads) {
            float m = sm.m[tid];
            for (int r = 0; r < kGaKeys; ++r) m = fmaxf(m, sm.s[tid][r]);
            const float ref = m == -INFINITY ? 0.0f : m;
            const float f = exp2f(sm.m[tid] - ref);
            float l = 0.0f;
            for (int r = 0; r < kGaKeys; ++r) {
                const float p = exp2f(sm.s[tid][r] - ref);
                sm.s[tid][r] = p;
                l += p;
            }
            sm.m[tid] = m;
            sm.l[tid] = sm.l[tid] * f + l;
            sm.f[tid] = f;
        }
        __syncthreads();
#pragma unroll 1
        for (int i = 0; i < kGaPer; ++i) {
            const int e = i * kGaThreads + tid, h = e / kDim, c = e % kDim;
            float a = 0.0f;
            for (int r = 0; r < kGaKeys; ++r) a = fmaf(sm.s[h][r], sm.k[r][c], a);
            acc[i] = acc[i] * sm.f[h] + a;
        }
    }
    __syncthreads();
    for (int i = 0; i < kGaPer; ++i) {
        const int e = i * kGaThreads + tid, h = e / kDim;
        const int64_t at = static_cast<int64_t>(tok) * kHeads * kDim + e;
        const float lo = A.lse_own ? A.lse_own[tok * kHeads + h] * 1.4426950408889634f : -INFINITY;
        const float m = fmaxf(sm.m[h], lo), ref = m == -INFINITY ? 0.0f : m;
        const float wk = exp2f(sm.m[h] - ref), wo = exp2f(lo - ref), l = sm.l[h] * wk + wo;
        const float o = acc[i] * wk + (wo > 0.0f ? wo * A.o_own[at] : 0.0f);
        A.out[at] = __float2bfloat16_rn(l == 0.0f ? 0.0f : o / l);   // a NaN stays one
        if (e % kDim == 0) A.lse[tok * kHeads + h] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
    }
}

}  // namespace csa2
