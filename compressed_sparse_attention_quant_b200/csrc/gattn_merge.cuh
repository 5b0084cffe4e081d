// gattn_merge.cuh -- K13: joins what K12 or K12b left in pieces.
#pragma once

#include "gattn_few.cuh"

namespace csa2 {

// ------------------------------------------------------------------ K13
// Joins the partials of the row tiles that the ranges cut, with the own part:
// with M the largest m, out = (sum_p 2^(m_p - M) O_p + 2^(own - M) o_own) / L,
// L = sum_p 2^(m_p - M) l_p + 2^(own - M), lse = M + log L. Memory-bound in
// principle (36,864 B per partial and token, from L2: 47 MB for 64 tokens over
// 32,768 keys, about 12 us), latency-bound per unit of work. So a unit is a
// slice of a token's channels, 192, 64 or 16 of them, the smaller the fewer
// tokens there are to fill the GPU, and the first partials are loaded together
// with the maxima and sums. A thread takes 4 channels of a head; with 16
// channels the four groups of 64 threads take every fourth partial each. The
// order of the additions is fixed: a call gives the same bits again.
constexpr int kGmThreads = 256;
constexpr int kGmCtasPerSm = 4;
constexpr int kGmSlices = kDim / 16;                               // 36, the most that a token is cut into
constexpr int kGmBatch = 8;                                        // partials loaded together

struct GmSmem {
    GaPlan::Tile first[kGaMaxCtas];
    alignas(16) float2 ml[kGaMaxCtas + 1][kHeads];                 // (m, l) of a partial, then (its weight, -)
    float red[2][kGmThreads / kHeads][kHeads];
    float4 sum[4][64];
    float2 fac[kHeads];                                            // of the joined sum: the entries', the own part's
    int before[kGaMaxCtas + 1];                                    // tokens up to a boundary
    int warp_sum[kGmThreads / 32];
};

// kPer x 64 channels of a token from col0 on, or (kPer = 0) 16 channels.
template <int kPer>
__device__ __forceinline__ void gm_slice(const GaArgs &A, GmSmem &sm, int c0, int n, int slot0, int tok, int64_t row,
                                         int col0, bool write_lse) {
    constexpr int kGroups = kPer == 0 ? 4 : 1, kV = kPer == 0 ? 1 : kPer, kAtOnce = kPer == 3 ? 2 : kGmBatch;
    const int tid = threadIdx.x, h = tid & (kHeads - 1), at = tid >> 4;
    // the thread's head and 4 channels of the outputs: neighbours lie together in the partials
    const int grp = kPer == 0 ? tid >> 6 : 0, in = kPer == 0 ? tid & 63 : tid, quads = kPer == 0 ? 4 : 16;
    const int oh = A.few ? in / quads : in % kHeads, c4 = col0 / 4 + (A.few ? in % quads : in / kHeads);
    const int kstep = A.few ? 16 : 16 * kHeads;
    const float4 *po = reinterpret_cast<const float4 *>(A.part_o) + static_cast<int64_t>(tok) * (kDim * kHeads / 4) +
                       (A.few ? oh * (kDim / 4) + c4 : c4 * kHeads + oh);
    auto slot = [&](int p) { return static_cast<int64_t>(p == 0 ? slot0 : 2 * (c0 + p)) * A.tok_slots; };
    float4 v[kAtOnce][kV];
    auto load = [&](int b) {                                       // partials b, b + kGroups, ..
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int p = min(b + i * kGroups, n - 1);             // past the end: the last one again, weight 0
#pragma unroll
            for (int k = 0; k < kV; ++k) v[i][k] = __ldcg(po + slot(p) * (kDim * kHeads / 4) + k * kstep);
        }
    };
    constexpr int kLanes = kGmThreads / kHeads;
    for (int p = at; p < n; p += kLanes)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;"
                     ::"r"(smem_u32(&sm.ml[p][h])), "l"(&A.part_ml[(slot(p) + tok) * kHeads + h]) : "memory");
    cp_async_commit();
    load(grp);
    // ---- weights
    const float own = A.lse_own ? __ldg(A.lse_own + row + h) * 1.4426950408889634f : -INFINITY;
    float mx = own;
    cp_async_wait<0>();
    for (int p = at; p < n; p += kLanes) mx = fmaxf(mx, sm.ml[p][h].x);
    sm.red[0][at][h] = mx;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kLanes; ++i) mx = fmaxf(mx, sm.red[0][i][h]);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float l = 0.0f;
    for (int p = at; p < n; p += kLanes) {
        const float w = ga_ex2(sm.ml[p][h].x - ref);
        l += sm.ml[p][h].y * w;
        sm.ml[p][h].x = w;
    }
    sm.red[1][at][h] = l;
    __syncthreads();
    const float wo = ga_ex2(own - ref);
    l = wo;
#pragma unroll
    for (int i = 0; i < kLanes; ++i) l += sm.red[1][i][h];
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;                 // a NaN stays one
    if (at == 0) sm.fac[h] = make_float2(inv, wo > 0.0f ? wo * inv : 0.0f);   // nothing to read without an own part
    if (write_lse && at == 0) A.lse[row + h] = l == 0.0f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
    __syncthreads();
    // ---- the channels
    const float2 fac = sm.fac[oh];
    float4 a[kV];
#pragma unroll
    for (int k = 0; k < kV; ++k) a[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int b = grp; b < n; b += kAtOnce * kGroups) {
        if (b != grp) load(b);
#pragma unroll
        for (int i = 0; i < kAtOnce; ++i) {
            const int p = b + i * kGroups;
            const float w = p < n ? sm.ml[p][oh].x : 0.0f;
#pragma unroll
            for (int k = 0; k < kV; ++k) {
                a[k].x += w * v[i][k].x;
                a[k].y += w * v[i][k].y;
                a[k].z += w * v[i][k].z;
                a[k].w += w * v[i][k].w;
            }
        }
    }
    if constexpr (kPer == 0) {
        sm.sum[grp][tid & 63] = a[0];
        __syncthreads();
        if (grp == 0)
#pragma unroll
            for (int i = 1; i < 4; ++i) {
                const float4 o = sm.sum[i][tid];
                a[0].x += o.x;
                a[0].y += o.y;
                a[0].z += o.z;
                a[0].w += o.w;
            }
    }
    if (grp == 0)
#pragma unroll
        for (int k = 0; k < kV; ++k) {
            const int64_t to = (row + oh) * kDim + (c4 + 16 * k) * 4;
            const float inv = fac.x, fo = fac.y;
            float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            if (fo != 0.0f) o = __ldg(reinterpret_cast<const float4 *>(A.o_own + to));
            const __nv_bfloat162 x = __floats2bfloat162_rn(a[k].x * inv + fo * o.x, a[k].y * inv + fo * o.y);
            const __nv_bfloat162 y = __floats2bfloat162_rn(a[k].z * inv + fo * o.z, a[k].w * inv + fo * o.w);
            *reinterpret_cast<uint2 *>(A.out + to) =
                make_uint2(*reinterpret_cast<const uint32_t *>(&x), *reinterpret_cast<const uint32_t *>(&y));
        }
    __syncthreads();
}

__global__ void __launch_bounds__(kGmThreads, kGmCtasPerSm)
group_attn_merge_kernel(const GaArgs A) {
    __shared__ GmSmem sm;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    pdl_wait();
    pdl_trigger();
    const int64_t total = __ldcg(&A.plan->total);
    const int ranges = __ldcg(&A.plan->ranges);
    GaPlan::Tile mine = {};
    if (tid < kGaMaxCtas) {                                        // beyond the ranges: whatever is there, not looked at
        mine.begin = __ldcg(&A.plan->first[tid].begin);
        mine.blocks = __ldcg(&A.plan->first[tid].blocks);
        mine.tok0 = __ldcg(&A.plan->first[tid].tok0);
        mine.ntok = __ldcg(&A.plan->first[tid].ntok);
        sm.first[tid] = mine;
    }
    // The range boundary c cuts the row tile of range c's first step when the
    // tile begins before it; the first such boundary of a tile stands for it.
    int incl = 0;
    if (tid > 0 && tid < ranges && mine.begin < ga_range(total, tid, ranges) && mine.begin >= ga_range(total, tid - 1, ranges))
        incl = mine.ntok;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < warp; ++w) incl += sm.warp_sum[w];
    if (tid < kGaMaxCtas) sm.before[tid + 1] = incl;
    if (tid == 0) sm.before[0] = 0;
    __syncthreads();
    const int tokens = sm.before[kGaMaxCtas];
    // slices of 16 channels while 36 of them per token fit one wave of CTAs, then of 64, then of 192
    const int grid = static_cast<int>(gridDim.x);
    const int per = tokens * kGmSlices <= grid ? kGmSlices : tokens * 9 <= 2 * grid ? 9 : 3;
    for (int unit = blockIdx.x; unit < tokens * per; unit += grid) {
        const int ut = unit / per, slice = unit - ut * per;
        int lo = 0, hi = kGaMaxCtas;                               // the boundary: before[c] <= ut < before[c + 1]
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (sm.before[mid] <= ut) lo = mid; else hi = mid;
        }
        const GaPlan::Tile &t = sm.first[lo];
        const int tok = ut - sm.before[lo];
        // ranges c0 = lo - 1 (which begins the tile) to the last c with total * c / ranges < the tile's end; a range's
        // first tile is in its slot 0
        const int c0 = lo - 1, n = static_cast<int>(((t.begin + t.blocks) * ranges - 1) / total) - c0 + 1;
        const int slot0 = 2 * c0 + (ga_range(total, c0, ranges) < t.begin - (A.few ? kGfGap : kGaGap) ? 1 : 0);
        const int64_t row = static_cast<int64_t>(t.tok0 + tok) * kHeads;
        if (per == kGmSlices) gm_slice<0>(A, sm, c0, n, slot0, tok, row, slice * 16, slice == 0);
        else if (per == 9) gm_slice<1>(A, sm, c0, n, slot0, tok, row, slice * 64, slice == 0);
        else gm_slice<3>(A, sm, c0, n, slot0, tok, row, slice * 192, slice == 0);
    }
}

// Workspace: the plan, then two partials per range.
inline size_t ga_plan_bytes() { return (sizeof(GaPlan) + 255) / 256 * 256; }
inline size_t ga_ml_bytes(int tok_slots) { return static_cast<size_t>(2 * kGaMaxCtas) * tok_slots * kHeads * sizeof(float2); }
inline size_t ga_ws_bytes(int tok_slots) {
    return ga_plan_bytes() + ga_ml_bytes(tok_slots) + static_cast<size_t>(2 * kGaMaxCtas) * tok_slots * kHeads * kDim * 4;
}

}  // namespace csa2
