// gattn_few.cuh -- K12b: group attention for groups of few tokens. K12's row
// tile has 128 rows; with one token per group seven of eight go unused, and an
// MMA takes the same 48 cycles for 16 columns as for 64. So here the entries
// are the rows of both products and the (token, head) pairs their columns:
//   S^T [112 x 64]    = K [112 x 576] . Q^T            (36 MMAs, M = 128, K = 16)
//   O^T [576 x 64]   += V^T [576 x 112] . P^T, V = K   (7 MMAs for each of 5 x 128 channels)
// for row tiles of 4 tokens x 16 heads and blocks of 112 keys: 71 MMAs where
// K12 takes 72 to 80 for 64 keys. Blocks of 128 keys would fill M, but with Q
// (73,728 B) and P the block would not fit in shared memory; the upper 16 rows
// of S^T read the next 8 channels' first keys and are not looked at. All of O
// fits in tensor memory (5 x 64 columns).
//
// Operands lie as in K12: slabs of 8 channels (16 bytes) per key, K-major for S
// and MN-major for O; P is written by the softmax threads as slabs of 8 rows
// (16 bytes) per key, MN-major.
//   warps 0-7   load the query tile, then per block the softmax: thread = key,
//               warps 0-3 the first half of the rows and 4-7 the other. A thread
//               does not see a row's other keys, and does not have to: it
//               compares its scores with the rows' references (K12's), and only
//               when one of them exceeds its row's maximum so far by more than
//               kGaSlack do all take the maxima over the keys (a transposing
//               butterfly) and rescale.
//               A row's sum is kept per key, 32 in registers, to the end. O is
//               moved out every kGfMove blocks, as in K12 (its code costs 1%).
//   warp 8      issues the MMAs, with 16 columns per token present.
//   warps 9-15  dequantise, 16 keys each (112 = 7 x 16; 16 keys share a page).
// The last 128 channels of O^T are 448 .. 575: 64 of them come twice. A tile's
// last scores read, its queries make room for the next tile's, so that those
// scores are there when the outputs have been written.
//
// Bound and measured: shared-memory bandwidth. With 64 columns a block moves
// 6 KB for each of 71 MMAs, 126 KB of entries and 14 KB of P, 4,400 cycles at
// 128 B each, and the softmax, in which nothing moves because no chunk of K is
// free before its MMAs, adds 1,400. Measured (slope over the length, at 1,965
// MHz) are 7,100 cycles for 112 keys when the entries come from L2 and 7,400
// from DRAM: the other 1,300 are hand-offs between the roles. With two tokens
// 6,500 and 6,900, with one 6,200 and 6,700; K12 takes 4,900 for 64 keys. 4
// tokens over 1M keys 262 us (K12 315): 237 for 63.3 blocks a CTA, the rest as
// in K12. 64 groups of 1 token over 4,096 keys each 74 us (K12 99.5). At 5 or
// more tokens a group takes two tiles here, and K12 wins: 32 groups of 5 over
// 4,096 keys 88 us against 70, of 4 61 against 69. The rule N <= 4 G takes the
// mean, so a popular group among many small or empty ones comes here too: 64
// tokens over 32,768 keys beside 20 groups of one over 4,096 take 167 us, and
// 133 beside 19, which K12 gets.
#pragma once

#include "gattn.cuh"

namespace csa2 {

constexpr int kGfTok = 4, kGfRows = kGfTok * kHeads;               // 64
constexpr int kGfBlk = 112, kGfGap = 2;                            // gaps 1, 2, 3, 5: 74.9, 74.9, 77.8, 80.6 us for 64 groups of one token
using GaFew = GaForm<kGfTok, kGfBlk, kGfGap>;
constexpr int kGfDeqWarps = 7;
constexpr int kGfQSlab = kGfRows * 16, kGfKSlab = kGfBlk * 16;     // 1,024 and 1,792 B
constexpr int kGfOCol = 64;                                        // S in columns 0-63, O^T from here on
constexpr int kGfTiles = 5;                                        // of 128 channels
// Chunks of 64 channels are filled, multiplied and released in rounds: two for
// each of O's first three tiles, three for the last two.
constexpr int kGfRounds = 4;
constexpr int kGfMove = 256;                                       // blocks (28,672 entries) that O adds up by itself
constexpr float kGfNone = 1e30f;                                   // reference of a row without keys yet: any score exceeds it

struct GfSmem {
    alignas(1024) uint8_t q[kGfRows * kDim * 2];
    alignas(1024) uint8_t k[kGfBlk * kDim * 2];
    alignas(16) uint8_t p[kGfRows * kGfBlk * 2];                   // behind k: S's unused rows read its first bytes
    uint64_t q_full, s_full, p_full;
    uint64_t k_full[kGfRounds], k_free[kGfRounds];                 // the last round's free: the block's O is complete too
    uint32_t tmem;
    alignas(16) float scale[kGfRows];                              // of a row: softmax scale (log2) times query exponent
    alignas(16) float nref[kGfRows];                               // minus its reference
    alignas(16) float fac[kGfRows], own[kGfRows];                  // factors of a rescaling, or of the entries and the own part
    float moved[kGfRows];                                          // factor of what was moved out
    float m[kGfRows];                                              // its reference, -inf without keys yet
    float col[4][kGfRows];                                         // a row's maximum or sum in each quarter of the keys
    int64_t scan[kGaThreads / 32], start, total;
    int start_g;
    GaWalk<GaFew> walk;
};
constexpr size_t kGfSmemBytes = sizeof(GfSmem);
static_assert(kGfSmemBytes <= 232448 && kGfRows * kGfBlk * 2 >= 256, "one CTA per SM");

// 32 lanes x 8 columns.
__device__ __forceinline__ void gf_tmem_ld8(uint32_t taddr, float (&v)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr) : "memory");
}
__device__ __forceinline__ void gf_tmem_st8(uint32_t taddr, const float (&v)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n\t"
                 "tcgen05.wait::st.sync.aligned;"
                 ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}

// K12's MMA from shared memory with the number of columns at run time: what
// the rows of absent tokens would read is left to the dequantising warps.
template <uint32_t kA, uint32_t kAHi, uint32_t kB, uint32_t kBHi>
__device__ __forceinline__ void gf_mma_ss(uint32_t one, uint32_t idesc, uint32_t d, uint32_t a_lo, uint32_t b_lo,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b32 a, b;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.u32 e, %9, 0;\n\tsetp.ne.u32 p, %2, 0;\n\tadd.u32 a, %0, %5;\n\tadd.u32 b, %1, %7;\n\t"
        "mov.b64 da, {a, %6};\n\tmov.b64 db, {b, %8};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%3], da, db, %4, p;\n\t}"
        ::"r"(a_lo), "r"(b_lo), "r"(accumulate), "r"(d), "r"(idesc), "n"(kA), "n"(kAHi), "n"(kB), "n"(kBHi), "r"(one)
        : "memory");
}

// Lane c < 8 n (n = 1 .. 4) gets the maximum (or sum) over the lanes of x[c]:
// each step halves the columns and doubles the lanes that a value stands for;
// with few columns the first steps come last, on one value.
template <bool kMax>
__device__ __forceinline__ float gf_across(float (&x)[32], int n, int lane) {
    auto join = [](float a, float b) { return kMax ? fmaxf(a, b) : a + b; };
    auto halve = [&](auto d_) {
        constexpr int d = decltype(d_)::value;
        const bool up = lane & d;
#pragma unroll
        for (int i = 0; i < d; ++i)
            x[i] = join(up ? x[i + d] : x[i], __shfl_xor_sync(0xffffffffu, up ? x[i] : x[i + d], d));
    };
    if (n > 2) halve(std::integral_constant<int, 16>{});
    if (n > 1) halve(std::integral_constant<int, 8>{});
    halve(std::integral_constant<int, 4>{});
    halve(std::integral_constant<int, 2>{});
    halve(std::integral_constant<int, 1>{});
    float v = x[0];
    if (n == 1) v = join(v, __shfl_xor_sync(0xffffffffu, v, 8));
    if (n <= 2) v = join(v, __shfl_xor_sync(0xffffffffu, v, 16));
    return v;
}

__device__ __forceinline__ void gf_bar() { asm volatile("bar.sync 5, 256;" ::: "memory"); }
__device__ __forceinline__ bool gf_any(bool v) {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbarrier.cta.red.or.pred q, 5, 256, p;\n\t"
                 "selp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"(static_cast<uint32_t>(v)) : "memory");
    return r != 0;
}

// Channel of O^T's tile t in tensor memory lane `at`.
__device__ __forceinline__ int gf_channel(int t, int at) { return (t < 4 ? 128 * t : 448) + at; }

template <bool kMoves>
__device__ __forceinline__ void gf_softmax(const GaArgs &A, GfSmem &sm, GaWalk<GaFew> walk, int warp, int lane) {
    const int quarter = warp & 3, half = warp >> 2, key = 32 * quarter + lane, tid = threadIdx.x;
    const uint32_t tm0 = sm.tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    GaWait wait;
    uint32_t blk = 0;
    auto find = [&](GaSeg &s, uint32_t &no) {                      // the next segment with entries; no counts all
        for (;; ++no) {
            if (!walk.next(A, s)) return false;
            if (s.T != 0) return true;
            ga_own_only<1>(A, s, warp, lane);                      // 2 and 4: 1 and 2% off every call, for the code alone
        }
    };
    auto load_q = [&](const GaSeg &s) {
        ga_load_q<kGfQSlab, 1>(A, sm.q, sm.scale, s, warp >> 1, 8 * (warp & 1), lane);
        fence_proxy_async_smem();
    };
    auto reset = [&]() {
        sm.m[tid] = -INFINITY;
        sm.nref[tid] = kGfNone;
        if constexpr (kMoves) sm.moved[tid] = 1.0f;
    };
    GaSeg s;
    uint32_t seg_no = 0;
    bool more = find(s, seg_no);
    if (!more) return;
    load_q(s);
    if (tid < kGfRows) reset();
    gf_bar();                                                      // the tile is whole
    if (tid == 0) mbar_arrive(&sm.q_full);
    while (more) {
        const int32_t *pages = A.page_table + static_cast<int64_t>(s.g) * A.max_pages;
        auto page_of = [&](int kb) {                               // of this thread's key, -1: it does not count
            const int pos = kb * kGfBlk + key;
            return key < kGfBlk && pos < s.T ? __ldg(pages + pos / kPage) : -1;
        };
        int page = page_of(s.k0);
        const int live = s.ntok, c0 = 8 * live * half;             // this warp's rows: live x 8 from c0 on
        const uint32_t tm = tm0 + c0;
        float2 l[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) l[i] = make_float2(0.0f, 0.0f);
        for (int kb = s.k0; kb < s.k1; ++kb, ++blk) {
            const bool ok = page >= 0 && page < A.num_pages;
            if (kb + 1 < s.k1) page = page_of(kb + 1);
            wait(&sm.s_full, blk & 1u);
            tc_fence_after();
            float x[32];
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
                bool over = false;
                ga_tmem_ld32(tm, x);
#pragma unroll
                for (int i = 0; i < 32; i += 4) {
                    const float4 sc = *reinterpret_cast<const float4 *>(sm.scale + c0 + i);
                    const float4 rf = *reinterpret_cast<const float4 *>(sm.nref + c0 + i);
                    const float2 a = ga_fma2(make_float2(x[i], x[i + 1]), make_float2(sc.x, sc.y), make_float2(rf.x, rf.y));
                    const float2 b = ga_fma2(make_float2(x[i + 2], x[i + 3]), make_float2(sc.z, sc.w), make_float2(rf.z, rf.w));
                    x[i] = ok ? a.x : -INFINITY;
                    x[i + 1] = ok ? a.y : -INFINITY;
                    x[i + 2] = ok ? b.x : -INFINITY;
                    x[i + 3] = ok ? b.y : -INFINITY;
                    if (i < 8 * live) over |= fmaxf(fmaxf(x[i], x[i + 1]), fmaxf(x[i + 2], x[i + 3])) > kGaHead + kGaSlack;
                }
                if (pass == 1 || !gf_any(over)) break;
                // new references: rows' maxima over the block's keys
                ga_tmem_ld32(tm, x);
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = ok ? x[i] : -INFINITY;
                const float top = gf_across<true>(x, live, lane);
                if (lane < 8 * live) sm.col[quarter][c0 + lane] = top;
                gf_bar();
                if (tid < kHeads * live) {
                    float mx = fmaxf(fmaxf(sm.col[0][tid], sm.col[1][tid]), fmaxf(sm.col[2][tid], sm.col[3][tid]));
                    mx = mx == -INFINITY ? mx : mx * sm.scale[tid];
                    const float m = sm.m[tid];
                    const bool raise = mx > m + (kGaHead + kGaSlack) || (m == -INFINITY && mx > m);
                    mx -= kGaHead;
                    const float f = raise ? ga_ex2(m - mx) : 1.0f; // 0 for the first keys of a row
                    sm.fac[tid] = f;
                    if constexpr (kMoves) sm.moved[tid] *= f;
                    if (raise) {
                        sm.m[tid] = mx;
                        sm.nref[tid] = -mx;
                    }
                }
                gf_bar();
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 f = *reinterpret_cast<const float2 *>(sm.fac + c0 + 2 * i);
                    l[i] = make_float2(l[i].x * f.x, l[i].y * f.y);
                }
                if (kb > s.k0) {                                   // O of the block before is complete
#pragma unroll 1
                    for (int c = kGfOCol; c < kGfOCol + kGfTiles * kGfRows; c += kGfRows)
#pragma unroll 1
                        for (int j = 0; j < 8 * live; j += 8) {
                            float a[8];
                            gf_tmem_ld8(tm + c + j, a);
#pragma unroll
                            for (int i = 0; i < 8; ++i) a[i] *= sm.fac[c0 + j + i];
                            gf_tmem_st8(tm + c + j, a);
                        }
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= live) break;
                uint32_t p[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 e = make_float2(ga_ex2(x[8 * j + 2 * i]), ga_ex2(x[8 * j + 2 * i + 1]));
                    l[4 * j + i] = ga_add2(l[4 * j + i], e);
                    p[i] = f32x2_f16x2(e.x, e.y);
                }
                if (key < kGfBlk)
                    *reinterpret_cast<uint4 *>(sm.p + (c0 / 8 + j) * kGfKSlab + key * 16) = make_uint4(p[0], p[1], p[2], p[3]);
            }
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full);
            if constexpr (!kMoves) continue;
            const int done = kb + 1 - s.k0;
            const bool last = kb + 1 == s.k1;
            if (last ? done > kGfMove : done % kGfMove == 0) {
                wait(&sm.k_free[kGfRounds - 1], blk & 1u);         // O is complete
                tc_fence_after();
                const int64_t row0 = (2 * blockIdx.x + (seg_no > 0)) * static_cast<int64_t>(A.tok_slots) * kHeads + c0;
#pragma unroll 1
                for (int t = 0; t < kGfTiles; ++t)
#pragma unroll 1
                    for (int j = 0; j < 8 * live; j += 4) {
                        if (t == kGfTiles - 1 && quarter < 2) break;       // channels 448-511 are in the tile before
                        float a[4], *out = A.part_o + (row0 + j) * kDim + gf_channel(t, 32 * quarter + lane);
                        const uint32_t at = tm + kGfOCol + t * kGfRows + j;
                        ga_tmem_ld4(at, a);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (done > kGfMove) a[i] += sm.moved[c0 + j + i] * out[i * kDim];
                            if (last) continue;
                            out[i * kDim] = a[i];
                            a[i] = 0.0f;
                        }
                        ga_tmem_st4(at, a);
                    }
                gf_bar();                                          // all have read their factors
                if (tid < kGfRows) sm.moved[tid] = 1.0f;
            }
        }
        // ---- end of the segment: the next one's queries first, so that its scores are computed meanwhile
        GaSeg n;
        uint32_t n_no = seg_no + 1;
        more = find(n, n_no);
        gf_bar();                                                  // all have read their scores and scales
        if (more) {
            load_q(n);
            gf_bar();
            if (tid == 0) mbar_arrive(&sm.q_full);
        }
        wait(&sm.k_free[kGfRounds - 1], (blk - 1) & 1u);
        tc_fence_after();
        float x[32];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[2 * i] = l[i].x, x[2 * i + 1] = l[i].y;
        const float part = gf_across<false>(x, live, lane);
        if (lane < 8 * live) sm.col[quarter][c0 + lane] = part;
        gf_bar();
        const bool whole = s.k0 == 0 && s.k1 == s.blocks;
        const int64_t slot = 2 * blockIdx.x + (seg_no > 0);
        if (tid < s.ntok * kHeads) {
            const float m = sm.m[tid], sum = (sm.col[0][tid] + sm.col[1][tid]) + (sm.col[2][tid] + sm.col[3][tid]);
            if (!whole) {
                A.part_ml[slot * A.tok_slots * kHeads + tid] = make_float2(m, sum);
            } else {
                const int64_t r = static_cast<int64_t>(s.tok0) * kHeads + tid;
                const float lo = A.lse_own ? __ldg(A.lse_own + r) * 1.4426950408889634f : -INFINITY;
                const float top = fmaxf(m, lo), ref = top == -INFINITY ? 0.0f : top;
                const float wk = ga_ex2(m - ref), wo = ga_ex2(lo - ref), all = sum * wk + wo;
                const float inv = all == 0.0f ? 0.0f : 1.0f / all; // a NaN stays one
                sm.fac[tid] = wk * inv;
                sm.own[tid] = wo > 0.0f ? wo * inv : 0.0f;         // nothing to read without an own part
                A.lse[r] = all == 0.0f ? -INFINITY : (ref + log2f(all)) * 0.6931471805599453f;
            }
        }
        if (tid < kGfRows) reset();
        gf_bar();
#pragma unroll 1
        for (int t = 0; t < kGfTiles; ++t) {
            if (t == kGfTiles - 1 && quarter < 2) break;           // channels 448-511 are in the tile before
            const int ch = gf_channel(t, 32 * quarter + lane);
#pragma unroll 1
            for (int j = 0; j < live; ++j) {
                const int row = c0 + 8 * j, tok = row / kHeads, h0 = row % kHeads;
                float a[8];
                gf_tmem_ld8(tm + kGfOCol + t * kGfRows + 8 * j, a);
                if (!whole) {
                    float *po = A.part_o + ((slot * A.tok_slots + tok) * kHeads + h0) * kDim + ch;
#pragma unroll
                    for (int h = 0; h < 8; ++h) po[h * kDim] = a[h];
                } else {
                    const int64_t to = (static_cast<int64_t>(s.tok0 + tok) * kHeads + h0) * kDim + ch;
#pragma unroll
                    for (int h = 0; h < 8; ++h) {
                        float v = a[h] * sm.fac[row + h];
                        const float fo = sm.own[row + h];
                        if (fo != 0.0f) v += fo * __ldg(A.o_own + to + h * kDim);
                        A.out[to + h * kDim] = __float2bfloat16_rn(v);
                    }
                }
            }
        }
        tc_fence_before();
        s = n;
        seg_no = n_no;
    }
}

// A warp's 16 keys of every block, one 16-byte load per lane and chunk; a
// chunk's load for the next block is issued as soon as it has been converted.
__device__ __forceinline__ void gf_dequant(const GaArgs &A, GfSmem &sm, GaWalk<GaFew> walk, int warp, int lane) {
    const int key = 16 * warp + (lane & 15), part = lane >> 4;
    uint8_t *const dst0 = sm.k + 4 * part * kGfKSlab + key * 16;
    constexpr int kChunks = kDim / kGaChunk;                       // 9
    GaWait wait;
    GaSeg s = {};
    int kb = 0, page = -1, left = 0;
    const uint8_t *codes = nullptr, *scales = nullptr;
    auto look = [&](int b) {                                       // the page of the warp's keys in block b
        const int pos = b * kGfBlk + 16 * warp;
        return pos < s.T ? __ldg(A.page_table + static_cast<int64_t>(s.g) * A.max_pages + pos / kPage) : -1;
    };
    auto segment = [&]() {
        do {
            if (!walk.next(A, s)) return false;
        } while (s.T == 0);
        kb = s.k0;
        page = look(kb);
        return true;
    };
    auto open = [&]() {                                            // the block at hand; the page of the next
        const int pos = kb * kGfBlk + 16 * warp;
        const bool there = page >= 0 && page < A.num_pages;
        if (!there && pos < s.T) flag_status(kStatusBounds);
        left = there ? s.T - pos - (lane & 15) : 0;
        const int64_t at = static_cast<int64_t>(there ? page : 0) * kPage + pos % kPage + (lane & 15);
        codes = A.kv_fp4 + at * kFp4Bytes + 16 * part;
        scales = A.kv_scale + at * kScaleBytes + 2 * part;
        if (kb + 1 < s.k1) page = look(kb + 1);
    };
    uint4 v[kChunks];
    uint32_t sc[kChunks];
    auto fetch = [&](int c) {
        // unconditional, so that nothing waits for it here: the rows are in the page whether they count or not
        v[c] = __ldg(reinterpret_cast<const uint4 *>(codes + 32 * c));
        sc[c] = __ldg(reinterpret_cast<const uint16_t *>(scales + 4 * c));
    };
    bool more = segment();
    if (!more) return;
    open();
#pragma unroll
    for (int c = 0; c < kChunks; ++c) fetch(c);
    uint32_t phase = 1u;                                           // of free: passes at once for the first block
    while (more) {
        const bool ok = left > 0;                                  // entries that do not count are zeros
        more = ++kb < s.k1 || segment();
        if (more) open();
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
            if (c < 8 && c % 2 == 0) wait(&sm.k_free[c / 2], phase);
            const uint32_t s2 = ok ? e4m3x2_to_f16x2(sc[c]) : 0u;
            const uint32_t sa = __byte_perm(s2, s2, 0x1010), sb = __byte_perm(s2, s2, 0x3232);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t f = i < 2 ? sa : sb;
                uint32_t h[4];
                ga_e2m1x8((&v[c].x)[i], h);
                *reinterpret_cast<uint4 *>(dst0 + (8 * c + i) * kGfKSlab) =
                    make_uint4(hmul2_u32(h[0], f), hmul2_u32(h[1], f), hmul2_u32(h[2], f), hmul2_u32(h[3], f));
            }
            if (more) fetch(c);
            if ((c < 6 && c % 2 == 1) || c == kChunks - 1) {
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.k_full[min(c / 2, kGfRounds - 1)]);
            }
        }
        phase ^= 1u;
    }
}

__device__ __forceinline__ void gf_mma(const GaArgs &A, GfSmem &sm, GaWalk<GaFew> walk) {
    const uint32_t one = ga_elect() ? 1u : 0u;
    const uint32_t d_q = ga_desc_lo(sm.q, kGfQSlab), d_k = ga_desc_lo(sm.k, kGfKSlab);
    const uint32_t d_v = ga_desc_lo(sm.k, 128), d_p = ga_desc_lo(sm.p, 128);
    GaWait wait;
    uint32_t blk = 0, tile_no = 0;
    GaSeg s;
    while (walk.next(A, s)) {
        if (s.T == 0) continue;
        wait(&sm.q_full, tile_no & 1u);
        ++tile_no;
        const uint32_t id_s = umma_idesc(128, kHeads * s.ntok, false, false), id_o = umma_idesc(128, kHeads * s.ntok, true, true);
        for (int kb = s.k0; kb < s.k1; ++kb, ++blk) {
            const uint32_t par = blk & 1u, acc = kb > s.k0;
            constexpr uint32_t hi = ga_desc_hi(128), hi_o = ga_desc_hi(kGfKSlab);
            constexpr uint32_t da = 2 * kGfKSlab >> 4, db = 2 * kGfQSlab >> 4;          // 16 channels
            // S's columns are free: p_full of the block before has been awaited
#pragma unroll 1
            for (int r = 0; r < kGfRounds; ++r) {
                wait(&sm.k_full[r], par);
                tc_fence_after();
#pragma unroll 1
                for (int c = 2 * r; c < (r < kGfRounds - 1 ? 2 * r + 2 : 9); ++c) {
                    const uint32_t a = d_k + c * (4 * da), b = d_q + c * (4 * db);
                    gf_mma_ss<0, hi, 0, hi>(one, id_s, 0u, a, b, c > 0);
                    gf_mma_ss<da, hi, db, hi>(one, id_s, 0u, a, b, 1u);
                    gf_mma_ss<2 * da, hi, 2 * db, hi>(one, id_s, 0u, a, b, 1u);
                    gf_mma_ss<3 * da, hi, 3 * db, hi>(one, id_s, 0u, a, b, 1u);
                }
            }
            ga_commit(one, &sm.s_full);
            wait(&sm.p_full, par);
            tc_fence_after();
#pragma unroll 1
            for (int t = 0; t < kGfTiles; ++t) {
                const uint32_t a = d_v + (t < 4 ? 16 * t : 56) * (kGfKSlab >> 4), d = kGfOCol + t * kGfRows;
                gf_mma_ss<0, hi_o, 0, hi_o>(one, id_o, d, a, d_p, acc);
                gf_mma_ss<16, hi_o, 16, hi_o>(one, id_o, d, a, d_p, 1u);
                gf_mma_ss<32, hi_o, 32, hi_o>(one, id_o, d, a, d_p, 1u);
                gf_mma_ss<48, hi_o, 48, hi_o>(one, id_o, d, a, d_p, 1u);
                gf_mma_ss<64, hi_o, 64, hi_o>(one, id_o, d, a, d_p, 1u);
                gf_mma_ss<80, hi_o, 80, hi_o>(one, id_o, d, a, d_p, 1u);
                gf_mma_ss<96, hi_o, 96, hi_o>(one, id_o, d, a, d_p, 1u);
                if (t < 3) ga_commit(one, &sm.k_free[t]);
            }
            ga_commit(one, &sm.k_free[kGfRounds - 1]);
        }
    }
    // every MMA of this CTA is done before tensor memory goes back
    if (blk > 0) wait(&sm.k_free[kGfRounds - 1], (blk - 1) & 1u);
}

template <bool kMoves>
__global__ void __launch_bounds__(kGaThreads, 1)
group_attn_few_kernel(const GaArgs A) {
    extern __shared__ __align__(1024) uint8_t ga_raw[];
    GfSmem &sm = *reinterpret_cast<GfSmem *>(ga_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.s_full, 1);
        mbar_init(&sm.p_full, kGaSoftWarps);
        for (int i = 0; i < kGfRounds; ++i) {
            mbar_init(&sm.k_full[i], kGfDeqWarps);
            mbar_init(&sm.k_free[i], 1);
        }
        fence_mbar_init();
    }
    pdl_wait();
    ga_locate<GaFew>(A, sm);
    __syncthreads();
    const int64_t total = sm.total;
    const int ranges = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total));
    if (blockIdx.x == 0 && tid == 0) {
        A.plan->total = total;
        A.plan->ranges = ranges;
    }
    if (static_cast<int>(blockIdx.x) >= ranges) return;
    if (tid == 0) ga_begin<GaFew>(A, sm, total, ranges);
    if (warp == kGaMmaWarp) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const GaWalk<GaFew> walk = sm.walk;
    if (warp < kGaSoftWarps) {
        ga_regs_up<kGaSoftRegs>();
        gf_softmax<kMoves>(A, sm, walk, warp, lane);
    } else {
        ga_regs_down<kGaOtherRegs>();
        if (warp == kGaMmaWarp)
            gf_mma(A, sm, walk);
        else
            gf_dequant(A, sm, walk, warp - kGaDeqWarp, lane);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    pdl_trigger();
    if (warp == kGaMmaWarp) {
        tc_fence_after();
        tmem_dealloc(sm.tmem, 512);
    }
}

}  // namespace csa2
