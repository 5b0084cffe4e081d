// gattn.cuh -- K12: group attention over the paged FP4 cache. Every query token
// of group g attends to the first kv_lens[g] entries of the group's pages
// (keys = values), and the result is joined with the token's own part. This is
// the form for many tokens per group; gattn_few.cuh has the one for few.
//
// Both products run on the tensor cores (tcgen05, accumulators in tensor
// memory) for row tiles of 8 tokens x 16 heads = 128 rows and blocks of 64
// keys (one page):
//   S [128 x 64]   = Q [128 x 576] . K^T              (36 MMAs, K = 16)
//   O [128 x 576] += P [128 x 64] . V, V = K          (4 MMAs per group of channels)
// What decides the layout: a row tile of 128 x 576 fp32 outputs (288 KB) is
// more than tensor memory (256 KB), Q (147,456 B) and one block of K
// (73,728 B) fill shared memory, and its bandwidth (128 B a cycle) is shared
// by the MMAs' operands and the dequantised entries. So 384 channels of O
// accumulate in tensor memory; the other 192 come out of the tensor cores
// block by block as pieces of 64, 32, 64 and 32 channels, two in S's columns
// (read by then) and two in columns of their own, and are added up in the
// registers of the softmax threads, 96 each. Splitting the channels over two
// CTAs would compute S twice. CTA pairs (cta_group::2) with each CTA
// dequantising half of the block took 111 us where single CTAs then took 124
// (64 tokens over 32,768 keys), but 646 against 378 (4 tokens over 1M keys): a
// hand-off between CTAs is about 1,000 cycles against 330 inside one. What they
// taught made single CTAs 103 and 315. Dequantising every block twice, so that
// S of the next could run during the softmax, took 7,400 cycles a block against
// 6,500 then.
//
// Q and K lie as slabs of 8 channels (16 bytes) per row: the K-major operand
// layout of S and the MN-major one of O, so a block is dequantised once for
// both. Tensor memory: O in columns 0-383, S 384-447, pieces 448-479, P (f16)
// 480-511.
//   warps 0-7   load the query tile, then per block the softmax: thread = row,
//               warps 0-3 the first 32 keys and 4-7 the others. Exp2 domain;
//               a row's reference is its maximum at some block minus kGaHead,
//               and rises only when a block exceeds that maximum by more than
//               kGaSlack (O is rescaled then). So a probability is 2^kGaHead
//               and at most 2^15 where it is largest, and f16, to which it is
//               rounded for the MMA, has its full 2^-11 (below the output's
//               bf16) down to 2^(-14 - kGaHead) of the largest one and steps of
//               2^(-24 - kGaHead) below: a flat tail of T entries behind one
//               dominant entry is off by at most T 2^(-25 - kGaHead) of its
//               values. With the largest one at 2^0 a million entries 17.4
//               below a sink were lost, 3% of the output. The sums are taken
//               before, in fp32. Then they add the pieces, and at the end of a
//               row tile write it. The tensor cores cut off what does not fit
//               when they add to O (sums of one sign were short by 1.1e-3 after
//               131,072 entries), so every kGaMove blocks O is moved out to the
//               range's partial, added up there with rounding, and begins at
//               zero again; after the last block the sum is brought back. The
//               code for it costs 2 to 3% (64 tokens over 32,768 keys 106.7 us
//               against 103.8), so calls whose ranges cannot be that long take
//               a kernel without it (kMoves).
//   warp 8      issues the MMAs, one lane under a predicate.
//   warps 9-14  dequantise: E2M1 x E4M3 is exact in f16. The codes of the next
//               block are in registers while this one is multiplied, and its
//               chunks are refilled in three rounds as O's MMAs release them.
// The roles' loops are kept rolled where they can be: 16 warps with five kinds
// of code press on the instruction cache (rolling the MMA loops took its misses
// from 669K to 63K and a tenth off the time).
//
// The work is one flat list of (row tile, block) steps, cut into equal
// contiguous ranges, one per CTA; a row tile that lies in several ranges is
// left as unnormalised partials (m, l, O) that K13 joins. Lengths and offsets
// are read on the device, so a captured call serves other lengths. Every wait
// is an mbarrier wait with a limit; a thread whose wait ran out goes on without
// waiting, so that all reach the end.
//
// Bound and measured: 4,900 cycles a block (the slope over the length, at 1,965
// MHz), of which S takes 2,150 (60 an MMA: its 6 KB of operands are 48 cycles of
// shared memory, and the block is being written meanwhile), the softmax 1,100 in
// which the tensor pipe idles (512 of them the exponentials), O 1,300 and the
// rest hand-offs. 64 tokens over 32,768 keys: 103 us, 750 TFLOP/s: 69 for 27.7
// blocks a CTA and 32 for query tiles in, partials out and K13.
#pragma once

#include "attn.cuh"
#include "common.cuh"

namespace csa2 {

constexpr int kGaMaxTokens = 1 << 20, kGaMaxGroups = 65535;
constexpr int kGaMaxCtas = 160;
constexpr int kGaTok = 8;                                          // tokens per row tile
constexpr int kGaRows = kGaTok * kHeads;                           // 128
constexpr int kGaBlk = kPage;                                      // keys per block
constexpr int kGaSoftWarps = 8, kGaMmaWarp = 8, kGaDeqWarp = 9, kGaDeqWarps = 6;
constexpr int kGaThreads = 16 * 32;                                // 512: whole warpgroups, for the register split
// Registers per thread: 128 at launch (512 x 128 = the SM's 65,536); the two
// softmax warpgroups take 168, the other two 88: (168 + 168 + 88 + 88) x 128
// threads = 65,536, the launch's own total.
constexpr int kGaSoftRegs = 168, kGaOtherRegs = 88;
constexpr int kGaChunk = 64;                                       // channels per chunk
constexpr int kGaQSlab = kGaRows * 16, kGaKSlab = kGaBlk * 16;     // 2,048 and 1,024 B: 8 channels of every row
constexpr int kGaTmemCh = 384;                                     // channels accumulated in tensor memory
constexpr int kGaSCol = kGaTmemCh, kGaDCol = kGaSCol + kGaBlk;     // 384, 448
constexpr int kGaPCol = kGaDCol + 32;                              // 480
constexpr int kGaRegs = (kDim - kGaTmemCh) / 2;                    // outputs a softmax thread holds: 96
// A block's nine chunks are filled, multiplied and released in three rounds, in
// the order in which O's MMAs are done with them: 2 r, 2 r + 1 and 6 + r.
constexpr int kGaRounds = 3;
constexpr int kGaMove = 512;                                       // blocks (32,768 entries) that O adds up by itself
constexpr int kGaGap = 5;                                          // 2: 93 us for 8 groups of 64 tokens, 5: 74
// log2 units: what a probability of the maximum is raised by, and a block may exceed that maximum by; f16 ends below 2^16.
constexpr float kGaHead = 7.0f, kGaSlack = 8.0f;                   // 11 and 4: 4 tokens x 1M entries of wide scores 322 us against 274
static_assert(kGaHead + kGaSlack <= 15.0f, "probabilities stay finite in f16");
static_assert(kGaPCol + kGaBlk / 2 == 512 && kGaRegs == 96, "tensor memory is full; pieces of 64, 32, 64 and 32 channels");

// A row tile of kT tokens, blocks of kB keys, and what a row tile costs beside
// its blocks (query in, result out), in blocks, so that ranges with many short
// tiles are not the longest.
template <int kT, int kB, int kG>
struct GaForm { static constexpr int kTok = kT, kBlk = kB, kGap = kG; };
using GaWide = GaForm<kGaTok, kGaBlk, kGaGap>;

struct GaArgs {
    const __nv_bfloat16 *q;            // [N][16][576]
    const uint8_t *kv_fp4, *kv_scale;
    int64_t num_pages;
    const int32_t *page_table;         // [G][max_pages]
    int max_pages;
    const int32_t *kv_lens;            // [G]
    const int32_t *q_offsets;          // [G + 1]
    int N, G;
    float scale_log2;                  // softmax scale * log2(e)
    const float *o_own, *lse_own;      // [N][16][576], [N][16], or null
    __nv_bfloat16 *out;                // [N][16][576]
    float *lse;                        // [N][16]
    struct GaPlan *plan;
    // [2 * ranges][tok_slots][144][16][4], 4 channels of 16 heads together; with few tokens [..][16][576]
    float *part_o;
    float2 *part_ml;                   // [2 * ranges][tok_slots * 16]: (the reference m in the log2 domain, l)
    int tok_slots;                     // min(8, N), with few tokens min(4, N)
    int few;                           // the form for few tokens per group
};

// What K13 has to know of K12's ranges.
struct GaPlan {
    int64_t total;                     // steps of all row tiles
    int ranges;
    // row tile of a range's first step; begin is the step of its first block
    struct Tile { int64_t begin; int blocks, tok0, ntok; } first[kGaMaxCtas];
};

// First step of range c (a 64-bit division only where 32 bits do not hold the product).
__device__ __forceinline__ int64_t ga_range(int64_t total, int c, int ranges) {
    if (total <= 0xffffffffll / kGaMaxCtas)
        return static_cast<uint32_t>(total) * static_cast<uint32_t>(c) / static_cast<uint32_t>(ranges);
    return total * c / ranges;
}

struct GaGroup { int tok0, n, T, blocks; };

// Group g as the kernel takes it: bounds outside [0, N] leave it without
// tokens, a bad length without entries. A group without entries still has one
// (empty) block per row tile, which writes its tokens' own parts.
template <class F>
__device__ __forceinline__ GaGroup ga_group(const GaArgs &A, int g, bool report) {
    GaGroup r;
    r.tok0 = __ldg(A.q_offsets + g);
    const int b = __ldg(A.q_offsets + g + 1);
    r.T = __ldg(A.kv_lens + g);
    bool bad = false;
    r.n = b - r.tok0;
    if (r.tok0 < 0 || b > A.N || b < r.tok0) {
        bad = true;
        r.n = 0;
    }
    if (r.T < 0 || r.T > A.max_pages * kPage) {
        bad = true;
        r.T = 0;
    }
    if (bad && report) flag_status(kStatusBounds);
    r.blocks = max(1, (r.T + F::kBlk - 1) / F::kBlk);
    return r;
}

// A group's steps: for each row tile its blocks, after the gap.
template <class F>
__device__ __forceinline__ int64_t ga_steps(const GaGroup &g) {
    return static_cast<int64_t>((g.n + F::kTok - 1) / F::kTok) * (F::kGap + g.blocks);
}

// One row tile's blocks [k0, k1) of a CTA's range.
struct GaSeg {
    int g, tok0, ntok, T, blocks, k0, k1;
};

// Walks a range segment by segment; every role of the CTA does so by itself.
template <class F>
struct GaWalk {
    int64_t left;                      // steps to go
    int g, tile, k;                    // group, row tile of the group, step of the row tile
    __device__ __forceinline__ bool next(const GaArgs &A, GaSeg &s) {
        while (left > 0) {
            GaGroup grp = ga_group<F>(A, g, false);
            while (tile * F::kTok >= grp.n) {
                if (++g >= A.G) return false;
                grp = ga_group<F>(A, g, false);
                tile = 0;
            }
            const int len = F::kGap + grp.blocks, end = left < len - k ? k + static_cast<int>(left) : len;
            s.g = g;
            s.tok0 = grp.tok0 + tile * F::kTok;
            s.ntok = min(F::kTok, grp.n - tile * F::kTok);
            s.T = grp.T;
            s.blocks = grp.blocks;
            s.k0 = max(0, k - F::kGap);
            s.k1 = max(0, end - F::kGap);
            left -= end - k;
            k = 0;
            ++tile;
            if (s.k1 > s.k0) return true;
        }
        return false;
    }
};

struct GaSmem {
    alignas(1024) uint8_t q[kGaRows * kDim * 2];
    alignas(1024) uint8_t k[kGaBlk * kDim * 2];
    uint64_t q_full;                   // query tile in
    uint64_t s_full;                   // scores in tensor memory
    uint64_t p_full;                   // probabilities in tensor memory, O rescaled
    uint64_t ds_full, ds_empty;        // a piece in S's columns; the first one read
    uint64_t dd_full, dd_empty;        // a piece in its own 32 columns; the first one read
    // A round's chunks: in (the first round's also says that S's columns are free), and multiplied (the last
    // round's also says that the block's O is complete).
    uint64_t k_full[kGaRounds], k_free[kGaRounds];
    uint32_t tmem;
    float scale[kGaRows];              // a row's softmax scale (log2) times its query exponent
    float mx[2][2][kGaRows];           // a row's maximum in each half of a block, by block parity
    float l[kGaRows];
    int64_t scan[kGaThreads / 32], start, total;
    int start_g;
    GaWalk<GaWide> walk;
};
constexpr size_t kGaSmemBytes = sizeof(GaSmem);
static_assert(kGaSmemBytes <= 232448, "one CTA per SM");

// ---------------------------------------------------------------- PTX
// One arrival when the MMAs issued so far by this lane have completed.
__device__ __forceinline__ void ga_commit(uint32_t one, uint64_t *bar) {
    asm volatile(
        "{\n\t.reg .pred e;\n\tsetp.ne.u32 e, %1, 0;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
        ::"r"(smem_u32(bar)), "r"(one) : "memory");
}

// MMAs are issued by the lane whose `one` is set; the warp stays together, so
// that the operands are uniform. A descriptor is its low word (address and
// leading offset) plus a constant under a constant high word.
template <uint32_t kIdesc, uint32_t kA, uint32_t kAHi, uint32_t kB, uint32_t kBHi>
__device__ __forceinline__ void ga_mma_ss(uint32_t one, uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b32 a, b;\n\t.reg .b64 da, db;\n\t"
        "setp.ne.u32 e, %9, 0;\n\tsetp.ne.u32 p, %2, 0;\n\tadd.u32 a, %0, %5;\n\tadd.u32 b, %1, %7;\n\t"
        "mov.b64 da, {a, %6};\n\tmov.b64 db, {b, %8};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%3], da, db, %4, p;\n\t}"
        ::"r"(a_lo), "r"(b_lo), "r"(accumulate), "r"(d), "n"(kIdesc), "n"(kA), "n"(kAHi), "n"(kB), "n"(kBHi), "r"(one)
        : "memory");
}

// A from tensor memory: lane = row, a 32-bit column holds two f16 of the K side.
template <uint32_t kIdesc, int kACol, uint32_t kB, uint32_t kBHi>
__device__ __forceinline__ void ga_mma_ts(uint32_t one, uint32_t d, uint32_t b_lo, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred e, p;\n\t.reg .b32 b;\n\t.reg .b64 db;\n\t"
        "setp.ne.u32 e, %7, 0;\n\tsetp.ne.u32 p, %1, 0;\n\tadd.u32 b, %0, %5;\n\tmov.b64 db, {b, %6};\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%2], [%3], db, %4, p;\n\t}"
        ::"r"(b_lo), "r"(accumulate), "r"(d), "r"(kACol), "n"(kIdesc), "n"(kB), "n"(kBHi), "r"(one) : "memory");
}

// Words of a descriptor without swizzle (umma_desc).
__device__ __forceinline__ uint32_t ga_desc_lo(const void *p, uint32_t lbo) { return (smem_u32(p) >> 4 & 0x3fffu) | lbo >> 4 << 16; }
__device__ __forceinline__ constexpr uint32_t ga_desc_hi(uint32_t sbo) { return sbo >> 4 | 1u << 14; }

__device__ __forceinline__ void ga_tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
          "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// 32 lanes x 4 columns.
__device__ __forceinline__ void ga_tmem_ld4(uint32_t taddr, float (&v)[4]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n\t"
                 "tcgen05.wait::ld.sync.aligned;"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]) : "r"(taddr) : "memory");
}
__device__ __forceinline__ void ga_tmem_st4(uint32_t taddr, const float (&v)[4]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n\t"
                 "tcgen05.wait::st.sync.aligned;"
                 ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]) : "memory");
}

// 32 lanes x 32 columns.
__device__ __forceinline__ void ga_tmem_ld32(uint32_t taddr, float (&v)[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ bool ga_elect() {
    uint32_t ok;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok != 0;
}

__device__ __forceinline__ float ga_ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

template <int N>
__device__ __forceinline__ void ga_regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void ga_regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ void ga_pair_bar(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id) : "memory"); }

// A wait that a thread gives up for good after its first timeout. Its limit is
// a number of probes of up to 1 us each (the sleeping probe's hint), 2 s in all:
// the roles' loops press on the instruction cache, so it is kept short.
struct GaWait {
    bool dead = false;
    __device__ __forceinline__ void operator()(uint64_t *bar, uint32_t parity) {
        for (int i = 0; i < (dead ? 1 : 2000000); ++i)
            if (mbar_try_wait_sleep(bar, parity, 1000u)) return;
        flag_status(kStatusTimeout);
        dead = true;
    }
};

// Two floats at once.
__device__ __forceinline__ float2 ga_fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}
__device__ __forceinline__ float2 ga_add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// ---------------------------------------------------------------- roles
// The first step of this CTA's range (its group, and that group's first step)
// and the total: a block scan over the groups, again over the chunks of 512
// when there are more.
template <class F, class Smem>
__device__ __forceinline__ void ga_locate(const GaArgs &A, Smem &sm) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kWarps = kGaThreads / 32;
    int64_t base = 0, begin = 0, mine = 0;
    auto scan = [&](int g0, bool report) {                // begin, mine of group g0 + tid; base moves past the chunk
        mine = g0 + tid < A.G ? ga_steps<F>(ga_group<F>(A, g0 + tid, report)) : 0;
        int64_t incl = mine;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
            if (lane >= d) incl += o;
        }
        if (lane == 31) sm.scan[warp] = incl;
        __syncthreads();
        int64_t before = lane < kWarps ? sm.scan[lane] : 0;
#pragma unroll
        for (int d = 1; d < kWarps; d <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, before, d);
            if (lane >= d) before += o;
        }
        begin = base + incl - mine + __shfl_sync(0xffffffffu, before, max(warp - 1, 0)) * (warp > 0);
        base += __shfl_sync(0xffffffffu, before, kWarps - 1);
        __syncthreads();
    };
    for (int g0 = 0; g0 < A.G; g0 += kGaThreads) scan(g0, blockIdx.x == 0);
    const int64_t total = base;
    const int ranges = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total)), range = blockIdx.x;
    const int64_t want = range < ranges ? ga_range(total, range, ranges) : -1;
    if (tid == 0) sm.total = total;
    base = 0;
    for (int g0 = 0; g0 < A.G; g0 += kGaThreads) {
        if (A.G > kGaThreads) scan(g0, false);
        if (want >= begin && want < begin + mine) {
            sm.start_g = g0 + tid;
            sm.start = begin;
        }
    }
}

// One thread: the walk of the CTA's range, complete after the next barrier,
// and what K13 has to know of its first row tile.
template <class F, class Smem>
__device__ __forceinline__ void ga_begin(const GaArgs &A, Smem &sm, int64_t total, int ranges) {
    const int range = blockIdx.x;
    const int64_t at = ga_range(total, range, ranges), local = at - sm.start;
    const GaGroup grp = ga_group<F>(A, sm.start_g, false);
    const int len = F::kGap + grp.blocks;
    GaWalk<F> w;
    w.left = ga_range(total, range + 1, ranges) - at;
    w.g = sm.start_g;
    w.tile = static_cast<int>(local / len);
    w.k = static_cast<int>(local - static_cast<int64_t>(w.tile) * len);
    sm.walk = w;
    GaPlan::Tile &t = A.plan->first[range];
    t.begin = at - w.k + F::kGap;
    t.blocks = grp.blocks;
    t.tok0 = grp.tok0 + w.tile * F::kTok;
    t.ntok = min(F::kTok, grp.n - w.tile * F::kTok);
}

// kHalves x 8 heads of a token of the query tile, from head0 on, -> f16 under a
// power-of-two exponent per row: a warp's loads are 64-byte runs of 8 rows and its stores whole 128-byte core
// matrices. The exponent is 0 as a rule, so the rows are stored as they come
// and again only where the largest magnitude asks for another one. Kept small:
// the code runs once per row tile, at the pace of the instruction fetch.
template <int kSlab, int kHalves>
__device__ __forceinline__ void ga_load_q(const GaArgs &A, uint8_t *tile, float *scale, const GaSeg &s, int tok, int head0,
                                          int lane) {
    const bool some = tok < s.ntok;
    // a negative softmax scale turns the query round, so that the largest score has the largest logit
    const float sign = copysignf(1.0f, A.scale_log2);
#pragma unroll 1
    for (int half = 0; half < kHalves; ++half) {
        const int h = head0 + half * 8 + (lane & 7), row = tok * kHeads + h, part = lane >> 3;
        const uint4 *src = reinterpret_cast<const uint4 *>(A.q + (static_cast<int64_t>(s.tok0 + (some ? tok : 0)) * kHeads + h) * kDim) + part;
        uint8_t *dst = tile + part * kSlab + row * 16;
        float mx, down = sign;
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
            uint32_t m2 = 0u;                                      // bf16 magnitudes order as integers
#pragma unroll 1
            for (int u0 = 0; u0 < 18; u0 += 9) {
                uint4 v[9];
#pragma unroll
                for (int u = 0; u < 9; ++u) v[u] = some ? __ldg(src + 4 * (u0 + u)) : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int u = 0; u < 9; ++u) {
                    uint32_t o[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t w = (&v[u].x)[e];
                        m2 = __vmaxu2(m2, w & 0x7fff7fffu);
                        const float2 f = bf16x2_f32(w);
                        o[e] = f32x2_f16x2(f.x * down, f.y * down);
                    }
                    *reinterpret_cast<uint4 *>(dst + 4 * (u0 + u) * kSlab) = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
            mx = __uint_as_float(max(m2 & 0xffff0000u, m2 << 16));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
            const int eq = mx < INFINITY ? f16_exponent(mx, 120) : 0;   // any finite row fits; one with inf or NaN stays one
            // never 0: entries that do not count have a score of -inf, which has to stay one
            if (part == 0) scale[row] = fmaxf(fabsf(A.scale_log2) * exp2f(static_cast<float>(eq)), 1e-30f);
            if (!__any_sync(0xffffffffu, eq != 0)) break;
            down = sign * exp2f(static_cast<float>(-eq));
        }
    }
}

// A segment of a group without entries: its tokens' own parts, or zeros, a
// token per warp, the loads of kAtOnce heads in flight (with one load at a time a tile
// took 26 us, 45 with the own parts in DRAM: longer than the other ranges, and
// 72 us instead of 50 for six groups of which one is empty).
template <int kAtOnce>
__device__ __forceinline__ void ga_own_only(const GaArgs &A, const GaSeg &s, int tok, int lane) {
    if (tok >= s.ntok) return;
    const int64_t r0 = static_cast<int64_t>(s.tok0 + tok) * kHeads;
#pragma unroll 1
    for (int h = 0; h < kHeads; h += kAtOnce) {
        const int64_t r = r0 + h;
        float2 v[9 * kAtOnce];
        float own[kAtOnce];
#pragma unroll
        for (int u = 0; u < 9 * kAtOnce; ++u)
            v[u] = A.o_own ? __ldg(reinterpret_cast<const float2 *>(A.o_own + r * kDim) + lane + 32 * u) : make_float2(0.0f, 0.0f);
#pragma unroll
        for (int u = 0; u < kAtOnce; ++u) {
            own[u] = A.lse_own ? __ldg(A.lse_own + r + u) : -INFINITY;
            if (lane == 0) A.lse[r + u] = own[u];
        }
#pragma unroll
        for (int u = 0; u < 9 * kAtOnce; ++u)
            reinterpret_cast<__nv_bfloat162 *>(A.out + r * kDim)[lane + 32 * u] =
                own[u / 9] != -INFINITY ? __floats2bfloat162_rn(v[u].x, v[u].y) : __floats2bfloat162_rn(0.0f, 0.0f);
    }
}

// Channel of a softmax thread's output register i (a multiple of 16): pieces
// of 64, 32, 64 and 32 channels from 384 on, half of each.
__device__ __forceinline__ constexpr int ga_reg_channel(int i, int half) {
    return i < 32 ? 384 + 32 * half + i : i < 48 ? 448 + 16 * half : i < 80 ? 480 + 32 * half + i - 48 : 544 + 16 * half;
}

// 16 channels of a row's result from ch on: the entries' sums times fk, the own part times fo.
__device__ __forceinline__ void ga_write16(const GaArgs &A, int64_t row, int ch, const float *a, float fk, float fo) {
    float v[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = a[i] * fk;
    if (fo != 0.0f) {
        const float4 *own = reinterpret_cast<const float4 *>(A.o_own + row * kDim + ch);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 o = __ldg(own + i);
            v[4 * i] += fo * o.x;
            v[4 * i + 1] += fo * o.y;
            v[4 * i + 2] += fo * o.z;
            v[4 * i + 3] += fo * o.w;
        }
    }
    uint32_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
        b[i] = *reinterpret_cast<const uint32_t *>(&t);
    }
    uint4 *dst = reinterpret_cast<uint4 *>(A.out + row * kDim + ch);
    dst[0] = make_uint4(b[0], b[1], b[2], b[3]);
    dst[1] = make_uint4(b[4], b[5], b[6], b[7]);
}

template <bool kMoves>
__device__ __forceinline__ void ga_softmax(const GaArgs &A, GaSmem &sm, GaWalk<GaWide> walk, int warp, int lane) {
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;      // keys 32 half ..; tile row
    const uint32_t tm = sm.tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const int pair_bar = 1 + (warp & 3);                           // the two warps of the same rows
    GaWait wait;
    uint32_t blk = 0, seg_no = 0;
    GaSeg s;
    if (lane == 0) mbar_arrive(&sm.k_full[0]);                     // S's columns are free for the first block
    while (walk.next(A, s)) {
        if (s.T == 0) {
            ga_own_only<4>(A, s, warp, lane);
            ++seg_no;
            continue;
        }
        const int32_t *pages = A.page_table + static_cast<int64_t>(s.g) * A.max_pages;
        int page = __ldg(pages + s.k0);
        ga_load_q<kGaQSlab, 2>(A, sm.q, sm.scale, s, warp, 0, lane);
        fence_proxy_async_smem();
        asm volatile("bar.sync 5, 256;" ::: "memory");             // scales of all rows; the tile is whole
        if (threadIdx.x == 0) mbar_arrive(&sm.q_full);
        const float scale = sm.scale[row];
        float m = -INFINITY, l = 0.0f;
        [[maybe_unused]] float moved = 1.0f;                       // factor of what was moved out
        float2 acc[kGaRegs / 2];
#pragma unroll
        for (int i = 0; i < kGaRegs / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
        // Part of a row tile, or what was moved out of one: unnormalised, 4 channels of a head together; only this
        // thread's own. The slot is free for a tile that lies whole in the range: the first one's own, then the last's.
        auto partial = [&]() {
            const int64_t slot = 2 * blockIdx.x + (seg_no > 0);
            return reinterpret_cast<float2 *>(A.part_o) + (slot * A.tok_slots + (row >> 4)) * (kDim * kHeads / 2) + 2 * (row & 15);
        };
        // adds this half's columns of a piece
        auto piece_add = [&](auto n_, int to, uint64_t *full, uint64_t *empty, int col, uint32_t parity) {
            constexpr int kN = decltype(n_)::value;
            wait(full, parity);
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < kN; c += 16) {
                float a[16];
                tmem_ld16(tm + col + kN * half + c, a);
                if (c + 16 == kN && empty != nullptr) {            // the columns are free
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(empty);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    acc[(to + c) / 2 + i] = ga_add2(acc[(to + c) / 2 + i], make_float2(a[2 * i], a[2 * i + 1]));
            }
        };
        for (int kb = s.k0; kb < s.k1; ++kb, ++blk) {
            const uint32_t par = blk & 1u;
            const int n = (page >= 0 && page < A.num_pages ? min(kGaBlk, s.T - kb * kGaBlk) : 0) - 32 * half;
            if (kb + 1 < s.k1) page = __ldg(pages + kb + 1);
            wait(&sm.s_full, par);
            tc_fence_after();
            float x[32];
            ga_tmem_ld32(tm + kGaSCol + 32 * half, x);
            if (n < 32) {
#pragma unroll
                for (int i = 0; i < 32; ++i) x[i] = i < n ? x[i] : -INFINITY;
            }
            float mx = fmaxf(x[0], x[1]);
#pragma unroll
            for (int i = 2; i < 32; i += 2) mx = fmaxf(mx, fmaxf(x[i], x[i + 1]));
            sm.mx[par][half][row] = mx;
            // with the reference as it stands; again if the block's maximum moves it
            uint32_t p[16];
            float2 sum;
#pragma unroll 1
            for (int pass = 0; pass < 2; ++pass) {
                const float ref = m == -INFINITY ? 0.0f : -m;
                const float2 sc = make_float2(scale, scale), rf = make_float2(ref, ref);
                sum = make_float2(0.0f, 0.0f);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float2 e = ga_fma2(make_float2(x[2 * i], x[2 * i + 1]), sc, rf);
                    e.x = ga_ex2(e.x);
                    e.y = ga_ex2(e.y);
                    sum = ga_add2(sum, e);
                    p[i] = f32x2_f16x2(e.x, e.y);
                }
                if (pass == 1) break;
                ga_pair_bar(pair_bar);
                mx = fmaxf(mx, sm.mx[par][half ^ 1][row]);
                mx = mx == -INFINITY ? mx : mx * scale;
                const bool raise = mx > m + (kGaHead + kGaSlack) || (m == -INFINITY && mx > m);
                if (!__any_sync(0xffffffffu, raise)) break;
                const float f = raise ? ga_ex2(m - (mx - kGaHead)) : 1.0f;   // 0 for the first keys of a row
                if (raise) m = mx - kGaHead;
                l *= f;
                if constexpr (kMoves) moved *= f;
#pragma unroll
                for (int i = 0; i < kGaRegs / 2; ++i) acc[i] = make_float2(acc[i].x * f, acc[i].y * f);
                if (kb > s.k0) {                                   // O of the block before is complete
#pragma unroll 1
                    for (int c = 0; c < kGaTmemCh / 2; c += 16) {
                        float a[16];
                        uint32_t o[16];
                        const uint32_t at = tm + half * (kGaTmemCh / 2) + c;
                        tmem_ld16(at, a);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(a[i] * f);
                        ga_tmem_st16(at, o);
                    }
                }
            }
            ga_tmem_st16(tm + kGaPCol + 16 * half, p);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.p_full);
            l += sum.x + sum.y;
            piece_add(std::integral_constant<int, 32>{}, 0, &sm.ds_full, &sm.ds_empty, kGaSCol, 0u);
            piece_add(std::integral_constant<int, 16>{}, 32, &sm.dd_full, &sm.dd_empty, kGaDCol, 0u);
            piece_add(std::integral_constant<int, 32>{}, 48, &sm.ds_full, &sm.k_full[0], kGaSCol, 1u);
            piece_add(std::integral_constant<int, 16>{}, 80, &sm.dd_full, nullptr, kGaDCol, 1u);   // p_full says it next
            if constexpr (!kMoves) continue;
            const int done = kb + 1 - s.k0;
            const bool last = kb + 1 == s.k1;
            if (last ? done > kGaMove : done % kGaMove == 0) {
                wait(&sm.k_free[kGaRounds - 1], par);              // O is complete
                tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < kGaTmemCh / 2; c += 4) {
                    const int ch = half * (kGaTmemCh / 2) + c;
                    float4 *const out = reinterpret_cast<float4 *>(partial() + ch / 4 * (2 * kHeads));
                    const bool live = (row >> 4) < s.ntok;
                    float a[4];
                    ga_tmem_ld4(tm + ch, a);
                    if (live && done > kGaMove) {
                        const float4 v = *out;
                        a[0] += moved * v.x;
                        a[1] += moved * v.y;
                        a[2] += moved * v.z;
                        a[3] += moved * v.w;
                    }
                    if (live && !last) *out = make_float4(a[0], a[1], a[2], a[3]);
                    if (!last) a[0] = a[1] = a[2] = a[3] = 0.0f;
                    ga_tmem_st4(tm + ch, a);
                }
                moved = 1.0f;
            }
        }
        // ---- end of the segment
        wait(&sm.k_free[kGaRounds - 1], (blk - 1) & 1u);
        tc_fence_after();
        const int tok = row >> 4, h = row & 15;
        const bool live = tok < s.ntok;
        if (half == 1) sm.l[row] = l;
        ga_pair_bar(pair_bar);
        if (half == 0) sm.l[row] = l += sm.l[row];
        ga_pair_bar(pair_bar);
        l = sm.l[row];
        if (s.k0 > 0 || s.k1 < s.blocks) {
            // the sums in registers leave in pairs: as fours they would cost spilled registers
            const int64_t slot = 2 * blockIdx.x + (seg_no > 0);
            float2 *po = partial();
            if (live && half == 0) A.part_ml[(slot * A.tok_slots + tok) * kHeads + h] = make_float2(m, l);
#pragma unroll 1
            for (int c = 0; c < kGaTmemCh / 2; c += 16) {
                float a[16];
                tmem_ld16(tm + half * (kGaTmemCh / 2) + c, a);
                float2 *to = po + (half * (kGaTmemCh / 2) + c) / 4 * (2 * kHeads);
                if (live)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        *reinterpret_cast<float4 *>(to + i * (2 * kHeads)) = make_float4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
            }
            if (live)
#pragma unroll
                for (int i = 0; i < kGaRegs / 2; ++i)
                    po[(ga_reg_channel(2 * i & ~15, half) + (2 * i & 15)) / 4 * (2 * kHeads) + (i & 1)] = acc[i];
        } else {
            // the whole row tile: join the token's own part and write it
            const int64_t r = static_cast<int64_t>(s.tok0 + (live ? tok : 0)) * kHeads + h;
            const float lo = A.lse_own ? __ldg(A.lse_own + r) * 1.4426950408889634f : -INFINITY;
            const float top = fmaxf(m, lo), ref = top == -INFINITY ? 0.0f : top;
            const float wk = ga_ex2(m - ref), wo = ga_ex2(lo - ref);
            const float sum = l * wk + wo;
            const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;     // a NaN stays one
            const float fk = wk * inv, fo = wo > 0.0f ? wo * inv : 0.0f;   // nothing to read without an own part
            if (live && half == 0)
                A.lse[r] = sum == 0.0f ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
#pragma unroll 1
            for (int c = 0; c < kGaTmemCh / 2; c += 16) {
                float a[16];
                tmem_ld16(tm + half * (kGaTmemCh / 2) + c, a);
                if (live) ga_write16(A, r, half * (kGaTmemCh / 2) + c, a, fk, fo);
            }
            if (live)
#pragma unroll
                for (int j = 0; j < kGaRegs; j += 16)
                    ga_write16(A, r, ga_reg_channel(j, half), reinterpret_cast<const float *>(acc) + j, fk, fo);
        }
        tc_fence_before();
        ++seg_no;
    }
}

// Walks the blocks of a range's segments with entries, one ahead with the page.
struct GaBlocks {
    GaWalk<GaWide> walk;
    GaSeg s;
    int kb, page;                      // the block at hand; its page
    __device__ __forceinline__ bool segment(const GaArgs &A) {
        do {
            if (!walk.next(A, s)) return false;
        } while (s.T == 0);
        kb = s.k0;
        page = __ldg(A.page_table + static_cast<int64_t>(s.g) * A.max_pages + kb);
        return true;
    }
    // The page of the block at hand (-1: none); moves the page on to the next block of the segment.
    __device__ __forceinline__ int take(const GaArgs &A) {
        const int now = page >= 0 && page < A.num_pages ? page : -1;
        if (kb + 1 < s.k1) page = __ldg(A.page_table + static_cast<int64_t>(s.g) * A.max_pages + kb + 1);
        return now;
    }
    __device__ __forceinline__ bool next(const GaArgs &A) { return ++kb < s.k1 || segment(A); }
};

// Six warps each fill the same half (32 keys) of one chunk of every round, two
// 16-byte loads per lane. A round's loads for the next block are issued as soon
// as it has been converted, so they have a block's time; with one round less in
// flight each round waited for L2 (900 cycles). A warp passes every phase of the
// barriers it waits for, so their parity is enough.
// Eight E2M1 codes of a word -> four f16x2, without moving the bytes apart first.
__device__ __forceinline__ void ga_e2m1x8(uint32_t w, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

struct GaRaw {
    uint4 v[2];                        // 32 channels of two keys
    uint32_t s[2];                     // their two scales each
};

__device__ __forceinline__ void ga_dequant(const GaArgs &A, GaSmem &sm, GaWalk<GaWide> walk, int warp, int lane) {
    const int place = warp % 3, key = 32 * (warp / 3) + (lane & 15), part = lane >> 4;   // the lane's first key, and 16 on
    uint8_t *const dst0 = sm.k + 4 * part * kGaKSlab + key * 16;
    auto chunk_of = [&](int round) { return place < 2 ? 2 * round + place : 6 + round; };
    const uint8_t *codes = nullptr, *scales = nullptr;
    GaWait wait;
    GaBlocks b = {walk, {}, 0, 0};
    int left = 0;
    auto open = [&]() {                                            // the block at hand
        const int page = b.take(A);
        if (page < 0 && b.s.T > b.kb * kGaBlk) flag_status(kStatusBounds);
        left = page < 0 ? 0 : b.s.T - b.kb * kGaBlk - key;
        const int64_t slot = static_cast<int64_t>(max(page, 0)) * kPage + key;
        codes = A.kv_fp4 + slot * kFp4Bytes + 16 * part;
        scales = A.kv_scale + slot * kScaleBytes + 2 * part;
    };
    GaRaw raw[kGaRounds];
    auto fetch = [&](int i) {
        const int c = chunk_of(i);
        // unconditional, so that nothing waits for them here: the rows are in the page whether they count or not
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            raw[i].v[k] = __ldg(reinterpret_cast<const uint4 *>(codes + 16 * k * kFp4Bytes + 32 * c));
            raw[i].s[k] = __ldg(reinterpret_cast<const uint16_t *>(scales + 16 * k * kScaleBytes + 4 * c));
        }
    };
    bool more = b.segment(A);
    if (!more) return;
    open();
#pragma unroll
    for (int i = 0; i < kGaRounds; ++i) fetch(i);
    uint32_t phase = 1u;                                           // of free: passes at once for the first block
    while (more) {
        const int count = left;                                    // keys that count from this lane's first on
        more = b.next(A);
        if (more) open();
#pragma unroll
        for (int i = 0; i < kGaRounds; ++i) {
            GaRaw &r = raw[i];
            wait(&sm.k_free[i], phase);
            uint8_t *dst = dst0 + chunk_of(i) * (8 * kGaKSlab);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const bool ok = count > 16 * k;                    // entries that do not count are zeros
                const uint32_t s2 = ok ? e4m3x2_to_f16x2(r.s[k]) : 0u;
                const uint32_t sa = __byte_perm(s2, s2, 0x1010), sb = __byte_perm(s2, s2, 0x3232);
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    const uint32_t w = (&r.v[k].x)[v], f = v < 2 ? sa : sb;
                    uint32_t h[4];
                    ga_e2m1x8(w, h);
                    *reinterpret_cast<uint4 *>(dst + v * kGaKSlab + k * 256) =
                        make_uint4(hmul2_u32(h[0], f), hmul2_u32(h[1], f), hmul2_u32(h[2], f), hmul2_u32(h[3], f));
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.k_full[i]);
            if (more) fetch(i);
        }
        phase ^= 1u;
    }
}

// The tensor memory address is 0: all of it is allocated. K-major operands:
// leading offset along K (8 channels), stride offset along the rows; MN-major
// (V): along the keys, along the channels.
// kN channels of V (at v_lo) into columns d, over the block's 64 keys.
template <int kN>
__device__ __forceinline__ void ga_pv(uint32_t one, uint32_t d, uint32_t v_lo, uint32_t accumulate) {
    constexpr uint32_t id = umma_idesc(kGaRows, kN, false, true), hi = ga_desc_hi(kGaKSlab);
    ga_mma_ts<id, kGaPCol, 0, hi>(one, d, v_lo, accumulate);
    ga_mma_ts<id, kGaPCol + 8, 16, hi>(one, d, v_lo, 1u);
    ga_mma_ts<id, kGaPCol + 16, 32, hi>(one, d, v_lo, 1u);
    ga_mma_ts<id, kGaPCol + 24, 48, hi>(one, d, v_lo, 1u);
}

__device__ __forceinline__ void ga_mma(const GaArgs &A, GaSmem &sm, GaWalk<GaWide> walk) {
    const uint32_t one = ga_elect() ? 1u : 0u;
    const uint32_t d_q = ga_desc_lo(sm.q, kGaQSlab), d_k = ga_desc_lo(sm.k, kGaKSlab), d_v = ga_desc_lo(sm.k, 128);
    GaWait wait;
    uint32_t blk = 0, tile_no = 0;
    GaSeg s;
    while (walk.next(A, s)) {
        if (s.T == 0) continue;
        wait(&sm.q_full, tile_no & 1u);
        ++tile_no;
        for (int kb = s.k0; kb < s.k1; ++kb, ++blk) {
            const uint32_t par = blk & 1u, acc = kb > s.k0;
            constexpr uint32_t id = umma_idesc(kGaRows, kGaBlk, false, false), hi = ga_desc_hi(128);
            constexpr uint32_t da = 2 * kGaQSlab >> 4, db = 2 * kGaKSlab >> 4, dv = 8 * kGaKSlab >> 4;   // 16, 16 and 64 channels
#pragma unroll 1
            for (int r = 0; r < kGaRounds; ++r) {
                wait(&sm.k_full[r], par);
                tc_fence_after();                                  // S's columns have been read
#pragma unroll 1
                for (int j = 0; j < 3; ++j) {
                    const int c = j < 2 ? 2 * r + j : 6 + r;
                    const uint32_t a = d_q + c * (4 * da), b = d_k + c * (4 * db);
                    ga_mma_ss<id, 0, hi, 0, hi>(one, kGaSCol, a, b, r + j > 0);
                    ga_mma_ss<id, da, hi, db, hi>(one, kGaSCol, a, b, 1u);
                    ga_mma_ss<id, 2 * da, hi, 2 * db, hi>(one, kGaSCol, a, b, 1u);
                    ga_mma_ss<id, 3 * da, hi, 3 * db, hi>(one, kGaSCol, a, b, 1u);
                }
            }
            ga_commit(one, &sm.s_full);
            wait(&sm.p_full, par);
            tc_fence_after();
            // O in parts of 128 channels between the pieces (64 columns of S's and 32 of their own, twice), so that
            // 400 cycles of other MMAs lie between a piece and the next use of its columns
#pragma unroll 1
            for (uint32_t h = 0; h < 2; ++h) {
                if (h > 0) {
                    wait(&sm.ds_empty, par);
                    tc_fence_after();
                }
                ga_pv<64>(one, kGaSCol, d_v + 6 * dv + h * (3 * dv / 2), 0u);
                ga_commit(one, &sm.ds_full);
                if (h > 0) {                                       // the first one: p_full said that it is free
                    wait(&sm.dd_empty, par);
                    tc_fence_after();
                }
                ga_pv<32>(one, kGaDCol, d_v + 7 * dv + h * (3 * dv / 2), 0u);
                ga_commit(one, &sm.dd_full);
                ga_pv<128>(one, 128 * h, d_v + h * (2 * dv), acc);
                ga_commit(one, &sm.k_free[h]);                     // chunks 2 h, 2 h + 1 and 6 + h
            }
            ga_pv<128>(one, 256, d_v + 4 * dv, acc);
            ga_commit(one, &sm.k_free[2]);                         // 4, 5 and 8
        }
    }
    // every MMA of this CTA is done before tensor memory goes back
    if (blk > 0) wait(&sm.k_free[kGaRounds - 1], (blk - 1) & 1u);
}

template <bool kMoves>
__global__ void __launch_bounds__(kGaThreads, 1)
group_attn_kernel(const GaArgs A) {
    extern __shared__ __align__(1024) uint8_t ga_raw[];
    GaSmem &sm = *reinterpret_cast<GaSmem *>(ga_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        mbar_init(&sm.q_full, 1);
        mbar_init(&sm.s_full, 1);
        mbar_init(&sm.p_full, kGaSoftWarps);
        mbar_init(&sm.ds_full, 1);
        mbar_init(&sm.ds_empty, kGaSoftWarps);
        mbar_init(&sm.dd_full, 1);
        mbar_init(&sm.dd_empty, kGaSoftWarps);
        for (int i = 0; i < kGaRounds; ++i) {
            mbar_init(&sm.k_full[i], i == 0 ? kGaDeqWarps + kGaSoftWarps : kGaDeqWarps);
            mbar_init(&sm.k_free[i], 1);
        }
        fence_mbar_init();
    }
    pdl_wait();
    ga_locate<GaWide>(A, sm);
    __syncthreads();
    const int64_t total = sm.total;
    const int ranges = static_cast<int>(min(static_cast<int64_t>(gridDim.x), total));
    if (blockIdx.x == 0 && tid == 0) {
        A.plan->total = total;
        A.plan->ranges = ranges;
    }
    if (static_cast<int>(blockIdx.x) >= ranges) return;
    if (tid == 0) ga_begin<GaWide>(A, sm, total, ranges);
    if (warp == kGaMmaWarp) {
        tmem_alloc(&sm.tmem, 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const GaWalk<GaWide> walk = sm.walk;
    if (warp < kGaSoftWarps) {
        ga_regs_up<kGaSoftRegs>();
        ga_softmax<kMoves>(A, sm, walk, warp, lane);
    } else {
        ga_regs_down<kGaOtherRegs>();
        if (warp == kGaMmaWarp)
            ga_mma(A, sm, walk);
        else if (warp < kGaDeqWarp + kGaDeqWarps)
            ga_dequant(A, sm, walk, warp - kGaDeqWarp, lane);
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
