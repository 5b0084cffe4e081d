// rope.cuh -- K10/K11: the position rotation. K10 rotates new tokens' latents
// and indexer keys by their position, quantises them and writes them to their
// slots of the paged cache in one launch; K11 rotates query rows.
//
// Pair i of a rotated row holds channels (a, b): (2i, 2i + 1) when the pairs
// are interleaved, (i, i + dim / 2) when the row is split in halves. With
// theta = position * inv_freq[i]:
//     a' = a cos(theta) - b sin(theta),   b' = a sin(theta) + b cos(theta).
// Angles reach 10^6 rad, where a binary32 product is off by a tenth of a
// radian, so angle, sine, cosine and products are binary64: the product of a
// position below 2^29 and a binary32 frequency is exact, and two fused steps
// of the reduction by 2 pi (its binary64 value, then what that misses) keep it
// to about 1e-16. The result is rounded to binary32 and then to bf16, the type
// of an unrotated row, so rotating and quantising in one launch gives the
// bytes of rotating first and quantising after.
#pragma once

#include "common.cuh"
#include "quant.cuh"

namespace csa2 {

constexpr int64_t kRopeMaxPos = INT64_C(1) << 29;

__device__ __forceinline__ void rope_sincos(int32_t pos, float freq, double &sn, double &cs) {
    const double p = static_cast<double>(pos) * static_cast<double>(freq);
    const double n = rint(p * 0.15915494309189535);                       // 1 / (2 pi)
    double r = fma(-n, 6.283185307179586, p);                             // 2 pi
    r = fma(-n, 2.4492935982947064e-16, r);                               // 2 pi - its binary64 value
    sincospi(r * 0.3183098861837907, &sn, &cs);                           // 1 / pi
}

__device__ __forceinline__ float bf16_f32(uint16_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }

// The rotated pair as two bf16, a' in the low half.
__device__ __forceinline__ uint32_t rope_pair(uint16_t a, uint16_t b, double sn, double cs) {
    const double x = bf16_f32(a), y = bf16_f32(b);
    const float ra = __double2float_rn(fma(x, cs, -(y * sn))), rb = __double2float_rn(fma(x, sn, y * cs));
    const __nv_bfloat162 v = __floats2bfloat162_rn(ra, rb);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Channel of pair i's first element and the distance to its second.
struct RopeArgs {
    const float *inv_freq;
    int half, offset;                  // dim / 2; first rotated channel
    int interleaved;
    __device__ __forceinline__ int first(int i) const { return offset + (interleaved ? 2 * i : i); }
    __device__ __forceinline__ int step() const { return interleaved ? 1 : half; }
};

// ------------------------------------------------------------------ K10
// A warp takes up to 4 tokens by itself, without a barrier: all their rows are
// on the way while it computes the angles. Rotated channels go through shared
// memory (a token at a time, a lane per pair), because a pair may lie in two
// groups and its angle serves the indexer key as well when both rows are
// rotated by the same frequencies. Then a lane quantises one 16-channel group
// of each token, and of the last step, with four groups and the key of every
// token left, 16 lanes take the groups and 16 the keys, 4 lanes per key.
//
// Bound and measured: 128K tokens with keys take 77 us, the HBM floor being 34
// (220 MB at the copy rate) and the instructions' 51 (456 a token at full
// issue, 148 of them for the 32 angles and pairs). A CTA of 8 tokens with a
// barrier between rotation and quantisation took 127; the same as a loop over
// resident CTAs, with the next rows on the way, 275: its one warp of keys held
// up the other nine. 4, 5, 6 and 7 CTAs per SM: 94, 83, 77 and 80 us (spills).
// 64 tokens: 3.9 us from launch to launch.
constexpr int kApTok = 4;
constexpr int kApWarps = 4;
constexpr int kApThreads = 32 * kApWarps;
constexpr int kApCtasPerSm = 6;

struct AppendArgs {
    const uint16_t *x;                 // [n][x_stride] bf16
    int64_t x_stride, n;
    int tokens;                        // per warp, 1 .. kApTok
    const int32_t *pos, *slots;
    RopeArgs rope;
    const uint16_t *k;                 // [n][k_stride] bf16, or null
    int64_t k_stride;
    RopeArgs krope;                    // half = 0: the key is not rotated
    int shared_angles;                 // the key's frequencies are the first ones of the latent's
    uint8_t *kv_fp4, *kv_scale, *kidx;
    float *kidx_scale;
    int64_t n_slots;
};

// Rounds a positive value to 12 significant bits. A sixth of a bf16 magnitude
// either equals a rounding midpoint of E4M3 or lies at least 2^-8 of it away
// (both sides are integers of at most 8 bits up to a power of two). So after
// this step the product with the rounded 1/6 sits exactly on its midpoint or on
// its right side, and the conversion's round-to-nearest-even decides as it
// would for the exact quotient.
__device__ __forceinline__ float snap12(float v) {
    return __uint_as_float((__float_as_uint(v) + 0x800u) & 0xfffff000u);
}

// The same for the quotients x / s, with an approximate reciprocal (2^-22) and
// a grid of 2^-13: E2M1's midpoints are multiples of 1/4, any other quotient is
// at least 2^-10 away from them, and one so large that the grid is coarser is
// far above 6, where the codes end.
__device__ __forceinline__ float2 snap_quotients(float2 x, float r) {
    constexpr float kGrid = 1536.0f;                              // binary32 values around it lie 2^-13 apart
    float2 v;
    asm("{.reg .b64 x, r, c, n, v;\n\t"
        "mov.b64 x, {%2, %3}; mov.b64 r, {%4, %4}; mov.b64 c, {%5, %5}; mov.b64 n, {%6, %6};\n\t"
        "fma.rn.f32x2 v, x, r, c; add.rn.f32x2 v, v, n;\n\t"
        "mov.b64 {%0, %1}, v;}"
        : "=f"(v.x), "=f"(v.y) : "f"(x.x), "f"(x.y), "f"(r), "f"(kGrid), "f"(-kGrid));
    return v;
}

// 16 bf16 channels (8 pairs) -> 8 bytes of E2M1 codes and the E4M3 scale byte.
__device__ __forceinline__ uint2 fp4_group(const uint32_t (&w)[8], uint32_t &scale_byte) {
    uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7fff7fffu));
    const float amax = __uint_as_float(max(m & 0xffff0000u, m << 16));
    scale_byte = static_cast<uint32_t>(__nv_cvt_float_to_fp8(snap12(amax * (1.0f / 6.0f)), __NV_SATFINITE, __NV_E4M3));
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(scale_byte), __NV_E4M3)));
    const float r = s > 0.0f ? rcp_approx(s) : 0.0f;
    uint32_t packed[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float2 q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            q[i] = snap_quotients(make_float2(__uint_as_float(w[4 * h + i] << 16), __uint_as_float(w[4 * h + i] & 0xffff0000u)), r);
        uint32_t c;
        asm("{.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1; cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5; cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};}"
            : "=r"(c) : "f"(q[0].x), "f"(q[0].y), "f"(q[1].x), "f"(q[1].y), "f"(q[2].x), "f"(q[2].y), "f"(q[3].x), "f"(q[3].y));
        const uint32_t mag = c & 0x77777777u;                     // a zero magnitude keeps no sign
        const uint32_t some = (mag | (mag >> 1) | (mag >> 2)) & 0x11111111u;
        packed[h] = mag | (c & (some << 3));
    }
    return make_uint2(packed[0], packed[1]);
}

// The rotated ones of channels [c0, c0 + 8) replace w[0 .. 3].
__device__ __forceinline__ void rope_replace(uint32_t *w, const uint16_t *rot, int c0, int lo, int hi) {
    if (c0 + 8 <= lo || c0 >= hi) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {                                 // offset and dim are even: pairs of channels
        const int c = c0 + 2 * i;
        if (c >= lo && c < hi) w[i] = *reinterpret_cast<const uint32_t *>(rot + c);
    }
}

__global__ void __launch_bounds__(kApThreads, kApCtasPerSm)
append_kv_rope_kernel(const AppendArgs A) {
    __shared__ uint16_t s_xs[kApWarps][kApTok][kDim];             // rotated channels, at their place
    __shared__ uint16_t s_ks[kApWarps][kApTok][kIdxDim];
    pdl_wait();
    pdl_trigger();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tok0 = (static_cast<int64_t>(blockIdx.x) * kApWarps + warp) * A.tokens;
    if (tok0 >= A.n) return;
    const int nt = static_cast<int>(min(static_cast<int64_t>(A.tokens), A.n - tok0));
    uint16_t (*s_x)[kDim] = s_xs[warp];
    uint16_t (*s_k)[kIdxDim] = s_ks[warp];

    // the rows; a key's quarter g is channels 8g .. 8g + 7 and 32 + 8g .. 32 + 8g + 7
    uint32_t w[kApTok][8], wm[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    auto load = [&](uint32_t (&to)[8], const uint16_t *row, int a, int b) {
        const uint4 v0 = __ldg(reinterpret_cast<const uint4 *>(row) + a), v1 = __ldg(reinterpret_cast<const uint4 *>(row) + b);
        to[0] = v0.x; to[1] = v0.y; to[2] = v0.z; to[3] = v0.w;
        to[4] = v1.x; to[5] = v1.y; to[6] = v1.z; to[7] = v1.w;
    };
    const int mt = (lane & 15) >> 2, g = lane & 3;                // token and group, or quarter, of the last step
#pragma unroll
    for (int t = 0; t < kApTok; ++t)
        if (t < nt) load(w[t], A.x + (tok0 + t) * A.x_stride, 2 * lane, 2 * lane + 1);
    if (mt < nt) {
        if (lane < 16)
            load(wm, A.x + (tok0 + mt) * A.x_stride, 64 + 2 * g, 65 + 2 * g);
        else if (A.k != nullptr)
            load(wm, A.k + (tok0 + mt) * A.k_stride, g, 4 + g);
    }
    int32_t slot = -1, pos = 0;                                   // of token `lane`
    if (lane < nt) {
        slot = A.slots[tok0 + lane];
        pos = A.pos[tok0 + lane];
        if (slot >= 0 && (slot >= A.n_slots || pos < 0 || pos >= kRopeMaxPos)) {
            flag_status(kStatusBounds);
            slot = -1;
        }
    }

    // rotation
    const int pairs = A.rope.half + (A.shared_angles ? 0 : A.krope.half);
    for (int p = lane; p < pairs; p += 32) {
        const bool of_x = p < A.rope.half;
        const int i = of_x ? p : p - A.rope.half;
        const bool of_k = !of_x || (A.shared_angles && i < A.krope.half);
        const int xc = A.rope.first(i), xd = A.rope.step(), kc = A.krope.first(i), kd = A.krope.step();
        const float freq = __ldg((of_x ? A.rope.inv_freq : A.krope.inv_freq) + i);
#pragma unroll 1
        for (int t = 0; t < nt; ++t) {
            const uint16_t *x = A.x + (tok0 + t) * A.x_stride + xc, *k = A.k + (tok0 + t) * A.k_stride + kc;
            uint16_t xa = 0, xb = 0, ka = 0, kb = 0;
            if (of_x) xa = __ldg(x), xb = __ldg(x + xd);
            if (of_k) ka = __ldg(k), kb = __ldg(k + kd);
            double sn, cs;
            rope_sincos(A.pos[tok0 + t], freq, sn, cs);
            if (of_x) {
                const uint32_t v = rope_pair(xa, xb, sn, cs);
                s_x[t][xc] = static_cast<uint16_t>(v);
                s_x[t][xc + xd] = static_cast<uint16_t>(v >> 16);
            }
            if (of_k) {
                const uint32_t v = rope_pair(ka, kb, sn, cs);
                s_k[t][kc] = static_cast<uint16_t>(v);
                s_k[t][kc + kd] = static_cast<uint16_t>(v >> 16);
            }
        }
    }
    __syncwarp();

    // rotated channels replace the loaded ones; quantise and write
    const int lo = A.rope.offset, hi = A.rope.offset + 2 * A.rope.half;
    auto put = [&](uint32_t (&v)[8], int t, int group, int64_t at) {
        rope_replace(v, s_x[t], 16 * group, lo, hi);
        rope_replace(v + 4, s_x[t], 16 * group + 8, lo, hi);
        uint32_t sb;
        const uint2 packed = fp4_group(v, sb);
        if (at < 0) return;
        *reinterpret_cast<uint2 *>(A.kv_fp4 + at * kFp4Bytes + group * 8) = packed;
        A.kv_scale[at * kScaleBytes + group] = static_cast<uint8_t>(sb);
    };
#pragma unroll
    for (int t = 0; t < kApTok; ++t) {
        const int32_t at = __shfl_sync(0xffffffffu, slot, t);
        if (t < nt) put(w[t], t, lane, at);
    }
    const int32_t at = __shfl_sync(0xffffffffu, slot, mt);
    if (lane < 16) {
        put(wm, mt, 32 + g, at);
    } else if (A.k != nullptr) {
        rope_replace(wm, s_k[mt], 8 * g, A.krope.offset, A.krope.offset + 2 * A.krope.half);
        rope_replace(wm + 4, s_k[mt], 32 + 8 * g, A.krope.offset, A.krope.offset + 2 * A.krope.half);
        float sigma;
        uint32_t o[4];
        fp8_row_codes(wm, 0xffff0000u, sigma, o);
        if (at >= 0) {
            const uint32_t page = static_cast<uint32_t>(at) / kPage, r = static_cast<uint32_t>(at) % kPage;
            uint8_t *dst = A.kidx + static_cast<int64_t>(page) * kKidxPageBytes + (r >> 3) * 512 + (r & 7) * 16;
            // quarter g of the row: 8 bytes of 16-channel block g / 2 and 8 of block 2 + g / 2
            *reinterpret_cast<uint2 *>(dst + (g >> 1) * 128 + (g & 1) * 8) = make_uint2(o[0], o[1]);
            *reinterpret_cast<uint2 *>(dst + (2 + (g >> 1)) * 128 + (g & 1) * 8) = make_uint2(o[2], o[3]);
            if (g == 0) A.kidx_scale[at] = sigma;
        }
    }
}

inline cudaError_t launch_append_kv_rope(AppendArgs A, int sm_count, cudaStream_t stream) {
    // more tokens per warp once the GPU is full of warps
    A.tokens = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kApTok, A.n / (kApCtasPerSm * kApWarps * sm_count))));
    const int64_t per = kApWarps * A.tokens;
    return launch_pdl(append_kv_rope_kernel, dim3(static_cast<unsigned>((A.n + per - 1) / per)), dim3(kApThreads), 0,
                      stream, A);
}

// ------------------------------------------------------------------ K11
// Query rows [n][heads][dim], in place or to another tensor. A token's angles
// serve all its heads, so a CTA computes them once for the tokens and heads it
// takes. Where the rotated range and the distance within a pair are multiples
// of 8 channels a thread turns 4 pairs at a time, 16 bytes or (when the row is
// split in halves) twice 8, and the first load is in flight while the angles
// are computed; otherwise it goes pair by pair. The other channels are
// copied, to another tensor only, before the angles. A token's heads are shared
// out over CTAs while there are fewer CTAs than the GPU holds.
//
// Measured: 64 tokens of 16 x 576 channels 2.6 us from launch to launch, 16,384
// tokens 134 us (93 by the bytes) and of 4 x 64 channels 8.6 us (2.6 by the
// bytes: three waves of CTAs whose time is the latency of the angles, and the
// conversions to and from binary64, four per pair). Without the early start of
// the next kernel they took 2.9, 135 and 9.7.
constexpr int kRrThreads = 256;
constexpr int kRrTokens = 8;
constexpr int kRrCtasPerSm = 6;                                   // without that start, 128K tokens of 4 x 64 channels: 5 72 us, 6 67, 8 63 but 64 tokens 3.3 against 2.9
constexpr int kRrPairs = 320;                                     // angles held by a CTA (dim / 2 <= 288)

struct RopeRowsArgs {
    const uint16_t *x;
    uint16_t *out;
    int64_t x_stride, out_stride, n;   // elements from token to token
    int heads, dim;
    int tokens, cta_heads;             // of a CTA
    const int32_t *pos;
    RopeArgs rope;
};

template <bool kWide>
__global__ void __launch_bounds__(kRrThreads, kRrCtasPerSm)
rope_rows_kernel(const RopeRowsArgs A) {
    __shared__ double2 s_cs[kRrPairs];                            // (cos, sin) of (token, pair)
    __shared__ bool s_ok[kRrTokens];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, half = A.rope.half, lo = A.rope.offset, h0 = blockIdx.y * A.cta_heads;
    const int nh = min(A.cta_heads, A.heads - h0);
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * A.tokens;
    const int nt = static_cast<int>(min(static_cast<int64_t>(A.tokens), A.n - tok0));
    const uint16_t *x = A.x + tok0 * A.x_stride + h0 * A.dim;
    uint16_t *out = A.out + tok0 * A.out_stride + h0 * A.dim;
    if (tid < nt) {
        const int32_t pos = A.pos[tok0 + tid];
        s_ok[tid] = pos >= 0 && pos < kRopeMaxPos;
        if (!s_ok[tid]) flag_status(kStatusBounds);
    }
    // this thread's first 16 bytes of rotated channels, or first pair
    const int per_row = kWide ? half / 4 : half, items = nt * nh * per_row;
    uint4 v;                                                      // 4 pairs, or one
    int t = 0, i = 0;
    int64_t from = 0, to = 0;
    auto load = [&](int p) {
        const int r = p / per_row, h = r % nh;
        t = r / nh;
        i = p - r * per_row;
        const int c = h * A.dim + (kWide ? lo + (A.rope.interleaved ? 8 : 4) * i : A.rope.first(i));
        from = t * A.x_stride + c;
        to = t * A.out_stride + c;
        if (!kWide) {
            v.x = x[from];
            v.y = x[from + A.rope.step()];
        } else if (A.rope.interleaved) {
            v = *reinterpret_cast<const uint4 *>(x + from);
        } else {
            const uint2 a = *reinterpret_cast<const uint2 *>(x + from), b = *reinterpret_cast<const uint2 *>(x + from + half);
            v = make_uint4(a.x, a.y, b.x, b.y);
        }
    };
    if (tid < items) load(tid);
    for (int p = tid; p < nt * half; p += kRrThreads) {
        const int at = p / half;
        double sn, cs;
        rope_sincos(A.pos[tok0 + at], __ldg(A.rope.inv_freq + p - at * half), sn, cs);
        s_cs[p] = make_double2(cs, sn);
    }
    __syncthreads();
    if (A.out != A.x) {
        if (kWide) {                                              // 8 channels at a time
            const int rest = (A.dim - 2 * half) / 8;
            for (int p = tid; p < nt * nh * rest; p += kRrThreads) {
                const int r = p / rest, ct = r / nh;
                int c = 8 * (p - r * rest);
                if (c >= lo) c += 2 * half;
                c += (r - ct * nh) * A.dim;
                if (s_ok[ct])
                    *reinterpret_cast<uint4 *>(out + ct * A.out_stride + c) = *reinterpret_cast<const uint4 *>(x + ct * A.x_stride + c);
            }
        } else {
            const int rest = A.dim / 2 - half;
            for (int p = tid; p < nt * nh * rest; p += kRrThreads) {
                const int r = p / rest, ct = r / nh;
                int c = 2 * (p - r * rest);
                if (c >= lo) c += 2 * half;
                c += (r - ct * nh) * A.dim;
                if (s_ok[ct])
                    *reinterpret_cast<uint32_t *>(out + ct * A.out_stride + c) = *reinterpret_cast<const uint32_t *>(x + ct * A.x_stride + c);
            }
        }
    }
    for (int p = tid; p < items; p += kRrThreads) {
        if (p != tid) load(p);
        if (!s_ok[t]) continue;
        const double2 *cs = s_cs + t * half + (kWide ? 4 * i : i);
        if (!kWide) {
            const uint32_t w = rope_pair(static_cast<uint16_t>(v.x), static_cast<uint16_t>(v.y), cs[0].y, cs[0].x);
            out[to] = static_cast<uint16_t>(w);
            out[to + A.rope.step()] = static_cast<uint16_t>(w >> 16);
        } else if (A.rope.interleaved) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t &w = (&v.x)[e];
                w = rope_pair(static_cast<uint16_t>(w), static_cast<uint16_t>(w >> 16), cs[e].y, cs[e].x);
            }
            *reinterpret_cast<uint4 *>(out + to) = v;
        } else {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                uint32_t &a = (&v.x)[e], &b = (&v.x)[2 + e];
                const double2 c0 = cs[2 * e], c1 = cs[2 * e + 1];
                const uint32_t v0 = rope_pair(static_cast<uint16_t>(a), static_cast<uint16_t>(b), c0.y, c0.x);
                const uint32_t v1 = rope_pair(static_cast<uint16_t>(a >> 16), static_cast<uint16_t>(b >> 16), c1.y, c1.x);
                a = __byte_perm(v0, v1, 0x5410);
                b = __byte_perm(v0, v1, 0x7632);
            }
            *reinterpret_cast<uint2 *>(out + to) = make_uint2(v.x, v.y);
            *reinterpret_cast<uint2 *>(out + to + half) = make_uint2(v.z, v.w);
        }
    }
}

inline cudaError_t launch_rope_rows(RopeRowsArgs A, int sm_count, cudaStream_t stream) {
    // Few CTAs: one token each and its heads shared out, until every SM has two. Many: several tokens each.
    const int64_t fill = 2 * sm_count;
    A.tokens = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>({A.n / (4 * fill), kRrPairs / A.rope.half, kRrTokens})));
    const int64_t ctas = (A.n + A.tokens - 1) / A.tokens;
    const int splits = static_cast<int>(std::min<int64_t>(A.heads, (fill + ctas - 1) / ctas));
    A.cta_heads = (A.heads + splits - 1) / splits;
    const dim3 grid(static_cast<unsigned>(ctas), (A.heads + A.cta_heads - 1) / A.cta_heads);
    const bool wide = A.rope.offset % 8 == 0 && (A.rope.interleaved ? 2 * A.rope.half : A.rope.half) % 8 == 0;
    return wide ? launch_pdl(rope_rows_kernel<true>, grid, dim3(kRrThreads), 0, stream, A)
                : launch_pdl(rope_rows_kernel<false>, grid, dim3(kRrThreads), 0, stream, A);
}

}  // namespace csa2
