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

#include <cuda_fp4.h>

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
// One CTA takes 8 tokens: 36 threads per token, one per 16-channel group, and
// one more warp whose 4 lanes per token take the indexer key. The rotated
// channels go through shared memory first (pair by pair, all threads), because
// a pair may lie in two groups and its angle serves the indexer key as well
// when both rows are rotated by the same frequencies.
constexpr int kApTok = 8;
constexpr int kApGroups = kDim / kGroup;                          // 36
constexpr int kApLatent = kApTok * kApGroups;                     // 288
constexpr int kApThreads = kApLatent + kApTok * 4;                // 320

struct AppendArgs {
    const uint16_t *x;                 // [n][x_stride] bf16
    int64_t x_stride, n;
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

// Rounds a positive value to 12 significant bits. A bf16 magnitude over an
// E4M3 scale, and a sixth of one, either equals a rounding midpoint of the
// code or lies at least 2^-8 of it away (both sides are integers of at most 8
// bits up to a power of two). So after this step a quotient taken with an
// approximate reciprocal (2^-22) sits exactly on its midpoint or on its right
// side, and the conversion's round-to-nearest-even decides as it would for the
// exact quotient.
__device__ __forceinline__ float snap12(float v) {
    return __uint_as_float((__float_as_uint(v) + 0x800u) & 0xfffff000u);
}

// 16 bf16 channels (8 pairs) -> 8 bytes of E2M1 codes and the E4M3 scale byte.
__device__ __forceinline__ uint2 fp4_group(const uint32_t (&w)[8], uint32_t &scale_byte) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    const float amax = __uint_as_float(max(m & 0xffff0000u, m << 16));
    scale_byte = static_cast<uint32_t>(__nv_cvt_float_to_fp8(snap12(amax * (1.0f / 6.0f)), __NV_SATFINITE, __NV_E4M3));
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(scale_byte), __NV_E4M3)));
    const float r = s > 0.0f ? rcp_approx(s) : 0.0f;
    uint32_t packed[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint32_t c = 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = w[4 * h + i];
            const float a = snap12(__uint_as_float(v << 16) * r), b = snap12(__uint_as_float(v & 0xffff0000u) * r);
            c |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest)) << (8 * i);
        }
        const uint32_t mag = c & 0x77777777u;                     // a zero magnitude keeps no sign
        const uint32_t some = (mag | (mag >> 1) | (mag >> 2)) & 0x11111111u;
        packed[h] = mag | (c & (some << 3));
    }
    return make_uint2(packed[0], packed[1]);
}

__global__ void __launch_bounds__(kApThreads)
append_kv_rope_kernel(const AppendArgs A) {
    __shared__ uint16_t s_x[kApTok][kDim];                        // rotated channels, at their place
    __shared__ uint16_t s_k[kApTok][kIdxDim];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x;
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * kApTok;
    const bool latent = tid < kApLatent;
    const int lt = latent ? tid / kApGroups : (tid - kApLatent) >> 2;    // token of the CTA
    const int g = latent ? tid - lt * kApGroups : tid & 3;               // 16-channel group, or quarter of the key
    const int64_t tok = tok0 + lt;

    // this thread's 16 channels (the key's quarter g: channels 8g .. 8g + 7 and 32 + 8g .. 32 + 8g + 7)
    uint32_t w[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
    int64_t slot = -1;
    const bool mine = tok < A.n && (latent || A.k != nullptr);
    if (mine) {
        const uint4 *src = reinterpret_cast<const uint4 *>(latent ? A.x + tok * A.x_stride : A.k + tok * A.k_stride);
        const uint4 v0 = __ldg(src + (latent ? 2 * g : g)), v1 = __ldg(src + (latent ? 2 * g + 1 : 4 + g));
        w[0] = v0.x; w[1] = v0.y; w[2] = v0.z; w[3] = v0.w;
        w[4] = v1.x; w[5] = v1.y; w[6] = v1.z; w[7] = v1.w;
        slot = A.slots[tok];
        const int32_t pos = A.pos[tok];
        if (slot >= 0 && (slot >= A.n_slots || pos < 0 || pos >= kRopeMaxPos)) {
            flag_status(kStatusBounds);
            slot = -1;
        }
    }

    // rotation, one pair per thread and pass
    const int pairs = A.rope.half + (A.shared_angles ? 0 : A.krope.half);
    for (int p = tid; p < kApTok * pairs; p += kApThreads) {
        const int t = p / pairs;
        int i = p - t * pairs;
        if (tok0 + t >= A.n) break;                               // later pairs lie in later tokens
        const int32_t pos = A.pos[tok0 + t];
        const bool of_x = i < A.rope.half;
        if (!of_x) i -= A.rope.half;
        double sn, cs;
        rope_sincos(pos, __ldg((of_x ? A.rope.inv_freq : A.krope.inv_freq) + i), sn, cs);
        if (of_x) {
            const int c = A.rope.first(i), d = A.rope.step();
            const uint16_t *src = A.x + (tok0 + t) * A.x_stride + c;
            const uint32_t v = rope_pair(__ldg(src), __ldg(src + d), sn, cs);
            s_x[t][c] = static_cast<uint16_t>(v);
            s_x[t][c + d] = static_cast<uint16_t>(v >> 16);
        }
        if (!of_x || (A.shared_angles && i < A.krope.half)) {
            const int c = A.krope.first(i), d = A.krope.step();
            const uint16_t *src = A.k + (tok0 + t) * A.k_stride + c;
            const uint32_t v = rope_pair(__ldg(src), __ldg(src + d), sn, cs);
            s_k[t][c] = static_cast<uint16_t>(v);
            s_k[t][c + d] = static_cast<uint16_t>(v >> 16);
        }
    }
    __syncthreads();

    // rotated channels replace the loaded ones
    {
        const RopeArgs &R = latent ? A.rope : A.krope;
        const int lo = R.offset, hi = R.offset + 2 * R.half;
        const uint16_t *rot = latent ? s_x[lt] : s_k[lt];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int c0 = latent ? 16 * g + 8 * h : 32 * h + 8 * g;
            if (c0 + 8 <= lo || c0 >= hi) continue;
#pragma unroll
            for (int i = 0; i < 4; ++i) {                         // offset and dim are even: pairs of channels
                const int c = c0 + 2 * i;
                if (c >= lo && c < hi) w[4 * h + i] = *reinterpret_cast<const uint32_t *>(rot + c);
            }
        }
    }
    if (latent) {
        if (slot < 0) return;
        uint32_t sb;
        const uint2 packed = fp4_group(w, sb);
        *reinterpret_cast<uint2 *>(A.kv_fp4 + slot * kFp4Bytes + g * 8) = packed;
        A.kv_scale[slot * kScaleBytes + g] = static_cast<uint8_t>(sb);
    } else if (A.k != nullptr) {                                  // the whole warp, for the shuffles of a row's lanes
        float sigma;
        uint32_t o[4];
        fp8_row_codes(w, 0xfu << (threadIdx.x & 28), sigma, o);
        if (slot < 0) return;
        const int r = static_cast<int>(slot % kPage);
        uint8_t *dst = A.kidx + (slot / kPage) * kKidxPageBytes + (r >> 3) * 512 + (r & 7) * 16;
        // quarter g of the row: 8 bytes of 16-channel block g / 2 and 8 of block 2 + g / 2
        *reinterpret_cast<uint2 *>(dst + (g >> 1) * 128 + (g & 1) * 8) = make_uint2(o[0], o[1]);
        *reinterpret_cast<uint2 *>(dst + (2 + (g >> 1)) * 128 + (g & 1) * 8) = make_uint2(o[2], o[3]);
        if (g == 0) A.kidx_scale[slot] = sigma;
    }
}

inline cudaError_t launch_append_kv_rope(const AppendArgs &A, cudaStream_t stream) {
    return launch_pdl(append_kv_rope_kernel, dim3(static_cast<unsigned>((A.n + kApTok - 1) / kApTok)), dim3(kApThreads),
                      0, stream, A);
}

// ------------------------------------------------------------------ K11
// Query rows [n][heads][dim], in place or to another tensor. A token's angles
// serve all its heads: a CTA computes them once for the tokens it takes, then
// rotates pair by pair and, to another tensor, copies the other channels.
constexpr int kRrThreads = 256;
constexpr int kRrPairs = 320;                                     // angles held by a CTA (dim / 2 <= 288)

struct RopeRowsArgs {
    const uint16_t *x;
    uint16_t *out;
    int64_t x_stride, out_stride, n;   // elements from token to token
    int heads, dim, tokens;            // tokens per CTA
    const int32_t *pos;
    RopeArgs rope;
};

__global__ void __launch_bounds__(kRrThreads)
rope_rows_kernel(const RopeRowsArgs A) {
    __shared__ double2 s_cs[kRrPairs];                            // (cos, sin) of (token, pair)
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, half = A.rope.half;
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * A.tokens;
    const int nt = static_cast<int>(min(static_cast<int64_t>(A.tokens), A.n - tok0));
    for (int p = tid; p < nt * half; p += kRrThreads) {
        const int t = p / half, i = p - t * half;
        const int32_t pos = A.pos[tok0 + t];
        if (i == 0 && (pos < 0 || pos >= kRopeMaxPos)) flag_status(kStatusBounds);
        double sn, cs;
        rope_sincos(pos, __ldg(A.rope.inv_freq + i), sn, cs);
        s_cs[p] = make_double2(cs, sn);
    }
    __syncthreads();
    auto ok = [&](int t) {
        const int32_t pos = A.pos[tok0 + t];
        return pos >= 0 && pos < kRopeMaxPos;
    };
    // pairs, head by head
    const int per_tok = A.heads * half;
    for (int p = tid; p < nt * per_tok; p += kRrThreads) {
        const int t = p / per_tok, q = p - t * per_tok, h = q / half, i = q - h * half;
        if (!ok(t)) continue;
        const int c = h * A.dim + A.rope.first(i), d = A.rope.step();
        const uint16_t *src = A.x + (tok0 + t) * A.x_stride + c;
        uint16_t *dst = A.out + (tok0 + t) * A.out_stride + c;
        const double2 a = s_cs[t * half + i];
        const uint32_t v = rope_pair(src[0], src[d], a.y, a.x);
        dst[0] = static_cast<uint16_t>(v);
        dst[d] = static_cast<uint16_t>(v >> 16);
    }
    if (A.out == A.x) return;
    // the channels that are not rotated
    const int lo = A.rope.offset, hi = lo + 2 * half, rest = A.dim - 2 * half;
    for (int p = tid; p < nt * A.heads * (rest / 2); p += kRrThreads) {
        const int t = p / (A.heads * (rest / 2)), q = p - t * A.heads * (rest / 2), h = q / (rest / 2);
        if (!ok(t)) continue;
        int c = 2 * (q - h * (rest / 2));
        if (c >= lo) c += hi - lo;
        *reinterpret_cast<uint32_t *>(A.out + (tok0 + t) * A.out_stride + h * A.dim + c) =
            *reinterpret_cast<const uint32_t *>(A.x + (tok0 + t) * A.x_stride + h * A.dim + c);
    }
}

inline cudaError_t launch_rope_rows(RopeRowsArgs A, cudaStream_t stream) {
    A.tokens = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kRrPairs / A.rope.half, 8)));
    return launch_pdl(rope_rows_kernel, dim3(static_cast<unsigned>((A.n + A.tokens - 1) / A.tokens)), dim3(kRrThreads),
                      0, stream, A);
}

}  // namespace csa2
