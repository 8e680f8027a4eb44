// mx_decode_bf16.cuh -- exact decode of block-float elements to bf16 in the
// 128-byte-swizzled K-major shared-memory layout that TMA produces and
// tcgen05.mma reads (the prefill GEMM's weights, the attention's MXFP8 cache).
#pragma once

#include "mx_common.cuh"

namespace mx {

__device__ __forceinline__ uint32_t scaled_bf16x2(uint32_t h2, float s)
{
    return f32x2_to_bf16x2(__fmul_rn(f16_lo_to_f32(h2), s), __fmul_rn(f16_hi_to_f32(h2), s));
}

// Exact f16x2 -> bf16x2 of (value * 2^-112) for values decoded from E2M1 or
// E4M3: those are zero or normal f16 numbers with at most 3 mantissa bits
// (f16 bits 7-9), so the f16 exponent and mantissa bits, moved 3 places
// right, are a normal bf16 number 2^-112 times the value (bf16 bias 127 =
// f16 bias 15 + 112) and zero stays zero; the signs are kept in place.
__device__ __forceinline__ uint32_t f16x2_to_bf16x2_m112(uint32_t h2)
{
    return ((h2 & 0x7F807F80u) >> 3) | (h2 & 0x80008000u);
}

__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b)
{
    uint32_t d;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// bf16x2 holding 2^(e-15) twice, for e in [-111, 142] (normal bf16).
__device__ __forceinline__ uint32_t bf16x2_pow2_m15(int e)
{
    const uint32_t b = (uint32_t)(e + 112) << 7;
    return b | (b << 16);
}

__device__ __forceinline__ void store_chunk(uint8_t *row_base, int chunk, int sw, uint32_t x, uint32_t y,
                                            uint32_t z, uint32_t w)
{
    *reinterpret_cast<uint4 *>(row_base + ((chunk ^ sw) << 4)) = make_uint4(x, y, z, w);
}

// Decode 32 elements of one weight row (half `half` of a 64-wide k-block)
// to bf16 and store them as chunks 4*half .. 4*half+3 of the row's 128 bytes
// at `row_base` (row r of a 128-byte-swizzled tile: chunk c at c ^ (r & 7)).
// w[]: the packed codes (4 words for E2M1, 8 for E4M3); sbits: the block
// scale byte (MX) or the two E4M3 scale bytes (NVFP4).
// Fast path: hardware cvt to f16, exact move to bf16 (scaled by 2^-112), one
// bf16 multiply by the block scale times 2^112 (exact: the result has at most
// 6 significant bits and stays a normal bf16 number).  Scales outside its
// range (E8M0 below 2 (10 for MXFP8) or above 142, NaN scales) use exact fp32
// products.
template <int FMT>
__device__ __forceinline__ void qhalf_store(const uint32_t *w, uint32_t sbits, uint8_t *row_base, int half, int sw)
{
    if constexpr (FMT == FMT_MXFP8) {
        const uint32_t e = sbits & 0xFFu;
        // An E4M3 NaN byte (S.1111.111) converts to an f16 NaN, which the
        // exact move would turn into a finite bf16: a half row holding one
        // takes the fp32 path, which keeps it NaN.  (b & 0x7F) + 1 sets bit 7
        // of its byte only for 0x7F, and never carries into the next byte.
        uint32_t nan_probe = 0u;
#pragma unroll
        for (int c = 0; c < 8; ++c) nan_probe |= (w[c] & 0x7F7F7F7Fu) + 0x01010101u;
        if (e - 10u <= 132u && (nan_probe & 0x80808080u) == 0u) {
            const uint32_t m = bf16x2_pow2_m15((int)e);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t h0, h1, h2, h3;
                e4m3x4_to_f16x2(w[2 * c], h0, h1);
                e4m3x4_to_f16x2(w[2 * c + 1], h2, h3);
                store_chunk(row_base, 4 * half + c, sw, bf16x2_mul(f16x2_to_bf16x2_m112(h0), m),
                            bf16x2_mul(f16x2_to_bf16x2_m112(h1), m), bf16x2_mul(f16x2_to_bf16x2_m112(h2), m),
                            bf16x2_mul(f16x2_to_bf16x2_m112(h3), m));
            }
            return;
        }
        const float s = e8m0_to_f32(e);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            store_chunk(row_base, 4 * half + c, sw, scaled_bf16x2(e4m3x2_to_f16x2(w[2 * c]), s),
                        scaled_bf16x2(e4m3x2_to_f16x2(w[2 * c] >> 16), s),
                        scaled_bf16x2(e4m3x2_to_f16x2(w[2 * c + 1]), s),
                        scaled_bf16x2(e4m3x2_to_f16x2(w[2 * c + 1] >> 16), s));
    } else {
        // multiplier of words 0-1 (m0) and 2-3 (m1): one 32-element E8M0
        // block, or two 16-element E4M3 blocks
        uint32_t m0, m1;
        bool fast;
        if constexpr (FMT == FMT_NVFP4) {
            // E4M3 scale s: bf16(s * 2^112) is exact (4 significant bits); NaN codes are 0x7F / 0xFF
            fast = (((sbits & 0x7F7Fu) + 0x0101u) & 0x8080u) == 0u;
            const uint32_t a2 = f16x2_to_bf16x2_m112(e4m3x2_to_f16x2(sbits));
            // a2 holds s * 2^-112: multiply by 2^112 twice to get s * 2^112
            const uint32_t p112 = bf16x2_pow2_m15(127);
            const uint32_t as = bf16x2_mul(bf16x2_mul(a2, p112), p112);
            m0 = (as & 0xFFFFu) | (as << 16);
            m1 = (as >> 16) | (as & 0xFFFF0000u);
        } else {
            const uint32_t e = sbits & 0xFFu;
            fast = e - 2u <= 140u;  // 2 <= e <= 142: products normal bf16
            m0 = m1 = bf16x2_pow2_m15((int)e);
        }
        if (fast) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // word j: elements 8j .. 8j+7 of the half row
                const uint32_t m = j < 2 ? m0 : m1;
                uint32_t h0, h1, h2, h3;
                e2m1x8_to_f16x2(w[j], h0, h1, h2, h3);
                store_chunk(row_base, 4 * half + j, sw, bf16x2_mul(f16x2_to_bf16x2_m112(h0), m),
                            bf16x2_mul(f16x2_to_bf16x2_m112(h1), m), bf16x2_mul(f16x2_to_bf16x2_m112(h2), m),
                            bf16x2_mul(f16x2_to_bf16x2_m112(h3), m));
            }
            return;
        }
        float s0, s1;
        if constexpr (FMT == FMT_NVFP4) {
            const uint32_t a = e4m3x2_to_f16x2(sbits);
            s0 = f16_lo_to_f32(a);
            s1 = f16_hi_to_f32(a);
        } else {
            s0 = s1 = e8m0_to_f32(sbits);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float s = j < 2 ? s0 : s1;
            store_chunk(row_base, 4 * half + j, sw, scaled_bf16x2(e2m1x2_to_f16x2(w[j]), s),
                        scaled_bf16x2(e2m1x2_to_f16x2(w[j] >> 8), s),
                        scaled_bf16x2(e2m1x2_to_f16x2(w[j] >> 16), s),
                        scaled_bf16x2(e2m1x2_to_f16x2(w[j] >> 24), s));
        }
    }
}

}  // namespace mx
