// pack_token.cuh -- one warp packs one token: optional RMSNorm and RoPE of its latent, then FP4 codes and
// E4M3 scales, the E4M3 indexer key and the FP8 window entry (pack.cu states the arithmetic).
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "convert.cuh"

namespace csa {

constexpr int kRopeRow = 64;   // floats of one rotation: 32 (cos, sin) pairs

// A token's inputs, loaded ahead of its arithmetic.
struct PackIn {
    uint4 a, b;     // latent channels 16 lane .. 16 lane + 15 (bf16)
    uint2 kw;       // indexer-key channels 4 lane .. 4 lane + 3 (bf16)
    int64_t s;      // main slot
    int32_t ss;     // window slot
};

// x / c where only its place among borders of few bits counts.  inv: 1 / c rounded, times 1 + 2^-20, so that the product is
// above the quotient, by less than 2^-19 of it; its first 11 significant bits are then those of a quotient that is a
// number t of at most 11 bits, and a quotient that is 2^-8 of itself away from t stays on its side of it.  Zeros keep their
// sign; infinities pass, and a NaN stays one (the product's NaN is 0x7FFFFFFF: rounding it by an addition would carry
// into the sign and leave a zero).
constexpr float kNearAbove = 1.f + 0x1p-20f;

__device__ __forceinline__ float near_quotient(float x, float inv)
{
    return __uint_as_float(__float_as_uint(__fmul_rn(x, inv)) & 0xFFFFE000u);
}

// Pack token `tok` (its number in a report of a bad slot).  kNorm: RMSNorm with weights norm_w first;
// kRope: then rotate channels 448..511 by rope_row, the token's 32 (cos, sin) pairs.
template <bool kNorm, bool kRope>
__device__ __forceinline__ void pack_token(const csa_kv_layer &layer, const PackIn &in, int tok, int lane, void *ws,
                                           const float *__restrict__ norm_w, const float *__restrict__ rope_row)
{
    const int64_t s = in.s;
    const int32_t ss = in.ss;
    const bool main_ok = s >= 0 && s < (int64_t)layer.num_pages * kPage;
    const bool swa_ok = ss >= 0 && ss < layer.num_rows * kWindow;
    if (lane == 0 && (!main_ok || (ss >= 0 && !swa_ok))) report(ws, CSA_ERR_DEVICE_DATA, tok);

    // 16 channels of group `lane`
    const uint32_t w[8] = {in.a.x, in.a.y, in.a.z, in.a.w, in.b.x, in.b.y, in.b.z, in.b.w};
    float x[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
    if (kNorm) {
        float acc = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) acc = __fmaf_rn(x[i], x[i], acc);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) acc = __fadd_rn(acc, __shfl_xor_sync(0xffffffffu, acc, d));
        const float r = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fmul_rn(acc, 1.0f / 512.0f), 1e-6f)));
        const float4 *wp = reinterpret_cast<const float4 *>(norm_w + 16 * lane);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 wv = wp[q];
            x[4 * q] = __fmul_rn(__fmul_rn(x[4 * q], r), wv.x);
            x[4 * q + 1] = __fmul_rn(__fmul_rn(x[4 * q + 1], r), wv.y);
            x[4 * q + 2] = __fmul_rn(__fmul_rn(x[4 * q + 2], r), wv.z);
            x[4 * q + 3] = __fmul_rn(__fmul_rn(x[4 * q + 3], r), wv.w);
        }
    }
    if (kRope && lane >= 28) {   // channels 448..511: pairs 8 (lane - 28) .. 8 (lane - 28) + 7
        const float4 *cp = reinterpret_cast<const float4 *>(rope_row + 16 * (lane - 28));
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float4 c2 = cp[q];   // (cos, sin) of two pairs
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float co = h ? c2.z : c2.x, si = h ? c2.w : c2.y;
                const int m = 2 * q + h;
                const float a = x[2 * m], b = x[2 * m + 1];
                x[2 * m] = __fsub_rn(__fmul_rn(a, co), __fmul_rn(b, si));
                x[2 * m + 1] = __fadd_rn(__fmul_rn(a, si), __fmul_rn(b, co));
            }
        }
    }
    if (kNorm || kRope) {
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __bfloat162float(__float2bfloat16_rn(x[i]));
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));

    if (main_ok) {
        // s = E4M3(amax / 6); codes = E2M1(x / s), or 0 when s decodes to 0, the quotients rounded to binary32
        // first.  near_quotient gives the same bytes as those: the formats' rounding borders t have at most 5
        // (E4M3) and 3 (E2M1) significant bits, so t * 6 and t * s have at most 7, x has 8 (it is a bf16 value),
        // and a quotient that is not exactly t is at least 2^-8 of it away.  (Seventeen divisions less per lane:
        // 65,536 tokens appended with norm and rotation: 80 -> 66 us.)
        const uint8_t sc = (uint8_t)(f32x2_to_e4m3x2(near_quotient(amax, kNearAbove / 6.0f), 0.f) & 0xFF);
        const float sd = e4m3_to_f32(sc);
        uint2 codes = make_uint2(0u, 0u);
        if (sd != 0.f) {
            const float inv = __fmul_rn(__frcp_rn(sd), kNearAbove);
            float y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) y[i] = near_quotient(x[i], inv);
            codes.x = f32x8_to_e2m1x8(y);
            codes.y = f32x8_to_e2m1x8(y + 8);
        }
        reinterpret_cast<uint2 *>(layer.codes + s * kCodeBytes)[lane] = codes;
        layer.scales[s * kScaleBytes + lane] = sc;

        // indexer key: channels 4*lane .. 4*lane+3, plain E4M3 cast
        const uint2 kw = in.kw;
        const uint32_t k01 = f32x2_to_e4m3x2(bf16_lo(kw.x), bf16_hi(kw.x));
        const uint32_t k23 = f32x2_to_e4m3x2(bf16_lo(kw.y), bf16_hi(kw.y));
        reinterpret_cast<uint32_t *>(layer.keys + s * kIdxDim)[lane] = k01 | (k23 << 16);
    }

    if (ss >= 0) {  // warp-uniform
        float m = amax;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (swa_ok) {
            const float scale = __fdiv_rn(m, 448.0f);
            uint32_t v[4] = {0u, 0u, 0u, 0u};
            if (scale != 0.f) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t lo = f32x2_to_e4m3x2(__fdiv_rn(x[4 * i], scale), __fdiv_rn(x[4 * i + 1], scale));
                    const uint32_t hi = f32x2_to_e4m3x2(__fdiv_rn(x[4 * i + 2], scale), __fdiv_rn(x[4 * i + 3], scale));
                    v[i] = lo | (hi << 16);
                }
            }
            reinterpret_cast<uint4 *>(layer.swa + (size_t)ss * kLatent)[lane] = make_uint4(v[0], v[1], v[2], v[3]);
            if (lane == 0) layer.swa_scale[ss] = scale;
        }
    }
}

}  // namespace csa
