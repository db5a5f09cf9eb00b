// cache_write_fp8.cuh -- the key rows of new tokens in 8 bits: the indexer key (e4m3 with an
// fp32 or a ue8m0 scale, or bf16) and the MLA latent (640 e4m3 codes and one ue8m0 scale).
// The norms and rotations are those of cache_write.cuh:
//   k   = RoPE_half(LayerNorm(k_raw) * ln_w + ln_b)            pairs (i, i + 32), i < 32
//   lat = kv_raw[:512] / rms * rms_w      rot = RoPE_interleaved(kv_raw[512:])
// and the quantisation, with Q = round to the nearest e4m3 number (ties to even):
//   s  = the smallest power of two with |lat| <= 448 s and |rot| <= 16 * 448 s
//   codes[0:512] = Q(lat / s)    hi = Q(rot / (16 s))    lo = Q(rot / (16 s) - hi)
// The RoPE dims take two codes (8 significant bits, like the bf16 they replace) because they
// carry positions in every head's score; the factor 16 keeps a token whose RoPE dims are
// larger than its normalised latent from coarsening the scale of the latent.
//
// A code is decided by which side of a border a value falls on; the codes are those of an
// evaluation in fp64.  The key and the RoPE dims (6 of a lane's 22 values) are evaluated in
// fp64 and rounded once: a value is taken to fp32 by rounding to odd, which cannot move it
// onto or across a border of the 4-bit significands, and from there (power-of-two scaling is
// exact) to e4m3.  The 512 latent dims go in fp32 with a bound on their error (below); a token
// with a value too near a border, or out of the bound's range, is evaluated again in fp64.
// The border cases are 2 % of the tokens; fp64 for all cost 29.4 us at 32768 tokens, much of
// it conversions between the formats, which run at 8 cycles a warp instruction.
// One warp per token; lane i owns RoPE pair i of both parts, so the angle it evaluates needs
// no exchange.  1.4 KB read and 0.8 KB written per token: 10.9 us at 32768 tokens and the copy
// bandwidth; measured 21.8 us, bound by issue (about 500 instructions a token, of them the fp64
// sine and cosine 1.5 us) and by what a token's chain of loads, sums and roots leaves uncovered.
// 64 tokens: 3.0 us.
#pragma once

#include "cache_write.cuh"
#include "dsa_common.cuh"

namespace dsa {
namespace cache {

constexpr int KV8_CODES = 640;        // 512 latent + 64 RoPE hi + 64 RoPE lo
constexpr float KV8_ROPE_GAIN = 16.0f;

__device__ __forceinline__ double warp_sum_d(double v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// fp64 -> fp32, rounded to odd (truncated, last bit set where that lost something).
__device__ __forceinline__ float round_odd(double v) {
    const float f = __double2float_rz(v);
    const uint32_t lost = (__double2loint(v) & 0x1fffffff) != 0 ? 1u : 0u;
    return __uint_as_float(__float_as_uint(f) | lost);
}

// Largest |v| as bits (NaN above infinity above every number), over the warp.
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t warp_max_u(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

// Biased exponent byte of the smallest power of two s with amax <= 448 s, at least 2^-126
// (byte 1); 255 (NaN) for a row that holds an infinity or a NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 255u;
    // 448 = 1.75 * 2^8: the exponent of amax less 8, one more where its significand is above 1.75
    const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return (uint32_t)(e < 1 ? 1 : e);
}
// 1 / 2^(byte - 127); NaN for the NaN byte.  Bytes 1 .. 247 (amax is finite) give 2^126 .. 2^-120.
__device__ __forceinline__ float scale_inverse(uint32_t byte) {
    return byte == 255u ? __uint_as_float(0x7fc00000u) : __uint_as_float((254u - byte) << 23);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float e4m3_value(uint32_t code) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
}

constexpr uint32_t WINDOW = 12;       // ulp: the largest error of a latent value in fp32

constexpr int FP8_WARPS = 4;          // (8: 24.4 us at 32768 tokens against 22.6)

enum KeyForm { KEY_BF16 = 0, KEY_E4M3 = 1, KEY_UE8M0 = 2 };

template <int FORM>
__global__ void __launch_bounds__(32 * FP8_WARPS, 8)
cache_write_fp8_kernel(int n, const __nv_bfloat16 *__restrict__ k_raw, const __nv_bfloat16 *__restrict__ kv_raw,
                       const int32_t *__restrict__ pos, const int32_t *__restrict__ rows,
                       const float *__restrict__ ln_w, const float *__restrict__ ln_b,
                       const float *__restrict__ rms_w, const float *__restrict__ inv_freq, float eps,
                       unsigned char *__restrict__ k_cache, void *__restrict__ k_scale,
                       unsigned char *__restrict__ kv_cache, unsigned char *__restrict__ kv_scale, int n_rows) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * FP8_WARPS + (threadIdx.x >> 5);
    if (t >= n) return;                                       // whole warp
    // ---- loads, all before the first use: indexer key dims lane + 32 j; latent dims 4 lane + 128 j
    // and the 3 after; RoPE pair `lane`
    const int64_t row = __ldg(rows + t);
    const int p = __ldg(pos + t);
    uint16_t xr[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) xr[j] = __ldg(reinterpret_cast<const uint16_t *>(k_raw) + (int64_t)t * 128 + lane + 32 * j);
    const uint2 *src = reinterpret_cast<const uint2 *>(kv_raw + (int64_t)t * 576);
    uint2 zw[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) zw[j] = __ldg(src + lane + 32 * j);
    const uint32_t zr = __ldg(reinterpret_cast<const uint32_t *>(src + 128) + lane);
    double sn, cs;
    sincos((double)p * (double)__ldg(inv_freq + lane), &sn, &cs);
    if (!row_in_cache(row, n_rows, lane)) return;
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __uint_as_float((uint32_t)xr[j] << 16);

    // ---- indexer key
    {
        // Sum x and sum x^2 in one reduction: lanes 0-15 end with the first, 16-31 with the second,
        // then they swap.  The variance loses nothing by the difference: while the exponents of x lie
        // within 15 binades both sums are exact (8-bit significands), and fma rounds once; beyond, some
        // x is far from the largest, the variance is at least 2^-9 of the mean square, and the error 2^-41.
        double y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = x[j];
        const double s1 = (y[0] + y[1]) + (y[2] + y[3]);
        const double s2 = fma(y[0], y[0], y[1] * y[1]) + fma(y[2], y[2], y[3] * y[3]);
        const bool upper = lane >= 16;
        double keep = (upper ? s2 : s1) + __shfl_xor_sync(0xffffffffu, upper ? s1 : s2, 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) keep += __shfl_xor_sync(0xffffffffu, keep, o);
        const double other = __shfl_xor_sync(0xffffffffu, keep, 16);
        const double sum = upper ? other : keep, sq = upper ? keep : other;
        const double mean = sum * (1.0 / 128.0);
        double var = fma(-sum, mean, sq) * (1.0 / 128.0);
        var = var < 0.0 ? 0.0 : var;                          // (a NaN stays)
        const double inv = rsqrt(var + (double)eps);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] -= mean;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = fma(y[j] * inv, (double)__ldg(ln_w + lane + 32 * j), (double)__ldg(ln_b + lane + 32 * j));
        const double u = y[0], v = y[1];
        y[0] = u * cs - v * sn;
        y[1] = v * cs + u * sn;
        if (FORM == KEY_BF16) {
            __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(k_cache) + row * 128;
#pragma unroll
            for (int j = 0; j < 4; ++j) dst[lane + 32 * j] = __float2bfloat16_rn(round_odd(y[j]));
        } else {
            float f[4];
            if (FORM == KEY_UE8M0) {
                uint32_t m = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    f[j] = round_odd(y[j]);
                    m = max(m, abs_bits(f[j]));
                }
                const uint32_t byte = scale_byte(warp_max_u(m));
                const float si = scale_inverse(byte);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] *= si;
                if (lane == 0) static_cast<unsigned char *>(k_scale)[row] = (unsigned char)byte;
            } else {
                // fp32 scale amax / 448 (1 for a zero row), from amax in fp64: the largest upper word,
                // then the largest lower word that goes with it; the codes of y / scale in fp64
                uint32_t h = 0, l = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) h = max(h, (uint32_t)__double2hiint(y[j]) & 0x7fffffffu);
                h = warp_max_u(h);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    l = max(l, ((uint32_t)__double2hiint(y[j]) & 0x7fffffffu) == h ? (uint32_t)__double2loint(y[j]) : 0u);
                const double am = __hiloint2double((int)h, (int)warp_max_u(l));
                float sc = am > 0.0 ? (float)(am / 448.0) : 1.0f;
                if (abs_bits((float)am) >= 0x7f800000u) sc = __uint_as_float(0x7fc00000u);
                const double si = 1.0 / (double)sc;
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = round_odd(y[j] * si);
                if (lane == 0) static_cast<float *>(k_scale)[row] = sc;
            }
            unsigned char *dst = k_cache + row * 128;
            const uint32_t c01 = e4m3x2(f[0], f[1]), c23 = e4m3x2(f[2], f[3]);
            dst[lane] = (unsigned char)c01;
            dst[lane + 32] = (unsigned char)(c01 >> 8);
            dst[lane + 64] = (unsigned char)c23;
            dst[lane + 96] = (unsigned char)(c23 >> 8);
        }
    }

    // ---- latent.  A lane's 16 dims lie 128 apart in fours, so that each load of the weights covers
    // whole lines: with 16 in a row the weights' loads alone were 64 of 73 L1 wavefronts a token.
    const double ru = __uint_as_float(zr << 16), rv = __uint_as_float(zr & 0xffff0000u);
    // rot / 16: an exact scaling, so the maximum over both parts is one maximum
    const float r0 = round_odd(ru * cs - rv * sn) * (1.0f / KV8_ROPE_GAIN);
    const float r1 = round_odd(rv * cs + ru * sn) * (1.0f / KV8_ROPE_GAIN);
    const uint32_t mr = max(abs_bits(r0), abs_bits(r1));
    const uint32_t w8[8] = {zw[0].x, zw[0].y, zw[1].x, zw[1].y, zw[2].x, zw[2].y, zw[3].x, zw[3].y};
    float2 z[8];
    float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        z[j] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w8[j]));
        acc[j & 1] = __ffma2_rn(z[j], z[j], acc[j & 1]);
    }
    // In units of 2^-24: the squares are exact, 3 sums here, 2 to one number, 5 over the warp, eps:
    // 11, halved by the square root; rsqrtf 2 ulp = 4; the two products 2: 11.5, or as many ulp.
    const float rinv = rsqrtf(warp_sum_f((acc[0].x + acc[1].x) + (acc[0].y + acc[1].y)) * (1.0f / 512.0f) + eps);
    const float2 rinv2 = make_float2(rinv, rinv);
    uint32_t near = 0xffffffffu;
    float zm = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 wt = __ldg(reinterpret_cast<const float4 *>(rms_w) + lane + 32 * j);
        z[2 * j] = __fmul2_rn(z[2 * j], __fmul2_rn(make_float2(wt.x, wt.y), rinv2));
        z[2 * j + 1] = __fmul2_rn(z[2 * j + 1], __fmul2_rn(make_float2(wt.z, wt.w), rinv2));
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        // every border (of codes and of the scale) has at most 5 significant bits, 19 zeros below;
        // so have infinities, and the NaN of a product, which fmaxf passes over, is 1 below that
        zm = fmaxf(zm, fmaxf(fabsf(z[j].x), fabsf(z[j].y)));
        near = min(near, min((__float_as_uint(z[j].x) + WINDOW) << 13, (__float_as_uint(z[j].y) + WINDOW) << 13));
    }
    uint32_t m = warp_max_u(max(mr, __float_as_uint(zm)));
    // The bound holds for the values that reach a code other than 0 (2^-20 of the largest) if nothing
    // on the way to them was below 2^-126: 2^-40 <= amax <= 2^100 and 2^-30 <= rinv <= 2^30 see to that.
    const bool unsure = near < (2 * WINDOW) << 13 || m < 0x2b800000u || m > 0x71800000u ||
                        !(rinv >= 0x1p-30f && rinv <= 0x1p30f);
    if (__any_sync(0xffffffffu, unsure)) {
        double ss = 0.0;
#pragma unroll 2
        for (int j = 0; j < 8; ++j) {
            const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w8[j]));
            ss = fma((double)v.x, (double)v.x, ss);
            ss = fma((double)v.y, (double)v.y, ss);
        }
        const double rd = 1.0 / sqrt(warp_sum_d(ss) * (1.0 / 512.0) + (double)eps);
        m = mr;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 v = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w8[j]));
            const float2 wt = __ldg(reinterpret_cast<const float2 *>(rms_w) + 2 * lane + 64 * (j >> 1) + (j & 1));
            z[j].x = round_odd((double)v.x * rd * (double)wt.x);
            z[j].y = round_odd((double)v.y * rd * (double)wt.y);
            m = max(m, max(abs_bits(z[j].x), abs_bits(z[j].y)));
        }
        m = warp_max_u(m);
    }
    const uint32_t byte = scale_byte(m);
    const float si = scale_inverse(byte);
    const float2 si2 = make_float2(si, si);
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = __fmul2_rn(z[j], si2);
    unsigned char *dst = kv_cache + row * KV8_CODES;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        reinterpret_cast<uint32_t *>(dst)[lane + 32 * j] =
            e4m3x2(z[2 * j].x, z[2 * j].y) | e4m3x2(z[2 * j + 1].x, z[2 * j + 1].y) << 16;
    const uint32_t hi = e4m3x2(r0 * si, r1 * si);
    // the remainders are exact in fp32 (r has 24 bits, hi the upper ones of them) except for the
    // odd-rounded last bit, far below a border of lo
    const uint32_t lo = e4m3x2(r0 * si - e4m3_value(hi & 0xffu), r1 * si - e4m3_value(hi >> 8));
    reinterpret_cast<uint16_t *>(dst + 512)[lane] = (uint16_t)hi;
    reinterpret_cast<uint16_t *>(dst + 576)[lane] = (uint16_t)lo;
    if (lane == 0) kv_scale[row] = (unsigned char)byte;
}

}  // namespace cache
}  // namespace dsa
