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
// A code is decided by which side of a border a value falls on, so everything up to the code
// is evaluated in fp64 and rounded once: a value is taken to fp32 by rounding to odd, which
// cannot move it onto or across a border of the 4-bit significands, and from there (power-of
// -two scaling is exact) to e4m3.  fp32 all the way would misplace about one code in a
// million.
// HBM-bound at its floor (1.4 KB read and about 0.8 KB written per token).  One warp per
// token; lane i owns RoPE pair i of both parts, so the angle it evaluates needs no exchange.
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

enum KeyForm { KEY_BF16 = 0, KEY_E4M3 = 1, KEY_UE8M0 = 2 };

template <int FORM>
__global__ void __launch_bounds__(32 * WARPS)
cache_write_fp8_kernel(int n, const __nv_bfloat16 *__restrict__ k_raw, const __nv_bfloat16 *__restrict__ kv_raw,
                       const int32_t *__restrict__ pos, const int32_t *__restrict__ rows,
                       const float *__restrict__ ln_w, const float *__restrict__ ln_b,
                       const float *__restrict__ rms_w, const float *__restrict__ inv_freq, float eps,
                       unsigned char *__restrict__ k_cache, void *__restrict__ k_scale,
                       unsigned char *__restrict__ kv_cache, unsigned char *__restrict__ kv_scale) {
    const int lane = threadIdx.x & 31;
    const int t = blockIdx.x * WARPS + (threadIdx.x >> 5);
    if (t >= n) return;                                       // whole warp
    const int64_t row = __ldg(rows + t);
    if (row < 0) return;                                      // a token without a row (padding)
    // ---- loads: indexer key dims lane + 32 j; 16 latent dims; RoPE pair `lane`
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __bfloat162float(k_raw[(int64_t)t * 128 + lane + 32 * j]);
    const uint4 *src = reinterpret_cast<const uint4 *>(kv_raw + (int64_t)t * 576) + 2 * lane;
    const uint4 za = __ldg(src), zb = __ldg(src + 1);
    const __nv_bfloat162 zr = reinterpret_cast<const __nv_bfloat162 *>(kv_raw + (int64_t)t * 576 + 512)[lane];
    double sn, cs;
    sincos((double)__ldg(pos + t) * (double)__ldg(inv_freq + lane), &sn, &cs);

    // ---- indexer key
    {
        const double mean = warp_sum_d(((double)x[0] + x[1]) + ((double)x[2] + x[3])) * (1.0 / 128.0);
        double y[4], ss = 0.0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            y[j] = x[j] - mean;
            ss = fma(y[j], y[j], ss);
        }
        const double inv = 1.0 / sqrt(warp_sum_d(ss) * (1.0 / 128.0) + (double)eps);
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
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (FORM == KEY_UE8M0) f[j] = round_odd(y[j]);
                else f[j] = (float)y[j];
                m = max(m, abs_bits(f[j]));
            }
            m = warp_max_u(m);
            if (FORM == KEY_UE8M0) {
                const uint32_t byte = scale_byte(m);
                const float si = scale_inverse(byte);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] *= si;
                if (lane == 0) static_cast<unsigned char *>(k_scale)[row] = (unsigned char)byte;
            } else {
                // fp32 scale amax / 448 (1 for a zero row): amax in fp64, the codes of y / scale in fp64
                double am = fmax(fmax(fabs(y[0]), fabs(y[1])), fmax(fabs(y[2]), fabs(y[3])));
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) am = fmax(am, __shfl_xor_sync(0xffffffffu, am, o));
                float sc = am > 0.0 ? (float)(am / 448.0) : 1.0f;
                if (m >= 0x7f800000u) sc = __uint_as_float(0x7fc00000u);
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

    // ---- latent: lane holds dims 16 lane .. 16 lane + 15 and RoPE pair `lane`
    const uint32_t w8[8] = {za.x, za.y, za.z, za.w, zb.x, zb.y, zb.z, zb.w};
    float z[16];
    double ss = 0.0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const __nv_bfloat162 h = *reinterpret_cast<const __nv_bfloat162 *>(&w8[j]);
        z[2 * j] = __low2float(h);
        z[2 * j + 1] = __high2float(h);
        ss = fma((double)z[2 * j], (double)z[2 * j], ss);
        ss = fma((double)z[2 * j + 1], (double)z[2 * j + 1], ss);
    }
    const double rinv = 1.0 / sqrt(warp_sum_d(ss) * (1.0 / 512.0) + (double)eps);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float4 wt = __ldg(reinterpret_cast<const float4 *>(rms_w + 16 * lane) + j);
        const float w4[4] = {wt.x, wt.y, wt.z, wt.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            z[4 * j + e] = round_odd((double)z[4 * j + e] * rinv * (double)w4[e]);
            m = max(m, abs_bits(z[4 * j + e]));
        }
    }
    const double ru = __low2float(zr), rv = __high2float(zr);
    // rot / 16: an exact scaling, so the maximum over both parts is one maximum
    const float r0 = round_odd(ru * cs - rv * sn) * (1.0f / KV8_ROPE_GAIN);
    const float r1 = round_odd(rv * cs + ru * sn) * (1.0f / KV8_ROPE_GAIN);
    m = warp_max_u(max(m, max(abs_bits(r0), abs_bits(r1))));
    const uint32_t byte = scale_byte(m);
    const float si = scale_inverse(byte);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        o[j] = e4m3x2(z[4 * j] * si, z[4 * j + 1] * si) | e4m3x2(z[4 * j + 2] * si, z[4 * j + 3] * si) << 16;
    unsigned char *dst = kv_cache + row * KV8_CODES;
    reinterpret_cast<uint4 *>(dst)[lane] = make_uint4(o[0], o[1], o[2], o[3]);
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
