// sparse_mla_fp8.cuh -- attention over the selected rows of the 8-bit latent cache
// (cache_write_fp8.cuh gives the row format): MLA in MQA mode, 128 heads, 576-d rows, the
// value is the 512-d latent.
//   z[t,h,i] = sm_scale * q[t,h,:] . kv[idx[t,i], :]     out = softmax(z) . kv[:, 0:512]
// Plain form: one CTA per (token, 16 heads), 32 keys at a time dequantised into shared
// memory, running maximum and sum per head.
#pragma once

#include "cache_write_fp8.cuh"
#include "dsa_common.cuh"
#include "sparse_mla_pair.cuh"

namespace dsa {
namespace mla8 {

constexpr int NT = 256, HG = 16, KC = 32, KVP = 577;
constexpr int SMEM = (HG * 576 + KC * KVP + HG * KC + 3 * HG + KC) * 4;

__global__ void __launch_bounds__(NT)
sparse_mla_fp8_plain_kernel(Problem P, const __nv_bfloat16 *__restrict__ q, const unsigned char *__restrict__ kv,
                            const unsigned char *__restrict__ kv_scale, const int32_t *__restrict__ idx,
                            __nv_bfloat16 *__restrict__ out, float *__restrict__ lse) {
    extern __shared__ float sm[];
    float *qs = sm, *ks = qs + HG * 576, *ps = ks + KC * KVP, *ms = ps + HG * KC, *ls = ms + HG, *fs = ls + HG;
    int *vis = reinterpret_cast<int *>(fs + HG);
    const int t = blockIdx.x >> 3, h0 = (blockIdx.x & 7) * HG, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const RowInfo ri = row_info(P, t);
    const bool row_live = row_ok(P, ri) && ri.pos < ri.len_k;
    for (int i = tid; i < HG * 576; i += NT) qs[i] = __bfloat162float(q[((int64_t)t * 128 + h0) * 576 + i]) * P.sm_scale;
    if (tid < HG) {
        ms[tid] = -INFINITY;
        ls[tid] = 0.f;
    }
    float acc[HG][2] = {};
    for (int k0 = 0; k0 < P.topk && row_live; k0 += KC) {
        __syncthreads();
        if (tid < KC) {
            const int e = k0 + tid < P.topk ? idx[(int64_t)t * P.topk + k0 + tid] : -1;
            vis[tid] = mla::pair_visible(e, ri) ? key_row(P, ri, e) : -1;
        }
        __syncthreads();
        for (int i = tid; i < KC * 576; i += NT) {
            const int k = i / 576, d = i - k * 576;
            float v = 0.f;
            if (vis[k] >= 0) {
                const unsigned char *r = kv + (int64_t)vis[k] * cache::KV8_CODES;
                const float s = ue8m0_to_float(kv_scale[vis[k]]);
                v = d < 512 ? cache::e4m3_value(r[d]) * s
                            : (cache::e4m3_value(r[d]) + cache::e4m3_value(r[d + 64])) * cache::KV8_ROPE_GAIN * s;
            }
            ks[k * KVP + d] = v;
        }
        __syncthreads();
        for (int h = warp; h < HG; h += NT / 32) {
            float z = 0.f;
            for (int d = 0; d < 576; ++d) z = fmaf(qs[h * 576 + d], ks[lane * KVP + d], z);
            if (vis[lane] < 0) z = -INFINITY;
            float m = z;
            for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
            const float mo = ms[h], mn = fmaxf(mo, m);
            const float p = vis[lane] < 0 ? 0.f : expf(z - mn);
            float l = p;
            for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            ps[h * KC + lane] = p;
            __syncwarp();
            if (lane == 0) {
                fs[h] = mo == -INFINITY ? 0.f : expf(mo - mn);
                ls[h] = ls[h] * fs[h] + l;
                ms[h] = mn;
            }
        }
        __syncthreads();
        for (int h = 0; h < HG; ++h) {
            acc[h][0] *= fs[h];
            acc[h][1] *= fs[h];
        }
        for (int k = 0; k < KC; ++k) {
            const float v0 = ks[k * KVP + tid], v1 = ks[k * KVP + tid + 256];
            for (int h = 0; h < HG; ++h) {
                acc[h][0] = fmaf(ps[h * KC + k], v0, acc[h][0]);
                acc[h][1] = fmaf(ps[h * KC + k], v1, acc[h][1]);
            }
        }
    }
    __syncthreads();
    for (int h = 0; h < HG; ++h) {
        const float inv = ls[h] == 0.f ? 0.f : 1.0f / ls[h];
        __nv_bfloat16 *o = out + ((int64_t)t * 128 + h0 + h) * 512;
        o[tid] = __float2bfloat16_rn(acc[h][0] * inv);
        o[tid + 256] = __float2bfloat16_rn(acc[h][1] * inv);
    }
    if (tid < HG) lse[(int64_t)t * 128 + h0 + tid] = ls[tid] == 0.f ? -INFINITY : ms[tid] + logf(ls[tid]);
}

}  // namespace mla8
}  // namespace dsa
