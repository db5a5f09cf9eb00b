// rope.cuh -- rotary positions on a part of each head of strided [tokens, heads, head_dim]
// tensors: the query side of the path (the cache-write kernels rotate the key side).
//
//   (u, v) -> scale * (u cos a - v sin a, v cos a + u sin a),   a = positions[t] * inv_freq[i]
// for the pairs i < rope_dim / 2 of dims rope_begin ..: (i, i + rope_dim / 2) in the half
// layout, (2i, 2i + 1) in the interleaved one.  `transposed` turns by -a, which is the
// rotation's transpose: the gradient of x from the gradient of out.  The other dims are
// copied (left alone in place).
//
// HBM-bound: every rotated element is read and written once.  Angles, cosines and sines are
// taken in fp64 (at position 163,840 an fp32 angle is off by 2^-7 rad) once per token and
// pair, times scale rounded to fp32 in shared memory; the heads of the token share them.  A
// CTA takes the heads of a few tokens, so that its 256 threads have about four 16-byte
// vectors each; their loads are issued before the angles are evaluated.
#pragma once

#include <cuda_fp16.h>

#include "dsa_common.cuh"

namespace dsa {
namespace rope {

constexpr int NT = 256;
constexpr int MAX_PAIRS = 512;       // (cos, sin) pairs kept per CTA
constexpr int MAX_TOKENS = 16;       // tokens per CTA

struct Args {
    const void *x;
    void *out;
    const int32_t *positions;
    const float *inv_freq;
    int n_tokens, n_heads, head_dim, begin, dim;
    int64_t x_token, x_head, out_token, out_head;   // strides in elements
    float scale;
    int transposed, in_place;
    int tokens_per_cta;
};

template <typename T> __device__ __forceinline__ float to_f(T v);
template <> __device__ __forceinline__ float to_f(float v) { return v; }
template <> __device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T> __device__ __forceinline__ T from_f(float v);
template <> __device__ __forceinline__ float from_f(float v) { return v; }
template <> __device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// A work item of a head is a rotation (V pairs in the half layout, V / 2 pairs of one vector
// in the interleaved one, one pair where V = 1) or the copy of V elements outside the
// rotated part.
template <typename T, int V, bool IL>
__global__ void __launch_bounds__(NT) rope_kernel(Args g) {
    constexpr int PER = IL ? (V == 1 ? 1 : V / 2) : V;   // pairs of a rotation item
    constexpr int UNROLL = 4;
    __shared__ float2 cs[MAX_PAIRS];
    const int half = g.dim >> 1;
    const int64_t t0 = (int64_t)blockIdx.x * g.tokens_per_cta;
    const int nt = (int)min((int64_t)g.tokens_per_cta, g.n_tokens - t0);
    const int rot = half / PER;                              // rotation items of a head
    const int cop = g.in_place ? 0 : (g.head_dim - g.dim) / V;
    const int per_head = rot + cop, per_token = per_head * g.n_heads;
    const int items = per_token * nt;
    const T *x = static_cast<const T *>(g.x);
    T *out = static_cast<T *>(g.out);

    struct Where {
        int64_t xi, oi;    // element offsets of the head's row
        int d, dp, pair;   // first dim, partner dim (half layout), index into cs (-1: a copy)
    };
    auto where = [&](int i) {
        const int t = i / per_token, r = i - t * per_token;
        const int h = r / per_head, k = r - h * per_head;
        Where w;
        w.xi = (t0 + t) * g.x_token + (int64_t)h * g.x_head;
        w.oi = (t0 + t) * g.out_token + (int64_t)h * g.out_head;
        if (k < rot) {
            w.d = g.begin + (IL ? 2 * PER * k : PER * k);
            w.dp = w.d + half;
            w.pair = t * half + PER * k;
        } else {
            const int c = (k - rot) * V;
            w.d = c < g.begin ? c : c + g.dim;
            w.dp = 0;
            w.pair = -1;
        }
        return w;
    };
    using VT = Vec<T, V>;
    for (int base = 0; base < items; base += NT * UNROLL) {
        VT a[UNROLL], b[UNROLL];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int i = base + u * NT + (int)threadIdx.x;
            if (i >= items) continue;
            const Where w = where(i);
            a[u] = *reinterpret_cast<const VT *>(x + w.xi + w.d);
            if (w.pair >= 0) {
                if (!IL) b[u] = *reinterpret_cast<const VT *>(x + w.xi + w.dp);
                else if (V == 1) b[u] = *reinterpret_cast<const VT *>(x + w.xi + w.d + 1);
            }
        }
        if (base == 0) {
            for (int k = threadIdx.x; k < nt * half; k += NT) {
                const int t = k / half;
                double s, c;
                sincos((double)__ldg(g.positions + t0 + t) * (double)__ldg(g.inv_freq + (k - t * half)), &s, &c);
                if (g.transposed) s = -s;
                cs[k] = make_float2((float)(c * g.scale), (float)(s * g.scale));
            }
            __syncthreads();
        }
#pragma unroll
        for (int u = 0; u < UNROLL; ++u) {
            const int i = base + u * NT + (int)threadIdx.x;
            if (i >= items) continue;
            const Where w = where(i);
            if (w.pair >= 0) {
                if (IL && V > 1) {
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const float2 q = cs[w.pair + j];
                        const float p0 = to_f(a[u].e[(2 * j) % V]), p1 = to_f(a[u].e[(2 * j + 1) % V]);
                        a[u].e[(2 * j) % V] = from_f<T>(p0 * q.x - p1 * q.y);
                        a[u].e[(2 * j + 1) % V] = from_f<T>(p1 * q.x + p0 * q.y);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < PER; ++j) {
                        const float2 q = cs[w.pair + j];
                        const float p0 = to_f(a[u].e[j]), p1 = to_f(b[u].e[j]);
                        a[u].e[j] = from_f<T>(p0 * q.x - p1 * q.y);
                        b[u].e[j] = from_f<T>(p1 * q.x + p0 * q.y);
                    }
                }
            }
            *reinterpret_cast<VT *>(out + w.oi + w.d) = a[u];
            if (w.pair >= 0) {
                if (!IL) *reinterpret_cast<VT *>(out + w.oi + w.dp) = b[u];
                else if (V == 1) *reinterpret_cast<VT *>(out + w.oi + w.d + 1) = b[u];
            }
        }
    }
}

}  // namespace rope
}  // namespace dsa
