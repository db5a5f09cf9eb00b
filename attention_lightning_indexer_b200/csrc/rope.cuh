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
// CTA takes whole tokens: as many as give its threads about four items each, or two where tokens
// have more than that and two still leave a full grid, so that all its warps evaluate angles at
// once and then stream without another barrier.
// A thread keeps its place within a head (one 16-byte vector, its pairs' cosines and sines in
// registers) and goes from head to head by adding strides: placing each vector by divisions
// cost more instructions (177 a vector) than rotating it.
// 8192 tokens x 128 heads x 64 dims out of [.., 192] rows into [.., 576] rows (268 MB, 41 us at
// the copy bandwidth): 53 us; 5003 x 64 heads of 128 dims, half of them copied: 35 us (164 MB, 25 us).
#pragma once

#include <cuda_fp16.h>

#include "dsa_common.cuh"

namespace dsa {
namespace rope {

constexpr int NT = 256;
constexpr int MAX_PAIRS = 512;       // (cos, sin) pairs kept per CTA
constexpr int MAX_TOKENS = 16;       // tokens per CTA
constexpr int FULL_GRID = 148 * 8;   // CTAs that keep every SM busy

// Heads a thread has in flight (kernel and launch).  8192 x 128 heads, interleaved: 57 us with 4
// and 4 CTAs per SM, 64 with 3 CTAs, 59 with 2 heads and 5, 66 with 6, 69 with 1 and 7 (59 as a
// copy without the rotation, with 3 CTAs; all with eight tokens per CTA).  5003 x 64 heads, half
// layout: 39 us with 1 head and 5 CTAs, 42 with 6; before the streamed stores 45 against 50 with
// 4 CTAs, 57 to 73 with 2 heads.  Single pairs (2000 x 40 heads of 150 dims at odd strides, 48 MB,
// interleaved): 22 us with 4 and 4 CTAs, 25 with 2, 27 with 6 CTAs, 37 without a bound on registers.
__host__ __device__ constexpr int heads_in_flight(bool vec, bool interleaved) { return !vec || interleaved ? 4 : 1; }

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

// 16-byte vectors are written as streamed (first to leave L2): 5 to 13 % faster at 50 MB and 134 MB.
template <typename T, int V>
__device__ __forceinline__ void store(T *p, const Vec<T, V> &v) {
    if constexpr (sizeof(v) == 16) __stcs(reinterpret_cast<uint4 *>(p), *reinterpret_cast<const uint4 *>(&v));
    else *reinterpret_cast<Vec<T, V> *>(p) = v;
}

// A work item of a head is a rotation (V pairs in the half layout, V / 2 pairs of one vector
// in the interleaved one, one pair where V = 1) or the copy of V elements outside the
// rotated part.  Threads beyond a whole number of heads idle.
template <typename T, int V, bool IL>
__global__ void __launch_bounds__(NT, V == 1 || IL ? 4 : 5) rope_kernel(Args g) {
    constexpr int PER = IL ? (V == 1 ? 1 : V / 2) : V;       // pairs of a rotation item
    constexpr bool TWO = !IL || V == 1;                      // an item has a second vector
    constexpr int U = heads_in_flight(V > 1, IL);
    using VT = Vec<T, V>;
    __shared__ __align__(16) float2 cs[MAX_PAIRS];
    const int threads = (int)blockDim.x;
    const int half = g.dim >> 1;
    const int64_t t0 = (int64_t)blockIdx.x * g.tokens_per_cta;
    const int nt = (int)min((int64_t)g.tokens_per_cta, g.n_tokens - t0);
    const int rot = half / PER;                              // rotation items of a head
    const int per_head = rot + (g.in_place ? 0 : (g.head_dim - g.dim) / V);
    // thread -> place within a head and first head; heads h0, h0 + step, h0 + 2 step, ..
    const int kp = min(per_head, threads), step = threads / kp;
    const int k0 = (int)threadIdx.x % kp, h0 = (int)threadIdx.x / kp;
    const int heads = h0 < step ? g.n_heads - h0 : 0;        // head h0 + i exists for i < heads
    const int rounds = (g.n_heads + U * step - 1) / (U * step);
    const int64_t xs = step * g.x_head, os = step * g.out_head;

    bool angles = false;
    for (int kb = 0; kb < per_head; kb += kp) {              // (once, unless a head has more items than the block)
        const int k = kb + k0;
        const bool turn = k < rot, mine = k < per_head;
        int d, second = 0;                                   // first element, its second vector
        if (turn) {
            d = g.begin + (IL ? 2 * PER * k : PER * k);
            second = IL ? 1 : half;
        } else {
            const int c = (k - rot) * V;
            d = c < g.begin ? c : c + g.dim;
        }
        const T *xt = static_cast<const T *>(g.x) + h0 * g.x_head + d;
        T *ot = static_cast<T *>(g.out) + h0 * g.out_head + d;
        const int n = mine ? heads : 0;
        VT a[U], b[TWO ? U : 1];
        auto load = [&](int ti, int rd) {
            const T *p = xt + ((t0 + ti) * g.x_token + rd * U * xs);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if ((rd * U + u) * step < n) {
                    a[u] = *reinterpret_cast<const VT *>(p + u * xs);
                    if (TWO && turn) b[TWO ? u : 0] = *reinterpret_cast<const VT *>(p + u * xs + second);
                }
            }
        };
        load(0, 0);
        if (!angles) {
            // the first loads are in flight: now the angles
            for (int i = threadIdx.x; i < nt * half; i += threads) {
                const int ti = i / half;
                double sn, cn;
                sincos((double)__ldg(g.positions + t0 + ti) * (double)__ldg(g.inv_freq + (i - ti * half)), &sn, &cn);
                if (g.transposed) sn = -sn;
                cs[i] = make_float2((float)(cn * g.scale), (float)(sn * g.scale));
            }
            __syncthreads();
            angles = true;
        }
        for (int ti = 0; ti < nt; ++ti) {
            float2 c[PER];
            if (turn) {
#pragma unroll
                for (int j = 0; j < PER; ++j) c[j] = cs[ti * half + PER * k + j];
            }
            for (int rd = 0; rd < rounds; ++rd) {
                T *o = ot + ((t0 + ti) * g.out_token + rd * U * os);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if ((rd * U + u) * step >= n) continue;
                    if (turn) {
#pragma unroll
                        for (int j = 0; j < PER; ++j) {
                            T &lo = IL && V > 1 ? a[u].e[(2 * j) % V] : a[u].e[j % V];
                            T &hi = IL && V > 1 ? a[u].e[(2 * j + 1) % V] : b[TWO ? u : 0].e[j % V];
                            const float p0 = to_f(lo), p1 = to_f(hi);
                            lo = from_f<T>(p0 * c[j].x - p1 * c[j].y);
                            hi = from_f<T>(p1 * c[j].x + p0 * c[j].y);
                        }
                    }
                    store<T, V>(o + u * os, a[u]);
                    if (TWO && turn) store<T, V>(o + u * os + second, b[TWO ? u : 0]);
                }
                // the next round's vectors (the next token's after the last)
                const bool wrap = rd + 1 == rounds;
                if (!wrap || ti + 1 < nt) load(wrap ? ti + 1 : ti, wrap ? 0 : rd + 1);
            }
        }
    }
}

}  // namespace rope
}  // namespace dsa
