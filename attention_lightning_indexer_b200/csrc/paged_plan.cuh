// paged_plan.cuh -- the sequence offsets, slot map and block-table entries of one step,
// made on the GPU from the requests' lengths (paged caches of 64-token pages,
// "DeepSeek-V3.2" (miles docs) §5.3).
//
//   total(b) = len_cached(b) + len_new(b)          pages(n) = ceil(n / 64)
//   cu_q = exclusive sums of len_new               cu_k = exclusive sums of total
//   need(b) = pages(total(b)) - pages(len_cached(b)), taken from the free list in order of
//   b: request b's j-th new page is free_pages[head + sum_{b' < b} need(b') + j]
//   token i of request b: position p = len_cached(b) + i, row = page(b, p / 64) * 64 + p % 64
//
// Latency-bound: a step's inputs are a few KB.  One launch; every CTA scans the lengths
// itself (a block scan of three 64-bit sums over at most 8192 requests, read from L2)
// instead of waiting for another launch, keeps the offsets in shared memory and places its
// own 1024 tokens by binary search there.  CTA 0 also writes the offsets and the counts.
// No atomics: what is written does not depend on the order in which CTAs run.
// 64 requests with one token each: 3.8 us; 500 requests with 33 thousand tokens: 5.5 us (launch
// and two dependent rounds of loads).
#pragma once

#include "dsa_common.cuh"

namespace dsa {
namespace plan {

constexpr int NT = 512;              // threads per CTA
constexpr int TOKENS = 1024;         // tokens placed by one CTA
constexpr int MAX_BATCH = 8192;      // three 4-byte offsets per request in shared memory

// Bits of counts[3].
constexpr int SHORT_PAGES = 1, NARROW_TABLE = 2, SHORT_AXIS = 4, BAD_LENGTH = 8;

inline size_t smem_bytes(int batch) { return 3u * 4u * (size_t)(batch + 1); }

struct Args {
    int batch, n_tokens, max_pages, n_free, n_pages;
    const int32_t *len_cached, *len_new;
    int32_t *block_table;
    const int32_t *free_pages, *free_head;
    int32_t *cu_q, *cu_k, *positions, *rows, *counts;
};

__device__ __forceinline__ int64_t pages_of(int64_t n) { return (n + 63) >> 6; }

__global__ void __launch_bounds__(NT) paged_plan_kernel(Args a) {
    extern __shared__ int32_t sm[];
    int32_t *s_q = sm;                        // [batch + 1] exclusive sums of len_new
    int32_t *s_pg = sm + (a.batch + 1);       // [batch + 1] exclusive sums of need
    int32_t *s_c = sm + 2 * (a.batch + 1);    // [batch] len_cached
    __shared__ int64_t w_sum[3][NT / 32];
    __shared__ int64_t w_max[NT / 32];
    __shared__ int w_err[NT / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    // ---- each thread sums a contiguous run of requests, then a block scan of the runs
    const int per = (a.batch + NT - 1) / NT;
    const int b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
    int64_t v[3] = {0, 0, 0}, longest = 0;
    int err = 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t c = __ldg(a.len_cached + b), n = __ldg(a.len_new + b);
        if (c < 0 || n < 0) err |= BAD_LENGTH;
        if (pages_of(c + n) > a.max_pages) err |= NARROW_TABLE;
        v[0] += n;
        v[1] += c + n;
        v[2] += pages_of(c + n) - pages_of(c);
        longest = longest > c + n ? longest : c + n;
        s_c[b] = (int32_t)c;
    }
    int64_t x[3] = {v[0], v[1], v[2]};
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x[k], o);
            if (lane >= o) x[k] += y;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const int64_t y = __shfl_xor_sync(0xffffffffu, longest, o);
        longest = longest > y ? longest : y;
        err |= __shfl_xor_sync(0xffffffffu, err, o);
    }
    if (lane == 31)
        for (int k = 0; k < 3; ++k) w_sum[k][warp] = x[k];
    if (lane == 0) {
        w_max[warp] = longest;
        w_err[warp] = err;
    }
    __syncthreads();
    int64_t run[3], total[3];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
        run[k] = x[k] - v[k];
        total[k] = 0;
    }
    longest = 0;
    err = 0;
    for (int w = 0; w < NT / 32; ++w) {
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (w < warp) run[k] += w_sum[k][w];
            total[k] += w_sum[k][w];
        }
        longest = longest > w_max[w] ? longest : w_max[w];
        err |= w_err[w];
    }
    const int64_t head = a.free_head != nullptr ? __ldg(a.free_head) : 0;
    if (total[0] > a.n_tokens || total[1] > 0x7fffffff) err |= SHORT_AXIS;
    if (head < 0 || head + total[2] > a.n_free) err |= SHORT_PAGES;

    // ---- offsets; a step that cannot be served leaves an empty batch and the table as it was
    const bool ok = err == 0;
    const bool lead = blockIdx.x == 0;
    for (int b = b0; b < b1; ++b) {
        const int64_t c = s_c[b], n = __ldg(a.len_new + b);
        s_q[b] = ok ? (int32_t)run[0] : 0;
        s_pg[b] = ok ? (int32_t)run[2] : 0;
        if (lead) {
            a.cu_q[b] = ok ? (int32_t)run[0] : 0;
            a.cu_k[b] = ok ? (int32_t)run[1] : 0;
        }
        run[0] += n;
        run[1] += c + n;
        run[2] += pages_of(c + n) - pages_of(c);
    }
    if (tid == 0) {
        s_q[a.batch] = ok ? (int32_t)total[0] : 0;
        if (lead) {
            a.cu_q[a.batch] = ok ? (int32_t)total[0] : 0;
            a.cu_k[a.batch] = ok ? (int32_t)total[1] : 0;
            a.counts[0] = ok ? (int32_t)total[0] : 0;
            a.counts[1] = ok ? (int32_t)total[2] : 0;
            a.counts[2] = ok ? (int32_t)longest : 0;
            a.counts[3] = err;
        }
    }
    __syncthreads();

    // ---- tokens
    const int n_live = s_q[a.batch];
    for (int i = tid; i < TOKENS; i += NT) {
        const int64_t t64 = (int64_t)blockIdx.x * TOKENS + i;
        if (t64 >= a.n_tokens) break;
        const int t = (int)t64;
        int pos = 0, row = -1;
        if (t < n_live) {
            int lo = 0, hi = a.batch - 1;     // the last b with s_q[b] <= t: requests without tokens are passed over
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (s_q[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            pos = s_c[lo] + (t - s_q[lo]);
            const int pg = pos >> 6;
            const int fresh = pg - (int)pages_of(s_c[lo]);
            int32_t *entry = a.block_table + (int64_t)lo * a.max_pages + pg;
            // (cached pages are not written by this launch)
            const int page = fresh >= 0 ? __ldg(a.free_pages + head + s_pg[lo] + fresh) : *entry;
            const bool real = page >= 0 && page < a.n_pages;
            // the page's first token stores it; -1 for one outside the pool, so that later steps reach
            // neither that number nor what the entry held before
            if (fresh >= 0 && (pos & 63) == 0) *entry = real ? page : -1;
            if (real) row = page * 64 + (pos & 63);
            else raise_error(ERR_BOUNDS);
        }
        a.positions[t] = pos;
        a.rows[t] = row;
    }
}

}  // namespace plan
}  // namespace dsa
