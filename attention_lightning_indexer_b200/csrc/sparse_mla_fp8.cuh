// sparse_mla_fp8.cuh -- attention over the selected rows of the 8-bit latent cache
// (cache_write_fp8.cuh gives the row format) on pairs of SMs: MLA in MQA mode, 128 heads over
// 576-d rows, the value is the 512-d latent.
//   z[t,h,i] = sm_scale * q[t,h,:] . kv[idx[t,i], :]     out = softmax(z) . kv[:, 0:512]
//
// Eight bits on the tensor cores: a bf16 number has 8 significant bits and e4m3 has 4, so q (and
// a probability) is the sum of two 8-bit numbers, hi = Q(x), e4m3, and lo = Q(x - hi), e5m2,
// and every product with a cached code is two kind::f8f6f4
// MMAs, each at twice the bf16 rate: the tensor time of the bf16 form, but the cached rows go
// from HBM into the MMA as they are.  Nothing is dequantised, the gathers move 144 KB per CTA and
// block instead of 272 KB, and a ring slot holds 128 dims of a key instead of 64.
//
// lo is e5m2 for its range, which reaches 2^-16.  For q, x - hi is at most 8 units of x's last bit,
// so 3 significant bits are enough (1 .. 8 are all among them): q is exact down to 2^-6 of a
// range that ends at 448, where an e4m3 lo was off by 2^-10 below 2^-2 (lse off by 1e-4 at the
// worst, since 16 times the RoPE dims sets the range; 9e-6 now).  A probability has more than 8
// bits: hi + lo is within 2^-8 of it above 2^-6 (as bf16 is), within 2^-14 below, 3 bits below
// 2^-10, and steps by 2^-16 at last.  An e4m3 lo is twice as near at the upper end but steps by
// 2^-9: 2047 keys at e^-10 beside one of weight 1 (9 % of the sum) were lost or doubled.
//
// The row's scale 2^e leaves the sums: S^T[key, h] is over codes, and its thread (which owns
// one key) multiplies by 2^e; for the values, the probability takes the scale with it, P' =
// p 2^(e - er + BASE), er the largest scale exponent among the keys this unit has read so far (of
// which p's reference takes account: see Probabilities).
// The RoPE dims are in the row as two codes of 64 dims at 16 times the row's scale, so q's
// RoPE dims are taken 16 times: the K axis is 4 atoms of latent codes and one atom [hi | lo],
// multiplied by the same 64 RoPE dims of q twice.
//
// Hand-overs between the CTAs avoid cluster-scope fences, which cost 1.5 to 2 us each beside
// the DSMEM traffic: the half of P'^T that belongs to the other CTA's heads goes there by
// st.async, which counts its bytes on that CTA's barrier p_in (the odd CTA's warp 7 relays it
// to the MMA thread), and the other arrivals carry nothing but the order of the tcgen05 and
// proxy fences before them.  Waits for what the other CTA sent acquire at cluster scope, which
// costs nothing measurable.
//
// The schedule is that of the bf16 kernel (sparse_mla_pair.cuh): persistent CTA pairs take
// (token, split) units in turn; blocks of 256 index slots, CTA c owns slots 128 c .. + 127 of
// each block and heads 64 c .. + 63;
//   QK_b   S^T[key, h], M = 256 keys (A: the gathered atoms of each CTA's own keys, K-major),
//          N = 128 heads (B: q hi / lo, 64 heads per CTA), K = 640 codes: 40 MMAs of K = 32
//   PV_b   O^T[d, h] += codes^T P'^T, M = 256 value dims twice (A: CTA c holds dims 256 i +
//          128 c .. + 127 of all 256 keys, MN-major), N = 128 heads (B: P'^T hi / lo, MN-major,
//          heads 64 c .. + 63 in CTA c), K = 256 keys: 32 MMAs
// with a 7-slot ring of 16 KB atoms (128 keys x 128 codes, tile::gather4, 128-byte swizzle) in
// MMA order QK_0, QK_1, PV_0, QK_2, PV_1, ...: five atoms for QK_b, four for PV_b (i = 0, 1 and
// key half h = 0, 1).  The order runs on across units: the next unit's QK_0 stands before a
// unit's last PV, so that the softmax need not wait between them.  A masked slot gathers a
// visible row of its token, so what lies in other rows never enters a sum.
//
// Probabilities: what is to be held well is the weight, a probability times its key's scale, so
// the reference m[h] is one of score + e - er (log2).  It moves up when a block's maximum exceeds
// it by more than TAU, so that P' <= 2^(TAU + BASE) < 448, and down when a block's maximum lies
// more than DOWN below it: many light keys beside a heavy one (a sequence's first token, for
// many heads) are then held as well as if it were not there, but for those in its own block.  In
// every block the largest P' is 2^(BASE - DOWN) = 1 or more (2^BASE in the heaviest).  A move
// sends columns of O^T through registers (0.1 to 0.9 us of a block's 4 to 5): 1024 queries took
// 621 us with TAU = 2.8 and BASE = 6, 565 with 4.8 and 4 (both before DOWN); with DOWN = 4 they
// take 566, with 6 555, without it 552 (scores of deviation 1.7, where it does little else).
// DEPTH ends the way down (what is 2^-20 of the heaviest so far needs no more), and SPAN bounds e -
// er from below, so that p and its sums stay below 2^90 whatever the scales.  The sum l takes p
// itself in fp32.
//
// Measured (graph replays): 1024 queries x 2048 keys 565 to 590 us (tensor floor 354 us; the bf16
// form 961 us), 64 queries 51 us (floor 22; bf16 85), one query over 8 pairs 18.5 us with the
// merge.  A block takes 4.9 us with all 74 pairs at work (tensor cores 3.2), of it the copy engine
// 3.5: 288 gather4 of 512 bytes per CTA at 12 ns; and shared memory 7400 of 9700 cycles: tensor
// cores 3456 wavefronts, loads and stores 2790, gathers 1152.  The chain QK, maxima, their
// exchange, P', PV has no slack beside those, and the SM clock falls to 1.73 GHz: leaving out any
// one of the gathers for PV, half of the QK or PV MMAs, or the split of P' saved 4 %.
//
// Warp roles (20 warps): 0-6 gather (one ring slot each), 7 issues the MMAs (even CTA), 8-11
// prepare (warp 8 also publishes each unit's block count; they split q into hi and lo, each head
// at its own power of two, while q_s is in use, into an image in the workspace that is copied to
// q_s as soon as the last QK has read it (the first unit's q: the softmax warps, in place); then
// they fetch the scales of the keys of each block, up to four blocks ahead, and write the
// previous unit's output), 12-19 softmax: TMEM lane quarter w % 4, head half (w - 12) / 4.
//
// The roles together are as much code as the instruction caches hold: what is not worth being
// unrolled is rolled, and the waits are short (1024 queries: 583 us before both, 553 after).
#pragma once

#include <type_traits>

#include "cache_write_fp8.cuh"
#include "dsa_common.cuh"
#include "sm100.cuh"
#include "sparse_mla_pair.cuh"

namespace dsa {
namespace mla8 {

struct Cfg {
    static constexpr int BLK = 256;                 // index slots per block (128 per CTA)
    static constexpr int ATOM = 128 * 128;          // one gathered atom: 128 keys x 128 codes
    static constexpr int QK_ATOMS = 5, PV_ATOMS = 4;
    static constexpr int QATOM = 64 * 128;          // 64 heads x 128 bytes
    static constexpr int NQ = 9;                    // raw: 9 x 64 dims; split: 4 hi, 4 lo, [RoPE hi | lo]
    static constexpr int NSLOT = 7, NLOAD = 7;
    static constexpr int NINFO = 4;                 // blocks of key scales kept ahead
    static constexpr int NQS = 4;                   // units of q scales kept
    static constexpr int QIMG = NQ * QATOM;         // bytes of a CTA's split q
    static constexpr int OFF_Q = 0;
    static constexpr int OFF_PH = OFF_Q + NQ * QATOM;           // P' hi [256 keys][64 heads]
    static constexpr int OFF_PL = OFF_PH + 256 * 64;            // P' lo
    static constexpr int OFF_RING = OFF_PL + 256 * 64;
    static constexpr int OFF_RED = OFF_RING + NSLOT * ATOM;     // [4][128] f32
    static constexpr int OFF_XM = OFF_RED + 4 * 128 * 4;        // [2][128] f32, peer block maxima
    static constexpr int OFF_XL = OFF_XM + 2 * 128 * 4;         // [128] f32, peer row sums
    static constexpr int OFF_MQ = OFF_XL + 128 * 4;             // [64] {-m, -m', qs, qs'} of a head pair
    static constexpr int OFF_FS = OFF_MQ + 64 * 16;             // [128] f32, rescale factor
    static constexpr int OFF_QS = OFF_FS + 128 * 4;             // [NQS][128] f32, 2^f[h] * sm_scale * log2 e
    static constexpr int OFF_INFO = OFF_QS + NQS * 128 * 4;     // [NINFO][128] f32, key scale or -1 (masked)
    static constexpr int OFF_ER = OFF_INFO + NINFO * 128 * 4;   // [NINFO][4] int, running maxima of exponents
    static constexpr int OFF_FO = OFF_ER + NINFO * 4 * 4;       // [2][128] f32, output factors of a unit
    static constexpr int OFF_MV = OFF_FO + 2 * 128 * 4;         // [4] u32, heads whose reference moved
    static constexpr int OFF_BAR = OFF_MV + 16;
    // empty[7] pfull[7] q_raw q_ready q_free s_full[2] s_free[2] p_full pv_done o_ready xbar[2] lbar
    // drain unit_full[2] unit_free[2] info_full[4] info_free[4] p_in fo_full[2] o_free qs_full[4] img_full
    static constexpr int NBARS = 2 * NSLOT + 3 + 2 + 2 + 3 + 2 + 2 + 2 + 2 + 2 * NINFO + 1 + 3 + NQS + 1;
    // [0] TMEM base, [1] abort, [2..3] unit blocks, [4..5] unit fallback keys, [6] peer's abort flag
    static constexpr int OFF_MISC = OFF_BAR + NBARS * 8;
    static constexpr int OFF_LASTPOS = OFF_MISC + 32;           // even CTA: [2][NSLOT] last ring position issued
    static constexpr int SMEM = OFF_LASTPOS + 2 * NSLOT * 4;
    static constexpr int PREP0 = 8, SOFT0 = 12, WARPS = 20, THREADS = 32 * WARPS;
    // all of the 640 x 96 registers of the launch: 256 x 64 + 128 x 80 + 256 x 136 = 61,440
    static constexpr int REG_LOAD = 64, REG_PREP = 80, REG_SOFT = 136;
    static constexpr int TMEM_S = 0, TMEM_O = 256;
    static constexpr float TAU = 4.8f;              // log2 units: the reference moves up beyond this,
    static constexpr float DOWN = 4.0f;             // down beyond this,
    static constexpr float DEPTH = 20.0f;           // and no lower than this below the largest so far
    static constexpr float SPAN = 24.0f;            // scales further below the largest count as this far in it
    static constexpr int BASE = 4;                  // 2^(TAU + BASE) = 446 < 448
    static constexpr int ER_MIN = BASE;             // exponent bytes below this count as this
    static_assert(SMEM <= 232448, "shared memory budget");
    static_assert(NLOAD == NSLOT, "one ring slot per gathering warp");
    static_assert(256 * REG_LOAD + 128 * REG_PREP + 256 * REG_SOFT <= 640 * 96, "register split");
};

// 2-SM MMA of e4m3 operands (see sm100::mma_f16_pair).
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// MN-major operand in the 64-byte swizzle: rows of 64 bytes along MN, 8-row (512-byte) groups
// along K, 16-byte chunk c of row r at chunk c ^ ((r >> 1) & 3) (layout 4 = SW64).
__device__ __forceinline__ uint64_t desc_sw64_mn(uint32_t smem_addr) {
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr & 0x3FFFFu) >> 4);
    d |= (uint64_t)1 << 16;
    d |= (uint64_t)(512 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)4 << 61;
    return d;
}

// Maximum over the warp of v (NaN passed over), in every lane.
__device__ __forceinline__ float warp_fmax(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// Two fp16 numbers as hi = Q(x), e4m3, and lo = Q(x - hi), e5m2 (two codes each).
__device__ __forceinline__ void split_8bit(__half2 x, uint32_t &hi, uint32_t &lo) {
    const __nv_fp8x2_storage_t h = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(x), __NV_SATFINITE, __NV_E4M3);
    const __half2 back = __half2(__nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3));
    hi = h;
    lo = __nv_cvt_halfraw2_to_fp8x2(static_cast<__half2_raw>(__hsub2(x, back)), __NV_SATFINITE, __NV_E5M2);
}

// Bounded waits of 0.2 s that raise no error: the role that gives up stops the pair by its flag, and
// the teardown of a pair that was stopped raises it and makes the pair's rows NaN.  The clock is
// read once in 4096 tries (how long a failed try suspends the warp is not specified; 1.5 us here):
// the 60 waits of the kernel with the clock and the error flag at each try were enough code to
// miss in the instruction caches (583 us instead of 556 for 1024 queries).
constexpr uint32_t WAIT_NS = 200000000u, WAIT_STRIDE = 4096u;
template <typename Try>
__device__ __forceinline__ bool wait_until(Try tried, uint32_t limit_ns) {
    uint32_t start = 0;
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        if (tried()) return true;
        if ((i & (WAIT_STRIDE - 1u)) == 0u) {
            const uint32_t now = sm100::globaltimer_lo();
            if (i == WAIT_STRIDE) start = now;
            else if (now - start > limit_ns) return false;
        }
    }
}
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, uint32_t limit_ns = WAIT_NS) {
    return wait_until([=] { return sm100::mbar_try_wait(bar, parity); }, limit_ns);
}
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity) {
    return wait_until([=] { return sm100::mbar_try_wait_cluster(bar, parity); }, WAIT_NS);
}

struct Unit {
    int nblocks;
    int fallback;   // a visible key of the token (position within its sequence)
};

// Blocks of one unit up to the last visible one of its slots first .. first + n - 1 of the index
// row, and that slot's key (the same in every lane of the warp).
__device__ __forceinline__ Unit unit_scan(const Problem &P, const RowInfo &ri, const int32_t *irow, int first, int n,
                                          int lane) {
    Unit u{0, 0};
    if (ri.pos >= ri.len_k || P.total_k == 0 || !row_ok(P, ri)) return u;   // behind the last sequence, or a bad row
    int last = -1;
    irow += first;                                        // a multiple of 256 slots
    if ((P.topk & 3) == 0) {
        const int n4 = n >> 2;
#pragma unroll 8
        for (int i4 = lane; i4 < n4; i4 += 32) {
            const int4 x = __ldg(reinterpret_cast<const int4 *>(irow) + i4);
            if (mla::pair_visible(x.x, ri)) last = 4 * i4;
            if (mla::pair_visible(x.y, ri)) last = 4 * i4 + 1;
            if (mla::pair_visible(x.z, ri)) last = 4 * i4 + 2;
            if (mla::pair_visible(x.w, ri)) last = 4 * i4 + 3;
        }
    } else {
        for (int i = lane; i < n; i += 32)
            if (mla::pair_visible(__ldg(irow + i), ri)) last = i;
    }
    last = __reduce_max_sync(0xffffffffu, last);
    if (last < 0) return u;
    u.nblocks = (last + Cfg::BLK) / Cfg::BLK;
    u.fallback = __ldg(irow + last);
    return u;
}

// 256 threads (st) fill CTA cr's part of a unit's output (2 x 128 dims of every head, the lse of 64
// heads) with one value each.
template <bool SPLIT>
__device__ __forceinline__ void fill_unit(const mla::SplitArgs &sp, __nv_bfloat16 *out, float *lse, int t, int split, int cr,
                                          int st, float o, float l) {
    const int64_t base = SPLIT ? ((int64_t)t * sp.nsplit + split) * 128 : (int64_t)t * 128;   // rows of 512
    const uint32_t w = sm100::pack_bf16x2(o, o);
#pragma unroll 1
    for (int e = st; e < 128 * 32; e += 256) {
        const int h = e >> 5, part = e & 31;                 // 32 x 8 dims per head
        const int64_t at = (base + h) * 512 + 256 * (part >> 4) + 128 * cr + 8 * (part & 15);
        if (SPLIT) {
            float4 *op = reinterpret_cast<float4 *>(sp.o_part + at);
            op[0] = make_float4(o, o, o, o);
            op[1] = make_float4(o, o, o, o);
        } else {
            *reinterpret_cast<uint4 *>(out + at) = make_uint4(w, w, w, w);
        }
    }
    if (st < 128 && (st >> 6) == cr) (SPLIT ? sp.lse_part : lse)[base + st] = l;
}

template <bool SPLIT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Cfg::THREADS, 1)
sparse_mla_fp8_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_kv, Problem P,
                      const unsigned char *__restrict__ kv_scale, const int32_t *__restrict__ idx,
                      const __nv_bfloat16 *__restrict__ q_rows, unsigned char *__restrict__ q_images,
                      __nv_bfloat16 *__restrict__ out, float *__restrict__ lse, mla::SplitArgs sp) {
    using C = Cfg;
    using namespace sm100;
    extern __shared__ __align__(1024) unsigned char smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cr = (int)cluster_ctarank();                   // 0: issues the MMAs
    const int peer = cr ^ 1;
    const int T = P.total_q, K = P.topk;
    const int nsplit = SPLIT ? sp.nsplit : 1;
    const int bps = SPLIT ? sp.bps : (1 << 22);
    const int units = T * nsplit;
    const int npairs = (int)(gridDim.x >> 1);
    const int pair0 = (int)(blockIdx.x >> 1);

    const uint32_t sbase = smem_u32(smem);
    const bool misaligned = (sbase & 1023u) != 0;           // uniform; no unit runs then
    const uint32_t q_s = sbase + C::OFF_Q;
    const uint32_t ph_s = sbase + C::OFF_PH;
    const uint32_t ring_s = sbase + C::OFF_RING;
    float *red = reinterpret_cast<float *>(smem + C::OFF_RED);
    float *xm = reinterpret_cast<float *>(smem + C::OFF_XM);
    float *xl = reinterpret_cast<float *>(smem + C::OFF_XL);
    float *mq = reinterpret_cast<float *>(smem + C::OFF_MQ);
    float *fs = reinterpret_cast<float *>(smem + C::OFF_FS);
    float *fo = reinterpret_cast<float *>(smem + C::OFF_FO);
    uint32_t *mvw = reinterpret_cast<uint32_t *>(smem + C::OFF_MV);
    float *qsc = reinterpret_cast<float *>(smem + C::OFF_QS);
    float *info = reinterpret_cast<float *>(smem + C::OFF_INFO);
    int *ers = reinterpret_cast<int *>(smem + C::OFF_ER);
    const uint32_t bar0 = sbase + C::OFF_BAR;
    auto empty = [&](int s) { return bar0 + 8u * s; };
    auto pfull = [&](int s) { return bar0 + 8u * (C::NSLOT + s); };
    const uint32_t q_raw = bar0 + 8u * (2 * C::NSLOT);       // this CTA's raw q landed
    const uint32_t q_ready = q_raw + 8;                      // even CTA: q of both CTAs split
    const uint32_t q_free = q_raw + 16;                      // the unit's last QK has read q_s
    auto s_full = [&](int b) { return q_raw + 24 + 8u * b; };
    auto s_free = [&](int b) { return q_raw + 40 + 8u * b; };
    const uint32_t p_full = q_raw + 56;                      // even CTA: P'^T in place, but for p_in
    const uint32_t pv_done = q_raw + 64;
    const uint32_t o_ready = q_raw + 72;
    auto xbar = [&](int b) { return q_raw + 80 + 8u * b; };
    const uint32_t lbar = q_raw + 96;
    const uint32_t drain = q_raw + 104;
    auto unit_full = [&](int i) { return q_raw + 112 + 8u * i; };
    auto unit_free = [&](int i) { return q_raw + 128 + 8u * i; };
    auto info_full = [&](int i) { return q_raw + 144 + 8u * i; };
    auto info_free = [&](int i) { return q_raw + 144 + 8u * (C::NINFO + i); };
    const uint32_t p_in = q_raw + 144 + 8u * (2 * C::NINFO); // P'^T rows of the peer's keys landed here
    auto fo_full = [&](int i) { return p_in + 8 + 8u * i; }; // a unit's output factors are in place
    const uint32_t o_free = p_in + 24;                       // even CTA: O^T of both CTAs read out
    auto qs_full = [&](int i) { return p_in + 32 + 8u * i; };   // a unit's q scales are in place
    const uint32_t img_full = p_in + 32 + 8u * C::NQS;       // the next unit's split q is in q_images
    volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + C::OFF_MISC);
    volatile int *unit_nb = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 8);
    volatile int *unit_fb = reinterpret_cast<volatile int *>(smem + C::OFF_MISC + 16);

    // ---- setup (every thread of both CTAs reaches the cluster barriers below)
    if (tid == 0 && !misaligned) {
        for (int s = 0; s < C::NSLOT; ++s) {
            mbar_init(empty(s), 1);
            mbar_init(pfull(s), 1);       // the even CTA's expect-tx for both CTAs' bytes
        }
        mbar_init(q_raw, 1);
        mbar_init(q_ready, 8);            // 4 preparing warps of each CTA
        mbar_init(q_free, 1);
        for (int b = 0; b < 2; ++b) {
            mbar_init(s_full(b), 1);
            mbar_init(s_free(b), 16);     // 8 softmax warps of each CTA
            mbar_init(xbar(b), 1);
            mbar_init(unit_full(b), 1);   // warp 8
            mbar_init(unit_free(b), C::NLOAD + 3 + 1 + 1);   // gathers, preparing warps, softmax, MMA or relay
        }
        mbar_init(p_full, 9);             // 4 warps of each CTA (own rows), the odd CTA's relay
        mbar_init(p_in, 1);
        mbar_init(fo_full(0), 4);         // the softmax warps of threads 0 .. 127
        mbar_init(fo_full(1), 4);
        mbar_init(o_free, 8);             // 4 preparing warps of each CTA
        for (int i = 0; i < C::NQS; ++i) mbar_init(qs_full(i), 4);   // own preparing warps (and the peer's bytes)
        mbar_init(img_full, 4);           // preparing warps
        mbar_init(pv_done, 1);
        mbar_init(o_ready, 1);
        mbar_init(lbar, 1);
        mbar_init(drain, 1);
        for (int i = 0; i < C::NINFO; ++i) {
            mbar_init(info_full(i), 4);
            mbar_init(info_free(i), 8);
        }
        misc[1] = 0;
        misc[6] = 0;
        for (int i = 0; i < 2 * C::NSLOT; ++i) reinterpret_cast<int *>(smem + C::OFF_LASTPOS)[i] = -1;
        fence_barrier_init();
    }
    if (tid == 0 && misaligned) {
        raise_error(ERR_SMEM_ALIGN);
        misc[1] = 1;
    }
    cluster_sync();   // both CTAs running, their barriers initialised
    if (warp == 0) tmem_alloc_pair(sbase + C::OFF_MISC, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = misc[0];   // 0: all 512 columns (the MMA warp counts on it)
    const bool run = !misaligned && tmem == 0;
    if (tid == 0 && tmem != 0) raise_error(ERR_SMEM_ALIGN);
    const uint32_t peer_misc1 = mapa_shared(sbase + C::OFF_MISC + 4, (uint32_t)peer);
    auto abort_pair = [&]() {                                // stop both CTAs of the pair
        raise_error(ERR_WAIT_TIMEOUT);
        misc[1] = 1;
        st_cluster_u32(peer_misc1, 1u);
    };

    const float sl2 = P.sm_scale * 1.4426950408889634f;
    const uint32_t q_ready_lead = mapa_shared(q_ready, 0);
    const uint32_t qsc_peer = mapa_shared(sbase + C::OFF_QS, (uint32_t)peer);
    const uint32_t qs_full_peer = mapa_shared(qs_full(0), (uint32_t)peer);
    // Split of q, head rows r0 .. r0 + 4 n - 1: 8 lanes per row, each the 16-byte chunk g of the row's nine
    // 128-byte lines (dims 64 a + 8 g ..); the split row takes nine lines of `to`.  In place: the raw rows
    // lie in q_s as TMA left them, else `rows` are rows of q.  scale(r, s) takes each row's scale in
    // one of its lanes.
    auto split_q = [&](auto in_place, unsigned char *to, const unsigned char *rows, int r0, int n, auto scale) {
        const int row_step = in_place.value ? 128 : 1152, line_step = in_place.value ? C::QATOM : 128;
        const int g8 = lane & 7;
#pragma unroll 1
        for (int it = 0; it < n; ++it) {
            const int r = r0 + 4 * it + (lane >> 3);
            unsigned char *line = to + r * 128;
            const unsigned char *raw = rows + r * row_step + ((g8 ^ (in_place.value ? r & 7 : 0)) << 4);
            uint4 x[C::NQ];
#pragma unroll
            for (int a = 0; a < C::NQ; ++a)
                x[a] = *reinterpret_cast<const uint4 *>(raw + a * line_step);
            auto absmax = [](const uint4 &v, __nv_bfloat162 m) {
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i])));
                return m;
            };
            __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
#pragma unroll
            for (int a = 0; a < 8; ++a) m = absmax(x[a], m);
            const __nv_bfloat162 mr2 = absmax(x[8], __floats2bfloat162_rn(0.f, 0.f));
            uint32_t top = max(max(cache::abs_bits(__low2float(m)), cache::abs_bits(__high2float(m))),
                               max(cache::abs_bits(__low2float(mr2) * cache::KV8_ROPE_GAIN),
                                   cache::abs_bits(__high2float(mr2) * cache::KV8_ROPE_GAIN)));
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const uint32_t byte = cache::scale_byte(top);
            const float inv = cache::scale_inverse(byte);
            __syncwarp();                                // the rows of this warp are read
#pragma unroll
            for (int a = 0; a < C::NQ; ++a) {
                const uint32_t w[4] = {x[a].x, x[a].y, x[a].z, x[a].w};
                const float gain = a == 8 ? cache::KV8_ROPE_GAIN : 1.0f;
                uint32_t hi[4], lo[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float v0 = __uint_as_float(w[i] << 16), v1 = __uint_as_float(w[i] & 0xffff0000u);
                    // fp16 holds the 8 significant bits of bf16 down to 2^-24
                    split_8bit(__floats2half2_rn(v0 * gain * inv, v1 * gain * inv), hi[i], lo[i]);
                }
                const uint2 h = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
                const uint2 l = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
                // line and 16-byte chunk of the split row: latent dims 128 A .. in atoms A and 4 + A,
                // the RoPE dims in atom 8 as [hi | lo]
                const int ah = a == 8 ? 8 : a >> 1, al = a == 8 ? 8 : 4 + (a >> 1);
                const int ch = (a == 8 ? 0 : (a & 1) * 4) + (g8 >> 1), cl = a == 8 ? 4 + (g8 >> 1) : ch;
                *reinterpret_cast<uint2 *>(line + ah * C::QATOM + ((ch ^ (r & 7)) << 4) + 8 * (g8 & 1)) = h;
                *reinterpret_cast<uint2 *>(line + al * C::QATOM + ((cl ^ (r & 7)) << 4) + 8 * (g8 & 1)) = l;
            }
            if (g8 == 0) scale(r, ue8m0_to_float(byte) * sl2);
        }
    };

    if (warp < C::PREP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_LOAD));
    if (warp < C::NLOAD) {
        // ------------------------------------------------ gathers (one ring slot per warp)
        const int lw = warp;
        const uint32_t lead_pfull = mapa_shared(pfull(lw), 0);
        const uint32_t slot_s = ring_s + lw * C::ATOM;
        if (lw == 0 && lane == 0) prefetch_tmap(&tm_kv);
        struct Ctx {                                         // a unit as its gathers see it
            RowInfo ri;
            const int32_t *irow;                             // its slots and how many there are
            int left, fb;                                    // fb: the cache row that stands in for masked slots
        };
        bool ok = run;
        int away = lw;                                       // ring positions up to this warp's next one (mod 7)
        int uses = 0;                                        // of this warp's slot
        // This warp's atom of the group, if it has one: value or key atom a, key half `half` of block b
        auto gather = [&](const Ctx &c, int b, int half, int a) {
            const int s0 = C::BLK * b + 128 * half + 4 * lane;
            int4 x;
            if ((K & 3) == 0 && s0 + 3 < c.left) {
                x = __ldg(reinterpret_cast<const int4 *>(c.irow + s0));
            } else {
                x.x = s0 < c.left ? __ldg(c.irow + s0) : -1;
                x.y = s0 + 1 < c.left ? __ldg(c.irow + s0 + 1) : -1;
                x.z = s0 + 2 < c.left ? __ldg(c.irow + s0 + 2) : -1;
                x.w = s0 + 3 < c.left ? __ldg(c.irow + s0 + 3) : -1;
            }
            auto row_of = [&](int e) {
                const int row = mla::pair_visible(e, c.ri) ? key_row_checked(P, c.ri, e) : -1;
                return row < 0 ? c.fb : row;
            };
            const int r0 = row_of(x.x), r1 = row_of(x.y), r2 = row_of(x.z), r3 = row_of(x.w);
            bool okw = true;
            if (lane == 0) {
                if (uses > 0) okw = wait(empty(lw), (uses - 1) & 1);
                if (okw && cr == 0) mbar_expect_tx(pfull(lw), 2 * C::ATOM);   // both CTAs' rows
            }
            if (!__shfl_sync(0xffffffffu, okw, 0) || misc[1]) return false;
            tma_gather4_pair(slot_s + 512 * lane, &tm_kv, lead_pfull, 128 * a, r0, r1, r2, r3);
            ++uses;
            return true;
        };
        Ctx cur = {}, old = {};
        int nb = 0, b = 0, old_b = -1;                       // the current block and the one whose PV is due
        for (int j = -1, u = pair0 - npairs; ok;) {
            bool have = true;                                // another block, of this unit or a later one
            for (++b; have && ok && b >= nb; ) {
                ++j;
                u += npairs;
                have = u < units;
                if (!have) break;
                const int t = T - 1 - u / nsplit;
                const int first = (u % nsplit) * bps * C::BLK;
                cur.ri = row_info_warp(P, t);
                cur.irow = idx + (int64_t)t * K + first;
                cur.left = K - first;
                const bool got = wait(unit_full(j & 1), (j >> 1) & 1);
                nb = got ? unit_nb[j & 1] : 0;
                cur.fb = got && nb > 0 ? key_row_checked(P, cur.ri, unit_fb[j & 1]) : 0;
                if (cur.fb < 0) {                            // on a page outside the pool: any key that is not
                    int other = 0;                           // (none: row 0, which the output leaves out)
#pragma unroll 1
                    for (int i = lane; i < min(cur.left, nb * C::BLK); i += 32) {
                        const int e = __ldg(cur.irow + i);
                        if (mla::pair_visible(e, cur.ri)) other = max(other, key_row_checked(P, cur.ri, e));
                    }
                    cur.fb = __reduce_max_sync(0xffffffffu, other);
                }
                ok = __all_sync(0xffffffffu, got);
                if (ok && lane == 0) mbar_arrive(unit_free(j & 1));
                b = 0;
            }
            if (!ok) break;
            // QK_b needs the CTA's own key half; PV of the block before: instruction i = m >> 1, key half
            // m & 1.  (One copy of the code for both: the instruction caches are short.)
#pragma unroll 1
            for (int part = have ? 0 : 1; ok && part < (old_b >= 0 ? 2 : 1); ++part) {
                const bool qk = part == 0;
                const int natoms = qk ? C::QK_ATOMS : C::PV_ATOMS;
                if (away < natoms)
                    ok = gather(qk ? cur : old, qk ? b : old_b, qk ? cr : away & 1, qk ? away : (away & 2) + cr);
                away -= natoms;
                away += away < 0 ? C::NLOAD : 0;
            }
            if (!have) break;
            old = cur;
            old_b = b;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok && lane == 0) abort_pair();
        // the last position issued into this warp's slot, recorded in the even CTA for the drain
        // after an abort
        if (lane == 0)
            st_cluster_u32(mapa_shared(sbase + C::OFF_LASTPOS + 4u * (uint32_t)(cr * C::NSLOT + lw), 0),
                           (uint32_t)(uses > 0 ? (uses - 1) * C::NSLOT + lw : -1));
    } else if (lane == 0 && cr == 1) {
        // ------------------------------------------------ relay (odd CTA): the peer's rows of P'^T
        const uint32_t p_full_lead = mapa_shared(p_full, 0);
        bool ok = run;
        int gb = 0;
        for (int j = 0, u = pair0; ok && u < units; ++j, u += npairs) {
            ok = wait(unit_full(j & 1), (j >> 1) & 1);
            const int nblocks = ok ? unit_nb[j & 1] : 0;
            if (ok) mbar_arrive(unit_free(j & 1));
            for (int b = 0; ok && b < nblocks; ++b, ++gb) {
                mbar_expect_tx(p_in, 128 * 128);
                ok = wait_cluster(p_in, gb & 1) && !misc[1];
                fence_proxy_async_smem();
                if (ok) mbar_arrive_remote(p_full_lead);
            }
        }
        if (!ok) abort_pair();
    } else if (cr == 0) {
        // ------------------------------------------------ MMA issuer (even CTA)
        // The whole warp runs the loop and one elected lane issues, so that descriptors stay in
        // uniform registers; a lane of its own spent as long on issuing an MMA as it takes to run.
        const uint32_t idesc_qk = idesc_e4m3(256, 128);
        const uint32_t idesc_qk_lo = idesc_qk | (1u << 10);                         // B e5m2
        const uint32_t idesc_pv = idesc_e4m3(256, 128) | (1u << 15) | (1u << 16);   // A and B MN-major
        const uint32_t idesc_pv_lo = idesc_pv | (1u << 10);                         // B e5m2
        // descriptors step by bytes / 16 in their low word
        const uint64_t dq = desc_sw128(q_s), da_k = desc_sw128(ring_s), da_mn = desc_sw128_mn(ring_s, C::ATOM);
        const uint64_t dph = desc_sw64_mn(ph_s);
        bool ok = run;
        bool issued = false;
        int slot = 0, phase = 0;                             // ring slot and its phase
        int gb = -1, nq = -1;                                // current block and unit with blocks, counted over all units
        int nb = 0, b = 0;                                   // blocks of the unit, the current one
        int old_b = -1, old_gb = 0, old_q = 0;               // the block whose PV is due, its unit
        bool old_last = false;
        for (int j = -1, u = pair0 - npairs; ok;) {
            bool have = true;                                // another block, of this unit or a later one
            for (++b; have && ok && b >= nb; ) {
                ++j;
                u += npairs;
                have = u < units;
                if (!have) break;
                ok = __all_sync(0xffffffffu, wait(unit_full(j & 1), (j >> 1) & 1));
                nb = ok ? __shfl_sync(0xffffffffu, unit_nb[j & 1], 0) : 0;
                if (ok && elect_one()) mbar_arrive(unit_free(j & 1));
                b = 0;
                if (nb > 0) {
                    ++nq;
                    ok = __all_sync(0xffffffffu, wait(q_ready, nq & 1));
                }
            }
            if (!ok) break;
            if (have) {                                      // QK_b -> S^T buffer gb & 1
                ++gb;
                bool okw = gb < 2 || wait(s_free(gb & 1), ((gb >> 1) - 1) & 1);
                tc_fence_after();
                const uint32_t d = C::TMEM_S + 128 * (gb & 1);
#pragma unroll 1
                for (int a = 0; a < C::QK_ATOMS; ++a) {
                    okw = okw && wait(pfull(slot), phase);
                    // q: hi and lo atoms of the same 128 dims; for the RoPE atom [hi | lo] of the
                    // keys, 64 dims of q hi and lo twice
                    constexpr int ROPE = C::QK_ATOMS - 1;
                    const uint64_t da = da_k + (uint64_t)(slot * (C::ATOM >> 4));
                    const uint64_t qh = dq + (uint64_t)((a == ROPE ? 8 : a) * (C::QATOM >> 4));
                    const uint64_t ql = a == ROPE ? qh + 4 : dq + (uint64_t)((4 + a) * (C::QATOM >> 4));
                    if (elect_one()) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk) {
                            const int qo = 2 * (a == ROPE ? (kk & 1) : kk);
                            mma_f8_pair(d, da + 2 * kk, qh + qo, idesc_qk, (a > 0 || kk > 0) ? 1u : 0u);
                            mma_f8_pair(d, da + 2 * kk, ql + qo, idesc_qk_lo, 1u);
                        }
                        mma_commit_pair_both(empty(slot));
                    }
                    if (++slot == C::NSLOT) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (elect_one()) {
                    if (b == nb - 1) mma_commit_pair_both(q_free);   // the unit's last read of q_s
                    mma_commit_pair_both(s_full(gb & 1));
                }
                issued = true;
                if (!__all_sync(0xffffffffu, okw && !misc[1])) ok = false;
            }
            if (ok && old_b >= 0) {                          // PV of the block before
                // the four atoms first: they landed long before P'^T as a rule
                bool okw = true;
                int sl = slot, ph = phase;
#pragma unroll
                for (int m = 0; m < C::PV_ATOMS; ++m) {
                    okw = okw && wait(pfull(sl), ph);
                    if (++sl == C::NSLOT) {
                        sl = 0;
                        ph ^= 1;
                    }
                }
                if (elect_one()) mbar_expect_tx(p_in, 128 * 128);
                // the previous unit's O^T has been read out
                if (old_b == 0 && old_q > 0) okw = okw && wait(o_free, (old_q - 1) & 1);
                okw = okw && wait_cluster(p_full, old_gb & 1) && wait_cluster(p_in, old_gb & 1);
                fence_proxy_async_smem();
                tc_fence_after();
#pragma unroll 1
                for (int m = 0; m < C::PV_ATOMS; ++m) {
                    const uint32_t d = C::TMEM_O + 128 * (m >> 1);
                    const uint64_t da = da_mn + (uint64_t)(slot * (C::ATOM >> 4));
                    const uint64_t db = dph + (uint64_t)((m & 1) * (128 * 64 >> 4));
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {    // 32 keys each
                            mma_f8_pair(d, da + k * (4096 >> 4), db + k * (2048 >> 4), idesc_pv,
                                        (old_b > 0 || (m & 1) || k > 0) ? 1u : 0u);
                            mma_f8_pair(d, da + k * (4096 >> 4), db + ((C::OFF_PL - C::OFF_PH) >> 4) + k * (2048 >> 4),
                                        idesc_pv_lo, 1u);
                        }
                        mma_commit_pair_both(empty(slot));
                    }
                    if (++slot == C::NSLOT) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
                if (elect_one()) {
                    mma_commit_pair_both(pv_done);
                    if (old_last) mma_commit_pair_both(o_ready);
                }
                issued = true;
                if (!__all_sync(0xffffffffu, okw && !misc[1])) ok = false;
            }
            if (!have) break;
            old_b = b;
            old_gb = gb;
            old_q = nq;
            old_last = b == nb - 1;
        }
        if (!ok) {
            if (lane == 0) abort_pair();
            if (issued) {                                    // nothing may be in flight at dealloc
                if (elect_one()) mma_commit_pair_both(drain);
                wait(drain, 0);
            }
        }
    }
    } else if (warp < C::SOFT0) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_PREP));
        // ------------------------------------------------ units, q, key scales, output
        const int pw = warp - C::PREP0;
        if (pw == 0 && lane == 0) prefetch_tmap(&tm_q);
        bool ok = run;
        int gb = 0;                                          // blocks so far
        int nq = 0;                                          // units with blocks so far
        int images = 0;                                      // units whose q went through the image
        unsigned char *const image = q_images + (int64_t)blockIdx.x * C::QIMG;
        int qslot = 0;                                       // where the unit's q scales go
        // ---- epilogue of a unit (token pt, split ps, the pn-th with blocks): O^T times its output
        // factors into out.  These warps do it, so that the softmax goes on with the next unit; its
        // first PV waits for o_free.
        const uint32_t o_free_lead = mapa_shared(o_free, 0);
        auto epilogue = [&](int pt, int ps, int pn) {
            bool fine = wait(fo_full(pn & 1), (pn >> 1) & 1);
            fine = wait(o_ready, pn & 1) && fine;
            if (!__all_sync(0xffffffffu, fine)) return false;
            tc_fence_after();
            const float *f = fo + 128 * (pn & 1);
            // no key had a row (its page was outside the pool), then for no head: zeros, whatever row 0 put
            // into O^T
            const bool none = f[0] == 0.f;
            // O^T block i: lanes = value dims 256 i + 128 cr + 32 pw + lane, columns = heads
            const bool odd = (lane & 1) != 0;
#pragma unroll 1
            for (int c8 = 0; c8 < 8; ++c8) {
                const int i = c8 >> 2, ch = c8 & 3;
                uint32_t o[32];
                tmem_ld32(tmem + ((uint32_t)(pw * 32) << 16) + C::TMEM_O + 32 * c8, o);
                tmem_wait_ld();
                if (none) {
#pragma unroll
                    for (int h = 0; h < 32; ++h) o[h] = 0u;
                }
                if (c8 == 7) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote(o_free_lead);
                }
                if (SPLIT) {   // fp32 partial rows (32 lanes: 128 bytes per head)
                    float *op = sp.o_part + (((int64_t)pt * nsplit + ps) * 128 + 32 * ch) * 512 + 256 * i + 128 * cr + 32 * pw + lane;
#pragma unroll
                    for (int h = 0; h < 32; ++h) op[(int64_t)h * 512] = __uint_as_float(o[h]) * f[32 * ch + h];
                } else {
                    // bf16 rows from registers: lanes 2m and 2m + 1 swap one value per head pair, so
                    // each stores two adjacent dims of one head (64 contiguous bytes per head per warp)
                    __nv_bfloat16 *orow = out + ((int64_t)pt * 128 + 32 * ch + (odd ? 1 : 0)) * 512 + 256 * i + 128 * cr +
                                          32 * pw + (lane & ~1);
#pragma unroll
                    for (int h = 0; h < 32; h += 2) {
                        const float2 f2 = reinterpret_cast<const float2 *>(f)[16 * ch + (h >> 1)];
                        const float v0 = __uint_as_float(o[h]) * f2.x, v1 = __uint_as_float(o[h + 1]) * f2.y;
                        const float recv = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
                        const uint32_t w = odd ? pack_bf16x2(recv, v1) : pack_bf16x2(v0, recv);
                        *reinterpret_cast<uint32_t *>(orow + (int64_t)h * 512) = w;
                    }
                }
            }
            return true;
        };
        int pt = -1, ps = 0;                                 // the unit whose epilogue is due (number nq - 1 or nq - 2)
        for (int j = 0, u = pair0; ok && u < units; ++j, u += npairs) {
            const int t = T - 1 - u / nsplit;
            const int split = u % nsplit;
            const RowInfo ri = row_info_warp(P, t);
            const int32_t *irow = idx + (int64_t)t * K;
            int nblocks;
            bool okw = true;
            if (pw == 0) {
                // The first unit's q goes ahead of the gathers, which would queue before it in the copy
                // engine (4.3 instead of 2 us); nothing holds q_s yet.
                if (j == 0 && lane == 0) {
                    mbar_expect_tx(q_raw, C::QIMG);
                    for (int a = 0; a < C::NQ; ++a) tma_load_2d(q_s + a * C::QATOM, &tm_q, q_raw, 64 * a, t * 128 + 64 * cr);
                }
                const int first = SPLIT ? split * bps * C::BLK : 0;   // < K: no split is empty
                const Unit un = unit_scan(P, ri, irow, first, SPLIT ? min(K - first, bps * C::BLK) : K, lane);
                nblocks = un.nblocks;
                if (lane == 0) {
                    if (j >= 2) okw = wait(unit_free(j & 1), ((j >> 1) - 1) & 1);
                    if (okw) {
                        unit_nb[j & 1] = nblocks;
                        unit_fb[j & 1] = un.fallback;
                        mbar_arrive(unit_full(j & 1));
                    }
                }
                okw = __shfl_sync(0xffffffffu, okw, 0);
            } else {
                okw = wait(unit_full(j & 1), (j >> 1) & 1);
                nblocks = okw ? unit_nb[j & 1] : 0;
                if (__all_sync(0xffffffffu, okw) && lane == 0) mbar_arrive(unit_free(j & 1));
            }
            // every load is waited for, whatever happens to its unit: none is in flight at the end
            if (j == 0) okw = wait(q_raw, 0) && okw;
            if (!__all_sync(0xffffffffu, okw) || misc[1]) {
                ok = false;
                break;
            }
            if (nblocks == 0) continue;
            // ---- q of a later unit (the first one's: the softmax warps), from its rows into the image while
            // q_s is in use
            if (j > 0) {
                // no unit had blocks: the softmax warps split the first one's q and scales all the same
                if (nq == 0 && j == 1) okw = wait(unit_free(0), 0);
                if (!__all_sync(0xffffffffu, okw)) {
                    ok = false;
                    break;
                }
                split_q(std::false_type{}, image,
                        reinterpret_cast<const unsigned char *>(q_rows) + ((int64_t)t * 128 + 64 * cr) * 1152, 16 * pw, 4,
                        [&](int r, float s) {
                            const int at = 128 * qslot + 64 * cr + r;
                            qsc[at] = s;
                            st_async_f32(qsc_peer + 4u * at, s, qs_full_peer + 8u * qslot);
                        });
                fence_proxy_async_global();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(img_full);
                    if (pw == 0) mbar_expect_tx(qs_full(qslot), 64 * 4);   // the scales of the peer's heads
                    else mbar_arrive(qs_full(qslot));
                }
                if (pw == 0) {                               // into q_s once the unit before has read it
                    if (lane == 0) {
                        okw = wait(img_full, images & 1);
                        if (okw && nq > 0) okw = wait(q_free, (nq - 1) & 1);
                        if (okw) {
                            fence_proxy_async_global();
                            mbar_expect_tx(q_raw, C::QIMG);
                            for (int a = 0; a < C::NQ; ++a) bulk_load(q_s + a * C::QATOM, image + a * C::QATOM, C::QATOM, q_raw);
                        }
                    }
                    okw = __shfl_sync(0xffffffffu, okw, 0);
                }
                ++images;
                if (okw) okw = wait(q_raw, images & 1);
                if (!__all_sync(0xffffffffu, okw)) {
                    ok = false;
                    break;
                }
                if (lane == 0) mbar_arrive_remote(q_ready_lead);
            }
            ++nq;
            qslot = qslot == C::NQS - 1 ? 0 : qslot + 1;
            // ---- scales of this CTA's keys (-1: masked) and the running largest exponent over both
            // CTAs' keys, block by block
            const int32_t *irow_s = irow + split * bps * C::BLK;
            const int ks_left = K - split * bps * C::BLK;
            const int s_own = 128 * cr + 32 * pw + lane, s_oth = 128 * peer + 32 * pw + lane;
            auto entry = [&](int s) { return s < ks_left ? __ldg(irow_s + s) : -1; };
            int e_own = entry(s_own), e_oth = entry(s_oth);
            int er = C::ER_MIN;
            for (int b = 0; b < nblocks; ++b, ++gb) {
                // a visible key without a row (a page outside the pool) is masked
                const bool s_vis = mla::pair_visible(e_own, ri);
                const int r_own = s_vis ? key_row_checked(P, ri, e_own) : -1;
                const int r_oth = mla::pair_visible(e_oth, ri) ? key_row_checked(P, ri, e_oth) : -1;
                const bool v_own = r_own >= 0, v_oth = r_oth >= 0;
                if (s_vis && !v_own) raise_error(ERR_BOUNDS);
                const uint32_t c_own = v_own ? __ldg(kv_scale + r_own) : 0u;
                const uint32_t c_oth = v_oth ? __ldg(kv_scale + r_oth) : 0u;
                if (b + 1 < nblocks) {
                    e_own = entry(s_own + C::BLK * (b + 1));
                    e_oth = entry(s_oth + C::BLK * (b + 1));
                }
                // a NaN scale (255) says nothing about the others'
                const uint32_t top = max(c_own == 255u ? 0u : c_own, c_oth == 255u ? 0u : c_oth);
                er = max(er, (int)__reduce_max_sync(0xffffffffu, top));
                const int sl = gb & (C::NINFO - 1);
                if (gb >= C::NINFO) okw = wait(info_free(sl), ((gb / C::NINFO) - 1) & 1);
                if (!__all_sync(0xffffffffu, okw) || misc[1]) {
                    ok = false;
                    break;
                }
                info[128 * sl + 32 * pw + lane] = v_own ? ue8m0_to_float(c_own) : -1.0f;
                if (lane == 0) ers[4 * sl + pw] = er;
                __syncwarp();
                if (lane == 0) mbar_arrive(info_full(sl));
                // the softmax has what it needs to start: the previous unit's epilogue
                if (b == 0 && pt >= 0 && !epilogue(pt, ps, nq - 2)) {
                    ok = false;
                    break;
                }
            }
            pt = t;
            ps = split;
        }
        if (ok && pt >= 0) ok = epilogue(pt, ps, nq - 1);
        if (!ok && lane == 0) abort_pair();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REG_SOFT));
        // ------------------------------------------------ softmax
        const int st = tid - 32 * C::SOFT0;                  // 0 .. 255
        const int quarter = warp & 3;
        const int h2 = (warp - C::SOFT0) >> 2;               // head half handled by this warp
        const int key = quarter * 32 + lane;                 // this thread's key among the CTA's 128
        const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
        const uint32_t xm_peer = mapa_shared(sbase + C::OFF_XM, (uint32_t)peer);
        const uint32_t xbar_peer = mapa_shared(xbar(0), (uint32_t)peer);
        const uint32_t s_free_lead = mapa_shared(s_free(0), 0);
        const uint32_t p_full_lead = mapa_shared(p_full, 0);
        const uint32_t p_in_peer = mapa_shared(p_in, (uint32_t)peer);
        // row 128 cr + key of the P'^T buffers of the CTA holding heads 64 h2 .. + 63
        const uint32_t prow = (uint32_t)(128 * cr + key);
        const uint32_t ph_row = (h2 == cr ? ph_s : mapa_shared(ph_s, (uint32_t)peer)) + prow * 64;
        const uint32_t pl_row = ph_row + (C::OFF_PL - C::OFF_PH);
        const uint32_t pswz = (prow >> 1) & 3;
        bool ok = run;
        int gb0 = 0;                                         // blocks of the earlier units
        int nq = 0;                                          // units with blocks so far
        int qslot = 0, qphase = 0;
        for (int j = 0, u = pair0; ok && u < units; ++j, u += npairs) {
            const int t = T - 1 - u / nsplit;
            const int split = u % nsplit;
            // The first unit's q is split here, where eight warps have nothing to do yet (2.4 us; the four
            // preparing warps took 3.8, with the gathers' rows waiting).
            bool got = true;
            float q_scale[2] = {0.f, 0.f};
            if (j == 0) {
                got = wait(q_raw, 0);
                if (__all_sync(0xffffffffu, got))
                    split_q(std::true_type{}, smem + C::OFF_Q, smem + C::OFF_Q, 8 * (warp - C::SOFT0), 2, [&](int r, float s) {
                        qsc[64 * cr + r] = s;
                        if ((r & 4) == 0) q_scale[0] = s;
                        else q_scale[1] = s;
                    });
                fence_proxy_async_smem();
            }
            got = wait(unit_full(j & 1), (j >> 1) & 1) && got;
            const int nblocks = got ? unit_nb[j & 1] : 0;
            if (named_bar_or(1, 256, !got || misc[1] != 0)) {
                ok = false;
                if (st == 0) abort_pair();
                break;
            }
            if (j == 0 && nblocks > 0) {                     // what the preparing warps do for later units
                if ((lane & 7) == 0) {
                    const int at = 64 * cr + 8 * (warp - C::SOFT0) + (lane >> 3);
                    st_async_f32(qsc_peer + 4u * at, q_scale[0], qs_full_peer);
                    st_async_f32(qsc_peer + 4u * (at + 4), q_scale[1], qs_full_peer);
                }
                if (lane == 0 && warp < C::SOFT0 + 4) {
                    mbar_arrive_remote(q_ready_lead);
                    if (warp == C::SOFT0) mbar_expect_tx(qs_full(0), 64 * 4);
                    else mbar_arrive(qs_full(0));
                }
            }
            if (st == 0) mbar_arrive(unit_free(j & 1));
            const int mqh = (st >> 1) * 4 + (st & 1);        // st < 128: this thread's head in mq
            if (st < 128) mq[mqh] = INFINITY;                // minus the reference maximum
            const float *qs = qsc + 128 * qslot;
            uint64_t l[32];                                  // row sums of head pairs
#pragma unroll
            for (int i = 0; i < 32; ++i) l[i] = 0ull;
            int er = C::ER_MIN;
            float m_top = -INFINITY, sunk = 0.f;             // st < 128: of this thread's head (below)
            for (int b = 0; b < nblocks; ++b) {
                const int gb = gb0 + b;
                const int sl = gb & (C::NINFO - 1);
                const bool fail = misc[1] != 0 || !wait(info_full(sl), (gb / C::NINFO) & 1) ||
                                  (b == 0 && !wait_cluster(qs_full(qslot), qphase)) ||
                                  !wait(s_full(gb & 1), (gb >> 1) & 1);
                __syncwarp();
                tc_fence_after();
                const float ks = info[128 * sl + key];
                const int4 er4 = reinterpret_cast<const int4 *>(ers)[sl];
                const int er_new = max(max(er4.x, er4.y), max(er4.z, er4.w));
                __syncwarp();
                if (lane == 0) mbar_arrive(info_free(sl));
                const bool vis = !(ks < 0.f);
                const uint32_t sb = t_lane + C::TMEM_S + 128 * (gb & 1) + 64 * h2;
                const bool all_vis = __all_sync(0xffffffffu, vis);
                // the key's scale against the largest so far (log2)
                const float de = fmaxf((float)((int)(__float_as_uint(ks) >> 23) - er_new), -C::SPAN);
                // ---- block maxima of score + scale of this CTA's keys (per head), then of the pair
#pragma unroll 1
                for (int jj = 0; jj < 2; ++jj) {
                    uint32_t sr[32];
                    tmem_ld32(sb + 32 * jj, sr);
                    tmem_wait_ld();
                    tmem_regs_ready(sr);
                    if (!all_vis) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) sr[i] = vis ? sr[i] : 0xff800000u;
                    }
                    const float k1 = vis ? ks : 1.0f;
                    float4 *r4 = reinterpret_cast<float4 *>(red + quarter * 128 + 64 * h2 + 32 * jj);
                    const float4 *q4 = reinterpret_cast<const float4 *>(qs + 64 * h2 + 32 * jj);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 q = q4[i];
                        float4 r;
                        r.x = warp_fmax(fmaf(__uint_as_float(sr[4 * i]) * k1, q.x, de));
                        r.y = warp_fmax(fmaf(__uint_as_float(sr[4 * i + 1]) * k1, q.y, de));
                        r.z = warp_fmax(fmaf(__uint_as_float(sr[4 * i + 2]) * k1, q.z, de));
                        r.w = warp_fmax(fmaf(__uint_as_float(sr[4 * i + 3]) * k1, q.w, de));
                        if (lane == 0) r4[i] = r;
                    }
                }
                // every exit decision is taken through a barrier, so the 8 warps stay together
                if (named_bar_or(1, 256, fail)) {
                    ok = false;
                    break;
                }
                if (st < 128) {
                    const int h = st;
                    const float m_cta = fmaxf(fmaxf(red[h], red[128 + h]), fmaxf(red[256 + h], red[384 + h]));
                    st_async_f32(xm_peer + 4u * (128 * (gb & 1) + h), m_cta, xbar_peer + 8u * (gb & 1));
                    if (st == 0) mbar_expect_tx(xbar(gb & 1), 128 * 4);
                    if (b == 0) mq[mqh + 2] = qs[h];
                    const float m_old = -mq[mqh];
                    const bool okx = wait_cluster(xbar(gb & 1), (gb >> 1) & 1);
                    const float m_blk = fmaxf(m_cta, okx ? xm[128 * (gb & 1) + h] : m_cta);
                    // the largest so far: what was seen before loses as much as the largest scale gained,
                    // SPAN at most (`sunk` so far)
                    const float gain = m_top == -INFINITY ? 0.f : fminf((float)(er_new - er), C::SPAN - sunk);
                    sunk += gain;
                    m_top = fmaxf(m_top - gain, m_blk);
                    // up where the block exceeds the reference by more than TAU, down where it lies more than
                    // DOWN below (a block without a visible key, or with NaN only, changes nothing)
                    const float m_new = fmaxf(m_blk, m_top - C::DEPTH);
                    const bool need = m_blk > -INFINITY && (m_blk > m_old + C::TAU || m_new < m_old - C::DOWN);
                    fs[h] = (need && m_old != -INFINITY) ? ex2_approx(m_old - m_new) : 1.0f;
                    if (need) mq[mqh] = -m_new;
                    if (!okx) misc[1] = 1;
                    const uint32_t w = __ballot_sync(0xffffffffu, need);
                    if (lane == 0) mvw[warp - C::SOFT0] = b > 0 ? w : 0u;   // warp i: heads 32 i .. + 31
                }
                named_bar(1, 256);
                // the previous PV (this unit's or the last one's) has read P'^T and, for a rescale, O^T is whole
                bool okp = true;
                if (gb > 0) okp = wait(pv_done, (gb - 1) & 1);
                if (!okp) misc[1] = 1;
                __syncwarp();
                const uint4 mv = *reinterpret_cast<const uint4 *>(mvw);
                if ((mv.x | mv.y | mv.z | mv.w) != 0u || (b > 0 && er_new != er)) {
                    tc_fence_after();
                    // the row sums of this warp's heads, 16 at a time
                    const uint32_t own[2] = {h2 ? mv.z : mv.x, h2 ? mv.w : mv.y};
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if ((own[c >> 1] >> (16 * (c & 1)) & 0xffffu) != 0u) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 w = reinterpret_cast<const float4 *>(fs)[16 * h2 + 4 * c + i];
                                l[8 * c + 2 * i] = mul_f32x2(l[8 * c + 2 * i], pack_f32x2(w.x, w.y));
                                l[8 * c + 2 * i + 1] = mul_f32x2(l[8 * c + 2 * i + 1], pack_f32x2(w.z, w.w));
                            }
                        }
                    }
                    // O^T: every column for a new exponent, else the groups of 16 heads with one that moved
                    const uint32_t oa = t_lane + C::TMEM_O + 128 * h2;
                    const float fe = exp2f((float)(er - er_new));
                    uint32_t groups = ((mv.x & 0xffffu) ? 1u : 0u) | ((mv.x >> 16) ? 2u : 0u) | ((mv.y & 0xffffu) ? 4u : 0u) |
                                      ((mv.y >> 16) ? 8u : 0u) | ((mv.z & 0xffffu) ? 16u : 0u) | ((mv.z >> 16) ? 32u : 0u) |
                                      ((mv.w & 0xffffu) ? 64u : 0u) | ((mv.w >> 16) ? 128u : 0u);
                    if (er_new != er) groups = 255u;
#pragma unroll 1
                    while (groups != 0u) {
                        const int c = __ffs(groups) - 1;
                        groups &= groups - 1u;
                        uint32_t o[16];
                        tmem_ld16(oa + 16 * c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float4 f = reinterpret_cast<const float4 *>(fs)[4 * c + i];
                            o[4 * i] = __float_as_uint(__uint_as_float(o[4 * i]) * (f.x * fe));
                            o[4 * i + 1] = __float_as_uint(__uint_as_float(o[4 * i + 1]) * (f.y * fe));
                            o[4 * i + 2] = __float_as_uint(__uint_as_float(o[4 * i + 2]) * (f.z * fe));
                            o[4 * i + 3] = __float_as_uint(__uint_as_float(o[4 * i + 3]) * (f.w * fe));
                        }
                        tmem_st16(oa + 16 * c, o);
                    }
                    tmem_wait_st();
                    // before the st.async below too: their bytes on p_in are all that the next PV waits for
                    // from the warps whose P' goes to the other CTA
                    tc_fence_before();
                }
                er = er_new;
                // ---- P'^T of this thread's key for its 64 heads, 16 heads at a time
                const float kf = vis ? ks * __uint_as_float((uint32_t)min(254 + C::BASE - er, 254) << 23) : 0.f;
                const uint64_t ks2 = pack_f32x2(ks, ks), kf2 = pack_f32x2(kf, kf);
                auto probabilities = [&](auto masked) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint32_t sr[16], hi[8], lo[8];
                        tmem_ld16(sb + 16 * v, sr);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float4 w = reinterpret_cast<const float4 *>(mq)[32 * h2 + 8 * v + i];
                            const uint64_t s2 = pack_f32x2(__uint_as_float(sr[2 * i]), __uint_as_float(sr[2 * i + 1]));
                            const uint64_t z2 = fma3_f32x2(mul_f32x2(s2, ks2), pack_f32x2(w.z, w.w), pack_f32x2(w.x, w.y));
                            float p0, p1;
                            unpack_f32x2(z2, p0, p1);
                            p0 = ex2_approx(p0);
                            p1 = ex2_approx(p1);
                            if (masked.value) {
                                p0 = vis ? p0 : 0.f;
                                p1 = vis ? p1 : 0.f;
                            }
                            const uint64_t p2 = pack_f32x2(p0, p1);
                            l[8 * v + i] = add_f32x2(l[8 * v + i], p2);
                            unpack_f32x2(mul_f32x2(p2, kf2), p0, p1);
                            split_8bit(__floats2half2_rn(p0, p1), hi[i], lo[i]);
                        }
                        uint32_t h[4], g[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            h[i] = __byte_perm(hi[2 * i], hi[2 * i + 1], 0x5410);
                            g[i] = __byte_perm(lo[2 * i], lo[2 * i + 1], 0x5410);
                        }
                        const uint32_t off = (v ^ pswz) << 4;
                        if (h2 == cr) {
                            st_shared_v4(ph_row + off, h[0], h[1], h[2], h[3]);
                            st_shared_v4(pl_row + off, g[0], g[1], g[2], g[3]);
                        } else {
                            st_async_v4(ph_row + off, h[0], h[1], h[2], h[3], p_in_peer);
                            st_async_v4(pl_row + off, g[0], g[1], g[2], g[3], p_in_peer);
                        }
                    }
                };
                if (all_vis) probabilities(std::false_type{});
                else probabilities(std::true_type{});
                tc_fence_before();
                if (h2 == cr) fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive_remote(s_free_lead + 8u * (gb & 1));    // S^T consumed
                    if (h2 == cr) mbar_arrive_remote(p_full_lead);      // this warp's 32 rows are in place
                }
            }
            if (!ok && st == 0) abort_pair();

            // ---- row sums of the pair: lse, and the output factors for the epilogue (after an abort the
            // teardown writes the rows)
            if (nblocks > 0 && ok) {
#pragma unroll
                for (int jj = 0; jj < 2; ++jj) {
                    float v[32];
#pragma unroll
                    for (int i = 0; i < 16; ++i) unpack_f32x2(l[16 * jj + i], v[2 * i], v[2 * i + 1]);
                    red[quarter * 128 + 64 * h2 + 32 * jj + lane] = mla::transpose_reduce32<false>(v, lane);
                }
                named_bar(1, 256);
                if (st < 128) {
                    const int h = st;
                    const float l_cta = (red[h] + red[128 + h]) + (red[256 + h] + red[384 + h]);
                    st_async_f32(mapa_shared(sbase + C::OFF_XL + 4u * h, (uint32_t)peer), l_cta,
                                 mapa_shared(lbar, (uint32_t)peer));
                    if (st == 0) mbar_expect_tx(lbar, 128 * 4);
                    const bool okl = wait_cluster(lbar, nq & 1);
                    if (!okl) misc[1] = 1;
                    // the two CTAs add the same two numbers in the same order
                    const float l_tot = cr == 0 ? l_cta + xl[h] : xl[h] + l_cta;
                    // O^T holds sum p 2^(e - er + BASE) code
                    fo[128 * (nq & 1) + h] =
                        !okl ? NAN : (l_tot != 0.f ? ue8m0_to_float((uint32_t)(er - C::BASE)) / l_tot : 0.f);
                    if ((h >> 6) == cr) {
                        const int64_t at = SPLIT ? ((int64_t)t * nsplit + split) * 128 + h : (int64_t)t * 128 + h;
                        const float lv =
                            okl ? (l_tot != 0.f ? (log2f(l_tot) - mq[mqh]) * 0.6931471805599453f : -INFINITY) : NAN;
                        (SPLIT ? sp.lse_part : lse)[at] = lv;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(fo_full(nq & 1));
                }
            } else {
                fill_unit<SPLIT>(sp, out, lse, t, split, cr, st, 0.f, -INFINITY);   // no visible slot
            }
            gb0 += nblocks;
            if (nblocks > 0) {
                ++nq;
                if (++qslot == C::NQS) {
                    qslot = 0;
                    qphase ^= 1;
                }
            }
        }
    }
    // ---- teardown: nothing of either CTA is in flight past this point.  After an abort
    // (either CTA's flag, so both take the same branch) the even CTA first waits, bounded,
    // until the last position either CTA issued into each slot has landed.  Each CTA hands
    // its final flag to the peer before the cluster barrier: past that barrier the peer may
    // already have exited, so nothing reads the peer's shared memory there.
    tc_fence_before();
    __syncthreads();                                         // this CTA's roles are done
    if (tid == 0) st_cluster_u32(mapa_shared(sbase + C::OFF_MISC + 24, (uint32_t)peer), misc[1]);
    cluster_sync();
    const bool aborted = misc[1] != 0u || misc[6] != 0u;     // the same in both CTAs
    if (aborted) {
        if (cr == 0 && run && tid < C::NSLOT) {
            const int *lp = reinterpret_cast<const int *>(smem + C::OFF_LASTPOS);
            const int pmax = max(lp[tid], lp[C::NSLOT + tid]);
            if (pmax >= 0) wait_cluster(pfull(tid), (uint32_t)(pmax / C::NSLOT) & 1u);
        }
        cluster_sync();
        // A wait that gave up may have left any of this pair's rows unwritten or wrong: all of them are NaN.
        if (tid == 0) raise_error(ERR_WAIT_TIMEOUT);
        int block, st;                                       // (read again: kept all along they cost spills)
        asm volatile("mov.u32 %0, %%ctaid.x;\n\tmov.u32 %1, %%tid.x;" : "=r"(block), "=r"(st));
        st -= 32 * C::SOFT0;
        const int parts = SPLIT ? sp.nsplit : 1;
        if (st >= 0)
            for (int u = block >> 1; u < P.total_q * parts; u += (int)(gridDim.x >> 1))
                fill_unit<SPLIT>(sp, out, lse, P.total_q - 1 - u / parts, u % parts, block & 1, st, NAN, NAN);
    }
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, 512);
    }
}

}  // namespace mla8
}  // namespace dsa
