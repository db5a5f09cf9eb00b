"""Attention over the 8-bit latent cache where most keys weigh little beside one of them (a
sink, as the first token of a sequence is for many heads), beside a key with a much larger
row scale, or beside another block of keys: what many small weights add up to must be kept."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_lightning_indexer_b200 as dsa
import serving_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
SM = 1 / 192 ** 0.5
BLOCK = 256                              # index slots that share a reference
HEADS = [0, 1, 63, 64, 100, 127]


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _rows(lat, score):
    """Cache rows (codes, scale bytes) of latents [n, 512] whose score against a query of
    _queries is `score` [n] (natural units, rounded to the RoPE dims' 8 bits)."""
    rot = np.zeros((len(lat), 64))
    rot[:, 5] = score
    return ref.quantise_latent(lat, rot)


def _queries(T, seed):
    """Latent part 0, one RoPE dim: the score of a key is its RoPE dim 5 times 0.8 to 1.2."""
    q = np.zeros((T, 128, 576))
    q[:, :, 512 + 5] = np.random.default_rng(seed).uniform(0.8, 1.2, (T, 128)) / SM
    return torch.from_numpy(q).to(DEV).to(torch.bfloat16)


def _rho(x):
    """Largest relative error of a weight as e4m3 + e5m2, for a weight of x times 2^4 at least: the
    first code leaves at most 2^-4 of the value above 2^-6, and 2^-10 below; the second keeps 3
    significant bits of that (an eighth, at most 2^-14 of what is below 2^-10) down to steps of
    2^-16.  And 2^-12 for the fp16 step before."""
    with np.errstate(divide="ignore"):
        return np.maximum(np.maximum(2.0 ** -8, np.minimum(2.0 ** -14 / x, 0.125)), np.minimum(2.0 ** -17 / x, 1.0)) + 2.0 ** -12


def _expected(q, codes, byte, order, heads):
    """out [H, 512], lse [H] of one query over the cache rows `order` (slot by slot) in 64 bits, and
    bounds on the kernel's error of both."""
    v = ref.cache_values(codes, byte)[order]
    e = byte[order].astype(np.float64) - 127
    qh = q.double().cpu().numpy()[heads]
    z = qh @ v.T * SM
    m = z.max(1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(1, keepdims=True)
    out, lse = p @ v[:, :512] / l, m[:, 0] + np.log(l[:, 0])
    # A weight is held times its row's scale, relative to a reference that is at most 2^4 above and
    # 2^4.8 below the largest such product of its block, and no lower than 2^-20 of the largest so far.
    c = z / np.log(2) + e[None, :]
    rho, top, hi = np.empty_like(z), np.full((len(heads), 1), -np.inf), -np.inf
    for b in range(0, len(order), BLOCK):
        s = slice(b, b + BLOCK)
        hi = max(hi, e[s].max())
        most = (z[:, s] / np.log(2) + np.maximum(e[s], hi - 24)[None, :]).max(1, keepdims=True)
        top = np.maximum(top, most)
        rho[:, s] = _rho(2.0 ** (c[:, s] - np.maximum(most, top - 20)))
    # q is exact here (one dim of 8 significant bits); the scores' sums are a few products of codes,
    # each step 2^-24: 2^-20 of the score, with the exponent's argument
    dz = 2.0 ** -20 * np.abs(z).max(1, keepdims=True) + 2.0 ** -20
    dp = p * (rho + 2 * dz)
    tol = (dp @ np.abs(v[:, :512]) + 128 * 2.0 ** -23 * (p @ np.abs(v[:, :512]))) / l + 2.0 ** -8 * np.abs(out) + 2.0 ** -30
    return out, lse, tol, dz[:, 0] + 2.0 ** -18


def _run(T, S, topk, q, codes, byte, idx):
    p = dsa.make_problem(1, T, S, T, S, topk)
    out, lse = torch.empty(T, 128, 512, dtype=torch.bfloat16, device=DEV), torch.empty(T, 128, device=DEV)
    ws = torch.full((max(256, dsa.dsa_sparse_mla_fp8_workspace_size(p)),), 255, dtype=torch.uint8, device=DEV)
    dsa.dsa_sparse_mla_fp8_fwd(p, q, dev(codes), dev(byte), dev(idx), out, lse, ws)
    dsa.dsa_check_device_errors()
    return out, lse


def _check(T, codes, byte, order, seed, most_tol=None, empty=0):
    """All T queries attend the slots `order` of a cache with T rows more (the queries' own), after
    `empty` blocks of slots without a key."""
    n = len(codes)
    codes = np.concatenate([codes, np.zeros((T, 640), np.uint8)])
    byte = np.concatenate([byte, np.full(T, 127, np.uint8)])
    q = _queries(T, seed)
    idx = np.tile(np.concatenate([np.full(empty * BLOCK, -1), order]).astype(np.int32), (T, 1))
    out, lse = _run(T, n + T, idx.shape[1], q, codes, byte, idx)
    for t in sorted({0, T // 2, T - 1}):
        o, s, tol, ltol = _expected(q[t], codes, byte, order, HEADS)
        go, gl = out[t].double().cpu().numpy()[HEADS], lse[t].double().cpu().numpy()[HEADS]
        assert np.all(np.abs(gl - s) <= ltol), (t, np.max(np.abs(gl - s) / ltol))
        assert np.all(np.abs(go - o) <= tol), (t, np.max(np.abs(go - o) / tol))
        if most_tol is not None:         # the bound says something: it is a part of the tail's output
            assert np.median(tol / np.abs(o)) <= most_tol


def _sink(seed, depth, spread, size, n=2047, direction=1.0):
    """A sink in slot 0 (latent `size` in dim 511, else 0) and n keys `depth` below it."""
    rng = np.random.default_rng(seed)
    lat = np.concatenate([np.zeros((1, 512)), direction + 0.3 * rng.standard_normal((n, 512))])
    lat[0, 511] = size
    return _rows(lat, np.concatenate([[0.0], -depth + spread * rng.standard_normal(n)]))


# one key and 2047 that together weigh 26 % to 1 % of it; sizes: the sink's row scale is far below
# the tail's, like it, and 2^5 above.  T: rows split over pairs (1, 37) and not (38, 200).
# What may be off: 2^-8 of the tail in seven of eight blocks; in the sink's own an eighth of its
# share, or all of it where the sink's scale puts it below 2^-21; and the output's rounding, 2^-8.
@pytest.mark.parametrize("T", [1, 37, 38, 200])
@pytest.mark.parametrize("depth,spread", [(8, 1), (9, 1), (10, 1), (11, 1), (12, 1), (9.5, 0), (10.4, 0), (11, 0)])
@pytest.mark.parametrize("size", [0.02, 2.0, 60.0])
def test_a_tail_beside_a_sink(T, depth, spread, size):
    codes, byte = _sink(int(10 * depth), depth, spread, size)
    _check(T, codes, byte, np.arange(2048), seed=T, most_tol=0.135)


@pytest.mark.parametrize("T", [2, 40])
def test_a_tail_without_a_direction(T):
    codes, byte = _sink(7, 10, 1, 2.0, direction=0.0)
    _check(T, codes, byte, np.arange(2048), seed=T)


# keys of a scale 2^n above the others' that weigh next to nothing themselves
@pytest.mark.parametrize("n", [1, 3, 8, 12])
@pytest.mark.parametrize("at", [0, 3, 700, 1999])
def test_a_light_key_with_a_large_scale(n, at):
    rng = np.random.default_rng(n)
    lat, score = rng.standard_normal((2000, 512)) + 0.5, 1.7 * rng.standard_normal(2000)
    lat[at] *= 2.0 ** n
    score[at] = -n - 3
    codes, byte = _rows(lat, score)
    assert byte[at] >= byte[at - 1] + n - 2
    _check(75, codes, byte, np.arange(2000), seed=n)
    _check(3, codes, byte, np.arange(2000), seed=n)


# block after block lower, or up and down: the reference follows both ways
@pytest.mark.parametrize("steps", [[0, -6, -12, -18, -24], [0, -9, 0, -9, 0, -9], [-20, 0, -20, 3, -40, -3], [0, -30, -60, -31, -33, -5]])
def test_blocks_of_unlike_weight(steps):
    rng = np.random.default_rng(len(steps))
    lat = 1 + 0.3 * rng.standard_normal((256 * len(steps), 512))
    codes, byte = _rows(lat, np.repeat(steps, 256) + 0.5 * rng.standard_normal(256 * len(steps)))
    for T in (1, 90):
        _check(T, codes, byte, np.arange(len(lat)), seed=T)


@pytest.mark.parametrize("empty", [0, 1, 2])
def test_scales_that_rise_after_blocks_without_keys(empty):
    # a heavy key with a value in one dim; a block of next to nothing with a large scale in it; a tail
    # at 2^-24: the large scale lowers all that was seen, which the empty blocks must not hide
    rng = np.random.default_rng(11)
    lat, score = 1 + 0.3 * rng.standard_normal((768, 512)), np.full(768, -60.0)
    lat[0], score[0] = 0, 0
    lat[0, 511] = 2
    lat[300] *= 2.0 ** 10
    score[512:] = -16.6              # equal weights: what rounding does to one it does to all
    codes, byte = _rows(lat, score)
    _check(80, codes, byte, np.arange(768), seed=12, most_tol=0.07, empty=empty)


def test_unlike_blocks_and_scales_with_masked_slots():
    rng = np.random.default_rng(3)
    n = 1500
    lat = (1 + 0.3 * rng.standard_normal((n, 512))) * 2.0 ** rng.integers(-6, 7, n)[:, None]
    codes, byte = _rows(lat, -3.0 * (np.arange(n) // 256 % 3) * 2 + rng.standard_normal(n))
    T, topk = 80, 1400
    idx = np.full((T, topk), -1, np.int32)
    rng_order = {}
    for t in range(T):
        keys = np.sort(rng.choice(n, 900, replace=False))
        at = np.sort(rng.choice(topk, 900, replace=False))
        idx[t, at] = keys
        rng_order[t] = (keys, at)
    idx[5, :300] = -1                    # an empty first block
    codes2 = np.concatenate([codes, np.zeros((T, 640), np.uint8)])
    byte2 = np.concatenate([byte, np.full(T, 127, np.uint8)])
    q = _queries(T, 4)
    out, lse = _run(T, n + T, topk, q, codes2, byte2, idx)
    for t in (0, 5, 41, 79):
        # slots as the kernel groups them: masked ones stand in as zero keys of no weight
        slots = idx[t]
        v = ref.cache_values(codes2, byte2)
        live = slots >= 0
        e = np.where(live, byte2[slots].astype(float) - 127, -np.inf)
        z = np.where(live, q[t].double().cpu().numpy()[HEADS] @ v[slots].T * SM, -np.inf)
        m = z.max(1, keepdims=True)
        p = np.exp(z - m)
        l = p.sum(1, keepdims=True)
        o, s = p @ v[slots][:, :512] / l, m[:, 0] + np.log(l[:, 0])
        c = z / np.log(2) + np.where(live, e, 0)
        rho, top = np.zeros_like(z), np.full((len(HEADS), 1), -np.inf)
        for b in range(0, topk, BLOCK):
            k = slice(b, b + BLOCK)
            most = c[:, k].max(1, keepdims=True)
            top = np.maximum(top, most)
            with np.errstate(invalid="ignore"):
                x = np.where(np.isfinite(c[:, k]), 2.0 ** (c[:, k] - np.maximum(most, top - 20)), 1.0)
            rho[:, k] = _rho(x)
        dz = 2.0 ** -20 * np.abs(z[:, live]).max(1, keepdims=True) + 2.0 ** -20
        av = np.abs(v[slots][:, :512])
        tol = ((p * (rho + 2 * dz)) @ av + 128 * 2.0 ** -23 * (p @ av)) / l + 2.0 ** -8 * np.abs(o) + 2.0 ** -30
        go, gl = out[t].double().cpu().numpy()[HEADS], lse[t].double().cpu().numpy()[HEADS]
        assert np.all(np.abs(gl - s) <= dz[:, 0] + 2.0 ** -18)
        assert np.all(np.abs(go - o) <= tol), (t, np.max(np.abs(go - o) / tol))
