"""Host-only checks of the serving operators: refusals before any launch, RoPE frequencies,
and pins of the 64-bit restatements the GPU parity tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attention_lightning_indexer_b200 as dsa
import serving_reference as ref
from attention_lightning_indexer_b200._native import DsaRope

FAKE = 1 << 20                       # aligned, never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


# ------------------------------------------------------------------ page plan

def _plan(batch=4, max_pages=8, n_free=2, n_pages=16, n_tokens=8, **ptr):
    p = dict(cached=FAKE, new=FAKE, table=FAKE, free=FAKE, head=None, cu_q=FAKE, cu_k=FAKE, pos=FAKE, rows=FAKE, counts=FAKE)
    p.update(ptr)
    return dsa.load().dsa_paged_plan(batch, p["cached"], p["new"], p["table"], max_pages, p["free"], n_free, p["head"],
                                     n_pages, p["cu_q"], p["cu_k"], p["pos"], p["rows"], n_tokens, p["counts"], None)


@pytest.mark.parametrize("kw", [dict(batch=0), dict(batch=-1), dict(max_pages=0), dict(n_free=-1), dict(n_pages=0),
                                dict(n_pages=1 << 25), dict(n_tokens=-1), dict(cached=None), dict(new=None),
                                dict(table=None), dict(cu_q=None), dict(cu_k=None), dict(counts=None), dict(free=None),
                                dict(pos=None), dict(rows=None), dict(cached=FAKE + 2), dict(head=FAKE + 1),
                                dict(head=FAKE + 4)])   # the last: the head may not be the count it is advanced by
def test_plan_refuses(kw):
    assert _plan(**kw) == INVALID


def test_plan_refuses_too_many_requests():
    assert _plan(batch=8193) == UNSUPPORTED


def test_plan_reference_by_hand():
    table = np.array([[3, -1, -1], [5, 6, -1], [-1, -1, -1]], np.int32)
    cu_q, cu_k, pos, rows, t, counts = ref.plan([63, 128, 0], [2, 1, 0], table, np.array([9, 1, 0], np.int32), 1, 16, 5)
    assert cu_q.tolist() == [0, 2, 3, 3] and cu_k.tolist() == [0, 65, 194, 194]
    assert pos.tolist() == [63, 64, 128, 0, 0]
    assert rows.tolist() == [3 * 64 + 63, 1 * 64, 0 * 64, -1, -1]
    assert t.tolist() == [[3, 1, -1], [5, 6, 0], [-1, -1, -1]]
    assert counts.tolist() == [3, 2, 129, 0]
    assert ref.plan([63], [2], table[:1], np.array([], np.int32), 0, 16, 5)[5].tolist() == [0, 0, 0, 1]


# ------------------------------------------------------------------ RoPE

def _rope(x=FAKE, pos=FAKE, freq=FAKE, out=FAKE + (1 << 16), **kw):
    d = dict(n_tokens=4, n_heads=2, head_dim=64, rope_begin=0, rope_dim=64, layout=0, dtype=0, x_token_stride=128,
             x_head_stride=64, out_token_stride=128, out_head_stride=64, scale=1.0, transposed=0)
    d.update(kw)
    r = DsaRope(*[d[n] for n, _ in DsaRope._fields_])
    return dsa.load().dsa_rope(ctypes.byref(r), x, pos, freq, out, None)


@pytest.mark.parametrize("kw", [dict(n_tokens=-1), dict(n_heads=-1), dict(head_dim=0), dict(rope_begin=-2),
                                dict(rope_dim=0), dict(rope_dim=63), dict(rope_begin=2), dict(layout=2),
                                dict(x_token_stride=-1), dict(out_head_stride=-1), dict(out_head_stride=63),
                                dict(out_token_stride=0), dict(out_token_stride=64), dict(out_token_stride=127),
                                dict(out_token_stride=64, out_head_stride=192), dict(scale=math.inf),
                                dict(scale=math.nan), dict(x=None),
                                dict(pos=None), dict(freq=None), dict(out=None), dict(x=FAKE + 1), dict(freq=FAKE + 2),
                                dict(dtype=2, out=FAKE + 2), dict(out=FAKE, x_head_stride=128)])
def test_rope_refuses(kw):
    assert _rope(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(head_dim=1026, rope_dim=1026, out_head_stride=1026, out_token_stride=4096)])
def test_rope_unsupported(kw):
    assert _rope(**kw) == UNSUPPORTED


def test_rope_without_tokens_or_heads_is_nothing():
    assert _rope(n_tokens=0) == OK and _rope(n_heads=0) == OK
    assert dsa.load().dsa_rope(None, FAKE, FAKE, FAKE, FAKE, None) == INVALID


def test_rope_frequencies():
    f, att = dsa.dsa_rope_frequencies(64)
    assert att == 1.0
    np.testing.assert_allclose(f.numpy(), 10000.0 ** (-np.arange(32) / 32), rtol=2.0 ** -23)
    g, att = dsa.dsa_rope_frequencies(64, 10000.0, 40.0, 4096.0, 32.0, 1.0)
    assert att == pytest.approx(0.1 * math.log(40) + 1, rel=1e-15)
    # ramp between the dims that turn 32 times and once in 4096 tokens: floor(10.47) and ceil(22.51)
    w = np.clip((np.arange(32) - 10) / 13, 0, 1)
    base = 10000.0 ** (-np.arange(32) / 32)
    np.testing.assert_allclose(g.numpy(), base * (w / 40 + 1 - w), rtol=2.0 ** -23)
    assert torch.equal(f[:11], g[:11])


@pytest.mark.parametrize("args", [(63,), (0,), (-2,), (64, 1.0), (64, 1e4, 0.5), (64, 1e4, 40.0, 0.0),
                                  (64, 1e4, 40.0, 4096.0, 1.0, 32.0), (64, 1e4, 40.0, 4096.0, 32.0, 0.0), (64, math.nan)])
def test_rope_frequencies_refuse(args):
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_rope_frequencies(*args)
    assert e.value.code == INVALID


def test_rope_reference_is_a_complex_rotation_and_its_transpose_undoes_it():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 3, 20))
    pos, freq = np.array([0, 1, 7, 4096, 163839]), rng.uniform(0.01, 1, 6).astype(np.float32)
    for layout in (0, 1):
        y = ref.rope(x, pos, freq, layout, 4, 12, scale=1.5)
        part = x[..., 4:16]
        u, v = (part[..., :6], part[..., 6:]) if layout == 0 else (part[..., 0::2], part[..., 1::2])
        w = (u + 1j * v) * 1.5 * np.exp(1j * pos[:, None] * freq.astype(np.float64))[:, None, :]
        got = y[..., 4:16]
        gu, gv = (got[..., :6], got[..., 6:]) if layout == 0 else (got[..., 0::2], got[..., 1::2])
        np.testing.assert_allclose(gu + 1j * gv, w, atol=1e-12)
        np.testing.assert_array_equal(y[..., :4], x[..., :4])
        np.testing.assert_allclose(ref.rope(y, pos, freq, layout, 4, 12, scale=1 / 1.5, transposed=True), x, atol=1e-12)
        # the transposed map is the gradient: <g, R x> = <R^T g, x>
        g = rng.standard_normal(x.shape)
        back = ref.rope(g, pos, freq, layout, 4, 12, scale=1.5, transposed=True)
        assert np.sum(g * y) == pytest.approx(np.sum(back * x), rel=1e-12)


# ------------------------------------------------------------------ 8-bit cache write

def _write(n=4, form=2, eps=1e-6, **ptr):
    names = ("k_raw", "kv_raw", "pos", "rows", "ln_w", "ln_b", "rms_w", "freq")
    p = {k: FAKE for k in names + ("kc", "ks", "kv", "kvs")}
    p.update(ptr)
    return dsa.load().dsa_cache_write_fp8(n, *[p[k] for k in names], eps, form, p["kc"], p["ks"], p["kv"], p["kvs"], None)


@pytest.mark.parametrize("kw", [dict(n=-1), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(k_raw=None),
                                dict(kv_raw=FAKE + 8), dict(rows=None), dict(freq=None), dict(kc=None), dict(kv=None),
                                dict(kv=FAKE + 8), dict(kvs=None), dict(ks=None), dict(form=0), dict(form=1, ks=FAKE + 2)])
def test_write_refuses(kw):
    assert _write(**kw) == INVALID


def test_write_unknown_key_type_and_no_tokens():
    assert _write(form=3) == UNSUPPORTED
    assert _write(n=0) == OK


def test_e4m3_rounding_reference():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(np.nan_to_num(t, nan=-1), np.nan_to_num(ref.E4M3, nan=-1))
    rng = np.random.default_rng(1)
    v = np.concatenate([rng.standard_normal(4000) * 50, ref.E4M3[:127], -ref.E4M3[:127],
                        (ref.E4M3[:126] + ref.E4M3[1:127]) / 2, [500.0, -1e9]]).astype(np.float32)
    want = torch.from_numpy(v).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.E4M3[ref.e4m3_nearest(v.astype(np.float64))], ref.E4M3[want])


def test_scale_is_the_smallest_power_that_holds_the_row():
    a = np.array([0.0, 448.0, np.nextafter(448.0, 500), 449.0, 224.0, 1.0, 1e-40, 3e38])
    e = ref.scale_exponent(a)
    assert e[:5].tolist() == [-126, 0, 1, 1, -1] and e[6] == -126
    assert np.all(a <= 448.0 * 2.0 ** e)
    assert all(x > 448.0 * 2.0 ** (k - 1) for x, k in zip(a, e) if k > -126)


def test_quantised_row_stands_for_its_values():
    rng = np.random.default_rng(2)
    lat, rot = rng.standard_normal((50, 512)), rng.standard_normal((50, 64)) * 5
    rot[7] *= 100                                   # RoPE dims that decide the scale
    codes, byte = ref.quantise_latent(lat, rot)
    got = ref.cache_values(codes, byte)
    s = 2.0 ** (byte.astype(np.float64) - 127)[:, None]
    # half a step: 2^-4 of the value (4 significant bits) or half the smallest step 2^-9 s
    assert np.all(np.abs(got[:, :512] - lat) <= np.maximum(2.0 ** -4 * np.abs(lat), 2.0 ** -10 * s))
    # the second code halves twice four bits more, down to half the smallest step of 16 s
    assert np.all(np.abs(got[:, 512:] - rot) <= np.maximum(2.0 ** -8 * np.abs(rot), 16 * 2.0 ** -10 * s))


# ------------------------------------------------------------------ attention

def _problem(**kw):
    args = dict(batch=1, total_q=128, total_k=128, max_len_q=128, max_len_k=128, topk=64)
    args.update(kw)
    return dsa.make_problem(**args)


def _mla(p, ws=None, ws_bytes=0, **ptr):
    a = dict(q=FAKE, kv=FAKE, ks=FAKE, idx=FAKE, out=FAKE, lse=FAKE)
    a.update(ptr)
    return dsa.load().dsa_sparse_mla_fp8_fwd(None if p is None else ctypes.byref(p), a["q"], a["kv"], a["ks"], a["idx"],
                                             a["out"], a["lse"], ws, ws_bytes, None)


def test_attention_refuses():
    assert _mla(None) == INVALID
    p = _problem()
    for kw in (dict(q=None), dict(kv=None), dict(ks=None), dict(idx=None), dict(out=None), dict(lse=None),
               dict(q=FAKE + 8), dict(kv=FAKE + 8), dict(idx=FAKE + 4), dict(out=FAKE + 8), dict(lse=FAKE + 4)):
        assert _mla(p, **kw) == INVALID, kw
    assert _mla(_problem(topk=0)) == INVALID
    assert _mla(_problem(topk=4096)) == UNSUPPORTED
    assert _mla(_problem(n_heads=64)) == UNSUPPORTED
    assert _mla(_problem(total_q=0, max_len_q=0), q=None) == OK      # no query row: nothing to do


def test_attention_workspace():
    small = _problem(total_q=1, max_len_q=1, total_k=4096, max_len_k=4096, topk=2048)
    need = dsa.dsa_sparse_mla_fp8_workspace_size(small)
    assert need > 0
    assert _mla(small) == WORKSPACE
    assert _mla(small, ws=FAKE, ws_bytes=need - 1) == WORKSPACE
    assert _mla(small, ws=FAKE + 16, ws_bytes=need) == WORKSPACE
    assert dsa.load().dsa_sparse_mla_fp8_workspace_size(None) == 0
    # many rows: the images of q of 74 pairs, however many rows there are
    many = dsa.dsa_sparse_mla_fp8_workspace_size(_problem(total_q=1000, max_len_q=1000, total_k=4096, max_len_k=4096, topk=2048))
    assert many == dsa.dsa_sparse_mla_fp8_workspace_size(_problem(total_q=4000, max_len_q=4000, total_k=4096, max_len_k=4096, topk=2048))
    assert many == 74 * 2 * 9 * 64 * 128
    assert dsa.dsa_sparse_mla_fp8_workspace_size(_problem(total_q=1, max_len_q=1, total_k=4096, max_len_k=4096, topk=256)) == 0


def test_attention_reference_against_plain_softmax():
    rng = np.random.default_rng(3)
    lat, rot = rng.standard_normal((40, 512)), rng.standard_normal((40, 64))
    codes, byte = ref.quantise_latent(lat, rot)
    kv = ref.cache_values(codes, byte)
    q = rng.standard_normal((4, 576))
    rows = np.array([3, 3, 17, 39, 0])
    o, l, ot, lt = ref.attention(q, rows, kv, byte, 0.07)
    z = torch.from_numpy(q @ kv[rows].T * 0.07)
    np.testing.assert_allclose(o, (torch.softmax(z, 1) @ torch.from_numpy(kv[rows, :512])).numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(l, torch.logsumexp(z, 1).numpy(), rtol=1e-12)
    o, l, _, _ = ref.attention(q, np.array([], int), kv, byte, 0.07)
    assert np.all(o == 0) and np.all(np.isneginf(l))


# ------------------------------------------------------------------ binding

def test_binding_refuses_host_tensors():
    z = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        dsa.dsa_paged_plan(z, z, z.view(4, 1), z, z, z, z, z, z, n_pages=4)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dsa.dsa_rope(x, z, torch.zeros(32), x)
    p = _problem()
    with pytest.raises(ValueError):
        dsa.dsa_sparse_mla_fp8_fwd(p, x, z, z, z, x, z)
