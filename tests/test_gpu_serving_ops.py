"""Parity of the serving operators (page plan, RoPE, 8-bit cache write, attention over the
8-bit latent cache) with their 64-bit restatements, at the sizes, layouts and masks where
they can go wrong, and a run of them together."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_lightning_indexer_b200 as dsa
import serving_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = torch.int32


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


# ------------------------------------------------------------------ page plan

def _run_plan(cached, new, table, free, head, n_pages, n_tokens, stream=None):
    B = len(cached)
    o = dict(cu_q=torch.full((B + 1,), 77, dtype=I32, device=DEV), cu_k=torch.full((B + 1,), 77, dtype=I32, device=DEV),
             positions=torch.full((n_tokens,), 77, dtype=I32, device=DEV), rows=torch.full((n_tokens,), 77, dtype=I32, device=DEV),
             counts=torch.full((4,), 77, dtype=I32, device=DEV))
    t = dev(table, I32)
    dsa.dsa_paged_plan(dev(np.array(cached), I32), dev(np.array(new), I32), t, dev(np.array(free, np.int32), I32), o["cu_q"],
                       o["cu_k"], o["positions"], o["rows"], o["counts"], n_pages=n_pages,
                       free_head=None if head is None else torch.tensor([head], dtype=I32, device=DEV))
    return o["cu_q"], o["cu_k"], o["positions"], o["rows"], t, o["counts"]


def _check_plan(cached, new, table, free, head, n_pages, n_tokens):
    got = _run_plan(cached, new, table, free, head, n_pages, n_tokens)
    want = ref.plan(cached, new, table, np.array(free, np.int32), head or 0, n_pages, n_tokens)
    for g, w, name in zip(got, want, ("cu_q", "cu_k", "positions", "rows", "table", "counts")):
        np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)


def _request_batch(B, ctx, most, seed, spare=3):
    rng = np.random.default_rng(seed)
    cached, new = rng.integers(0, ctx + 1, B), rng.integers(0, most + 1, B)
    width = -(-(ctx + most) // 64) + 1
    old = -(-cached // 64)
    extra = -(-(cached + new) // 64) - old
    n_pages = int(old.sum() + extra.sum()) + spare
    perm = rng.permutation(n_pages).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :old[b]] = perm[at:at + old[b]]
        at += old[b]
    return cached, new, table, perm[at:], n_pages


@pytest.mark.parametrize("B,ctx,most,pad", [(1, 0, 1, 0), (1, 63, 1, 5), (1, 64, 200, 0), (7, 300, 0, 3), (33, 200, 3, 0),
                                            (511, 500, 70, 9), (513, 130, 1, 0), (1024, 64, 5, 1), (8192, 130, 2, 100)])
def test_plan_matches_reference(B, ctx, most, pad):
    cached, new, table, free, n_pages = _request_batch(B, ctx, most, seed=B + ctx)
    _check_plan(cached, new, table, free, None, n_pages, int(new.sum()) + pad)


def test_plan_page_borders_and_free_head():
    table = np.array([[4, -1, -1], [5, -1, -1], [6, 7, -1], [-1, -1, -1]], np.int32)
    _check_plan([63, 64, 65, 0], [1, 1, 64, 129], table, [9, 8, 1, 0, 2, 3, 11], 1, 12, 300)


def test_plan_long_sequence_and_many_tokens():
    # one request of 20,000 new tokens (several CTAs) beside empty ones
    cached, new = np.array([5, 0, 100000, 7]), np.array([0, 20000, 1, 0])
    width = 1600
    rng = np.random.default_rng(5)
    perm = rng.permutation(4000).astype(np.int32)
    table = np.full((4, width), -1, np.int32)
    table[0, :1], table[2, :1563], table[3, :1] = perm[:1], perm[1:1564], perm[1564:1565]
    _check_plan(cached, new, table, perm[1565:], None, 4000, 20001)


@pytest.mark.parametrize("case", ["pages", "head", "table", "axis", "negative", "keys"])
def test_plan_that_cannot_be_served_is_an_empty_batch(case):
    cached, new, table, free, n_pages = _request_batch(9, 200, 70, seed=3, spare=0)
    head, T = 0, int(new.sum())
    if case == "pages":
        free = free[:-1]
    elif case == "head":
        head = 1
    elif case == "table":
        table = np.ascontiguousarray(table[:, :2])
    elif case == "axis":
        T -= 1
    elif case == "negative":
        new = new.copy()
        new[4] = -1
    elif case == "keys":
        cached = np.full(9, 2 ** 31 - 100)
        new = np.ones(9, int)
    _check_plan(cached, new, table, free, head, n_pages, T)


def test_plan_page_numbers_outside_the_pool_give_no_row():
    dsa.dsa_check_device_errors()
    table = np.array([[40, -1]], np.int32)
    cu_q, cu_k, pos, rows, t, counts = _run_plan([10], [60], table, [-3], None, 16, 60)
    assert rows.cpu().tolist() == [-1] * 60 and counts.cpu().tolist() == [60, 1, 70, 0]
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_check_device_errors()
    assert e.value.code == 6
    dsa.dsa_check_device_errors()


def test_plan_captured_steps_follow_the_lengths():
    cached = torch.tensor([60, 0, 127], dtype=I32, device=DEV)
    new = torch.ones(3, dtype=I32, device=DEV)
    table = torch.full((3, 4), -1, dtype=I32, device=DEV)
    table[0, 0], table[2, 0], table[2, 1] = 8, 6, 7
    free = torch.arange(5, -1, -1, dtype=I32, device=DEV)
    head = torch.zeros(1, dtype=I32, device=DEV)
    cu_q, cu_k = (torch.empty(4, dtype=I32, device=DEV) for _ in range(2))
    pos, rows = (torch.empty(4, dtype=I32, device=DEV) for _ in range(2))
    counts = torch.zeros(4, dtype=I32, device=DEV)

    def step():
        dsa.dsa_paged_plan(cached, new, table, free, cu_q, cu_k, pos, rows, counts, n_pages=9, free_head=head)
        cached.add_(new)
        head.add_(counts[1:2])

    want_c, want_t, want_h = cached.cpu().numpy(), table.cpu().numpy(), 0
    step()                                     # warm-up: the first step
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(6):
        if k > 0:
            g.replay()
        r = ref.plan(want_c, np.ones(3, int), want_t, free.cpu().numpy(), want_h, 9, 4)
        for got, w in zip((cu_q, cu_k, pos, rows, table, counts), r):
            np.testing.assert_array_equal(got.cpu().numpy(), w)
        want_c, want_t, want_h = want_c + 1, r[4], want_h + int(r[5][1])


# ------------------------------------------------------------------ RoPE

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _check_rope(x, out, pos, freq, layout, begin, dim, scale=1.0, transposed=False):
    x64 = x.double().cpu().numpy().copy()
    dsa.dsa_rope(x, pos, freq, out, layout=layout, rope_begin=begin, rope_dim=dim, scale=scale, transposed=transposed)
    got = out.double().cpu().numpy()
    want = ref.rope(x64, pos.cpu().numpy(), freq.cpu().numpy(), layout, begin, dim, scale, transposed)
    # the copied dims are the same bits; a rotated one is one rounding (half a step of its type,
    # or of the smallest subnormal) from products in fp32: cosine, product and sum each 2^-24
    eps, tiny = torch.finfo(x.dtype).eps / 2, torch.finfo(x.dtype).smallest_normal * torch.finfo(x.dtype).eps / 2
    rot = np.zeros(x.shape[-1], bool)
    rot[begin:begin + dim] = True
    np.testing.assert_array_equal(got[..., ~rot], x64[..., ~rot])
    mag = ref.rope(np.abs(x64), np.zeros(len(pos)), freq.cpu().numpy(), layout, begin, dim, scale)
    iu = begin + (np.arange(dim // 2) if layout == 0 else 2 * np.arange(dim // 2))
    iv = iu + (dim // 2 if layout == 0 else 1)
    both = np.zeros_like(mag)
    both[..., iu] = both[..., iv] = mag[..., iu] + mag[..., iv]
    err = np.abs(got - want)[..., rot]
    lim = (eps * np.abs(want) + 3 * 2.0 ** -24 * (1 + eps) * both + tiny)[..., rot]
    assert np.all(err <= lim), f"worst {np.max(err / lim)}"


def _inputs(T, H, D, dtype, seed=0, dim=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(T, H, D, generator=g, device=DEV).to(dtype)
    pos = torch.randint(0, 163840, (T,), generator=g, device=DEV).to(I32)
    pos[0] = 0
    pos[-1] = 163839
    freq = dsa.dsa_rope_frequencies(dim or D, factor=40.0)[0].to(DEV)
    return x, pos, freq


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("T,H,D,begin,dim", [(1, 1, 2, 0, 2), (1, 128, 64, 0, 64), (3, 64, 128, 0, 64), (17, 5, 128, 64, 64),
                                             (40, 7, 80, 16, 48), (33, 3, 37, 5, 22), (130, 2, 1056, 16, 1024), (5, 300, 6, 1, 4)])
def test_rope_sizes_types_and_layouts(dtype, layout, T, H, D, begin, dim):
    x, pos, freq = _inputs(T, H, D, TYPES[dtype], seed=T + D, dim=dim)
    for transposed in (False, True):
        _check_rope(x, torch.full_like(x, 7), pos, freq, layout, begin, dim, scale=1.37, transposed=transposed)


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("dim", [64, 22])
def test_rope_in_place_equals_out_of_place(layout, dim):
    x, pos, freq = _inputs(29, 6, 96, torch.bfloat16, dim=dim)
    out = torch.empty_like(x)
    dsa.dsa_rope(x, pos, freq, out, layout=layout, rope_begin=32, rope_dim=dim)
    dsa.dsa_rope(x, pos, freq, x, layout=layout, rope_begin=32, rope_dim=dim)
    assert torch.equal(x, out)


def test_rope_slices_of_wider_tensors_leave_the_rest_alone():
    # the query's RoPE part out of the projection's rows into the absorbed query
    g = torch.Generator(device=DEV).manual_seed(9)
    src = torch.randn(50, 128, 192, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.full((50, 128, 576), 3.0, dtype=torch.bfloat16, device=DEV)
    _, pos, freq = _inputs(50, 1, 64, torch.bfloat16)
    _check_rope(src[..., 128:], q[..., 512:], pos, freq, 1, 0, 64)
    assert torch.all(q[..., :512] == 3)
    # heads outside tokens (a transposed tensor), unaligned starts
    x = torch.randn(9, 31, 70, generator=g, device=DEV).transpose(0, 1)[..., 3:69]
    out = torch.zeros(31, 9, 71, device=DEV)[..., 1:67]
    _, pos, freq = _inputs(31, 1, 66, torch.float32)
    _check_rope(x, out, pos, freq, 0, 0, 66)
    # one head broadcast over all heads of the output
    x = torch.randn(31, 1, 64, generator=g, device=DEV).expand(31, 6, 64)
    _, pos, freq = _inputs(31, 1, 64, torch.float32)
    _check_rope(x, torch.zeros(31, 6, 64, device=DEV), pos, freq, 1, 0, 64)


def test_rope_large_tensor_offsets_pass_32_bits():
    T, H = 12_000, 2
    wide = torch.zeros(T, 100_000, dtype=torch.int32, device=DEV).view(torch.float32)   # 4.8 GB: 1.2e9 elements
    x = wide.as_strided((T, H, 64), (100_000, 64, 1))
    x.normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    wide2 = torch.zeros(T, 200_000, dtype=torch.bfloat16, device=DEV)                   # 2.4e9 elements
    y = wide2.as_strided((T, H, 64), (200_000, 64, 1))
    y.copy_(x)
    _, pos, freq = _inputs(T, 1, 64, torch.bfloat16)
    out = torch.empty(T, H, 64, dtype=torch.bfloat16, device=DEV)
    _check_rope(y, out, pos, freq, 1, 0, 64)


def test_rope_transposed_is_the_gradient():
    x, pos, freq = _inputs(6, 3, 64, torch.float32, dim=32)
    pos = (pos % 50).contiguous()
    kw = dict(layout=0, rope_begin=16, rope_dim=32, scale=1.2)
    g, y, dx = torch.randn_like(x), torch.empty_like(x), torch.empty_like(x)
    dsa.dsa_rope(g, pos, freq, dx, transposed=True, **kw)
    d = torch.randn_like(x)
    dsa.dsa_rope(d, pos, freq, y, **kw)      # the map is linear: its difference along d is R d
    # 3 x 2^-24 per rotated element (test above), summed over the 1152 elements' magnitudes
    lim = 2 * 3 * 2.0 ** -24 * 1.2 * float((g.abs().double().sum() * d.abs().max() * 2))
    assert abs(float((g.double() * y.double()).sum() - (dx.double() * d.double()).sum())) <= lim


def test_binding_checks_shapes_and_types():
    x, pos, freq = _inputs(4, 2, 64, torch.bfloat16)
    for bad in (lambda: dsa.dsa_rope(x, pos.long(), freq, x), lambda: dsa.dsa_rope(x, pos[:3], freq, x),
                lambda: dsa.dsa_rope(x, pos, freq[:-1], x), lambda: dsa.dsa_rope(x, pos, freq, x.float()),
                lambda: dsa.dsa_rope(x[0], pos, freq, x[0]), lambda: dsa.dsa_rope(x.double(), pos, freq, x.double()),
                lambda: dsa.dsa_rope(x.transpose(1, 2), pos, freq[:1], x.transpose(1, 2))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(dsa.DsaError):
        dsa.dsa_rope(x, pos, freq, x, layout=5)


# ------------------------------------------------------------------ 8-bit cache write

FORMS = {"bf16": dsa.DSA_BF16, "e4m3": dsa.DSA_E4M3, "ue8m0": dsa.DSA_E4M3_UE8M0}


def _write_inputs(n, rows, seed=0, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    place = torch.randperm(rows, generator=g, device=DEV)[:n].to(I32)
    pos = torch.randint(0, 163840, (n,), generator=g, device=DEV).to(I32)
    return dict(k_raw=(2 * r(n, 128) + 0.5).to(torch.bfloat16), kv_raw=(std * r(n, 576)).to(torch.bfloat16), pos=pos, rows=place,
                ln_w=torch.rand(128, generator=g, device=DEV) + 0.5, ln_b=0.1 * r(128),
                rms_w=torch.rand(512, generator=g, device=DEV) + 0.5, freq=dsa.dsa_rope_frequencies(64, factor=40.0)[0].to(DEV))


def _caches(rows, form):
    k = torch.full((rows, 128), 5, dtype=torch.bfloat16 if form == "bf16" else torch.uint8, device=DEV)
    ks = None if form == "bf16" else torch.full((rows,), 9, dtype=torch.float32 if form == "e4m3" else torch.uint8, device=DEV)
    return k, ks, torch.full((rows, 640), 5, dtype=torch.uint8, device=DEV), torch.full((rows,), 9, dtype=torch.uint8, device=DEV)


def _write(i, c, form, eps=1e-6):
    dsa.dsa_cache_write_fp8(i["k_raw"], i["kv_raw"], i["pos"], i["rows"], i["ln_w"], i["ln_b"], i["rms_w"], i["freq"], *c,
                            idx_dtype=FORMS[form], eps=eps)


def _check_write(i, n_rows, form, eps=1e-6):
    c = _caches(n_rows, form)
    before = [None if t is None else t.clone() for t in c]
    _write(i, c, form, eps)
    f = lambda k: i[k].double().cpu().numpy()  # noqa: E731
    live = i["rows"].cpu().numpy() >= 0
    at = torch.from_numpy(i["rows"].cpu().numpy()[live].astype(np.int64)).to(DEV)
    k, lat, rot = ref.write_rows(f("k_raw")[live], f("kv_raw")[live], i["pos"].cpu().numpy()[live], f("ln_w"), f("ln_b"),
                                 f("rms_w"), i["freq"].cpu().numpy(), float(np.float32(eps)))
    codes, byte = ref.quantise_latent(lat, rot)
    # codes are compared as numbers (-0 is 0): each is the nearest one to the 64-bit value
    np.testing.assert_array_equal(c[3][at].cpu().numpy(), byte)
    np.testing.assert_array_equal(ref.E4M3[c[2][at].cpu().numpy()], ref.E4M3[codes])
    got = c[0][at]
    if form == "bf16":
        g64 = got.double().cpu().numpy()
        assert np.all(np.abs(g64 - k) <= 2.0 ** -8 * np.abs(k) + 1e-12)
    elif form == "ue8m0":
        e = ref.scale_exponent(np.abs(k).max(1))
        np.testing.assert_array_equal(c[1][at].cpu().numpy(), (e + 127).astype(np.uint8))
        np.testing.assert_array_equal(ref.E4M3[got.cpu().numpy()], ref.E4M3[ref.e4m3_nearest(k / 2.0 ** e[:, None])])
    else:
        s = np.where(np.abs(k).max(1) > 0, np.abs(k).max(1) / 448, 1).astype(np.float32)
        np.testing.assert_array_equal(c[1][at].cpu().numpy(), s)
        np.testing.assert_array_equal(ref.E4M3[got.cpu().numpy()], ref.E4M3[ref.e4m3_nearest(k / s.astype(np.float64)[:, None])])
    other = torch.ones(n_rows, dtype=torch.bool, device=DEV)
    other[at] = False
    for a, b in zip(c, before):
        assert a is None or torch.equal(a[other], b[other])


@pytest.mark.parametrize("form", list(FORMS))
@pytest.mark.parametrize("n,n_rows", [(1, 64), (7, 64), (8, 128), (257, 320), (3001, 4096)])
def test_write_codes_and_scales(form, n, n_rows):
    _check_write(_write_inputs(n, n_rows, seed=n), n_rows, form)


@pytest.mark.parametrize("form", list(FORMS))
def test_write_passes_over_tokens_without_a_row(form):
    i = _write_inputs(100, 256, seed=4)
    i["rows"][40:90] = -1
    i["rows"][3] = -7
    _check_write(i, 256, form)
    i["rows"][:] = -1
    _check_write(i, 256, form)


def test_bf16_write_passes_over_tokens_without_a_row():
    i = _write_inputs(40, 64, seed=5)
    i["rows"][10:] = -1
    kc, kv = (torch.full((64, d), 5.0, dtype=torch.bfloat16, device=DEV) for d in (128, 576))
    dsa.dsa_cache_write(i["k_raw"], i["kv_raw"], i["pos"], i["rows"], i["ln_w"], i["ln_b"], i["rms_w"], i["freq"], kc, kv)
    other = torch.ones(64, dtype=torch.bool, device=DEV)
    other[i["rows"][:10].long()] = False
    assert torch.all(kc[other] == 5) and torch.all(kv[other] == 5) and not torch.any(torch.all(kv[~other] == 5, dim=1))


@pytest.mark.parametrize("form", ["e4m3", "ue8m0"])
def test_write_scales_of_unusual_rows(form):
    i = _write_inputs(12, 64, seed=6)
    i["kv_raw"][0, 512:] *= 50          # RoPE dims decide the scale
    i["kv_raw"][1] = 0                  # a zero latent and zero RoPE dims
    i["kv_raw"][2, :512] = 0
    i["kv_raw"][2, 5] = 1               # one spike: 22.6 times the rms
    i["kv_raw"][3, 512:] = 0
    i["kv_raw"][4] *= 1e-30
    i["k_raw"][5] = 1                   # no variance: the key is the bias, rotated
    i["ln_b"][:] = 0
    _check_write(i, 64, form)
    i["ln_w"][:] = 0                    # zero keys
    _check_write(i, 64, form)


def test_write_values_on_and_next_to_code_borders():
    """The latent dims are evaluated in fp32 where that decides the code: values that lie on a border
    between two codes, or one unit in the last place beside it, must come out as in 64 bits."""
    i = _write_inputs(8, 64, seed=8)
    sign = torch.sign(torch.randn(8, 512, device=DEV))
    i["kv_raw"][:, :512] = sign * 2.0 ** torch.arange(-3, 5, device=DEV)[:, None]   # |z| / rms is 1 exactly
    i["kv_raw"][:, 512:] = 0
    ties = ref.E4M3[:127]
    ties = (ties[1:] + ties[:-1]) / 2                          # 126 borders, 2^-10 .. 432
    w = np.concatenate([ties, np.nextafter(ties.astype(np.float32), np.float32(0)),
                        np.nextafter(ties.astype(np.float32), np.float32(1e9)), ref.E4M3[:126], [1, 2, 3, 5, 7, 1, 1, 0]])
    for top in (448.0, np.nextafter(np.float32(448), np.float32(1e9))):   # the scale's own border
        w[-3:-1] = top, top
        i["rms_w"] = torch.tensor(w[:512].astype(np.float32), device=DEV)
        assert i["rms_w"].numel() == 512
        _check_write(i, 64, "ue8m0", eps=0.0)
    i["rms_w"] = i["rms_w"] * 2.0 ** -100                      # out of the range that fp32 decides
    _check_write(i, 64, "ue8m0", eps=0.0)


def test_write_many_tokens_have_the_codes_of_64_bits():
    _check_write(_write_inputs(16400, 20000, seed=9), 20000, "e4m3")


def test_write_rows_with_nan_or_infinity_get_a_nan_scale():
    i = _write_inputs(6, 64, seed=7)
    i["kv_raw"][0, 3] = float("nan")
    i["kv_raw"][1, 600 - 64] = float("inf")
    i["k_raw"][2, 9] = float("nan")
    c = _caches(64, "ue8m0")
    _write(i, c, "ue8m0")
    at = i["rows"].long()
    assert c[3][at].cpu().tolist()[:2] == [255, 255] and c[1][at].cpu().tolist()[2] == 255
    assert 255 not in c[3][at].cpu().tolist()[2:]
    codes = c[2][at].view(torch.float8_e4m3fn).float()
    assert torch.isnan(codes[:2]).all() and not torch.isnan(codes[2:]).any()
    assert torch.isnan(c[0][at].view(torch.float8_e4m3fn).float()[2]).all()


def test_write_far_rows_pass_32_bit_offsets():
    n_rows = 3_600_000                  # 2.3 GB of latent codes
    i = _write_inputs(64, 64, seed=8)
    i["rows"] = (n_rows - 1 - i["rows"] * 1000).to(I32)
    c = _caches(n_rows, "ue8m0")
    _write(i, c, "ue8m0")
    small = _caches(64, "ue8m0")
    j = dict(i, rows=torch.arange(64, dtype=I32, device=DEV))
    _write(j, small, "ue8m0")
    for a, b in zip(c, small):
        assert torch.equal(a[i["rows"].long()], b)


def test_binding_checks_the_caches():
    i = _write_inputs(4, 64)
    k, ks, kv, kvs = _caches(64, "ue8m0")
    for bad in ((k, ks.float(), kv, kvs), (k, None, kv, kvs), (k.view(torch.int8), ks, kv, kvs), (k, ks, kv[:, :576].contiguous(), kvs),
                (k, ks, kv, kvs[:60]), (k, ks[:60], kv, kvs)):
        with pytest.raises(ValueError):
            _write(i, bad, "ue8m0")


# ------------------------------------------------------------------ attention

def _cache(S, seed=0, spread=0.0, std=1.0):
    """A random 8-bit cache (codes, scale bytes); ``spread``: scales differ by 2^+-spread."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    kv = std * torch.randn(S, 576, generator=g, device=DEV)
    if spread:
        kv *= torch.exp2(spread * (2 * torch.rand(S, 1, generator=g, device=DEV) - 1))
    amax = torch.maximum(kv[:, :512].abs().amax(1), kv[:, 512:].abs().amax(1) / 16)
    e = torch.ceil(torch.log2(amax / 448)).clamp(-126, 120)
    y = kv / torch.exp2(e)[:, None]
    q = lambda v: v.clamp(-448, 448).to(torch.float8_e4m3fn)  # noqa: E731
    hi = q(y[:, 512:] / 16)
    codes = torch.cat([q(y[:, :512]).view(torch.uint8), hi.view(torch.uint8),
                       q(y[:, 512:] / 16 - hi.float()).view(torch.uint8)], 1)
    return codes.contiguous(), (e + 127).to(torch.uint8)


def _queries(T, seed=0, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(100 + seed)
    return (std * torch.randn(T, 128, 576, generator=g, device=DEV)).to(torch.bfloat16)


def _random_idx(T, topk, pos, seed=0, holes=0.0):
    """Ascending distinct visible keys, -1 behind; some entries replaced by -1."""
    rng = np.random.default_rng(seed)
    idx = np.full((T, topk), -1, np.int32)
    for t in range(T):
        n = min(topk, int(pos[t]) + 1)
        idx[t, :n] = np.sort(rng.choice(int(pos[t]) + 1, n, replace=False))
        if holes:
            idx[t, rng.random(topk) < holes] = -1
    return idx


def _run_mla(p, q, codes, byte, idx, ws=None):
    T = q.shape[0]
    out = torch.full((T, 128, 512), 7, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((T, 128), 7.0, device=DEV)
    if ws is None:
        ws = torch.full((dsa.dsa_sparse_mla_fp8_workspace_size(p),), 255, dtype=torch.uint8, device=DEV)   # NaN bytes
    dsa.dsa_sparse_mla_fp8_fwd(p, q, codes, byte, idx, out, lse, ws)
    dsa.dsa_check_device_errors()
    return out, lse


def _check_rows(q, codes, byte, rows_of, out, lse, tokens, heads=slice(None), scale=1 / 192 ** 0.5):
    """rows_of(t): cache rows of token t's live slots."""
    c, b = codes.cpu().numpy(), byte.cpu().numpy()
    for t in tokens:
        rows = rows_of(t)
        used, at = np.unique(rows, return_inverse=True) if len(rows) else (np.array([], int), np.array([], int))
        values = ref.cache_values(c[used], b[used])
        o, l, ot, lt = ref.attention(q[t].double().cpu().numpy()[heads], at, values, b[used], scale)
        go, gl = out[t].double().cpu().numpy()[heads], lse[t].double().cpu().numpy()[heads]
        if len(rows) == 0:
            assert np.all(go == 0) and np.all(np.isneginf(gl)), t
            continue
        assert np.all(np.isfinite(go)) and np.all(np.abs(gl - l) <= lt), (t, np.max(np.abs(gl - l) / lt))
        assert np.all(np.abs(go - o) <= ot), (t, np.max(np.abs(go - o) / ot))


def _packed(T, S, topk, **kw):
    return dsa.make_problem(1, T, S, T, S, topk, **kw)


@pytest.mark.parametrize("T,S,topk", [(1, 1, 1), (1, 5, 2048), (2, 300, 64), (3, 700, 255), (5, 700, 256), (4, 900, 257),
                                      (1, 3000, 2048), (9, 2500, 2047), (40, 600, 130), (75, 400, 300), (160, 500, 256),
                                      (230, 2600, 520)])
def test_attention_sizes(T, S, topk):
    codes, byte = _cache(S, seed=T)
    q = _queries(T, seed=S)
    pos = S - T + np.arange(T)
    idx = _random_idx(T, topk, pos, seed=topk)
    out, lse = _run_mla(_packed(T, S, topk), q, codes, byte, dev(idx))
    tokens = range(T) if T <= 9 else sorted({0, 1, T // 2, T - 2, T - 1, *range(70, min(T, 78))})
    _check_rows(q, codes, byte, lambda t: idx[t][idx[t] >= 0], out, lse, tokens)


@pytest.mark.parametrize("T", [3, 200])
def test_attention_masks(T):
    S, topk = 900, 600
    codes, byte = _cache(S, seed=1)
    q = _queries(T, seed=2)
    pos = S - T + np.arange(T)
    idx = _random_idx(T, topk, pos, seed=3, holes=0.3)
    idx[0] = -1                                             # nothing
    idx[1] = -1
    idx[1, 599] = 5                                         # the last slot only
    idx[2] = S + 50                                         # out of range only
    idx[2, 300] = 2 ** 31 - 1
    if T > 3:
        idx[3, :] = pos[3] + 1                              # the future only
        idx[4] = -1
        idx[4, 0] = pos[4]                                  # one key: its own
        idx[5, :] = 7                                       # one key 600 times
        idx[6, 256:] = -1                                   # a whole first block, then nothing
        idx[7, :256] = -1                                   # an empty first block
        idx[8, :] = -2 ** 31
    out, lse = _run_mla(_packed(T, S, topk), q, codes, byte, dev(idx))

    def rows(t):
        e = idx[t].astype(np.int64)
        return e[(e >= 0) & (e <= pos[t])]

    _check_rows(q, codes, byte, rows, out, lse, range(min(T, 12)))


@pytest.mark.parametrize("tail", [0, 90])
def test_attention_rows_of_unlike_lengths_in_turn(tail):
    """Several rows per SM pair, of 0 to 3 blocks: empty rows first, last and between, rows of one key."""
    S, T, topk = 1500, 330, 700
    codes, byte = _cache(S, seed=21)
    q = _queries(T, seed=22)
    pos = S - T + np.arange(T)
    idx = _random_idx(T, topk, pos, seed=23)
    keep = np.random.default_rng(24).choice([0, 0, 1, 200, 256, 257, 512, 513, 700], T)
    keep[T - tail:] = 0                                     # the rows that are taken first
    keep[:5] = [0, 700, 0, 1, 0]
    idx[np.arange(topk)[None, :] >= keep[:, None]] = -1
    out, lse = _run_mla(_packed(T, S, topk), q, codes, byte, dev(idx))
    _check_rows(q, codes, byte, lambda t: idx[t][idx[t] >= 0], out, lse, range(0, T, 3), heads=slice(0, 128, 9))
    again, lse2 = _run_mla(_packed(T, S, topk), q, codes, byte, dev(idx))
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_attention_masked_rows_may_hold_anything():
    S, T, topk = 400, 90, 128
    codes, byte = _cache(S, seed=4)
    codes[0] = 0x7F                                         # NaN codes at key 0, NaN scale at key 1
    byte[1] = 255
    codes[S - 1] = 0x7E
    byte[S - 1] = 254                                       # a huge last key
    q = _queries(T, seed=4)
    pos = S - T + np.arange(T)
    idx = np.full((T, topk), -1, np.int32)
    for t in range(T):
        idx[t, ::3] = 2 + (np.arange(len(idx[t, ::3])) * 2 + t) % 290
    idx[5] = -1
    idx[:, 1] = S - 1                                       # in the future of all but the last token
    out, lse = _run_mla(_packed(T, S, topk), q, codes, byte, dev(idx))

    def rows(t):
        e = idx[t]
        return e[(e >= 0) & (e <= pos[t])]

    _check_rows(q, codes, byte, rows, out, lse, [0, 1, 5, 40, T - 2])
    idx[7, 100] = 0                                         # a NaN row that is attended
    out, lse = _run_mla(_packed(T, S, topk), q, codes, byte, dev(idx))
    assert torch.isnan(lse[7]).all() and torch.isnan(out[7]).all()
    assert not torch.isnan(out[6]).any() and not torch.isnan(out[8]).any()


@pytest.mark.parametrize("spread", [1.5, 6.0, 30.0])
def test_attention_scales_that_differ(spread):
    S, T, topk = 1500, 4, 1024
    codes, byte = _cache(S, seed=5, spread=spread, std=2.0 ** -spread)
    byte[3], codes[3] = 1, 0                                # a zero key (the smallest scale) takes part in the sum
    q = _queries(T, seed=5)
    pos = S - T + np.arange(T)
    idx = _random_idx(T, topk, pos, seed=5)
    idx[:, 0] = 3
    out, lse = _run_mla(_packed(T, S, topk), q, codes, byte, dev(idx))
    _check_rows(q, codes, byte, lambda t: idx[t][idx[t] >= 0], out, lse, range(T))


@pytest.mark.parametrize("kind", ["sharp", "flat", "zero", "tiny", "outlier"])
def test_attention_score_ranges(kind):
    S, T, topk = 900, 3, 700
    codes, byte = _cache(S, seed=6)
    q = _queries(T, seed=6)
    if kind == "sharp":
        q *= 30                                             # one key takes nearly all
    elif kind == "flat":
        q *= 1e-3
    elif kind == "zero":
        q.zero_()
    elif kind == "tiny":
        q *= 2.0 ** -100
    else:
        q[:, :, 7] = 60.0                                   # one dim decides q's scale
        q[:, 3, 540] = -90.0
    pos = S - T + np.arange(T)
    idx = _random_idx(T, topk, pos, seed=6)
    out, lse = _run_mla(_packed(T, S, topk), q, codes, byte, dev(idx))
    _check_rows(q, codes, byte, lambda t: idx[t][idx[t] >= 0], out, lse, range(T))


def test_attention_rising_maxima():
    # keys whose scores rise block after block move the running maximum every time
    S, T, topk = 2100, 2, 2048
    codes, byte = _cache(S, seed=7, std=0.3)
    q = _queries(T, seed=7)
    kv = ref.cache_values(codes.cpu().numpy(), byte.cpu().numpy())
    z = kv @ q[0, 0].double().cpu().numpy()
    order = np.argsort(z[:S - T]).astype(np.int32)[:topk]
    idx = np.stack([order, order[::-1]])
    q[1] = q[0] * 8
    out, lse = _run_mla(_packed(T, S, topk), q, codes, byte, dev(idx))
    _check_rows(q, codes, byte, lambda t: idx[t], out, lse, range(T))


def _ragged(lens, queries, topk, seed, paged, pad_rows=0):
    B = len(lens)
    cu_q = np.concatenate([[0], np.cumsum(queries)]).astype(np.int32)
    cu_k = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu_q[-1])
    seq = np.repeat(np.arange(B), queries)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, queries)]) if T else np.array([], int)
    idx = _random_idx(T, topk, pos, seed=seed, holes=0.1)
    table, S = None, int(cu_k[-1])
    if paged:
        pages = [-(-n // 64) for n in lens]
        rng = np.random.default_rng(seed)
        perm = rng.permutation(sum(pages) + 3).astype(np.int32)
        table = np.full((B, max(max(pages), 1)), -1, np.int32)
        at = 0
        for b in range(B):
            table[b, :pages[b]] = perm[at:at + pages[b]]
            at += pages[b]
        S = 64 * (sum(pages) + 3)
    if pad_rows:
        idx = np.concatenate([idx, np.tile(np.arange(topk, dtype=np.int32), (pad_rows, 1))])
    on_gpu = dev(cu_q), dev(cu_k), None if table is None else dev(table)
    p = dsa.make_problem(B, T + pad_rows, S, int(max(queries)), int(max(lens)), topk, cu_q=on_gpu[0], cu_k=on_gpu[1],
                         block_table=on_gpu[2])
    p.tensors = on_gpu                 # the problem holds addresses only

    def rows(t):
        if t >= T:
            return np.array([], int)
        e = idx[t].astype(np.int64)
        e = e[(e >= 0) & (e <= pos[t])]
        return cu_k[seq[t]] + e if table is None else table[seq[t], e // 64].astype(np.int64) * 64 + e % 64

    return p, T + pad_rows, S, idx, rows


@pytest.mark.parametrize("paged", [False, True])
def test_attention_ragged_batches_with_empty_sequences(paged):
    lens, queries = [700, 64, 65, 1, 300, 128, 2000], [2, 0, 3, 1, 0, 1, 3]
    p, T, S, idx, rows = _ragged(lens, queries, 512, 11, paged)
    codes, byte = _cache(S, seed=8)
    q = _queries(T, seed=8)
    out, lse = _run_mla(p, q, codes, byte, dev(idx))
    _check_rows(q, codes, byte, rows, out, lse, range(T))


@pytest.mark.parametrize("paged", [False, True])
def test_attention_rows_behind_the_last_sequence(paged):
    p, T, S, idx, rows = _ragged([300, 500], [1, 2], 256, 12, paged, pad_rows=80)
    codes, byte = _cache(S, seed=9)
    q = _queries(T, seed=9)
    q[3:] = float("nan")
    out, lse = _run_mla(p, q, codes, byte, dev(idx))
    _check_rows(q, codes, byte, rows, out, lse, range(T))


def test_attention_empty_plan_is_all_empty_rows():
    z = torch.zeros(4, dtype=I32, device=DEV)
    table = torch.full((3, 2), -1, dtype=I32, device=DEV)
    p = dsa.make_problem(3, 5, 64, 1, 128, 64, cu_q=z, cu_k=z, block_table=table)
    codes, byte = _cache(64)
    idx = torch.arange(64, dtype=I32, device=DEV).repeat(5, 1)
    out, lse = _run_mla(p, _queries(5), codes, byte, idx)
    assert torch.all(out == 0) and torch.all(torch.isneginf(lse))


def test_attention_far_rows_pass_32_bit_offsets():
    S, topk = 3_600_000, 300                                # 2.3 GB of codes
    codes, byte = torch.zeros(S, 640, dtype=torch.uint8, device=DEV), torch.full((S,), 127, dtype=torch.uint8, device=DEV)
    c, b = _cache(2000, seed=10)
    codes[-2000:], byte[-2000:] = c, b
    q = _queries(2, seed=10)
    idx = np.stack([np.sort(np.random.default_rng(t).choice(1990, topk, replace=False)) for t in range(2)]).astype(np.int32)
    out, lse = _run_mla(_packed(2, S, topk), q, codes, byte, dev(idx + (S - 2000)))
    _check_rows(q, c, b, lambda t: idx[t], out, lse, range(2))


@pytest.mark.parametrize("T", [1, 6, 100])
def test_attention_is_deterministic_captured_and_on_other_streams(T):
    S, topk = 1200, 600
    codes, byte = _cache(S, seed=13)
    q = _queries(T, seed=13)
    idx = dev(_random_idx(T, topk, S - T + np.arange(T), seed=13))
    p = _packed(T, S, topk)
    out, lse = _run_mla(p, q, codes, byte, idx)
    ws = torch.empty(max(256, dsa.dsa_sparse_mla_fp8_workspace_size(p)), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        dsa.dsa_sparse_mla_fp8_fwd(p, q, codes, byte, idx, o2, l2, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dsa.dsa_sparse_mla_fp8_fwd(p, q, codes, byte, idx, o2, l2, ws)
    for seed in (14, 15):
        q.copy_(_queries(T, seed=seed))
        o2.zero_()
        g.replay()
        o3, l3 = _run_mla(p, q, codes, byte, idx)
        assert torch.equal(o3, o2) and torch.equal(l3, l2)


def test_attention_two_calls_at_once_with_their_own_workspaces():
    S, topk = 3000, 2048
    codes, byte = _cache(S, seed=16)
    p = _packed(2, S, topk)
    idx = dev(_random_idx(2, topk, S - 2 + np.arange(2), seed=16))
    qs = [_queries(2, seed=s) for s in range(4)]
    want = [_run_mla(p, q, codes, byte, idx) for q in qs]
    got = [(torch.empty_like(o), torch.empty_like(l)) for o, l in want]
    wss = [torch.empty(dsa.dsa_sparse_mla_fp8_workspace_size(p), dtype=torch.uint8, device=DEV) for _ in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(5):
        for q, (o, l), ws, s in zip(qs, got, wss, streams):
            dsa.dsa_sparse_mla_fp8_fwd(p, q, codes, byte, idx, o, l, ws, stream=s)
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)


def test_attention_near_the_bf16_cache_form():
    # the same values in a bf16 cache (e4m3 times a power of two is exact in bf16; RoPE dims with
    # a zero second code) through dsa_sparse_mla_fwd: both within their own bounds of the definition
    S, T, topk = 1500, 120, 512
    codes, byte = _cache(S, seed=17)
    codes[:, 576:] = 0
    kv = torch.from_numpy(ref.cache_values(codes.cpu().numpy(), byte.cpu().numpy())).to(DEV)
    assert torch.equal(kv.to(torch.bfloat16).double(), kv)
    q = _queries(T, seed=17)
    idx = dev(_random_idx(T, topk, S - T + np.arange(T), seed=17))
    p = _packed(T, S, topk)
    out, lse = _run_mla(p, q, codes, byte, idx)
    o2, l2 = torch.empty_like(out), torch.empty_like(lse)
    dsa.dsa_sparse_mla_fwd(p, q, kv.to(torch.bfloat16).contiguous(), idx, o2, l2)
    # |values| < 448 * max scale; each side's p error <= 2^-8 + 2^-12 and rounding 2^-8 relative to sum p|v|
    lim = 2 * (2.0 ** -8 + 2.0 ** -12 + 2.0 ** -8) * kv.abs().max().item()
    assert torch.max(torch.abs(out.float() - o2.float())).item() <= lim
    assert torch.max(torch.abs(lse - l2)).item() <= 2e-3


def test_attention_debug_checks_skip_bad_rows():
    codes, byte = _cache(640, seed=18)
    cu_q, cu_k = dev(np.array([0, 1, 2], np.int32)), dev(np.array([0, 100, 200], np.int32))
    table = dev(np.array([[3, 1], [999, -1]], np.int32))
    p = dsa.make_problem(2, 2, 640, 1, 128, 64, cu_q=cu_q, cu_k=cu_k, block_table=table)
    q, idx = _queries(2), dev(np.tile(np.arange(64, dtype=np.int32), (2, 1)))
    out, lse = torch.empty(2, 128, 512, dtype=torch.bfloat16, device=DEV), torch.empty(2, 128, device=DEV)
    ws = torch.empty(dsa.dsa_sparse_mla_fp8_workspace_size(p) + 256, dtype=torch.uint8, device=DEV)
    dsa.dsa_check_device_errors()
    dsa.dsa_set_debug_checks(True)
    try:
        dsa.dsa_sparse_mla_fp8_fwd(p, q, codes, byte, idx, out, lse, ws)
        with pytest.raises(dsa.DsaError) as e:
            dsa.dsa_check_device_errors()
        assert e.value.code == 6
    finally:
        dsa.dsa_set_debug_checks(False)
    assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1])) and torch.isfinite(lse[0]).all()


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("form", list(FORMS))
def test_serving_steps_together(form):
    """Three requests prefill and decode: plan -> cache write -> query RoPE -> indexer -> top-k ->
    attention, every step through the operators, against the 64-bit definitions on the caches'
    history kept by the test."""
    topk, eps, B, n_pages = 128, 1e-6, 3, 24
    g = torch.Generator(device=DEV).manual_seed(21)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    ln_w, ln_b = torch.rand(128, generator=g, device=DEV) + 0.5, 0.1 * r(128)
    rms_w, freq = torch.rand(512, generator=g, device=DEV) + 0.5, dsa.dsa_rope_frequencies(64, factor=40.0)[0].to(DEV)
    k_cache, k_scale, kv_cache, kv_scale = _caches(n_pages * 64, form)
    table = torch.full((B, 8), -1, dtype=I32, device=DEV)
    free = torch.randperm(n_pages, generator=g, device=DEV).to(I32)
    head, cached = torch.zeros(1, dtype=I32, device=DEV), torch.zeros(B, dtype=I32, device=DEV)
    history = [(np.zeros((0, 640), np.uint8), np.zeros(0, np.uint8)) for _ in range(B)]
    for new in ([130, 0, 70], [1, 200, 1], [1, 1, 1], [1, 0, 60]):
        T = sum(new) + 5
        n = torch.tensor(new, dtype=I32, device=DEV)
        cu_q, cu_k = (torch.empty(B + 1, dtype=I32, device=DEV) for _ in range(2))
        pos, rows = (torch.empty(T, dtype=I32, device=DEV) for _ in range(2))
        counts = torch.empty(4, dtype=I32, device=DEV)
        dsa.dsa_paged_plan(cached, n, table, free, cu_q, cu_k, pos, rows, counts, n_pages=n_pages, free_head=head)
        assert counts.cpu().tolist()[3] == 0
        k_raw, kv_raw = r(T, 128).to(torch.bfloat16), r(T, 576).to(torch.bfloat16)
        dsa.dsa_cache_write_fp8(k_raw, kv_raw, pos, rows, ln_w, ln_b, rms_w, freq, k_cache, k_scale, kv_cache, kv_scale,
                                idx_dtype=FORMS[form], eps=eps)
        # queries: absorbed part beside the rotated part, the indexer's rotated on their first 64 dims
        q = torch.empty(T, 128, 576, dtype=torch.bfloat16, device=DEV)
        q[..., :512] = r(T, 128, 512)
        dsa.dsa_rope(r(T, 128, 192).to(torch.bfloat16)[..., 128:], pos, freq, q[..., 512:])
        q_idx = r(T, 64, 128).to(torch.bfloat16)
        dsa.dsa_rope(q_idx, pos, freq, q_idx, layout=dsa.DSA_ROPE_HALF, rope_begin=0, rope_dim=64)
        w = r(T, 64) / 8
        longest = int(counts[2])
        p = dsa.make_problem(B, T, n_pages * 64, max(new), longest, topk, cu_q=cu_q, cu_k=cu_k, block_table=table,
                             idx_dtype=FORMS[form])
        kw = {}
        if form == "e4m3":
            am = q_idx.float().abs().amax((1, 2)) / 448
            q_idx, kw = (q_idx.float() / am[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), dict(q_scale=am, k_scale=k_scale)
        elif form == "ue8m0":
            e = torch.ceil(torch.log2(q_idx.float().abs().amax(2) / 448))
            q_idx = (q_idx.float() / torch.exp2(e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            kw = dict(q_scale=(e + 127).to(torch.uint8), k_scale=k_scale)
        live = sum(new)
        sc = torch.zeros(T, dsa.scores_ld(longest), device=DEV)
        dsa.dsa_indexer_scores(p, q_idx.contiguous(), k_cache, w, sc, row_count=live, **kw)
        idx = torch.full((T, topk), 3, dtype=I32, device=DEV)     # padding rows keep what was there
        dsa.dsa_topk(p, sc, idx, row_count=live)
        out, lse = _run_mla(p, q, kv_cache, kv_scale, idx)
        # the cache's history, from the definitions
        f = lambda t: t.double().cpu().numpy()  # noqa: E731
        _, lat, rot = ref.write_rows(f(k_raw), f(kv_raw), pos.cpu().numpy(), f(ln_w), f(ln_b), f(rms_w), freq.cpu().numpy(),
                                     float(np.float32(eps)))
        codes, byte = ref.quantise_latent(lat, rot)
        at = 0
        ix = idx.cpu().numpy()
        for b in range(B):
            history[b] = (np.concatenate([history[b][0], codes[at:at + new[b]]]), np.concatenate([history[b][1], byte[at:at + new[b]]]))
            length = len(history[b][1])
            for t in sorted({at, at + new[b] // 2, at + new[b] - 1} if new[b] else set()):
                mine = length - new[b] + (t - at)
                assert np.count_nonzero(ix[t] >= 0) == min(topk, mine + 1) and ix[t].max() <= mine
                hc, hb = (torch.from_numpy(v) for v in history[b])
                _check_rows(q, hc, hb, lambda t_: ix[t_][ix[t_] >= 0], out, lse, [t], heads=slice(0, 128, 17))
            at += new[b]
        assert torch.all(out[live:] == 0) and torch.all(torch.isneginf(lse[live:]))
        cached += n
        head += counts[1:2]
    dsa.dsa_check_device_errors()


def test_serving_step_captured_and_replayed():
    """A step's calls in one graph, replayed with other lengths and inputs, give what the calls give eagerly."""
    B, T, n_pages, topk = 3, 40, 24, 64
    g = torch.Generator(device=DEV).manual_seed(31)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    weights = [torch.ones(128, device=DEV), torch.zeros(128, device=DEV), torch.ones(512, device=DEV)]
    freq = dsa.dsa_rope_frequencies(64)[0].to(DEV)
    free = torch.randperm(n_pages, generator=g, device=DEV).to(I32)

    def state():
        z = lambda *s, dtype=I32: torch.zeros(*s, dtype=dtype, device=DEV)  # noqa: E731
        s = dict(cached=z(B), new=z(B), table=torch.full((B, 8), -1, dtype=I32, device=DEV), head=z(1), cu_q=z(B + 1),
                 cu_k=z(B + 1), pos=z(T), rows=z(T), counts=z(4), k_raw=z(T, 128, dtype=torch.bfloat16),
                 kv_raw=z(T, 576, dtype=torch.bfloat16), x=z(T, 128, 192, dtype=torch.bfloat16),
                 q=z(T, 128, 576, dtype=torch.bfloat16), out=z(T, 128, 512, dtype=torch.bfloat16), lse=z(T, 128, dtype=torch.float32),
                 q_idx=z(T, 64, 128, dtype=torch.bfloat16), rotated=z(T, 64, 128, dtype=torch.bfloat16), w=z(T, 64, dtype=torch.float32),
                 scores=z(T, dsa.scores_ld(512), dtype=torch.float32), idx=z(T, topk), caches=_caches(n_pages * 64, "bf16"))
        s["p"] = dsa.make_problem(B, T, n_pages * 64, T, 512, topk, cu_q=s["cu_q"], cu_k=s["cu_k"], block_table=s["table"],
                                  idx_dtype=dsa.DSA_BF16)
        s["ws"] = z(dsa.dsa_sparse_mla_fp8_workspace_size(s["p"]), dtype=torch.uint8)
        return s

    def step(s):
        dsa.dsa_paged_plan(s["cached"], s["new"], s["table"], free, s["cu_q"], s["cu_k"], s["pos"], s["rows"], s["counts"],
                           n_pages=n_pages, free_head=s["head"])
        dsa.dsa_cache_write_fp8(s["k_raw"], s["kv_raw"], s["pos"], s["rows"], *weights, freq, *s["caches"], idx_dtype=dsa.DSA_BF16)
        dsa.dsa_rope(s["x"][..., 128:], s["pos"], freq, s["q"][..., 512:])
        dsa.dsa_rope(s["q_idx"], s["pos"], freq, s["rotated"], layout=dsa.DSA_ROPE_HALF, rope_dim=64)
        dsa.dsa_indexer_scores(s["p"], s["rotated"], s["caches"][0], s["w"], s["scores"])
        dsa.dsa_topk(s["p"], s["scores"], s["idx"])
        dsa.dsa_sparse_mla_fp8_fwd(s["p"], s["q"], s["caches"][2], s["caches"][3], s["idx"], s["out"], s["lse"], s["ws"])

    eager, captured = state(), state()
    step(captured)                                          # an empty batch: no lengths yet
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(captured)
    for new in ([20, 0, 13], [1, 17, 1], [1, 1, 38], [0, 0, 0]):
        drawn = dict(new=torch.tensor(new, dtype=I32, device=DEV), k_raw=r(T, 128), kv_raw=r(T, 576), x=r(T, 128, 192),
                     q_idx=r(T, 64, 128), w=r(T, 64))
        q = r(T, 128, 512).to(torch.bfloat16)
        for s in (eager, captured):
            for k, v in drawn.items():
                s[k].copy_(v)
            s["q"][..., :512] = q
        step(eager)
        graph.replay()
        for k in ("table", "cu_q", "cu_k", "pos", "rows", "counts", "q", "out", "lse"):
            assert torch.equal(eager[k], captured[k]), k
        assert all(torch.equal(eager["caches"][i], captured["caches"][i]) for i in (0, 2, 3))
        live = sum(new)
        assert torch.equal(eager["idx"][:live], captured["idx"][:live])
        assert torch.all(torch.isneginf(eager["lse"][live:])) and torch.all(torch.isfinite(eager["lse"][:live]))
        for s in (eager, captured):
            s["cached"] += s["new"]
            s["head"] += s["counts"][1:2]
    dsa.dsa_check_device_errors()
