"""Block tables and free lists that name pages outside the pool: nothing is read or written
outside the caches, the error is reported, and the other sequences' results do not change."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_lightning_indexer_b200 as dsa
import serving_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BAD = [-1, 12, 1 << 24, 2 ** 31 - 1, -2 ** 31, 2 ** 26]      # 12 pages; the last two times 64 pass 32 bits


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
    return t if dtype is None else t.to(dtype)


def _expect_bounds():
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_check_device_errors()
    assert e.value.code == 6
    dsa.dsa_check_device_errors()


def _problem(table, lens, topk, form, repeat):
    B = len(lens)
    t = dev(np.arange(0, B * repeat + 1, repeat), torch.int32), dev(np.concatenate([[0], np.cumsum(lens)]), torch.int32), dev(table, torch.int32)
    p = dsa.make_problem(B, B * repeat, 12 * 64, repeat, max(lens), topk, cu_q=t[0], cu_k=t[1], block_table=t[2], idx_dtype=form)
    p.tensors = t
    return p


@pytest.mark.parametrize("repeat", [1, 30])
@pytest.mark.parametrize("page", [1, 2])                     # a page of sequence 1: keys 64 .., or its last keys
@pytest.mark.parametrize("bad", BAD)
def test_attention_masks_keys_on_pages_outside_the_pool(bad, page, repeat):
    rng = np.random.default_rng(1)
    lens, topk = [200, 150, 700 - 64 * 3], 600
    good = np.full((3, 8), -1, np.int64)
    good[0, :4], good[1, :3], good[2, :7] = [0, 1, 2, 3], [4, 5, 6], [7, 8, 9, 10, 11, 0, 1]
    lens[2] = 448
    table = good.copy()
    table[1, page] = bad
    codes, byte = ref.quantise_latent(rng.standard_normal((768, 512)), rng.standard_normal((768, 64)))
    codes[0] = 0x7F                          # (key 0 of sequence 0 is NaN: listed by nobody below)
    T = 3 * repeat
    q = torch.randn(T, 128, 576, generator=torch.Generator(device=DEV).manual_seed(1), device=DEV).to(torch.bfloat16)
    seq = np.repeat(np.arange(3), repeat)
    idx = np.full((T, topk), -1, np.int32)
    for t in range(T):
        n = lens[seq[t]] - repeat + t % repeat + 1
        idx[t, 1:n] = np.arange(1, n)
    idx[seq == 2] = np.where(idx[seq == 2] == 320, -1, idx[seq == 2])   # (its key 320 is the same row)
    outs = []
    for tab, ix in ((table, idx), (good, np.where((seq == 1)[:, None] & (idx // 64 == page), -1, idx))):
        p = _problem(tab, lens, topk, dsa.DSA_BF16, repeat)
        out, lse = torch.zeros(T, 128, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(T, 128, device=DEV)
        ws = torch.zeros(max(256, dsa.dsa_sparse_mla_fp8_workspace_size(p)), dtype=torch.uint8, device=DEV)
        dsa.dsa_sparse_mla_fp8_fwd(p, q, dev(codes), dev(byte), dev(ix), out, lse, ws)
        if tab is table:
            _expect_bounds()
        dsa.dsa_check_device_errors()
        outs.append((out, lse))
    # as if the keys had not been listed
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.isfinite(outs[0][1]).all()


@pytest.mark.parametrize("topk", [128, 600])
@pytest.mark.parametrize("bad", BAD)
def test_attention_of_a_token_whose_pages_are_all_bad_changes_no_other(bad, topk):
    rng = np.random.default_rng(2)
    codes, byte = ref.quantise_latent(rng.standard_normal((768, 512)), rng.standard_normal((768, 64)))
    codes[0], byte[1] = 0x7F, 255            # what row 0 holds must not matter
    table = np.array([[3, 4], [bad, bad], [5, 6]])
    p = _problem(table, [100, 100, 100], topk, dsa.DSA_BF16, 1)
    q = torch.randn(3, 128, 576, generator=torch.Generator(device=DEV).manual_seed(2), device=DEV).to(torch.bfloat16)
    idx = np.tile(np.where(np.arange(topk) < 100, np.arange(topk), -1).astype(np.int32), (3, 1))
    out, lse = torch.zeros(3, 128, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(3, 128, device=DEV)
    ws = torch.zeros(max(256, dsa.dsa_sparse_mla_fp8_workspace_size(p)), dtype=torch.uint8, device=DEV)
    dsa.dsa_sparse_mla_fp8_fwd(p, q, dev(codes), dev(byte), dev(idx), out, lse, ws)
    _expect_bounds()
    assert torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))
    values = ref.cache_values(codes, byte)
    for t, first in ((0, 3 * 64), (2, 5 * 64)):
        o, l, ot, lt = ref.attention(q[t].double().cpu().numpy(), np.arange(first, first + 100), values, byte, 1 / 192 ** 0.5)
        assert np.all(np.abs(out[t].double().cpu().numpy() - o) <= ot) and np.all(np.abs(lse[t].double().cpu().numpy() - l) <= lt)


@pytest.mark.parametrize("T", [2, 60])
def test_attention_of_a_part_whose_pages_are_all_bad(T):
    """A split of the index row (few tokens) or a whole block of it lists keys on bad pages only."""
    rng = np.random.default_rng(4)
    codes, byte = ref.quantise_latent(rng.standard_normal((768, 512)), rng.standard_normal((768, 64)))
    codes[0] = 0x7F
    table = np.full((T, 11), 11)
    table[:] = np.arange(1, 12)
    table[1, 4:8] = -1                       # keys 256 .. 511 of token 1
    lens = [704] * T
    q = torch.randn(T, 128, 576, generator=torch.Generator(device=DEV).manual_seed(5), device=DEV).to(torch.bfloat16)
    values = ref.cache_values(codes, byte)
    for topk in (512, 704):                  # the bad block last, and between others
        p = _problem(table, lens, topk, dsa.DSA_BF16, 1)
        idx = np.tile(np.arange(topk, dtype=np.int32), (T, 1))
        out, lse = torch.zeros(T, 128, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(T, 128, device=DEV)
        ws = torch.zeros(max(256, dsa.dsa_sparse_mla_fp8_workspace_size(p)), dtype=torch.uint8, device=DEV)
        dsa.dsa_sparse_mla_fp8_fwd(p, q, dev(codes), dev(byte), dev(idx), out, lse, ws)
        _expect_bounds()
        for t in (0, 1, T - 1):
            keys = np.array([k for k in range(topk) if t != 1 or not 256 <= k < 512])
            o, l, ot, lt = ref.attention(q[t].double().cpu().numpy(), keys + 64, values, byte, 1 / 192 ** 0.5)
            assert np.all(np.abs(out[t].double().cpu().numpy() - o) <= ot), (topk, t)
            assert np.all(np.abs(lse[t].double().cpu().numpy() - l) <= lt), (topk, t)


@pytest.mark.parametrize("form", [dsa.DSA_BF16, dsa.DSA_E4M3, dsa.DSA_E4M3_UE8M0])
@pytest.mark.parametrize("bad", BAD)
def test_indexer_scores_keys_on_pages_outside_the_pool_zero(form, bad):
    g = torch.Generator(device=DEV).manual_seed(3)
    lens, B = [300, 130, 64], 3
    good = np.full((3, 6), -1, np.int64)
    good[0, :5], good[1, :3], good[2, 0] = [0, 1, 2, 3, 4], [5, 6, 7], 8
    table = good.copy()
    table[0, 1] = table[1, 2] = bad
    e8 = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
    q, k, w = e8(B, 64, 128), e8(768, 128), torch.randn(B, 64, generator=g, device=DEV)
    qs = ks = None
    if form == dsa.DSA_BF16:
        q, k = (x.view(torch.float8_e4m3fn).to(torch.bfloat16) for x in (q, k))
    elif form == dsa.DSA_E4M3:
        qs, ks = torch.rand(B, generator=g, device=DEV) + 0.5, torch.rand(768, generator=g, device=DEV) + 0.5
    else:
        qs = torch.randint(120, 130, (B, 64), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
        ks = torch.randint(120, 130, (768,), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
    got = []
    for tab in (table, good):
        p = _problem(tab, lens, 64, form, 1)
        sc = torch.full((B, dsa.scores_ld(300)), 7.0, device=DEV)
        dsa.dsa_indexer_scores(p, q, k, w, sc, q_scale=qs, k_scale=ks)
        if tab is table and form != dsa.DSA_BF16:   # (bf16 keys come by tile loads only, which give zeros)
            _expect_bounds()
        dsa.dsa_check_device_errors()
        got.append(sc)
    want = got[1].clone()
    want[0, 64:128] = 0
    want[1, 128:130] = 0
    assert torch.equal(got[0], want)


@pytest.mark.parametrize("bad", BAD)
def test_plan_stores_no_page_outside_the_pool(bad):
    B, n_pages = 2, 12
    cached, new = dev([10, 60], torch.int32), dev([60, 140], torch.int32)
    table = dev([[3, 7, 9, 9], [4, 7, 9, 9]], torch.int32)        # stale numbers behind the cached pages
    free = dev([5, bad, 6, 8], torch.int32)
    z = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    cu_q, cu_k, pos, rows, counts = z(B + 1), z(B + 1), z(200), z(200), z(4)
    dsa.dsa_paged_plan(cached, new, table, free, cu_q, cu_k, pos, rows, counts, n_pages=n_pages)
    _expect_bounds()
    # request 0 takes page 5; request 1 takes the bad number, 6 and 8
    assert table.cpu().tolist() == [[3, 5, 9, 9], [4, -1, 6, 8]]
    r = rows.cpu().numpy()
    want = np.concatenate([3 * 64 + np.arange(10, 64), 5 * 64 + np.arange(6), 4 * 64 + np.arange(60, 64), np.full(64, -1),
                           6 * 64 + np.arange(64), 8 * 64 + np.arange(8)])
    np.testing.assert_array_equal(r, want)
    assert counts.cpu().tolist() == [200, 4, 200, 0]
    # the next step: a token on the page that has none gets no row
    cached, new = dev([70, 110], torch.int32), dev([0, 1], torch.int32)
    dsa.dsa_paged_plan(cached, new, table, free, cu_q, cu_k, pos[:1], rows[:1], counts, n_pages=n_pages, free_head=dev([4], torch.int32))
    _expect_bounds()
    assert rows[0].item() == -1 and pos[0].item() == 110
