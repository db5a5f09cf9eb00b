"""The cache writes pass over rows past the caches' end, report them, and write the others."""
from __future__ import annotations

import pytest
import torch

import attention_lightning_indexer_b200 as dsa

pytestmark = pytest.mark.gpu
DEV = "cuda"
N, ROWS = 50, 64
FAR = [64, 65, 10_000, 2 ** 31 - 1]      # rows past the end; 2^31 - 1 is 1.4 TB away


def _inputs():
    g = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    return (r(N, 128).to(torch.bfloat16), r(N, 576).to(torch.bfloat16), torch.arange(N, dtype=torch.int32, device=DEV),
            torch.randperm(ROWS, generator=g, device=DEV)[:N].to(torch.int32), torch.ones(128, device=DEV),
            torch.zeros(128, device=DEV), torch.ones(512, device=DEV), dsa.dsa_rope_frequencies(64)[0].to(DEV))


def _caches(form, spare):
    """Caches of ROWS rows, with rows behind them that must stay as they are."""
    n = ROWS + spare
    if form is None:
        return [torch.full((n, d), 5.0, dtype=torch.bfloat16, device=DEV) for d in (128, 576)]
    u8 = lambda *s: torch.full(s, 5, dtype=torch.uint8, device=DEV)  # noqa: E731
    key = torch.full((n, 128), 5.0, dtype=torch.bfloat16, device=DEV) if form == dsa.DSA_BF16 else u8(n, 128)
    scale = {dsa.DSA_BF16: None, dsa.DSA_E4M3: torch.full((n,), 5.0, device=DEV), dsa.DSA_E4M3_UE8M0: u8(n)}[form]
    return [key, scale, u8(n, 640), u8(n)]


def _write(form, inputs, caches):
    if form is None:
        dsa.dsa_cache_write(*inputs, *caches)
    else:
        dsa.dsa_cache_write_fp8(*inputs, *caches, idx_dtype=form)


@pytest.mark.parametrize("form", [None, dsa.DSA_BF16, dsa.DSA_E4M3, dsa.DSA_E4M3_UE8M0])
@pytest.mark.parametrize("short", [False, True])
def test_rows_past_the_end_are_passed_over_and_reported(form, short):
    k_raw, kv_raw, pos, rows, *weights = _inputs()
    want = _caches(form, 100)
    _write(form, (k_raw, kv_raw, pos, rows, *weights), [None if c is None else c[:ROWS] for c in want])
    dsa.dsa_check_device_errors()
    # the same rows, with four tokens sent past the end (two of one warp's CTA, the last one)
    lost = torch.tensor([0, 1, 20, N - 1], device=DEV)
    bad = rows.clone()
    bad[lost] = torch.tensor(FAR, dtype=torch.int32, device=DEV)
    got = _caches(form, 100)
    views = [None if c is None else c[:ROWS] for c in got]
    if short:                            # the first cache (and its scales) has rows enough, the other not
        views[0] = got[0]
        if form is not None and got[1] is not None:
            views[1] = got[1]
    _write(form, (k_raw, kv_raw, pos, bad, *weights), views)
    with pytest.raises(dsa.DsaError) as e:
        dsa.dsa_check_device_errors()
    assert e.value.code == 6
    for w in want:
        if w is not None:
            w[rows[lost].long()] = 5
    for g, w in zip(got, want):
        assert g is None or torch.equal(g, w)
    dsa.dsa_check_device_errors()


def test_padding_rows_are_no_error():
    k_raw, kv_raw, pos, rows, *weights = _inputs()
    rows[10:] = -1
    for form in (None, dsa.DSA_E4M3):
        caches = _caches(form, 0)
        _write(form, (k_raw, kv_raw, pos, rows, *weights), caches)
    dsa.dsa_check_device_errors()
