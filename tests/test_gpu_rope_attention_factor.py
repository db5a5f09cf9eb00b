"""Where the attention factor of stretched frequencies goes: with cached keys as the cache writes
leave them, its square on the queries' rotated dims gives the scores of the definition."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_lightning_indexer_b200 as dsa
import serving_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fp8", [False, True])
def test_the_square_on_the_queries_gives_the_definitions_scores(fp8):
    n, H = 48, 8
    g = torch.Generator(device=DEV).manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)  # noqa: E731
    freq, factor = dsa.dsa_rope_frequencies(64, factor=40.0)
    freq_d = freq.to(DEV)
    pos = torch.randint(0, 163840, (n,), generator=g, device=DEV).to(torch.int32)
    rows = torch.arange(n, dtype=torch.int32, device=DEV)
    k_raw, kv_raw, q = r(n, 128), r(n, 576), r(n, H, 64)
    weights = torch.ones(128, device=DEV), torch.zeros(128, device=DEV), torch.ones(512, device=DEV)
    if fp8:
        caches = [torch.zeros(n, *s, dtype=torch.uint8, device=DEV) for s in ((128,), (), (640,), ())]
        dsa.dsa_cache_write_fp8(k_raw, kv_raw, pos, rows, *weights, freq_d, *caches)
        keys = ref.cache_values(caches[2].cpu().numpy(), caches[3].cpu().numpy())[:, 512:]
    else:
        caches = [torch.zeros(n, d, dtype=torch.bfloat16, device=DEV) for d in (128, 576)]
        dsa.dsa_cache_write(k_raw, kv_raw, pos, rows, *weights, freq_d, *caches)
        keys = caches[1][:, 512:].double().cpu().numpy()
    turned = torch.empty_like(q)
    dsa.dsa_rope(q, pos, freq_d, turned, scale=factor ** 2)
    got = np.einsum("thd,sd->ths", turned.double().cpu().numpy(), keys)
    # the definition: cosine and sine times the factor on both sides
    p, f = pos.cpu().numpy(), freq.numpy()
    qd = ref.rope(q.double().cpu().numpy(), p, f, 1, 0, 64, scale=factor)
    kd = ref.rope(kv_raw[:, None, 512:].double().cpu().numpy(), p, f, 1, 0, 64, scale=factor)[:, 0]
    want = np.einsum("thd,sd->ths", qd, kd)
    # a query dim and a key dim (bf16, or two e4m3 codes) are each one rounding of 2^-8; the rotation in
    # fp32 adds 2^-22, and 8-bit RoPE dims step by 2^-9 at 16 times the scale, half of it an error
    step = 0.0 if not fp8 else 16 * 2.0 ** -10 * 2.0 ** (caches[3].double().cpu().numpy() - 127)
    mag = np.einsum("thd,sd->ths", np.abs(qd), np.abs(kd))
    lim = mag * (2 * 2.0 ** -8 + 2.0 ** -16 + 2.0 ** -20) + np.abs(qd).sum(2)[:, :, None] * factor * step * 1.01
    # magnitudes before the rotation bound the rotated ones' rounding
    assert np.all(np.abs(got - want) <= lim + 2.0 ** -20 * 64 * 25), np.max(np.abs(got - want) / lim)
