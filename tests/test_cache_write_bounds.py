"""Host-only checks of the bounded cache writes: refusals, and what the binding passes on."""
import pytest
import torch

import attention_lightning_indexer_b200 as dsa
from attention_lightning_indexer_b200 import _native

FAKE = 1 << 20                       # aligned, never dereferenced: validation fails first
OK, INVALID, UNSUPPORTED = 0, 1, 2


def test_bounded_writes_refuse():
    lib = dsa.load()
    write = lambda n=4, rows=64, kc=FAKE, eps=1e-6: lib.dsa_cache_write_bounded(n, *[FAKE] * 8, eps, kc, FAKE, rows, None)  # noqa: E731
    fp8 = lambda n=4, rows=64, kc=FAKE, form=2: lib.dsa_cache_write_fp8_bounded(n, *[FAKE] * 8, 1e-6, form, kc, FAKE, FAKE, FAKE, rows, None)  # noqa: E731
    assert write(rows=-1) == INVALID and write(kc=None) == INVALID and write(eps=-1.0) == INVALID and write(n=-1) == INVALID
    assert fp8(rows=-1) == INVALID and fp8(kc=FAKE + 8) == INVALID and fp8(form=3) == UNSUPPORTED
    assert write(n=0) == OK and fp8(n=0) == OK


@pytest.mark.parametrize("k_rows,kv_rows", [(64, 64), (128, 64), (64, 128)])
def test_binding_passes_the_shorter_cache(monkeypatch, k_rows, kv_rows):
    seen = {}

    class Lib:
        def dsa_cache_write_bounded(self, *a):
            seen["bf16"] = a[-2]
            return 0

        def dsa_cache_write_fp8_bounded(self, *a):
            seen["fp8"] = a[-2]
            return 0

    monkeypatch.setattr(_native, "load", lambda: Lib())
    monkeypatch.setattr(_native, "_ptr", lambda t: None)
    monkeypatch.setattr(_native, "_stream", lambda s: None)
    monkeypatch.setattr(_native, "_raw_stream", lambda s: None)
    monkeypatch.setattr(_native, "_addresses", lambda where, *tt: [None] * len(tt))
    f, i = torch.zeros, torch.int32
    common = (f(3, 128), f(3, 576), f(3, dtype=i), f(3, dtype=i), f(128), f(128), f(512), f(32))
    dsa.dsa_cache_write(*common, f(k_rows, 128), f(kv_rows, 576))
    dsa.dsa_cache_write_fp8(*common, f(k_rows, 128), f(k_rows), f(kv_rows, 640), f(kv_rows))
    assert seen == {"bf16": min(k_rows, kv_rows), "fp8": min(k_rows, kv_rows)}
