"""A NaN in a query or in an attended cache row comes out as NaN, however many SM pairs the
row is split over, and changes no other row or head."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import attention_lightning_indexer_b200 as dsa
import dsa_synth

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _fp8(T, S, topk, idx, poison_q=None, poison_row=None):
    g = torch.Generator(device=DEV).manual_seed(T)
    codes = torch.randn(S, 640, generator=g, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    byte = torch.full((S,), 127, dtype=torch.uint8, device=DEV)
    q = torch.randn(T, 128, 576, generator=g, device=DEV).to(torch.bfloat16)
    if poison_q is not None:
        q[poison_q + (9,)] = float("nan")
    if poison_row is not None:
        codes[poison_row, 100] = 0x7F
    p = dsa.make_problem(1, T, S, T, S, topk)
    out, lse = torch.zeros(T, 128, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(T, 128, device=DEV)
    ws = torch.zeros(max(256, dsa.dsa_sparse_mla_fp8_workspace_size(p)), dtype=torch.uint8, device=DEV)
    dsa.dsa_sparse_mla_fp8_fwd(p, q, codes, byte, idx, out, lse, ws)
    dsa.dsa_check_device_errors()
    return out, lse


def _only(out, lse, t, h):
    """NaN at token t, heads h, and nowhere else."""
    bad = torch.zeros(lse.shape, dtype=torch.bool, device=DEV)
    bad[t, h] = True
    assert torch.equal(torch.isnan(lse), bad)
    assert torch.equal(torch.isnan(out).all(-1), bad) and torch.equal(torch.isnan(out).any(-1), bad)
    assert torch.isfinite(lse[~bad]).all()


@pytest.mark.parametrize("T", [1, 9, 37, 38, 90])
def test_a_nan_query_head(T):
    S, topk = 3000, 2048
    idx = torch.arange(topk, dtype=torch.int32, device=DEV).repeat(T, 1)
    out, lse = _fp8(T, S, topk, idx, poison_q=(T // 2, 77))
    _only(out, lse, T // 2, 77)


@pytest.mark.parametrize("T", [1, 9, 37, 38, 90])
@pytest.mark.parametrize("slots", [1, 200, 2048])
@pytest.mark.parametrize("at", [0, 1500])
def test_a_nan_cache_row_that_is_attended(T, slots, at):
    S, topk = 3000, 2048                     # slots < 257: one part has the NaN, the others nothing
    idx = torch.full((T, topk), -1, dtype=torch.int32, device=DEV)
    first = min(at, topk - slots)
    idx[:, first:first + slots] = torch.arange(slots, dtype=torch.int32, device=DEV) + 5
    t = T - 1
    idx[t, first] = 2900                     # this token alone attends the row
    out, lse = _fp8(T, S, topk, idx, poison_row=2900)
    # a NaN code makes the value dim of its row NaN and, by the score, the whole output
    _only(out, lse, t, slice(None))


@pytest.mark.parametrize("batch", [2, 37, 80])
def test_a_nan_query_head_over_the_bf16_cache(batch):
    inp = dsa_synth.make_decode(batch, 4000, 4200, topk=1024, seed=batch, device=DEV)
    p = dsa.problem_from_inputs(inp)
    inp["q"][1, 3, 5] = float("nan")
    out, lse = torch.zeros(batch, 128, 512, dtype=torch.bfloat16, device=DEV), torch.zeros(batch, 128, device=DEV)
    ws = torch.zeros(dsa.dsa_forward_workspace_size(p, 0), dtype=torch.uint8, device=DEV)
    idx = torch.zeros(batch, 1024, dtype=torch.int32, device=DEV)
    dsa.dsa_forward(p, inp["q_idx"], inp["k_idx"], inp["w"], inp["q"], inp["kv"], out, lse, ws, idx_out=idx)
    _only(out, lse, 1, 3)
    dsa.dsa_sparse_mla_fwd(p, inp["q"], inp["kv"], idx, out, lse)
    _only(out, lse, 1, 3)
    # an attended key: every head of the row that lists it
    inp["q"][1, 3, 5] = 0
    own = int(inp["cu_k"][2]) - 1 - int(inp["cu_k"][1])
    idx[1:] = -1
    idx[1:, 0] = own - 3000
    idx[1, 700] = own
    inp["kv"][int(inp["cu_k"][1]) + own] = float("nan")
    dsa.dsa_sparse_mla_fwd(p, inp["q"], inp["kv"], idx, out, lse)
    _only(out, lse, 1, slice(None))
    dsa.dsa_check_device_errors()


def test_rows_without_a_visible_slot_beside_nan_rows():
    T, S, topk = 9, 3000, 2048
    idx = torch.arange(topk, dtype=torch.int32, device=DEV).repeat(T, 1)
    idx[4] = -1
    out, lse = _fp8(T, S, topk, idx, poison_q=(4, 7))
    assert torch.all(out[4] == 0) and torch.all(torch.isneginf(lse[4]))
    assert torch.isfinite(lse[[0, 3, 5, 8]]).all()
