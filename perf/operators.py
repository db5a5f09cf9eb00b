"""The serving operators around the DSA path, as cases that can be timed and compared.

Four operators, in the order in which one step of a server runs them:

  plan    block tables and slot maps from the requests' lengths (``dsa_paged_plan``)
  rope    rotary positions on the queries' RoPE dims (``dsa_rope``)
  write   new tokens' indexer keys and latents into the 8-bit cache (``dsa_cache_write_fp8``)
  mla     attention over the selected rows of the 8-bit latent cache (``dsa_sparse_mla_fp8_fwd``)

With ``own`` false, ``run`` computes an operator in plain torch operations; with ``own``
true it makes the package's call.  ``exact`` gives the same outputs from the definitions in
64 bits.

The 8-bit latent cache: row r holds 640 e4m3 codes and one power-of-two scale
s = 2^(kv_scale[r] - 127).  Codes 0..511 times s are the latent; RoPE dim i stands as
(code[512 + i] + code[576 + i]) * 16 * s.
"""
import math

import torch

own = False

PAGE = 64            # tokens per cache page
HEADS = 128          # query heads
LATENT, ROPE = 512, 64
CODES = LATENT + 2 * ROPE
ROPE_GAIN = 16.0
IDX_HEADS, IDX_DIM = 64, 128
SM_SCALE = 1.0 / math.sqrt(192.0)
MAX_POS = 163840     # positions of the long-context configuration
EPS = 1e-6
DEV = "cuda"


# ------------------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 64 running requests: one token each, some cross into a new page
        {"name": "plan decode 64", "op": "plan", "batch": 64, "new_min": 1, "new_max": 1, "ctx_max": 65536, "pad": 0},
        # a mixed step: 500 requests, prompts being prefilled beside decodes, a padded token axis
        {"name": "plan mixed 500", "op": "plan", "batch": 500, "new_min": 0, "new_max": 131, "ctx_max": 8192, "pad": 77},
        # queries of a decode step: the RoPE part of 128 heads out of the projection's rows
        # ([.., 192] per head) into the absorbed query's last 64 dims ([.., 576])
        {"name": "rope query decode 64", "op": "rope", "tokens": 64, "heads": HEADS, "src": 192, "src_at": 128,
         "dst": 576, "dst_at": 512, "head": 64, "begin": 0, "dim": 64, "interleaved": True, "dtype": "bf16", "back": False},
        # the same for one 8192-query chunk of a long prefill
        {"name": "rope query chunk 8192", "op": "rope", "tokens": 8192, "heads": HEADS, "src": 192, "src_at": 128,
         "dst": 576, "dst_at": 512, "head": 64, "begin": 0, "dim": 64, "interleaved": True, "dtype": "bf16", "back": False},
        # the indexer's queries of an odd-sized chunk: half layout on the first 64 of 128 dims,
        # the rest copied
        {"name": "rope indexer 5003", "op": "rope", "tokens": 5003, "heads": IDX_HEADS, "src": 128, "src_at": 0,
         "dst": 128, "dst_at": 0, "head": 128, "begin": 0, "dim": 64, "interleaved": False, "dtype": "bf16", "back": False},
        # cache rows of a decode step's tokens
        {"name": "write decode 64", "op": "write", "tokens": 64, "rows": 4096, "index": "ue8m0", "pad": 0},
        # an odd chunk with padding rows, indexer keys with fp32 scales
        {"name": "write chunk 4099", "op": "write", "tokens": 4099, "rows": 8192, "index": "e4m3", "pad": 61},
        # a whole 32K prefill
        {"name": "write prefill 32768", "op": "write", "tokens": 32768, "rows": 40960, "index": "ue8m0", "pad": 0},
        # one request decoding at 32K: latency
        {"name": "mla decode 1", "op": "mla", "batch": 1, "ctx_min": 32768, "ctx_max": 32768, "queries": 1, "topk": 2048, "paged": True},
        # a small ragged batch with several queries each and short selections
        {"name": "mla ragged 9x3", "op": "mla", "batch": 9, "ctx_min": 300, "ctx_max": 4001, "queries": 3, "topk": 512, "paged": True},
        # the decode workload: 64 requests, contexts 8K to 64K
        {"name": "mla decode 64", "op": "mla", "batch": 64, "ctx_min": 8192, "ctx_max": 65536, "queries": 1, "topk": 2048, "paged": True},
        # a 1024-query chunk of a 32K prefill, packed cache
        {"name": "mla chunk 1024", "op": "mla", "batch": 1, "ctx_min": 32768, "ctx_max": 32768, "queries": 1024, "topk": 2048, "paged": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "rope", "write", "mla", "mla"])
    if op == "plan":
        hi = _log(rng, 1, 500)
        return {"op": op, "batch": _log(rng, 1, 500), "new_min": rng.choice([0, 1]), "new_max": min(hi, 131),
                "ctx_max": _log(rng, 64, 65536), "pad": rng.choice([0, rng.randint(1, 300)])}
    if op == "rope":
        kind = rng.randint(0, 2)
        if kind == 0:
            return {"op": op, "tokens": _log(rng, 1, 8000), "heads": HEADS, "src": 192, "src_at": 128, "dst": 576,
                    "dst_at": 512, "head": 64, "begin": 0, "dim": 64, "interleaved": True, "dtype": "bf16",
                    "back": rng.random() < 0.3}
        if kind == 1:
            return {"op": op, "tokens": _log(rng, 1, 8000), "heads": IDX_HEADS, "src": 128, "src_at": 0, "dst": 128,
                    "dst_at": 0, "head": 128, "begin": 0, "dim": 64, "interleaved": False,
                    "dtype": rng.choice(["bf16", "fp16", "fp32"]), "back": rng.random() < 0.3}
        dim = 2 * rng.randint(1, 64)
        head = dim + rng.randint(0, 100)
        return {"op": op, "tokens": _log(rng, 1, 2000), "heads": rng.randint(1, 40), "src": head + rng.randint(0, 30),
                "src_at": 0, "dst": head, "dst_at": 0, "head": head, "begin": rng.randint(0, head - dim), "dim": dim,
                "interleaved": rng.random() < 0.5, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "back": rng.random() < 0.3}
    if op == "write":
        n = _log(rng, 1, 32000)
        return {"op": op, "tokens": n, "rows": (n + 64 + rng.randint(0, 8000)) // 64 * 64 + 64,
                "index": rng.choice(["ue8m0", "e4m3", "bf16"]), "pad": rng.choice([0, rng.randint(0, n // 2)])}
    ctx = _log(rng, 1100, 32000)
    if rng.random() < 0.5:
        return {"op": op, "batch": _log(rng, 1, 64), "ctx_min": max(1, ctx // rng.randint(2, 9)), "ctx_max": ctx,
                "queries": rng.randint(1, 3), "topk": rng.choice([2048, 2048, rng.randint(1, 2048)]), "paged": True}
    return {"op": op, "batch": 1, "ctx_min": ctx, "ctx_max": ctx, "queries": _log(rng, 1, 1000),
            "topk": rng.choice([2048, 2048, rng.randint(1, 2048)]), "paged": False}


# ------------------------------------------------------------------------------ inputs

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _frequencies(dim):
    """RoPE frequencies of ``dim`` rotated dims, base 10000, stretched 40 times over a 4096-token
    training length with the usual ramp between 32 and 1 turns (the long-context schedule)."""
    i = torch.arange(dim // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / dim)
    at = [dim * math.log(4096 / (turns * 2 * math.pi)) / (2 * math.log(10000.0)) for turns in (32.0, 1.0)]
    lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), dim - 1)
    ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
    return (f / 40.0 * ramp + f * (1 - ramp)).to(torch.float32).to(DEV)


def _codes(x):
    x = x.clamp(-448.0, 448.0)
    if x.dtype == torch.float64:   # rounded once, to the nearest code: torch's cast goes through 32 bits
        unit = torch.exp2((torch.frexp(x).exponent - 4).clamp(min=-9).double())
        x = torch.round(x / unit) * unit
    return x.to(torch.float8_e4m3fn)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 13)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)

    def ints(lo, hi, *shape, dtype=torch.int32):   # lo .. hi
        return torch.randint(lo, hi + 1, shape, generator=g, device=DEV, dtype=torch.int64).to(dtype)

    s = dict(case)
    if case["op"] == "plan":
        B = case["batch"]
        cached = ints(0, case["ctx_max"], B)
        new = ints(case["new_min"], case["new_max"], B)
        new[0] = max(1, case["new_min"])
        width = (case["ctx_max"] + case["new_max"] + 1 + PAGE - 1) // PAGE
        old = (cached.long() + PAGE - 1) // PAGE
        extra = (cached.long() + new + PAGE - 1) // PAGE - old
        n_old, n_new = int(old.sum()), int(extra.sum())
        pages = n_old + n_new + 5
        perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
        table = torch.full((B, width), -1, dtype=torch.int32, device=DEV)
        table[torch.arange(width, device=DEV)[None, :] < old[:, None]] = perm[:n_old]
        T = B * case["new_max"] + case["pad"]   # the token axis a captured step is sized for
        s.update(cached=cached, new=new, table=table, free=perm[n_old:].contiguous(), pages=pages, T=T,
                 cu_q=torch.empty(B + 1, dtype=torch.int32, device=DEV), cu_k=torch.empty(B + 1, dtype=torch.int32, device=DEV),
                 positions=torch.empty(T, dtype=torch.int32, device=DEV), slots=torch.empty(T, dtype=torch.int32, device=DEV),
                 counts=torch.empty(4, dtype=torch.int32, device=DEV))
    elif case["op"] == "rope":
        t = _TYPES[case["dtype"]]
        x = normal(case["tokens"], case["heads"], case["src"]).to(t)
        out = torch.zeros(case["tokens"], case["heads"], case["dst"], dtype=t, device=DEV)
        s.update(x=x[..., case["src_at"]:case["src_at"] + case["head"]], out=out[..., case["dst_at"]:case["dst_at"] + case["head"]],
                 positions=ints(0, MAX_POS - 1, case["tokens"]), inv_freq=_frequencies(case["dim"]),
                 gain=0.1 * math.log(40.0) + 1.0)
    elif case["op"] == "write":
        n, rows = case["tokens"], case["rows"]
        place = torch.randperm(rows, generator=g, device=DEV)[:n].to(torch.int32)
        if case["pad"]:
            place[n - case["pad"]:] = -1   # a padded batch: these tokens have no row
        s.update(k_raw=(2.0 * normal(n, IDX_DIM) + 0.5).to(torch.bfloat16), kv_raw=normal(n, LATENT + ROPE).to(torch.bfloat16),
                 positions=ints(0, MAX_POS - 1, n), place=place, ln_w=torch.rand(IDX_DIM, generator=g, device=DEV) + 0.5,
                 ln_b=0.1 * normal(IDX_DIM), rms_w=torch.rand(LATENT, generator=g, device=DEV) + 0.5, inv_freq=_frequencies(ROPE),
                 k_cache=torch.zeros(rows, IDX_DIM, dtype=torch.bfloat16 if case["index"] == "bf16" else torch.uint8, device=DEV),
                 k_scale=None if case["index"] == "bf16" else torch.zeros(rows, dtype=torch.float32 if case["index"] == "e4m3" else torch.uint8, device=DEV),
                 kv_cache=torch.zeros(rows, CODES, dtype=torch.uint8, device=DEV), kv_scale=torch.zeros(rows, dtype=torch.uint8, device=DEV))
    else:
        B, K, Q = case["batch"], case["topk"], case["queries"]
        lens = ints(case["ctx_min"], case["ctx_max"], B)
        host = [max(int(v), Q) for v in lens.tolist()]
        lens = torch.tensor(host, dtype=torch.int32, device=DEV)
        T = B * Q
        pages = [(n + PAGE - 1) // PAGE for n in host]
        S = sum(pages) * PAGE if case["paged"] else sum(host)
        # cached rows: normalised latents and rotated keys, quantised with a scale for each row
        kv = normal(S, LATENT + ROPE, dtype=torch.bfloat16).float() * (0.5 + torch.rand(S, 1, generator=g, device=DEV))
        amax = torch.maximum(kv[:, :LATENT].abs().amax(1), kv[:, LATENT:].abs().amax(1) / ROPE_GAIN)
        scale = torch.exp2(torch.ceil(torch.log2(amax / 448.0)))
        codes = torch.empty(S, CODES, dtype=torch.float8_e4m3fn, device=DEV)
        codes[:, :LATENT] = _codes(kv[:, :LATENT] / scale[:, None])
        r = kv[:, LATENT:] / (ROPE_GAIN * scale[:, None])
        codes[:, LATENT:LATENT + ROPE] = _codes(r)
        codes[:, LATENT + ROPE:] = _codes(r - codes[:, LATENT:LATENT + ROPE].float())
        del kv, r
        pos = (lens.long()[:, None] - Q + torch.arange(Q, device=DEV)[None, :]).reshape(-1)      # of each query
        # the selected keys, ascending, -1 behind them (what the top-k writes)
        u = torch.rand(T, max(host), generator=g, device=DEV)
        u.masked_fill_(torch.arange(max(host), device=DEV)[None, :] > pos[:, None], -1.0)
        best = u.topk(min(K, max(host)), dim=1)
        idx = torch.where(best.values >= 0, best.indices, max(host)).sort(dim=1).values
        idx = torch.where(idx == max(host), -1, idx).to(torch.int32)
        if idx.shape[1] < K:
            idx = torch.cat([idx, idx.new_full((T, K - idx.shape[1]), -1)], 1)
        del u, best
        table = None
        if case["paged"]:
            perm = torch.randperm(sum(pages), generator=g, device=DEV).to(torch.int32)
            table = torch.full((B, max(pages)), -1, dtype=torch.int32, device=DEV)
            table[torch.arange(max(pages), device=DEV)[None, :] < torch.tensor(pages, device=DEV)[:, None]] = perm
        zero = torch.zeros(1, dtype=torch.int32, device=DEV)
        s.update(T=T, S=S, longest=max(host), q=normal(T, HEADS, LATENT + ROPE).to(torch.bfloat16), codes=codes.view(torch.uint8),
                 kv_scale=(torch.log2(scale) + 127.0).to(torch.uint8), idx=idx.contiguous(), table=table,
                 cu_q=torch.arange(0, T + 1, Q, dtype=torch.int32, device=DEV),
                 cu_k=torch.cat([zero, lens.cumsum(0).to(torch.int32)]), out=torch.empty(T, HEADS, LATENT, dtype=torch.bfloat16, device=DEV),
                 lse=torch.empty(T, HEADS, dtype=torch.float32, device=DEV))
    return s


# ------------------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _own(state)
    return {"plan": _plan, "rope": _rope, "write": _write, "mla": _mla}[state["op"]](state)


def _own(s):
    import attention_lightning_indexer_b200 as dsa

    if s["op"] == "plan":
        dsa.dsa_paged_plan(s["cached"], s["new"], s["table"], s["free"], s["cu_q"], s["cu_k"], s["positions"], s["slots"],
                           s["counts"], n_pages=s["pages"])
        return _plan_outputs(s)
    if s["op"] == "rope":
        dsa.dsa_rope(s["x"], s["positions"], s["inv_freq"], s["out"],
                     layout=dsa.DSA_ROPE_INTERLEAVED if s["interleaved"] else dsa.DSA_ROPE_HALF, rope_begin=s["begin"],
                     rope_dim=s["dim"], scale=s["gain"], transposed=s["back"])
        return s["out"]
    if s["op"] == "write":
        kind = {"bf16": dsa.DSA_BF16, "e4m3": dsa.DSA_E4M3, "ue8m0": dsa.DSA_E4M3_UE8M0}[s["index"]]
        dsa.dsa_cache_write_fp8(s["k_raw"], s["kv_raw"], s["positions"], s["place"], s["ln_w"], s["ln_b"], s["rms_w"],
                                s["inv_freq"], s["k_cache"], s["k_scale"], s["kv_cache"], s["kv_scale"], idx_dtype=kind, eps=EPS)
        return _write_outputs(s)
    if "problem" not in s:   # a server keeps its problem description and workspace over the layers of a step
        Q, packed = s["queries"], s["table"] is None
        s["problem"] = dsa.make_problem(s["batch"], s["T"], s["S"], Q, s["longest"], s["topk"], cu_q=None if packed else s["cu_q"],
                                        cu_k=None if packed else s["cu_k"], sm_scale=SM_SCALE, block_table=s["table"])
        s["workspace"] = torch.empty(dsa.dsa_sparse_mla_fp8_workspace_size(s["problem"]), dtype=torch.uint8, device=DEV)
    dsa.dsa_sparse_mla_fp8_fwd(s["problem"], s["q"], s["codes"], s["kv_scale"], s["idx"], s["out"], s["lse"], s["workspace"])
    return s["out"], s["lse"]


def _plan_outputs(s):
    return {k: s[k] for k in ("cu_q", "cu_k", "positions", "slots", "table", "counts")}


def _write_outputs(s):
    """8-bit codes as the numbers they are, beside their scales."""
    k = s["k_cache"] if s["index"] == "bf16" else s["k_cache"].view(torch.float8_e4m3fn)
    return {"k": k, "k_scale": s["k_scale"], "kv": s["kv_cache"].view(torch.float8_e4m3fn), "kv_scale": s["kv_scale"]}


def _plan(s):
    cached, new, T = s["cached"].long(), s["new"].long(), s["T"]
    total = cached + new
    q_end, k_end = new.cumsum(0), total.cumsum(0)
    s["cu_q"][0] = 0
    s["cu_q"][1:] = q_end
    s["cu_k"][0] = 0
    s["cu_k"][1:] = k_end
    old = (cached + PAGE - 1) // PAGE
    need = (total + PAGE - 1) // PAGE - old
    first = need.cumsum(0) - need
    t = torch.arange(T, device=DEV)
    live = t < q_end[-1]
    u = torch.minimum(t, q_end[-1] - 1)
    b = torch.searchsorted(q_end, u, right=True)
    pos = cached[b] + u - (q_end - new)[b]
    page = pos // PAGE
    fresh = page - old[b]
    number = torch.where(fresh >= 0, s["free"][(first[b] + fresh).clamp(min=0)], s["table"][b, page])
    s["table"].index_put_((b, page), number)
    s["positions"].copy_(torch.where(live, pos, 0))
    s["slots"].copy_(torch.where(live, number.long() * PAGE + pos % PAGE, -1))
    s["counts"].copy_(torch.stack([q_end[-1], need.sum(), total.max(), torch.zeros_like(q_end[-1])]))
    return _plan_outputs(s)


def _angles(s, dim):
    a = s["positions"].double()[:, None] * s["inv_freq"].double()[None, :]
    return torch.cos(a), torch.sin(a)


def _rope(s):
    c, n = (v.float()[:, None, :] * s["gain"] for v in _angles(s, s["dim"]))
    if s["back"]:
        n = -n
    x, b, d = s["x"], s["begin"], s["dim"]
    part = x[..., b:b + d].float()
    if s["interleaved"]:
        u, v = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([u * c - v * n, v * c + u * n], -1).flatten(-2)
    else:
        u, v = part[..., :d // 2], part[..., d // 2:]
        turned = torch.cat([u * c - v * n, v * c + u * n], -1)
    out = s["out"]
    out[..., :b] = x[..., :b]
    out[..., b:b + d] = turned
    out[..., b + d:] = x[..., b + d:]
    return out


def _exponent(amax):
    """The exponent of the smallest power of two s with amax / s <= 448 (at least 2^-126)."""
    m, e = torch.frexp(amax)
    e = e - 9 + (m > 0.875)
    return torch.where(amax > 0, e, -126).clamp(-126, 127)


def _write(s):
    # in 64 bits: a value next to a border between two codes decides which code is written
    x = s["k_raw"].double()
    x = x - x.mean(1, keepdim=True)
    x = x / torch.sqrt(x.square().mean(1, keepdim=True) + EPS) * s["ln_w"].double() + s["ln_b"].double()
    c, n = _angles(s, ROPE)
    u, v = x[:, :32], x[:, 32:64]
    x = torch.cat([u * c - v * n, v * c + u * n, x[:, 64:]], 1)
    z = s["kv_raw"].double()
    lat = z[:, :LATENT]
    lat = lat / torch.sqrt(lat.square().mean(1, keepdim=True) + EPS) * s["rms_w"].double()
    u, v = z[:, LATENT::2], z[:, LATENT + 1::2]
    rot = torch.stack([u * c - v * n, v * c + u * n], -1).flatten(-2)

    # tokens without a row go to a row behind the cache, which is dropped
    rows = s["kv_scale"].shape[0]
    at = torch.where(s["place"] < 0, rows, s["place"]).long()

    def put(name, values):
        full = torch.cat([s[name], s[name].new_zeros((1,) + s[name].shape[1:])])
        full.index_copy_(0, at, values)
        s[name].copy_(full[:rows])

    if s["index"] == "bf16":
        put("k_cache", x.to(torch.bfloat16))
    else:
        amax = x.abs().amax(1)
        if s["index"] == "ue8m0":
            e = _exponent(amax)
            put("k_scale", (e + 127).to(torch.uint8))
            div = torch.exp2(e.double())
        else:
            div = torch.where(amax > 0, amax / 448.0, 1.0).float()
            put("k_scale", div)
            div = div.double()
        put("k_cache", _codes(x / div[:, None]).view(torch.uint8))
    e = _exponent(torch.maximum(lat.abs().amax(1), rot.abs().amax(1) / ROPE_GAIN))
    div = torch.exp2(e.double())[:, None]
    r = rot / (ROPE_GAIN * div)
    hi = _codes(r)
    put("kv_scale", (e + 127).to(torch.uint8))
    put("kv_cache", torch.cat([_codes(lat / div), hi, _codes(r - hi.double())], 1).view(torch.uint8))
    return _write_outputs(s)


def _key_rows(s):
    """Cache row of every selected key and whether the slot is live."""
    live = s["idx"] >= 0
    at = s["idx"].clamp(min=0).long()
    b = torch.arange(s["T"], device=DEV)[:, None] // s["queries"]
    if s["table"] is not None:
        return s["table"][b, at // PAGE].long() * PAGE + at % PAGE, live
    return s["cu_k"][b].long() + at, live


def _mla(s):
    rows, live = _key_rows(s)
    c = s["codes"][rows].view(torch.float8_e4m3fn).float()
    kv = torch.cat([c[..., :LATENT], (c[..., LATENT:LATENT + ROPE] + c[..., LATENT + ROPE:]) * ROPE_GAIN], -1)
    kv *= torch.exp2(s["kv_scale"][rows].float() - 127.0)[..., None]
    z = torch.bmm(s["q"].float(), kv.transpose(1, 2)) * SM_SCALE
    z.masked_fill_(~live[:, None, :], float("-inf"))
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    total = p.sum(-1, keepdim=True)
    out = torch.bmm(p, kv[..., :LATENT]) / total
    return out.to(torch.bfloat16), (m + torch.log(total))[..., 0]


# ------------------------------------------------------------------------------ work

def work(case):
    if case["op"] == "plan":
        tokens, axis = case["batch"] * (case["new_min"] + case["new_max"]) / 2, case["batch"] * case["new_max"] + case["pad"]
        return {"bytes": 4 * (2 * case["batch"] + 2 * axis + 2 * tokens / PAGE + 3 * case["batch"]), "flops": 0}
    if case["op"] == "rope":
        size = 4 if case["dtype"] == "fp32" else 2
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * case["head"] * size + 4 * case["tokens"], "flops": 3 * n * case["dim"]}
    if case["op"] == "write":
        n, live = case["tokens"], case["tokens"] - case["pad"]
        k = 256 if case["index"] == "bf16" else 128 + (4 if case["index"] == "e4m3" else 1)
        return {"bytes": live * (1408 + 4 + k + CODES + 1) + 4 * n, "flops": 8 * live * 704}
    T = case["batch"] * case["queries"]
    mean = (case["ctx_min"] + case["ctx_max"]) / 2
    keys = T * min(case["topk"], mean)
    distinct = min(keys, case["batch"] * mean)   # each cached row read once
    return {"bytes": distinct * (CODES + 1) + 4 * T * case["topk"] + T * HEADS * (2 * 576 + 2 * 512 + 4),
            "flops": 2 * keys * HEADS * (576 + 512)}


# ------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None   # whole numbers only
    if case["op"] == "rope":
        x, d, b = s["x"].double(), case["dim"], case["begin"]
        turn = torch.polar(torch.full((1,), s["gain"], dtype=torch.float64, device=DEV),
                           s["positions"].double()[:, None] * s["inv_freq"].double())[:, None, :]
        if case["back"]:
            turn = turn.conj()
        out = x.clone()
        part = x[..., b:b + d]
        if case["interleaved"]:
            out[..., b:b + d] = torch.view_as_real(torch.view_as_complex(part.reshape(*part.shape[:-1], d // 2, 2).contiguous()) * turn).flatten(-2)
        else:
            w = torch.complex(part[..., :d // 2].contiguous(), part[..., d // 2:].contiguous()) * turn
            out[..., b:b + d] = torch.cat([w.real, w.imag], -1)
        return out
    if case["op"] == "write":
        return _exact_write(case, s)
    out, lse = [], []
    step = max(1, (1 << 17) // case["topk"])
    table = s["table"]
    for t0 in range(0, s["T"], step):
        o, l = [], []
        ix = s["idx"][t0:t0 + step].long()
        seq = torch.arange(t0, t0 + ix.shape[0], device=DEV) // case["queries"]
        sel = ix.clamp(min=0)
        rows = s["cu_k"].long()[seq][:, None] + sel if table is None else table.long()[seq].gather(1, sel // PAGE) * PAGE + sel % PAGE
        code = s["codes"].view(torch.float8_e4m3fn)[rows.reshape(-1)].double().reshape(*rows.shape, CODES)
        code *= torch.pow(2.0, s["kv_scale"][rows].double() - 127)[..., None]
        val = code[..., :LATENT]
        rot = 16.0 * code[..., LATENT:].unflatten(-1, (2, ROPE)).sum(-2)
        qd = s["q"][t0:t0 + step].double()
        z = (torch.einsum("thd,tkd->thk", qd[..., :LATENT], val) + torch.einsum("thd,tkd->thk", qd[..., LATENT:], rot)) / math.sqrt(192.0)
        z = torch.where(ix[:, None, :] < 0, float("-inf"), z)
        l = torch.logsumexp(z, -1)
        o = torch.einsum("thk,tkd->thd", torch.exp(z - l[..., None]), val)
        out.append(o)
        lse.append(l)
    return torch.cat(out), torch.cat(lse)


def _exact_write(case, s):
    def nearest(v):   # the e4m3 number nearest to v, ties to the even code
        a = v.abs().clamp(max=448.0)
        step = torch.exp2((torch.frexp(a).exponent - 4).clamp(min=-9).double())
        return torch.sign(v) * torch.round(a / step) * step

    def scale_of(top):
        e = torch.ceil(torch.log2(top.clamp(min=2.0 ** -126 * 448) / 448.0))
        return torch.exp2(torch.where(top <= 448.0 * torch.exp2(e - 1), e - 1, e).clamp(-126, 127))

    live = s["place"] >= 0
    at = s["place"][live].long()
    ang = (s["positions"].double()[:, None] * s["inv_freq"].double())[live]
    turn = torch.polar(torch.ones_like(ang), ang)
    x = s["k_raw"][live].double()
    mu = x.sum(1, keepdim=True) / IDX_DIM
    x = (x - mu) * ((x - mu).pow(2).sum(1, keepdim=True) / IDX_DIM + EPS).pow(-0.5) * s["ln_w"].double() + s["ln_b"].double()
    w = torch.complex(x[:, :32].contiguous(), x[:, 32:64].contiguous()) * turn
    x = torch.cat([w.real, w.imag, x[:, 64:]], 1)
    z = s["kv_raw"][live].double()
    lat = z[:, :LATENT] * (z[:, :LATENT].pow(2).sum(1, keepdim=True) / LATENT + EPS).pow(-0.5) * s["rms_w"].double()
    rot = torch.view_as_real(torch.view_as_complex(z[:, LATENT:].reshape(-1, 32, 2).contiguous()) * turn).flatten(-2)

    def whole(values, width):
        full = torch.zeros((case["rows"], width), dtype=torch.float64, device=DEV)
        full[at] = values
        return full

    k_scale = None
    if case["index"] == "ue8m0":
        x = nearest(x / scale_of(x.abs().amax(1, keepdim=True)))
    elif case["index"] == "e4m3":
        k_scale = x.abs().amax(1, keepdim=True) / 448.0
        x = nearest(x / k_scale.float().double())
        k_scale = whole(k_scale, 1)[:, 0]
    div = scale_of(torch.maximum(lat.abs().amax(1, keepdim=True), rot.abs().amax(1, keepdim=True) / 16))
    r = rot / (16 * div)
    hi = nearest(r)
    return {"k": whole(x, IDX_DIM), "k_scale": k_scale, "kv": whole(torch.cat([nearest(lat / div), hi, nearest(r - hi)], 1), CODES),
            "kv_scale": None}
