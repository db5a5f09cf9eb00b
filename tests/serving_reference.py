"""64-bit restatements of the serving operators (page plan, RoPE, 8-bit cache write, attention
over the 8-bit latent cache), one definition at a time in numpy, for the parity tests."""
from __future__ import annotations

import math

import numpy as np

PAGE = 64


def e4m3_table() -> np.ndarray:
    """The number each e4m3 code stands for (fp64; codes 0x7f and 0xff are NaN)."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = math.nan if (e == 15 and m == 7) else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if s else v
    return out


E4M3 = e4m3_table()
_POS = E4M3[:127]                        # 0 .. 448, ascending


def e4m3_nearest(v: np.ndarray) -> np.ndarray:
    """Codes of the e4m3 numbers nearest to v (|v| <= 448 after clipping), ties to the even code."""
    a = np.minimum(np.abs(v), 448.0)
    hi = np.searchsorted(_POS, a)        # first code with value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[np.minimum(hi, 126)] - a
    take_hi = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = np.where(hi == 0, 0, np.where(take_hi, hi, lo)).astype(np.uint8)
    return np.where(np.signbit(v), code | 0x80, code).astype(np.uint8)


def scale_exponent(amax: np.ndarray) -> np.ndarray:
    """Smallest e >= -126 with amax <= 448 * 2^e, by trying exponents."""
    e = np.full(amax.shape, -126)
    for k in range(-126, 120):
        e = np.where(amax > 448.0 * 2.0 ** k, k + 1, e)
    return e


def rope(x, positions, inv_freq, layout, begin, dim, scale=1.0, transposed=False) -> np.ndarray:
    """x fp64 [T, H, D]; layout 0 half, 1 interleaved."""
    a = positions.astype(np.float64)[:, None] * inv_freq.astype(np.float64)[None, :]
    c, s = np.cos(a)[:, None, :] * scale, np.sin(a)[:, None, :] * scale
    if transposed:
        s = -s
    iu = begin + (np.arange(dim // 2) if layout == 0 else 2 * np.arange(dim // 2))
    iv = iu + (dim // 2 if layout == 0 else 1)
    out = x.copy()
    out[..., iu] = x[..., iu] * c - x[..., iv] * s
    out[..., iv] = x[..., iv] * c + x[..., iu] * s
    return out


def write_rows(k_raw, kv_raw, positions, ln_w, ln_b, rms_w, inv_freq, eps):
    """Indexer keys [n, 128], latents [n, 512] and rotated RoPE dims [n, 64] in fp64."""
    x = k_raw - k_raw.mean(1, keepdims=True)
    x = x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * ln_w + ln_b
    k = rope(x[:, None, :], positions, inv_freq, 0, 0, 64)[:, 0]
    lat = kv_raw[:, :512]
    lat = lat / np.sqrt((lat * lat).mean(1, keepdims=True) + eps) * rms_w
    rot = rope(kv_raw[:, None, 512:], positions, inv_freq, 1, 0, 64)[:, 0]
    return k, lat, rot


def quantise_latent(lat, rot):
    """(codes uint8 [n, 640], scale bytes uint8 [n])."""
    e = scale_exponent(np.maximum(np.abs(lat).max(1), np.abs(rot).max(1) / 16))
    s = 2.0 ** e[:, None]
    r = rot / (16 * s)
    hi = e4m3_nearest(r)
    lo = e4m3_nearest(r - E4M3[hi])
    return np.concatenate([e4m3_nearest(lat / s), hi, lo], 1), (e + 127).astype(np.uint8)


def cache_values(codes, scale_bytes) -> np.ndarray:
    """fp64 [rows, 576]: what 8-bit latent rows stand for."""
    v = E4M3[codes]
    s = 2.0 ** (scale_bytes.astype(np.float64) - 127)
    return np.concatenate([v[:, :512], (v[:, 512:576] + v[:, 576:]) * 16], 1) * s[:, None]


def plan(cached, new, table, free, head, n_pages, n_tokens):
    """(cu_q, cu_k, positions, rows, table, counts), request by request."""
    B, width = table.shape
    table = table.copy()
    pages = [-(-int(c) // PAGE) for c in cached]
    need = [-(-(int(c) + int(n)) // PAGE) for c, n in zip(cached, new)]
    err = 0
    if sum(max(0, b - a) for a, b in zip(pages, need)) + head > len(free) or head < 0:
        err |= 1
    if any(b > width for b in need):
        err |= 2
    if sum(int(n) for n in new) > n_tokens or sum(int(c) + int(n) for c, n in zip(cached, new)) > 2 ** 31 - 1:
        err |= 4
    if any(c < 0 for c in cached) or any(n < 0 for n in new):
        err |= 8
    pos, rows = np.zeros(n_tokens, np.int32), np.full(n_tokens, -1, np.int32)
    if err:
        z = np.zeros(B + 1, np.int32)
        return z, z.copy(), pos, rows, table, np.array([0, 0, 0, err], np.int32)
    cu_q, cu_k, at = [0], [0], head
    for b in range(B):
        for j in range(pages[b], need[b]):
            table[b, j] = free[at]
            at += 1
        for i in range(int(new[b])):
            p, t = int(cached[b]) + i, cu_q[-1] + i
            page = int(table[b, p // PAGE])
            pos[t] = p
            rows[t] = page * PAGE + p % PAGE if 0 <= page < n_pages else -1
        cu_q.append(cu_q[-1] + int(new[b]))
        cu_k.append(cu_k[-1] + int(cached[b]) + int(new[b]))
    longest = max(int(c) + int(n) for c, n in zip(cached, new))
    return (np.array(cu_q, np.int32), np.array(cu_k, np.int32), pos, rows, table,
            np.array([cu_q[-1], at - head, longest, 0], np.int32))


def attention(q, key_rows, values, scale_bytes, sm_scale):
    """One query row: q fp64 [H, 576], key_rows the cache rows of its live slots.  Returns out
    [H, 512], lse [H], and bounds on what the kernel's roundings may change of each (below)."""
    H = q.shape[0]
    if len(key_rows) == 0:
        return np.zeros((H, 512)), np.full(H, -np.inf), np.zeros((H, 512)), np.zeros(H)
    kv = values[key_rows]
    z = q @ kv.T * sm_scale
    m = z.max(1, keepdims=True)
    p = np.exp(z - m)
    l = p.sum(1, keepdims=True)
    out = p @ kv[:, :512] / l
    # Bounds.
    # (1) q as hi (e4m3) + lo (e5m2) at scale 2^f, the smallest with max(|q_lat|, 16 |q_rope|) <= 448 * 2^f:
    #     from 2^-6 * 2^f on hi has 4 significant bits and the rest is at most 8 units of the 8th bit,
    #     which e5m2's 3 bits hold; below, hi steps by 2^-9, the rest is at most 2^-10 and half its step
    #     in e5m2 at most 2^-14 (times 2^f; for 16 * q_rope: 2^-18 on q_rope).
    top = np.maximum(np.abs(q[:, :512]).max(1), 16 * np.abs(q[:, 512:]).max(1))
    f = 2.0 ** scale_exponent(top)[:, None]
    dq = np.concatenate([np.where(np.abs(q[:, :512]) < 2.0 ** -6 * f, 2.0 ** -14 * f, 0),
                         np.where(np.abs(16 * q[:, 512:]) < 2.0 ** -6 * f, 2.0 ** -18 * f, 0)], 1)
    # (2) 1280 products summed in fp32, added up 32 at a time: 40 additions at 2^-23 of the sum
    #     of magnitudes; the scaling and the exponent's argument add a few more.
    dz = sm_scale * (dq @ np.abs(kv).T + 48 * 2.0 ** -23 * (np.abs(q) @ np.abs(kv).T)) + 2.0 ** -22 * (np.abs(z) + np.abs(m))
    dzmax = dz.max(1, keepdims=True)
    lse_tol = dzmax[:, 0] + 2.0 ** -20 + 2.0 ** -23 * np.abs(m[:, 0] + np.log(l[:, 0]))
    # (3) p as two e4m3 numbers: relative 2^-8 (4 + 4 significant bits; 2^-12 for the fp16 step
    #     between), or half the smallest step.  p is held as p * 2^(4 + its scale's exponent less the
    #     largest one) relative to a reference that no p' of the row is below 1 against, and e4m3
    #     steps by 2^-9 at the least: 2^-10 / 2^4 = 2^-14 of the row's largest p, times the ratio of
    #     the largest scale to the key's.
    s = 2.0 ** (scale_bytes[key_rows].astype(np.float64) - 127)
    dp = p * (2.0 ** -8 + 2.0 ** -12 + 2 * dzmax) + 2.0 ** -14 * (s.max() / s)[None, :]
    # (4) the sums over keys in fp32, and the one rounding to bf16.
    av = np.abs(kv[:, :512])
    out_tol = (dp @ av + 128 * 2.0 ** -23 * (p @ av)) / l + 2.0 ** -8 * np.abs(out) + 2.0 ** -30
    return out, m[:, 0] + np.log(l[:, 0]), out_tol, lse_tol
