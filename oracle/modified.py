"""fp64 CPU oracle of attention with modified scores, of the 8-bit key/value
cache and of decoding from it -- TEST INFRASTRUCTURE ONLY (see oracle/attention.py).

Plain definitions in float64, one head at a time, with dense truth values for
the mask and the full score matrix; nothing here is tiled or taken as intervals.
"""
from __future__ import annotations

import numpy as np

__all__ = ["visible", "mod_head_fwd", "mod_head_bwd", "mod_attn_fwd", "mod_attn_bwd", "e4m3_values", "quantise_row",
           "cache_values", "cache_decode_ref"]


def visible(N, causal=False, window=0, doc_ids=None, prefix=0):
    """[N, N] truth values: query i sees key j (one batch entry)."""
    see = np.zeros((N, N), bool)
    ids = None if doc_ids is None else [int(x) for x in doc_ids]
    run = [0] * N
    for i in range(1, N):
        run[i] = run[i - 1] + (0 if ids is None or ids[i] == ids[i - 1] else 1)
    for i in range(N):
        for j in range(N):
            ok = run[i] == run[j] and not (ids is not None and ids[i] < 0)
            if causal and j > i and j >= prefix:
                ok = False
            if window and abs(i - j) >= window:
                ok = False
            see[i, j] = ok
    return see


def _logits(q, k, scale, softcap, slope, away):
    """(z, dz/dx) of the scores x = scale q k^T."""
    x = scale * (np.asarray(q, np.float64) @ np.asarray(k, np.float64).T)
    dz = np.ones_like(x)
    if softcap:
        t = np.tanh(x / softcap)
        x, dz = softcap * t, 1.0 - t * t
    if slope:
        x = x - slope * away
    return x, dz


def _weights(z, see):
    z = np.where(see, z, -np.inf)
    some = see.any(1)
    m = np.where(some, np.max(z, 1, initial=-np.inf), 0.0)
    e = np.exp(z - m[:, None])
    s = e.sum(1)
    with np.errstate(divide="ignore", invalid="ignore"):
        lse = np.where(some, m + np.log(s), -np.inf)
        p = np.where(some[:, None], e / s[:, None], 0.0)
    return p, lse


def mod_head_fwd(q, k, v, see, scale, softcap=0.0, slope=0.0, away=None):
    """One head: O [N, d], LSE [N] and P of queries q against keys k, values v."""
    if away is None:
        away = np.abs(np.arange(len(q))[:, None] - np.arange(len(k))[None, :])
    z, _ = _logits(q, k, scale, softcap, slope, away)
    p, lse = _weights(z, see)
    return p @ np.asarray(v, np.float64), lse, p


def mod_head_bwd(q, k, v, do, see, scale, softcap=0.0, slope=0.0):
    """One head: dQ, dK, dV by the softmax Jacobian and the tanh's derivative."""
    q, k, v, do = (np.asarray(t, np.float64) for t in (q, k, v, do))
    away = np.abs(np.arange(len(q))[:, None] - np.arange(len(k))[None, :])
    z, dz = _logits(q, k, scale, softcap, slope, away)
    p, _ = _weights(z, see)
    dp = do @ v.T
    ds = p * (dp - (p * dp).sum(1, keepdims=True)) * dz
    return scale * ds @ k, scale * ds.T @ q, p.T @ do


def mod_attn_fwd(q, k, v, see, scale, softcap=0.0, slopes=None):
    """q [B, N, H, d], k, v [B, N, Hkv, d], see [B, N, N] -> O, LSE [B, H, N]."""
    B, N, H, d = q.shape
    G = H // k.shape[2]
    O, LSE = np.zeros((B, N, H, d)), np.zeros((B, H, N))
    for b in range(B):
        for h in range(H):
            O[b, :, h], LSE[b, h], _ = mod_head_fwd(q[b, :, h], k[b, :, h // G], v[b, :, h // G], see[b], scale,
                                                    softcap, 0.0 if slopes is None else slopes[h])
    return O, LSE


def mod_attn_bwd(q, k, v, do, see, scale, softcap=0.0, slopes=None):
    B, N, H, d = q.shape
    G = H // k.shape[2]
    dq, dk, dv = np.zeros(q.shape), np.zeros(k.shape), np.zeros(v.shape)
    for b in range(B):
        for h in range(H):
            g = mod_head_bwd(q[b, :, h], k[b, :, h // G], v[b, :, h // G], do[b, :, h], see[b], scale, softcap,
                             0.0 if slopes is None else slopes[h])
            dq[b, :, h] = g[0]
            dk[b, :, h // G] += g[1]
            dv[b, :, h // G] += g[2]
    return dq, dk, dv


def e4m3_values():
    """The 256 values of the OCP e4m3 code: sign, 4 exponent bits (bias 7), 3
    mantissa bits; 0x7f and 0xff are NaN, there are no infinities."""
    out = np.zeros(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = np.nan if (c & 0x7f) == 0x7f else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[c] = -v if s else v
    return out


_POS = e4m3_values()[:127]  # the non-negative finite values, in increasing order


def quantise_row(x):
    """Codes (uint8) and exponent byte of one row, by search: the smallest byte
    e >= 1 with amax <= 448 2^(e - 127); nearest code, ties to the even code.
    Finite values beyond 1.875 2^127 are taken as that."""
    x = np.asarray(x, np.float64)
    x = np.where(np.isfinite(x), np.clip(x, -1.875 * 2.0 ** 127, 1.875 * 2.0 ** 127), x)
    fin = np.abs(x[np.isfinite(x)])
    amax = fin.max() if fin.size else 0.0
    e = 127 if amax == 0.0 else next(e for e in range(1, 255) if amax <= 448.0 * 2.0 ** (e - 127))
    codes = np.zeros(x.shape, np.uint8)
    for i, v in enumerate(x):
        if np.isnan(v):
            codes[i] = 0x7f
            continue
        a = min(abs(v) * 2.0 ** (127 - e), 448.0)
        gap = np.abs(_POS - a)
        best = np.flatnonzero(gap == gap.min())
        c = best[0] if len(best) == 1 or best[0] % 2 == 0 else best[1]
        codes[i] = c | (0x80 if np.signbit(v) else 0)
    return codes, e


def cache_values(codes, exps):
    """codes uint8 [B, Nk, Hkv, d], exps uint8 [B, Hkv, Nk] -> float64 values."""
    scale = np.where(exps == 255, np.nan, 2.0 ** (exps.astype(np.float64) - 127))
    return e4m3_values()[codes] * scale.transpose(0, 2, 1)[..., None]


def cache_decode_ref(q, k, v, lens, scale, causal=False, softcap=0.0, slopes=None, window=0):
    """q [B, Nq, H, d] against float64 cached values k, v [B, Nk, Hkv, d]."""
    B, nq, H, d = q.shape
    G = H // k.shape[2]
    O, LSE = np.zeros(q.shape), np.zeros((B, H, nq))
    for b in range(B):
        L = int(lens[b])
        away = (L - nq + np.arange(nq))[:, None] - np.arange(L)[None, :]
        see = np.ones(away.shape, bool)
        if causal:
            see &= away >= 0
        if window:
            see &= np.abs(away) < window
        for h in range(H):
            O[b, :, h], LSE[b, h], _ = mod_head_fwd(q[b, :, h], k[b, :L, h // G], v[b, :L, h // G], see, scale, softcap,
                                                    0.0 if slopes is None else slopes[h], np.abs(away))
    return O, LSE
