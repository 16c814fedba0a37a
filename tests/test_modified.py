"""Attention with modified scores (mask_plan, mod_fwd, mod_bwd, mod_attention).

On the CPU: the oracle against finite differences, loops and the plain oracle,
and every refusal.  On the GPU: parity with the oracle over masks, caps, biases,
grouped heads, odd and tiny lengths, against bounds derived from the kernels'
roundings (see ``bounds``); rows and keys that see nothing; reproducibility;
streams; graph capture; autograd."""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_95_b200 as fa
import oracle
from exact_io_aware_95_b200 import build as fabuild
from oracle import modified as om
from tests.common import f64, rel_fro

U = 2.0 ** -8     # a rounding to bf16 is off by at most this, relative to the value
H16 = 2.0 ** -11  # a rounding to fp16


@pytest.fixture(scope="module", autouse=True)
def built():
    fabuild.build()


# ------------------------------------------------------------------ inputs
def make(B, N, H, Hkv, d, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)
    return {"q": (r(B, N, H, d) * gain).bfloat16(), "k": r(B, N, Hkv, d).bfloat16(), "v": r(B, N, Hkv, d).bfloat16(),
            "do": r(B, N, H, d).bfloat16()}


def slopes_of(H):
    return torch.pow(2.0, -8.0 * torch.arange(1, H + 1, dtype=torch.float32) / H)


def docs_of(B, N, seed, mean):
    """Documents of about `mean` tokens; entry 0 ends in padding, the last entry starts with some."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.cumsum(torch.rand(B, N, generator=g) < 1.0 / mean, 1).int()
    ids[0, N - N // 5:] = -1
    ids[-1, :N // 7] = -3
    return ids


def see_of(mask, B, N):
    return np.stack([om.visible(N, mask.get("causal", False), mask.get("window", 0),
                                None if mask.get("doc_ids") is None else mask["doc_ids"][b].tolist(),
                                int(mask["prefix"][b]) if mask.get("prefix") is not None else 0) for b in range(B)])


def plan_of(mask, B, N):
    m = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in mask.items()}
    return fa.mask_plan(B, N, device="cuda", **m)


# ------------------------------------------------------------------ bounds
def bounds(x, see, scale, softcap, slopes):
    """Element bounds of the kernels' error, from their roundings:

    z     fp32 sum of d products (d 2^-24 of sum |q k|), the cap's tanh (4.5e-7 at most
          absolute) and a few fp32 operations on |z| and the bias
    O     each weight rounded to bf16 (U, numerator and normaliser: 2 U), the
          error of z in both (2 dz), O rounded to bf16 (U)
    D     O with its residual: the weights' 2 U and 2 dz, residual rounded (U^2)
    dV    P rounded (U), P's own dz, dV rounded (U)
    dS    P (1 - t^2) 2^15 rounded to fp16 (2^-11, or half of its smallest step
          2^-24, which is 2^-40 of P's scale, where that is more), the result to
          bf16 (U), dz in P and in 1 - t^2 (its derivative is at most 2 / cap), D
    dQ,dK sums of dS, rounded (U)
    fp32 sums over N terms add N 2^-24 of the absolute sums, inside the slack
    of 2^-16 taken on every absolute sum."""
    q, k, v, do = (f64(x[n]) for n in ("q", "k", "v", "do"))
    B, N, H, d = q.shape
    G = H // k.shape[2]
    out = {n: np.zeros(q.shape) for n in ("o", "dq")}
    out |= {n: np.zeros(k.shape) for n in ("dk", "dv")}
    out["lse"] = np.zeros((B, H, N))
    away = np.abs(np.arange(N)[:, None] - np.arange(N)[None, :])
    for b in range(B):
        for h in range(H):
            sl = 0.0 if slopes is None else float(slopes[h])
            qh, kh, vh, gh = q[b, :, h], k[b, :, h // G], v[b, :, h // G], do[b, :, h]
            mag = abs(scale) * (np.abs(qh) @ np.abs(kh).T)
            dz = d * 2.0 ** -24 * mag + 4.5e-7 * softcap + 2.0 ** -21 * (np.minimum(mag, softcap or np.inf) + sl * away) + 2.0 ** -20
            dz = np.where(see[b], dz, 0.0).max(1, initial=0.0)[:, None]
            O, lse, p = om.mod_head_fwd(qh, kh, vh, see[b], scale, softcap, sl)
            slack = 2.0 ** -16
            o_in = (2 * U + 2 * dz + slack) * (p @ np.abs(vh))
            out["o"][b, :, h] = o_in + U * (np.abs(O) + o_in)
            out["lse"][b, h] = dz[:, 0] + 2.0 ** -21 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0.0)))
            x_ = scale * qh @ kh.T
            f = 1 - np.tanh(x_ / softcap) ** 2 if softcap else np.ones_like(x_)
            dp = gh @ vh.T
            D = (gh * O).sum(1, keepdims=True)
            dD = (np.abs(gh) * (o_in + U * U * np.abs(O))).sum(1, keepdims=True)
            ddp = d * 2.0 ** -23 * (np.abs(gh) @ np.abs(vh).T)
            df = 2 * dz / softcap if softcap else 0.0
            e = p * (f * ((U + H16 + 2 * dz + slack) * np.abs(dp - D) + (1 + 2 * U) * (dD + ddp)) + df * np.abs(dp - D))
            e = e + np.where(see[b], 2.0 ** -40 * (1 + U) * np.abs(dp - D), 0.0)
            ds = np.abs(p * f * (dp - D))
            g = om.mod_head_bwd(qh, kh, vh, gh, see[b], scale, softcap, sl)
            s = abs(scale)
            eq = s * (e + slack * ds) @ np.abs(kh)
            out["dq"][b, :, h] = eq + U * (np.abs(g[0]) + eq) + 1e-30
            ek = s * (e + slack * ds).T @ np.abs(qh)
            out["dk"][b, :, h // G] += ek * (1 + U) + U * np.abs(g[1])
            out["dv"][b, :, h // G] += ((U + 2 * dz + slack) * p).T @ np.abs(gh) * (1 + U) + U * np.abs(g[2])
    return out


# Frobenius bar of a gradient: two roundings to bf16 of at most U each (dS, the
# result) and one to fp16 stand between the inputs and dQ or dK, two for dV.
FRO = {"o": 2 * U, "dq": 2 * U + H16, "dk": 2 * U + H16, "dv": 2 * U}


def check(x, mask, softcap=0.0, slopes=None, low=True):
    B, N, H, d = x["q"].shape
    scale = 1 / math.sqrt(d)
    see = see_of(mask, B, N)
    sl = None if slopes is None else slopes.double().numpy()
    g = {n: t.cuda() for n, t in x.items()}
    plan = plan_of(mask, B, N)
    how = {"softcap": softcap, "slopes": None if slopes is None else slopes.cuda()}
    outs = [torch.full_like(g["q"], float("nan")) for _ in range(2)]
    lse = torch.full((B, H, N), float("nan"), device="cuda")
    r = fa.mod_fwd(g["q"], g["k"], g["v"], plan, out=outs[0], lse=lse, out_low=outs[1] if low else None, **how)
    grads = [torch.full_like(g[n], float("nan")) for n in ("q", "k", "v")]
    fa.mod_bwd(g["q"], g["k"], g["v"], outs[0], lse, g["do"], plan, o_low=outs[1] if low else None, dq=grads[0],
               dk=grads[1], dv=grads[2], **how)
    det = [torch.full_like(g[n], float("nan")) for n in ("q", "k", "v")]
    fa.mod_bwd(g["q"], g["k"], g["v"], outs[0], lse, g["do"], plan, o_low=outs[1] if low else None, dq=det[0],
               dk=det[1], dv=det[2], deterministic=True, **how)
    fa.check_device_error()
    assert len(r) == (3 if low else 2)
    # the fixed-order pass: the same dK and dV, and dQ from the same terms
    assert torch.equal(det[1], grads[1]) and torch.equal(det[2], grads[2])
    if low:
        assert not torch.isnan(det[0]).any()
        again = fa.mod_bwd(g["q"], g["k"], g["v"], outs[0], lse, g["do"], plan, o_low=outs[1], deterministic=True, **how)
        assert all(torch.equal(a, b) for a, b in zip(again, det))
    got = dict(zip(("o", "dq", "dk", "dv"), (f64(t) for t in (outs[0], *grads))))
    a = [f64(x[n]) for n in ("q", "k", "v")]
    want = {}
    want["o"], L = om.mod_attn_fwd(*a, see, scale, softcap, sl)
    want["dq"], want["dk"], want["dv"] = om.mod_attn_bwd(*a, f64(x["do"]), see, scale, softcap, sl)
    tol = bounds(x, see, scale, softcap, sl)
    l64 = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(l64), np.isneginf(L))
    fin = np.isfinite(L)
    assert np.all(np.abs(l64[fin] - L[fin]) <= tol["lse"][fin])
    if low:
        assert (np.abs(f64(det[0]) - want["dq"]) - tol["dq"]).max() <= 0
    for n in want:
        if low or n in ("o", "dv"):
            over = np.abs(got[n] - want[n]) - tol[n]
            assert not np.isnan(got[n]).any() and over.max() <= 0, (n, over.max())
        # a gradient that vanishes (one visible key) has no relative error
        if np.linalg.norm(want[n]) > 1e-3 * np.linalg.norm(tol[n]) / U:
            assert rel_fro(got[n], want[n]) <= FRO[n] * (1 if low else 4), n
    if low:  # O + its residual is O to 16 bits more than bf16 alone, up to the weights' rounding
        both = got["o"] + f64(outs[1])
        assert np.all(np.abs(f64(outs[1])) <= U * np.abs(got["o"]) * (1 + U) + 1e-38)
        assert np.all(np.abs(both - want["o"]) <= tol["o"])
    return outs[0], lse, grads


# -------------------------------------------------------------- CPU: oracle
def test_oracle_gradients_are_the_differences():
    rng = np.random.default_rng(0)
    N, d = 6, 4
    q, k, v, do = (rng.standard_normal((N, d)) for _ in range(4))
    see = om.visible(N, causal=True, doc_ids=[0, 0, 0, 1, 1, 1])
    f = lambda: (om.mod_head_fwd(q, k, v, see, 0.7, 1.3, 0.2)[0] * do).sum()
    for t, g in zip((q, k, v), om.mod_head_bwd(q, k, v, do, see, 0.7, 1.3, 0.2)):
        for i in range(N):
            for c in range(d):
                t0, h = t[i, c], 1e-5
                t[i, c] = t0 + h
                up = f()
                t[i, c] = t0 - h
                down = f()
                t[i, c] = t0
                assert abs((up - down) / (2 * h) - g[i, c]) < 1e-8


def test_oracle_without_modifications_is_the_plain_oracle():
    rng = np.random.default_rng(1)
    q, k, v, do = (rng.standard_normal((1, 9, 2, 8)) for _ in range(4))
    for causal in (False, True):
        see = om.visible(9, causal)[None]
        O, L = om.mod_attn_fwd(q, k, v, see, 0.3)
        O2, L2 = oracle.attn_fwd_ref(q, k, v, 0.3, causal)
        assert np.allclose(O, O2, atol=1e-13) and np.allclose(L, L2, atol=1e-13)
        for a, b in zip(om.mod_attn_bwd(q, k, v, do, see, 0.3), oracle.attn_bwd_ref(q, k, v, do, 0.3, causal)):
            assert np.allclose(a, b, atol=1e-12)


def test_oracle_masks_by_hand():
    see = om.visible(5, causal=True, prefix=3)
    assert see.astype(int).tolist() == [[1, 1, 1, 0, 0], [1, 1, 1, 0, 0], [1, 1, 1, 0, 0], [1, 1, 1, 1, 0], [1] * 5]
    see = om.visible(5, doc_ids=[2, 2, -1, 2, 2], window=2)
    assert see.astype(int).tolist() == [[1, 1, 0, 0, 0], [1, 1, 0, 0, 0], [0] * 5, [0, 0, 0, 1, 1], [0, 0, 0, 1, 1]]


# ------------------------------------------------------------ CPU: refusals
def bf(*s):
    return torch.zeros(*s, dtype=torch.bfloat16)


def cpu_plan(B, N):
    return fa.MaskPlan(torch.zeros(fa.lib().fa_mask_plan_size(B, N), dtype=torch.uint8), B, N)


def test_mod_calls_refuse_bad_arguments():
    q, k, p = bf(2, 64, 4, 64), bf(2, 64, 2, 64), cpu_plan(2, 64)
    lse = torch.zeros(2, 4, 64)
    bad = [((bf(2, 64, 4, 64).float(), k, k, p), TypeError), ((q, bf(2, 64, 3, 64), bf(2, 64, 3, 64), p), ValueError),
           ((q, bf(2, 63, 2, 64), bf(2, 63, 2, 64), p), ValueError), ((q, k, bf(2, 64, 1, 64), p), ValueError),
           ((q, k, k, cpu_plan(2, 65)), ValueError), ((q, k, k, None), TypeError),
           ((q, bf(2, 2, 64, 64).transpose(1, 2), k, p), ValueError), ((q, k, k, p), ValueError)]  # the last: CPU tensors
    for args, err in bad:
        with pytest.raises(err):
            fa.mod_fwd(*args)
        with pytest.raises(err):
            fa.mod_bwd(*args[:3], q, lse, q, args[3])
    for kw in ({"softcap": -1.0}, {"softcap": float("inf")}, {"softcap": float("nan")}, {"slopes": torch.zeros(3)},
               {"slopes": torch.zeros(4, dtype=torch.float64)}, {"slopes": torch.zeros(4, requires_grad=True)}):
        with pytest.raises((ValueError, TypeError)):
            fa.mod_fwd(q, k, k, p, **kw)
        with pytest.raises((ValueError, TypeError)):
            fa.mod_bwd(q, k, k, q, lse, q, p, **kw)
        with pytest.raises((ValueError, TypeError)):
            fa.mod_attention(q, k, k, p, **kw)
    with pytest.raises(ValueError):
        fa.mod_fwd(q, k, k, p, out_low=bf(2, 64, 2, 64))
    with pytest.raises(ValueError):
        fa.mod_bwd(q, k, k, q, lse, q, p, dk=bf(2, 64, 4, 64))
    with pytest.raises(fa.FaError) as e:
        fa.mod_bwd(q, k, k, q, lse, q, p, workspace=torch.zeros(256, dtype=torch.uint8))
    assert e.value.status == fa.FA_ERR_WORKSPACE


def test_mask_plan_refuses_bad_arguments():
    for B, N in ((0, 4), (4, 0), (1, 2**24 + 1)):
        with pytest.raises(ValueError):
            fa.mask_plan(B, N, device="cpu")
    for kw in ({"window": -1}, {"window": 2**31}, {"window": 1.5}, {"doc_ids": torch.zeros(2, 5, dtype=torch.int64)},
               {"doc_ids": torch.zeros(2, 4, dtype=torch.int32)}, {"prefix": torch.zeros(3, dtype=torch.int32)},
               {"prefix": torch.zeros(2, dtype=torch.int32)}):  # the last: right, but on the CPU
        with pytest.raises((ValueError, TypeError)):
            fa.mask_plan(2, 5, **kw)


def test_library_refuses_bad_arguments():
    L, P = fa.lib(), 4096
    inv, uns, wsp = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_WORKSPACE
    need = L.fa_mask_plan_size(2, 300)
    # rows [2, 300] of 8 bytes, query tiles [2, 3] of 32, key tiles [2, 3] of 8, each part in 256-byte units
    assert need == 4864 + 256 + 256
    assert L.fa_mask_plan_size(0, 3) == 0 and L.fa_mask_plan_size(1, 2**24 + 1) == 0
    assert L.fa_mask_plan(P, need - 1, None, None, 2, 300, 0, 0, None) == wsp
    assert L.fa_mask_plan(None, need, None, None, 2, 300, 0, 0, None) == inv
    assert L.fa_mask_plan(P + 16, need, None, None, 2, 300, 0, 0, None) == inv
    assert L.fa_mask_plan(P, need, None, None, 2, 300, -1, 0, None) == inv
    assert L.fa_mask_plan(P, need, P + 2, None, 2, 300, 0, 0, None) == inv
    assert L.fa_mask_plan(P, need, None, None, 2, 300, 0, 2, None) == inv
    assert L.fa_mask_plan(P, 2**40, None, None, 2**10, 2**22, 0, 0, None) == inv
    f = [P, P, P, P, None, P, P, None]  # q k v o o_low lse plan slopes
    at = lambda a, i, x: a[:i] + [x] + a[i + 1:]
    for i in (0, 1, 2, 3, 5, 6):
        assert L.fa_mod_fwd(*at(f, i, None), 1, 8, 2, 1, 64, 1.0, 0.0, None) == inv
    assert L.fa_mod_fwd(*at(f, 4, P + 8), 1, 8, 2, 1, 64, 1.0, 0.0, None) == inv
    assert L.fa_mod_fwd(*at(f, 6, P + 16), 1, 8, 2, 1, 64, 1.0, 0.0, None) == inv
    assert L.fa_mod_fwd(*f, 1, 8, 3, 2, 64, 1.0, 0.0, None) == inv
    assert L.fa_mod_fwd(*f, 1, 8, 2, 1, 96, 1.0, 0.0, None) == uns
    assert L.fa_mod_fwd(*f, 1, 8, 2, 1, 64, float("inf"), 0.0, None) == inv
    assert L.fa_mod_fwd(*f, 1, 8, 2, 1, 64, 1.0, -1.0, None) == inv
    assert L.fa_mod_fwd(*f, 1, 8, 2, 1, 64, 1.0, 1e-40, None) == inv  # scale / softcap is infinite
    assert L.fa_mod_fwd(*f, 1, 8, 2, 1, 64, 1.0, 2e38, None) == inv   # and here subnormal
    assert L.fa_mod_fwd(*f, 1, 8, 2, 1, 64, -1.0, 0.0, None) == inv
    assert L.fa_mod_fwd(*f, 65536, 8, 2, 1, 64, 1.0, 0.0, None) == inv
    ws = L.fa_mod_bwd_workspace_size(1, 8, 2, 1, 64)
    # dQ accumulator, D, and partial dK and dV where the group's heads are split; nothing of them with enough items
    assert ws == 4096 + 256 + 2 * 4096 and L.fa_mod_bwd_workspace_size(1, 8, 3, 2, 64) == 0
    assert L.fa_mod_bwd_workspace_size(8, 8192, 2, 1, 64) == L.fa_bwd_workspace_size(8, 8192, 2, 64)
    b = [P] * 4 + [None] + [P] * 6 + [None, P]  # q k v o o_low lse dO dq dk dv plan slopes workspace
    assert L.fa_mod_bwd(*b, ws - 1, 1, 8, 2, 1, 64, 1.0, 0.0, None) == wsp
    assert L.fa_mod_bwd(*at(b, 12, P + 16), ws, 1, 8, 2, 1, 64, 1.0, 0.0, None) == inv
    for i in (0, 1, 2, 3, 5, 6, 7, 8, 9, 10, 12):
        assert L.fa_mod_bwd(*at(b, i, None), ws, 1, 8, 2, 1, 64, 1.0, 0.0, None) == inv
        assert L.fa_mod_bwd_deterministic(*at(b, i, None), ws, 1, 8, 2, 1, 64, 1.0, 0.0, None) == inv


# --------------------------------------------------------------- GPU: parity
MASKS = {
    "full": lambda B, N: {},
    "causal": lambda B, N: {"causal": True},
    "window": lambda B, N: {"causal": True, "window": max(1, N // 5)},
    "window_both": lambda B, N: {"window": 70},
    "documents": lambda B, N: {"causal": True, "doc_ids": docs_of(B, N, 3, 60)},
    "documents_both": lambda B, N: {"doc_ids": docs_of(B, N, 4, 150)},
    "prefix": lambda B, N: {"causal": True, "prefix": torch.tensor([N // 2, 1][:B], dtype=torch.int32)},
    "all": lambda B, N: {"causal": True, "window": 90, "doc_ids": docs_of(B, N, 5, 100),
                         "prefix": torch.tensor([N // 3, 2 * N][:B], dtype=torch.int32)},
}


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (0.0, True), (20.0, False), (2.0, True)])
@pytest.mark.parametrize("mask", sorted(MASKS))
def test_parity(mask, cap, bias, d):
    B, N, H, Hkv = 2, 333, 4, 2
    check(make(B, N, H, Hkv, d, 7, gain=2.0), MASKS[mask](B, N), cap, slopes_of(H) if bias else None)


@pytest.mark.gpu
@pytest.mark.parametrize("N", [1, 2, 63, 128, 129, 256, 257, 700])
@pytest.mark.parametrize("mask", ["causal", "documents", "prefix"])
def test_lengths(N, mask):
    check(make(2, N, 3, 1, 64, N), MASKS[mask](2, N), 30.0, slopes_of(3))


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hkv", [(1, 1), (6, 6), (6, 3), (8, 1), (14, 2)])
def test_heads(H, Hkv):
    check(make(2, 200, H, Hkv, 128, 11), {"causal": True}, 50.0, slopes_of(H))


@pytest.mark.gpu
@pytest.mark.parametrize("B,N,H,Hkv", [(8, 400, 16, 8), (1, 1300, 16, 4), (2, 140, 12, 1)])
def test_groups_whole_and_split(B, N, H, Hkv):
    """A group's heads in one item, in two or four, and each in its own."""
    ws = fa.mod_bwd_workspace_size(B, N, H, Hkv, 64)
    plain = fa.workspace_size(B, N, H, 64)
    assert (ws == plain) == ((B, H) == (8, 16))
    check(make(B, N, H, Hkv, 64, 19), {"causal": True}, 30.0, slopes_of(H))


@pytest.mark.gpu
@pytest.mark.parametrize("gain,cap", [(8.0, 0.0), (30.0, 5.0), (40.0, 50.0)])
def test_scores_far_beyond_the_cap_and_peaked_rows(gain, cap):
    check(make(1, 300, 2, 2, 128, 12, gain=gain), {"causal": True}, cap)


@pytest.mark.gpu
def test_without_the_residual():
    check(make(2, 150, 2, 1, 64, 13), {"causal": True}, 30.0, low=False)


@pytest.mark.gpu
def test_negative_and_large_slopes():
    check(make(1, 300, 3, 1, 64, 14), {"causal": True, "prefix": torch.tensor([200], dtype=torch.int32)}, 0.0,
          torch.tensor([-0.05, 3.0, 0.0]))


@pytest.mark.gpu
def test_everything_masked():
    x = make(1, 260, 2, 1, 64, 15)
    o, lse, grads = check(x, {"doc_ids": torch.full((1, 260), -1, dtype=torch.int32)}, 30.0, slopes_of(2))
    assert (o == 0).all() and torch.isneginf(lse).all() and all((t == 0).all() for t in grads)


@pytest.mark.gpu
def test_gaps_between_tiles():
    """Whole 128-row tiles of padding between documents: query tiles without keys
    next to tiles with, key tiles no query sees."""
    N = 1100
    ids = torch.full((1, N), -1, dtype=torch.int32)
    ids[:, 5:140] = 1
    ids[:, 530:600] = 2
    ids[:, 1000:1090] = 2
    check(make(1, N, 2, 1, 64, 16), {"doc_ids": ids})
    check(make(1, N, 2, 1, 128, 17), {"doc_ids": ids, "causal": True}, 30.0, slopes_of(2))


@pytest.mark.gpu
def test_gradients_against_differences():
    """A directional derivative of sum(dO O) through the kernels' forward pass
    (both sides in the kernels' arithmetic; see the bound)."""
    x = make(1, 160, 2, 1, 64, 18)
    plan = fa.mask_plan(1, 160, causal=True, device="cuda")
    sl = slopes_of(2).cuda()
    g = {n: t.cuda() for n, t in x.items()}
    o, lse, low = fa.mod_fwd(g["q"], g["k"], g["v"], plan, softcap=5.0, slopes=sl, low=True)
    grads = fa.mod_bwd(g["q"], g["k"], g["v"], o, lse, g["do"], plan, softcap=5.0, slopes=sl, o_low=low)
    do = g["do"].double()
    for n, gr in zip(("q", "k", "v"), grads):
        h = 2.0 ** -3
        dirn = torch.sign(gr.float())  # every element adds to the sum
        vals = []
        for s in (1, -1):
            y = dict(g)
            y[n] = (g[n].float() + s * h * dirn).bfloat16()
            step = (y[n].double() - g[n].double())
            oo, _, ll = fa.mod_fwd(y["q"], y["k"], y["v"], plan, softcap=5.0, slopes=sl, low=True)
            vals.append((((oo.double() + ll.double()) * do).sum(), (gr.double() * step).sum()))
        got, want = vals[0][0] - vals[1][0], vals[0][1] - vals[1][1]
        # third-order term of a step of 1/8 in unit-size inputs plus 3 U: a few per cent
        assert abs(got - want) <= 0.05 * abs(want), n


# ------------------------------------------------------------ GPU: behaviour
@pytest.mark.gpu
def test_no_modification_agrees_with_the_plain_forward_and_backward():
    x = {n: t.cuda() for n, t in make(2, 400, 3, 3, 128, 20).items()}
    plan = fa.mask_plan(2, 400, causal=True, device="cuda")
    o, lse = fa.mod_fwd(x["q"], x["k"], x["v"], plan)
    o2, lse2 = fa.fwd(x["q"], x["k"], x["v"], causal=True)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g = fa.mod_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], plan)
    g2 = fa.bwd(x["q"], x["k"], x["v"], o, lse, x["do"], causal=True)
    for a, b in zip(g, g2):
        assert rel_fro(f64(a), f64(b)) <= U


@pytest.mark.gpu
def test_documents_equal_the_packed_call():
    lens = [70, 1, 200, 129]
    N = sum(lens)
    x = {n: t.cuda() for n, t in make(1, N, 2, 2, 64, 21).items()}
    ids = torch.repeat_interleave(torch.arange(4), torch.tensor(lens)).int()[None].cuda()
    plan = fa.mask_plan(1, N, causal=True, doc_ids=ids)
    o, lse = fa.mod_fwd(x["q"], x["k"], x["v"], plan)
    cu = torch.tensor([0, 70, 71, 271, 400], dtype=torch.int32, device="cuda")
    o2, lse2 = fa.varlen_fwd(x["q"][0], x["k"][0], x["v"][0], cu, 200, causal=True)
    assert (o[0].float() - o2.float()).abs().max() <= 2 * U * o2.float().abs().max()
    assert (lse[0] - lse2).abs().max() <= 1e-5


@pytest.mark.gpu
def test_dk_dv_are_reproducible_and_plan_is_reused():
    x = {n: t.cuda() for n, t in make(2, 500, 4, 1, 128, 22).items()}
    plan = fa.mask_plan(2, 500, causal=True, window=100, device="cuda")
    runs = []
    for _ in range(3):
        o, lse, low = fa.mod_fwd(x["q"], x["k"], x["v"], plan, softcap=20.0, low=True)
        runs.append((o, lse, low, *fa.mod_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], plan, softcap=20.0, o_low=low)[1:]))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))


@pytest.mark.gpu
def test_nan_row_stays_in_its_row():
    x = make(1, 200, 2, 1, 64, 23)
    x["q"][0, 50, 1] = float("nan")
    plan = fa.mask_plan(1, 200, causal=True, device="cuda")
    for cap in (0.0, 30.0):
        o, lse = fa.mod_fwd(*(x[n].cuda() for n in ("q", "k", "v")), plan, softcap=cap)
        assert torch.isnan(o[0, 50, 1]).all() and torch.isnan(lse[0, 1, 50])
        o[0, 50, 1] = 0
        lse[0, 1, 50] = 0
        assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
def test_another_stream_and_a_captured_step():
    x = {n: t.cuda() for n, t in make(2, 300, 4, 2, 64, 24).items()}
    ids = docs_of(2, 300, 6, 80).cuda()
    sl = slopes_of(4).cuda()

    def step():
        plan = fa.mask_plan(2, 300, causal=True, doc_ids=ids)
        o, lse, low = fa.mod_fwd(x["q"], x["k"], x["v"], plan, softcap=30.0, slopes=sl, low=True)
        return (o, lse) + fa.mod_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], plan, softcap=30.0, slopes=sl, o_low=low)

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    x["q"].mul_(0.5)
    want2 = step()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in ((other, want), (held, want2)):
        for i in (0, 1, 3, 4):
            assert torch.equal(a[i], b[i])
        assert rel_fro(f64(a[2]), f64(b[2])) <= U


@pytest.mark.gpu
def test_autograd():
    x = make(2, 210, 4, 2, 64, 25)
    q, k, v = (x[n].cuda().requires_grad_(True) for n in ("q", "k", "v"))
    sl = slopes_of(4).cuda()
    plan = fa.mask_plan(2, 210, causal=True, device="cuda")
    o = fa.mod_attention(q, k, v, plan, softcap=30.0, slopes=sl)
    o.transpose(1, 2).backward(x["do"].cuda().transpose(1, 2))  # a gradient that is not contiguous
    with torch.no_grad():
        o1, lse, low = fa.mod_fwd(q, k, v, plan, softcap=30.0, slopes=sl, low=True)
        g = fa.mod_bwd(q, k, v, o1, lse, x["do"].cuda(), plan, softcap=30.0, slopes=sl, o_low=low)
        assert torch.equal(fa.mod_attention(q, k, v, plan, softcap=30.0, slopes=sl), o)
    assert torch.equal(o, o1)
    assert torch.equal(k.grad, g[1]) and torch.equal(v.grad, g[2]) and rel_fro(f64(q.grad), f64(g[0])) <= U


@pytest.mark.gpu
def test_deterministic_gradients():
    # many key tiles add into each dQ row, so an order that varied would show
    x = make(2, 1500, 8, 2, 64, 31)
    q, k, v = (x[n].cuda().requires_grad_(True) for n in ("q", "k", "v"))
    do, sl = x["do"].cuda(), slopes_of(8).cuda()
    ids = docs_of(2, 1500, 9, 900).cuda()

    def step():
        plan = fa.mask_plan(2, 1500, doc_ids=ids)
        o = fa.mod_attention(q, k, v, plan, softcap=20.0, slopes=sl, deterministic=True)
        return torch.autograd.grad(o, (q, k, v), do)

    want = step()
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(step(), want))
    with torch.no_grad():
        plan = fa.mask_plan(2, 1500, doc_ids=ids)
        o, lse, low = fa.mod_fwd(q, k, v, plan, softcap=20.0, slopes=sl, low=True)

        def back():
            return fa.mod_bwd(q, k, v, o, lse, do, plan, softcap=20.0, slopes=sl, o_low=low, deterministic=True)

        assert all(torch.equal(a, b) for a, b in zip(back(), want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = back()
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))


@pytest.mark.gpu
def test_autograd_refuses_a_second_derivative():
    x = make(1, 40, 2, 1, 64, 27)
    q, k, v = (x[n].cuda().requires_grad_(True) for n in ("q", "k", "v"))
    o = fa.mod_attention(q, k, v, fa.mask_plan(1, 40, device="cuda"))
    (g,) = torch.autograd.grad(o, q, x["do"].cuda(), create_graph=True)
    with pytest.raises(RuntimeError):
        g.float().sum().backward()


@pytest.mark.gpu
def test_two_calls_at_once_and_from_a_new_host_thread():
    import threading
    x = {n: t.cuda() for n, t in make(2, 500, 4, 2, 64, 28).items()}
    plan = fa.mask_plan(2, 500, causal=True, device="cuda")

    def step():
        o, lse, low = fa.mod_fwd(x["q"], x["k"], x["v"], plan, softcap=20.0, low=True)
        return (o, lse) + fa.mod_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], plan, softcap=20.0, o_low=low)

    want = step()
    torch.cuda.synchronize()
    got = {}

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(4):
                got[i] = step()
            torch.cuda.current_stream().synchronize()

    ts = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert len(got) == 3
    for g in got.values():
        assert all(torch.equal(g[i], want[i]) for i in (0, 1, 3, 4)) and rel_fro(f64(g[2]), f64(want[2])) <= U


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """Tensors of more than 2^31 elements: the last rows of a windowed batch
    against the oracle on those rows alone."""
    N, H, Hkv, d, W, S = 140000, 128, 2, 128, 50, 300
    assert N * H * d > 2**31
    g = torch.Generator(device="cuda").manual_seed(29)
    rand = lambda h: torch.randn(1, N, h, d, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k, v, do = rand(H), rand(Hkv), rand(Hkv), rand(H)
    plan = fa.mask_plan(1, N, causal=True, window=W, device="cuda")
    o, lse, low = fa.mod_fwd(q, k, v, plan, softcap=30.0, low=True)
    dq, dk, dv = fa.mod_bwd(q, k, v, o, lse, do, plan, softcap=30.0, o_low=low)
    fa.check_device_error()
    x = {"q": q[:, -S:, -64:], "k": k[:, -S:, 1:], "v": v[:, -S:, 1:], "do": do[:, -S:, -64:]}  # the last key head's group
    x = {n: t.cpu() for n, t in x.items()}
    see = see_of({"causal": True, "window": W}, 1, S)
    want = dict(zip(("dq", "dk", "dv"), om.mod_attn_bwd(*(f64(x[n]) for n in ("q", "k", "v", "do")), see, 1 / math.sqrt(d), 30.0)))
    want["o"], _ = om.mod_attn_fwd(*(f64(x[n]) for n in ("q", "k", "v")), see, 1 / math.sqrt(d), 30.0)
    tol = bounds(x, see, 1 / math.sqrt(d), 30.0, None)
    got = {"o": o[:, -S:, -64:], "dq": dq[:, -S:, -64:], "dk": dk[:, -S:, 1:], "dv": dv[:, -S:, 1:]}
    for n, t in got.items():  # rows whose whole window lies in the slice
        e = np.abs(f64(t) - want[n])[:, W:] - tol[n][:, W:]
        assert e.max() <= 0, (n, e.max())


@pytest.mark.gpu
def test_plan_of_a_long_batch():
    """Documents that begin and end in other blocks of rows than theirs, one of
    them over two whole blocks and more, against the definition row by row."""
    N = 10300
    g = torch.Generator().manual_seed(26)
    ids = torch.cumsum(torch.rand(2, N, generator=g) < 0.01, 1).int()
    ids[1, 1500:9000] = 7
    ids[0, 4000:4100] = -1
    ids[0, 10250:] = -2
    plan = fa.mask_plan(2, N, causal=True, window=300, doc_ids=ids.cuda(), prefix=torch.tensor([0, 3000], dtype=torch.int32).cuda())
    rows = plan.data[:2 * N * 8].view(torch.int32).view(2, N, 2).cpu()
    for b in range(2):
        a = ids[b].tolist()
        first, last = [0] * N, [N] * N
        for i in range(1, N):
            first[i] = first[i - 1] if a[i] == a[i - 1] else i
        for i in range(N - 2, -1, -1):
            last[i] = last[i + 1] if a[i] == a[i + 1] else i + 1
        for i in range(N):
            lo, hi = max(first[i], i - 299), min(last[i], max(i + 1, [0, 3000][b]), i + 300)
            want = (0, 0) if a[i] < 0 or lo >= hi else (lo, hi)
            assert tuple(rows[b, i].tolist()) == want, (b, i)
