"""Modified scores over the documented range of their arguments: explicit scales,
slopes of any size, plans that do not hold what they claim, forward-mode
derivatives, schedules of many short sequences, and decoding with each of them.

Helpers and bounds are those of test_modified.py and test_cache.py."""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_95_b200 as fa
from exact_io_aware_95_b200 import build as fabuild
from oracle import modified as om
from tests.common import f64, rel_fro
from tests.test_cache import check_decode, empty_cache, filled, query
from tests.test_modified import FRO, MASKS, U, bf, bounds, cpu_plan, make, plan_of, see_of, slopes_of


@pytest.fixture(scope="module", autouse=True)
def built():
    fabuild.build()


def against(x, mask, see, scale, softcap=0.0, slopes=None, oracle_slopes=None, elements=True, extra=0.0, least=0.0):
    """The kernels under `mask` and `slopes` against the oracle over the pairs `see`
    with `oracle_slopes`: element by element within bounds(), and (where an error
    relative to the whole means something) in the Frobenius norm, with `extra` on its bar.
    `least`: absolute bound of one rounding of a result, where it is more than relative ones."""
    B, N, H, d = x["q"].shape
    g = {n: t.cuda() for n, t in x.items()}
    plan = plan_of(mask, B, N)
    how = {"softcap": softcap, "slopes": None if slopes is None else slopes.cuda(), "scale": scale}
    o, lse, low = fa.mod_fwd(g["q"], g["k"], g["v"], plan, low=True, **how)
    grads = fa.mod_bwd(g["q"], g["k"], g["v"], o, lse, g["do"], plan, o_low=low, **how)
    det = fa.mod_bwd(g["q"], g["k"], g["v"], o, lse, g["do"], plan, o_low=low, deterministic=True, **how)
    fa.check_device_error()
    osl = None if oracle_slopes is None else oracle_slopes.double().numpy()
    a = [f64(x[n]) for n in ("q", "k", "v")]
    want = {}
    want["o"], L = om.mod_attn_fwd(*a, see, scale, softcap, osl)
    want["dq"], want["dk"], want["dv"] = om.mod_attn_bwd(*a, f64(x["do"]), see, scale, softcap, osl)
    tol = bounds(x, see, scale, softcap, osl)
    l64 = lse.double().cpu().numpy()
    assert np.array_equal(np.isneginf(l64), np.isneginf(L)) and not np.isnan(l64).any()
    fin = np.isfinite(L)
    if elements:
        assert np.all(np.abs(l64[fin] - L[fin]) <= tol["lse"][fin])
    got = dict(zip(("o", "dq", "dk", "dv"), (f64(t) for t in (o, *grads))))
    for name, t in [*got.items(), ("dq", f64(det[0])), ("dk", f64(det[1])), ("dv", f64(det[2]))]:
        assert np.isfinite(t).all(), name
        if elements:
            over = np.abs(t - want[name]) - tol[name] - least
            assert over.max() <= 0, (name, over.max())
        if np.linalg.norm(want[name]) > 1e-3 * np.linalg.norm(tol[name]) / U:
            floor = least * math.sqrt(want[name].size) / np.linalg.norm(want[name])  # every element off by `least`
            assert rel_fro(t, want[name]) <= FRO[name] + extra + floor, name


# ------------------------------------------------------------------ scales
@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (0.0, True), (20.0, False), (20.0, True)])
@pytest.mark.parametrize("scale", [0.0, 0.01, 1.0])
@pytest.mark.parametrize("mask", ["causal", "documents", "full"])
def test_explicit_scales(mask, scale, cap, bias, d):
    """scale 0: every visible key has the weight of its bias; N is no multiple of a tile."""
    B, N, H, Hkv = 2, 201, 4, 2
    m, sl = MASKS[mask](B, N), slopes_of(H) if bias else None
    against(make(B, N, H, Hkv, d, 41), m, see_of(m, B, N), scale, cap, sl, sl)


@pytest.mark.gpu
def test_a_scale_below_the_normal_numbers():
    """dQ and dK are of the scale's size, where bf16's step is 2^-133 and fp32's 2^-149:
    two roundings of half a step."""
    m = {"causal": True}
    against(make(1, 140, 2, 1, 64, 42), m, see_of(m, 1, 140), 1e-40, least=2.0 ** -134 + 2.0 ** -150)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("softcap,bias", [(0.0, False), (30.0, True)])
def test_decode_scales(softcap, bias, d):
    """A scale of s 2^k is the default scale s with q 2^k, bit for bit (both are exact
    scalings of the same fp16 operands), and the right side is checked within its
    bounds; so are scale 0 against queries of 0 and -s against -q."""
    c = filled(3, 150, 2, d, 43)
    lens = torch.tensor([150, 64, 3], dtype=torch.int32)
    q = query(3, 2, 8, d, 44)
    sl = torch.tensor([0.5, 0.1, 0.02, 0.0] * 2) if bias else None
    s = 1 / math.sqrt(d)
    for scale, mul in ((0.0, 0.0), (8 * s, 8.0), (s / 16, 1 / 16), (-s, -1.0)):
        want = check_decode(q * mul, c, lens, softcap=softcap, slopes=sl)
        got = fa.cache_decode_fwd(q.cuda(), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], lens.cuda(), causal=True,
                                  scale=scale, softcap=softcap, slopes=None if sl is None else sl.cuda())
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), scale


# ------------------------------------------------------------------ scales out of range
def test_scales_out_of_range_are_refused():
    """What the kernels multiply scores by has to be finite: scale log2(e), and with a
    cap 2 log2(e) times scale / cap and cap."""
    L, P, inv = fa.lib(), 4096, fa.FA_ERR_INVALID_ARG
    f = [P, P, P, P, None, P, P, None]
    b = [P] * 4 + [None] + [P] * 6 + [None, P]
    c = [P] * 7 + [None, None, P]
    ws, wc = L.fa_mod_bwd_workspace_size(1, 8, 2, 1, 64), L.fa_cache_decode_workspace_size(1, 1, 64, 2, 1, 64)
    for scale, cap in ((3e38, 0.0), (float("inf"), 0.0), (float("nan"), 0.0), (2e38, 1.0), (1e30, 2e38)):
        assert L.fa_mod_fwd(*f, 1, 8, 2, 1, 64, scale, cap, None) == inv
        for call in (L.fa_mod_bwd, L.fa_mod_bwd_deterministic):
            assert call(*b, ws, 1, 8, 2, 1, 64, scale, cap, None) == inv
        for x in (scale, -scale):
            assert L.fa_cache_decode_fwd(*c, wc, 1, 1, 64, 2, 1, 64, x, cap, 0, 0, None) == inv


# ------------------------------------------------------------------ slopes
@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mask", ["causal", "full", "prefix", "documents"])
@pytest.mark.parametrize("cap", [0.0, 5.0])
@pytest.mark.parametrize("slope", [300.0, 3e3, 3e4, 1e6, 1e9, 3e38])
def test_slopes_that_leave_one_key(slope, cap, mask, d):
    """Scores here differ by less than 60, so any other key's weight is below e^-240,
    which is 0 in fp32: the row attends to itself alone, with weight 1, and the
    oracle of that is the attention over the diagonal."""
    B, N, H, Hkv = 2, 201, 2, 1
    m = MASKS[mask](B, N)
    see = see_of(m, B, N) & np.eye(N, dtype=bool)
    x = make(B, N, H, Hkv, d, 45)
    q, k = f64(x["q"]), np.repeat(f64(x["k"]), H // Hkv, 2)
    scores = np.einsum("bihc,bjhc->bhij", q, k) / math.sqrt(d)
    assert np.abs(scores).max() < 30
    against(x, m, see, 1 / math.sqrt(d), cap, torch.full((H,), slope))


@pytest.mark.gpu
@pytest.mark.parametrize("mask", ["causal", "full", "prefix", "documents_both"])
@pytest.mark.parametrize("slope", [3.9, 4.1, 20.0])
def test_steep_slopes(slope, mask):
    """On both sides of the size from which the backward pass takes the distance
    element by element; large scores, so that several keys of a row count."""
    B, N, H = 2, 260, 2
    m, sl = MASKS[mask](B, N), torch.tensor([slope, slope / 2])
    against(make(B, N, H, 1, 64, 46, gain=20.0), m, see_of(m, B, N), 1 / 8, 0.0, sl, sl)


@pytest.mark.gpu
@pytest.mark.parametrize("mask", ["causal", "full", "prefix"])
def test_steep_negative_slopes(mask):
    """Far keys win, and the scores reach 260 x 20 = 5200, 7503 in base 2: below 2^13,
    so a rounding of one is off by at most 2^-11, 3.4e-4 of a weight.  The recomputed
    P has four of them (the forward's logsumexp, half of whose last place is 2^-12,
    and its product with log2 e; the bias; the sum), 1.3e-3, and the forward's weights
    two, 7e-4: 2e-3 on the bar.  Elements have no bound of bounds(), which takes
    the bias as positive."""
    B, N, H = 2, 260, 2
    m, sl = MASKS[mask](B, N), torch.tensor([-20.0, -5.0])
    against(make(B, N, H, 1, 64, 47), m, see_of(m, B, N), 1 / 8, 0.0, sl, sl, elements=False, extra=2e-3)


@pytest.mark.gpu
@pytest.mark.parametrize("slope", [3e3, 1e9, 3e38])
def test_decode_slopes_that_leave_one_key(slope):
    """Each query sees its own key alone (see above): O is that key's value."""
    c = filled(3, 150, 1, 64, 48)
    lens = torch.tensor([150, 64, 3], dtype=torch.int32)
    q = query(3, 2, 2, 64, 49)
    for cap in (0.0, 20.0):
        o, lse = fa.cache_decode_fwd(q.cuda(), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], lens.cuda(),
                                     causal=True, softcap=cap, slopes=torch.full((2,), slope).cuda())
        v = fa.cache_read(c["v_cache"], c["v_scale"])
        for b in range(3):
            for i in range(2):
                assert torch.equal(o[b, i], v[b, int(lens[b]) - 2 + i].expand(2, 64)) and torch.isfinite(lse).all()


# ------------------------------------------------------------------ the plan
def test_a_plan_of_other_bytes_is_refused():
    q, k, lse = bf(2, 64, 4, 64), bf(2, 64, 2, 64), torch.zeros(2, 4, 64)
    data = cpu_plan(2, 64).data
    for bad in (data[:-1], data[:0], torch.zeros(1, dtype=torch.uint8), data.to(torch.int32), data.view(2, -1),
                data.repeat_interleave(2)[::2], data.tolist(), None):
        plan = fa.MaskPlan(bad, 2, 64)
        for call in (lambda: fa.mod_fwd(q, k, k, plan), lambda: fa.mod_bwd(q, k, k, q, lse, q, plan),
                     lambda: fa.mod_attention(q, k, k, plan),
                     lambda: fa.mod_attention(q.clone().requires_grad_(True), k, k, plan)):
            with pytest.raises((ValueError, TypeError), match="plan"):
                call()


# ------------------------------------------------------------------ derivatives that it lacks
def test_forward_mode_is_refused(monkeypatch):
    """A dual tensor asks for no gradient in the reverse sense; its tangent must not
    get lost silently."""
    import torch.autograd.forward_ad as fwad
    from exact_io_aware_95_b200 import modified
    monkeypatch.setattr(modified, "mod_fwd", lambda q, k, v, plan, **kw: tuple(q.clone() for _ in range(2 + kw.get("low", False))))
    q, k, plan = bf(1, 8, 2, 64), bf(1, 8, 1, 64), cpu_plan(1, 8)
    with fwad.dual_level():
        for i in range(3):
            args = [q, k, k]
            args[i] = fwad.make_dual(args[i], torch.ones_like(args[i]))
            with pytest.raises(RuntimeError):
                fa.mod_attention(*args, plan)
    assert not fa.mod_attention(q, k, k, plan).requires_grad
    with torch.no_grad():
        assert not fa.mod_attention(q.clone().requires_grad_(True), k, k, plan).requires_grad


def test_what_rounding_lost_is_kept_for_a_backward_only(monkeypatch):
    """mod_attention asks mod_fwd for the residual of O when a gradient may follow."""
    from exact_io_aware_95_b200 import modified
    asked = []

    def fake(q, k, v, plan, **kw):
        asked.append(bool(kw.get("low")))
        return tuple(q.clone() for _ in range(2 + bool(kw.get("low"))))

    monkeypatch.setattr(modified, "mod_fwd", fake)
    q, k, plan = bf(1, 8, 2, 64), bf(1, 8, 1, 64), cpu_plan(1, 8)
    leaf = q.clone().requires_grad_(True)
    fa.mod_attention(q, k, k, plan)
    fa.mod_attention(leaf, k, k, plan)
    fa.mod_attention(q, k, k.clone().requires_grad_(True), plan)
    with torch.no_grad():
        fa.mod_attention(leaf, k, k, plan)
    assert asked == [False, True, True, False]


# ------------------------------------------------------------------ schedules
@pytest.mark.gpu
def test_backward_items_in_groups():
    """More than 4096 items of the backward pass go in groups of heads whose rows fit
    the L2 cache, the last group shorter than the others: the same gradients as in
    calls of one group.  Each dQ row has two terms, so their order does not show."""
    B, N, H, d, part = 300, 130, 7, 64, 50
    group = (48 << 20) // (N * d * 8)
    assert B * H * 2 > 4096 and group < B * H and (B * H) % group and part * H * 2 <= 4096
    g = torch.Generator(device="cuda").manual_seed(50)
    q, k, v, do = (torch.randn(B, N, H, d, generator=g, device="cuda").bfloat16() for _ in range(4))
    how = {"softcap": 20.0, "slopes": slopes_of(H).cuda()}

    def step(x):
        plan = fa.mask_plan(len(x[0]), N, causal=True, device="cuda")
        o, lse, low = fa.mod_fwd(*x[:3], plan, low=True, **how)
        outs = [torch.full_like(t, float("nan")) for t in x[:3]]
        fa.mod_bwd(*x[:3], o, lse, x[3], plan, o_low=low, dq=outs[0], dk=outs[1], dv=outs[2], **how)
        return o, lse, *outs

    whole = step((q, k, v, do))
    for b in range(0, B, part):
        for a, c in zip(step(tuple(t[b:b + part] for t in (q, k, v, do))), whole):
            assert torch.equal(a, c[b:b + part])
    x = {n: t[-2:].cpu() for n, t in zip(("q", "k", "v", "do"), (q, k, v, do))}  # of the last group
    see = see_of({"causal": True}, 2, N)
    tol = bounds(x, see, 1 / 8, 20.0, how["slopes"].double().cpu().numpy())
    want = om.mod_attn_bwd(*(f64(x[n]) for n in ("q", "k", "v", "do")), see, 1 / 8, 20.0, how["slopes"].double().cpu().numpy())
    for n, t, w in zip(("dq", "dk", "dv"), whole[2:], want):
        assert (np.abs(f64(t[-2:]) - w) - tol[n]).max() <= 0, n


# ------------------------------------------------------------------ decoding
@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window", [0, 50])
def test_capped_decode_ignores_rows_no_query_sees(window, d):
    """Rows past the length and before the window hold zeros, or large finite values
    whose scores are far beyond the cap: the same bits."""
    c = filled(3, 333, 2, d, 51)
    lens = torch.tensor([333, 100, 7], dtype=torch.int32)
    for Nq in (1, 5):
        q = query(3, Nq, 4, d, 52)
        outs = []
        for code, exp in ((0x00, 127), (0x7e, 160)):  # 0; 448 2^33
            held = {n: t.clone() for n, t in c.items()}
            for b, L in enumerate(lens.tolist()):
                for part in (slice(L, None), slice(0, max(0, L - Nq + 1 - window) if window else 0)):
                    for n in ("k", "v"):
                        held[n + "_cache"].view(torch.uint8)[b, part] = code
                        held[n + "_scale"][b, :, part] = exp
            outs.append(check_decode(q, held, lens, softcap=30.0, window=window))
        assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


# ------------------------------------------------------------------ cache blocks
@pytest.mark.gpu
@pytest.mark.parametrize("Hkv", [1, 63, 64, 65, 255, 256, 257, 513])
def test_cache_rows_around_a_block(Hkv):
    """Head counts around those where a block's share of rows changes: values that
    e4m3 holds exactly come back as they went in."""
    B, T, d = 2, 3, 64
    g = torch.Generator().manual_seed(53)
    x = torch.randint(-8, 9, (2, B, T, Hkv, d), generator=g) * torch.exp2(torch.randint(-20, 20, (2, B, T, Hkv, 1), generator=g).float())
    x = x.bfloat16().cuda()
    c = empty_cache(B, T + 4, Hkv, d)
    before = {n: t.clone() for n, t in c.items()}
    fa.cache_append(x[0], x[1], c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"],
                    torch.tensor([1, 4], dtype=torch.int32).cuda())
    for i, n in enumerate("kv"):
        out = fa.cache_read(c[n + "_cache"], c[n + "_scale"])
        old = fa.cache_read(before[n + "_cache"], before[n + "_scale"])
        old[0, 1:4], old[1, 4:7] = x[i, 0], x[i, 1]
        assert torch.equal(out, old)
    fa.check_device_error()


# ------------------------------------------------------------------ infinities
@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_scores_under_a_cap(d):
    """tanh(inf) = 1: a capped score of an infinite product is the cap, as it is of one
    far beyond it (e^(2x) is infinite in both); masked ones stay out."""
    cap, m = 2.0, {"causal": True}
    x = make(1, 200, 2, 1, d, 54)
    plan = plan_of(m, 1, 200)
    outs = []
    for big in (float("inf"), 1e30):
        y = {n: t.clone() for n, t in x.items()}
        y["q"][0, 50, 1, 3], y["q"][0, 150, 0, 7] = big, -big
        y["k"][0, 70, 0, 5], y["k"][0, 130, 0, 1] = big, -big
        # every score that meets two of them is a sum of infinities of either sign
        o, lse = fa.mod_fwd(*(y[n].cuda() for n in ("q", "k", "v")), plan, softcap=cap)
        outs.append((f64(o), lse.double().cpu().numpy()))
    O, L = om.mod_attn_fwd(f64(y["q"]), f64(y["k"]), f64(x["v"]), see_of(m, 1, 200), 1 / math.sqrt(d), cap)
    rows = np.ones((1, 200, 2), bool)
    rows[0, 150, 0] = False  # row 150 of head 0 sees both infinite keys, with an infinite query
    fin = rows.transpose(0, 2, 1)
    assert np.array_equal(outs[0][0][rows], outs[1][0][rows]) and np.array_equal(outs[0][1][fin], outs[1][1][fin])
    # weights rounded to bf16 (2 U of the sum of p |v|) and O (U); the products' sums: d 2^-24
    # of scale sum |q k|, which is below 12 where it is finite
    assert (np.abs(outs[0][0] - O)[rows] <= 4 * U * np.abs(f64(x["v"])).max()).all()
    assert (np.abs(outs[0][1] - L)[fin] <= 2.0 ** -13).all()


@pytest.mark.gpu
@pytest.mark.parametrize("bias", [False, True])
def test_an_infinite_query_stays_in_its_row(bias):
    x = make(1, 200, 2, 1, 64, 55)
    sl = slopes_of(2).cuda() if bias else None
    plan = plan_of({"causal": True}, 1, 200)
    want = fa.mod_fwd(*(x[n].cuda() for n in ("q", "k", "v")), plan, slopes=sl)
    x["q"][0, 60, 1, 3] = float("inf")
    o, lse = fa.mod_fwd(*(x[n].cuda() for n in ("q", "k", "v")), plan, slopes=sl)
    assert not torch.isfinite(lse[0, 1, 60])  # +inf where the products have one sign, NaN else
    o[0, 60, 1], lse[0, 1, 60] = want[0][0, 60, 1], want[1][0, 1, 60]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
