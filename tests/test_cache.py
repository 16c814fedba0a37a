"""The 8-bit key/value cache (cache_append, cache_read) and the decoding that
reads it (cache_decode_fwd).

On the CPU: the oracle's number format and quantiser, every refusal.  On the
GPU: append bit for bit against the oracle, reading back exactly, rows outside
left as they were, decoding against the oracle within bounds derived from the
kernel's roundings, the whole path together with the modified-score attention
of the same sequence, bad lengths, streams and graph capture."""
import math

import numpy as np
import pytest
import torch

import exact_io_aware_95_b200 as fa
from exact_io_aware_95_b200 import build as fabuild
from oracle import modified as om
from tests.common import f64

U = 2.0 ** -8    # rounding to bf16
H16 = 2.0 ** -11  # rounding to fp16


@pytest.fixture(scope="module", autouse=True)
def built():
    fabuild.build()


def empty_cache(B, Nk, Hkv, d, device="cuda", fill=0x55):
    """Caches full of a recognisable pattern."""
    return {n: torch.full((B, Nk, Hkv, d), fill, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
            for n in ("k_cache", "v_cache")} | \
           {n: torch.full((B, Hkv, Nk), 0x77, dtype=torch.uint8, device=device) for n in ("k_scale", "v_scale")}


def rows(B, T, Hkv, d, seed, spread=3.0):
    """Rows whose sizes differ by powers of two, with some special values."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, T, Hkv, d, generator=g) * torch.exp2(spread * torch.randn(B, T, Hkv, 1, generator=g))
    return x.bfloat16()


def np8(t):
    return t.view(torch.uint8).cpu().numpy()


# --------------------------------------------------------------- CPU: oracle
def test_format_is_torch_s():
    all_codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    mine = om.e4m3_values()
    assert np.array_equal(np.isnan(all_codes), np.isnan(mine))
    assert np.array_equal(all_codes[~np.isnan(mine)], mine[~np.isnan(mine)])


def test_oracle_quantiser():
    for amax, e in ((448.0, 127), (449.0, 128), (224.0, 126), (1.75, 119), (1.7501, 120), (2.0 ** -140, 1), (0.0, 127)):
        assert om.quantise_row([amax, 0.0])[1] == e
    g = torch.Generator().manual_seed(0)
    x = torch.randn(64, generator=g)
    codes, e = om.quantise_row(x.numpy())
    assert np.array_equal(codes, np8((x * 2.0 ** (127 - e)).to(torch.float8_e4m3fn)))
    assert om.quantise_row([np.inf, -np.inf, np.nan, 1.0])[0][:3].tolist() == [0x7e, 0xfe, 0x7f]


# ------------------------------------------------------------- CPU: refusals
def test_cache_calls_refuse_bad_arguments():
    B, T, Nk, H, Hkv, d = 2, 3, 20, 4, 2, 64
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    c = empty_cache(B, Nk, Hkv, d, "cpu")
    kv, st = bf(B, T, Hkv, d), torch.zeros(B, dtype=torch.int32)
    ok = [kv, kv, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], st, st]
    other = empty_cache(B, Nk - 1, Hkv, d, "cpu")
    for i, bad in ((0, kv.float()), (1, bf(B, T, Hkv, d // 2)), (1, bf(B, T + 1, Hkv, d)), (2, other["k_cache"]),
                   (3, other["v_cache"]), (2, c["k_cache"].view(torch.uint8)), (4, other["k_scale"]),
                   (5, c["v_scale"].float()), (6, st.long()), (6, st[:1]), (7, st[:1]),
                   (4, c["k_scale"].transpose(1, 2).contiguous().transpose(1, 2)), (0, kv)):  # the last: CPU tensors
        with pytest.raises((ValueError, TypeError)):
            fa.cache_append(*ok[:i], bad, *ok[i + 1:])
    for args in ((other["k_cache"], c["k_scale"]), (c["k_cache"], c["k_scale"], st[:1]),
                 (c["k_cache"], c["k_scale"], None, bf(B, Nk, Hkv, d // 2)), (c["k_cache"], c["k_scale"])):
        with pytest.raises((ValueError, TypeError)):
            fa.cache_read(*args)
    q = bf(B, 1, H, d)
    ok = [q, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], st]
    for i, bad in ((0, bf(B, 1, 3, d)), (0, bf(B + 1, 1, H, d)), (0, bf(B, 1, H, 128)), (2, other["v_cache"]),
                   (4, other["v_scale"]), (5, st[:1]), (5, st.long()), (0, q)):
        with pytest.raises((ValueError, TypeError)):
            fa.cache_decode_fwd(*ok[:i], bad, *ok[i + 1:])
    for kw in ({"softcap": -1.0}, {"window": -1}, {"window": 2**31}, {"slopes": torch.zeros(3)},
               {"slopes": torch.zeros(4, requires_grad=True)}, {"out": bf(B, 2, H, d)}, {"lse": torch.zeros(B, 1, H)}):
        with pytest.raises((ValueError, TypeError)):
            fa.cache_decode_fwd(*ok, **kw)
    with pytest.raises(fa.FaError) as e:
        fa.cache_decode_fwd(*ok, workspace=torch.zeros(16, dtype=torch.uint8))
    assert e.value.status == fa.FA_ERR_WORKSPACE


def test_library_refuses_bad_arguments():
    L, P = fa.lib(), 4096
    inv, uns, wsp = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_WORKSPACE
    at = lambda a, i, x: a[:i] + [x] + a[i + 1:]
    a = [P] * 8  # k v k_cache v_cache k_scale v_scale start count; then B T Nk Hkv d
    for i in range(7):
        assert L.fa_cache_append(*at(a, i, None), 1, 2, 8, 1, 64, None) == inv
    assert L.fa_cache_append(*at(a, 2, P + 8), 1, 2, 8, 1, 64, None) == inv
    assert L.fa_cache_append(*at(a, 6, P + 2), 1, 2, 8, 1, 64, None) == inv
    assert L.fa_cache_append(*a, 1, 9, 8, 1, 64, None) == inv        # T > Nk
    assert L.fa_cache_append(*a, 1, 0, 8, 1, 64, None) == inv
    assert L.fa_cache_append(*a, 65536, 2, 8, 1, 64, None) == inv
    assert L.fa_cache_append(*a, 1, 2, 2**30, 2, 64, None) == inv
    assert L.fa_cache_append(*a, 1, 2, 8, 1, 96, None) == uns
    r = [P, P, P, P]  # cache scale seqlens out
    for i in (0, 1, 3):
        assert L.fa_cache_read(*at(r, i, None), 1, 8, 1, 64, None) == inv
    assert L.fa_cache_read(*at(r, 3, P + 8), 1, 8, 1, 64, None) == inv
    assert L.fa_cache_read(*r, 1, 8, 1, 32, None) == uns
    ws = L.fa_cache_decode_workspace_size(1, 1, 64, 2, 1, 64)
    assert ws > 0 and L.fa_cache_decode_workspace_size(1, 17, 64, 2, 1, 64) == 0
    assert L.fa_cache_decode_workspace_size(1, 1, 64, 3, 2, 64) == 0
    assert ws == L.fa_cache_decode_workspace_size(1, 16, 4096, 8, 1, 64)
    d = [P] * 7 + [None, None, P]  # q kc vc ks vs o lse seqlens slopes ws; ws_bytes B Nq Nk H Hkv d scale cap window causal
    tail = [1, 1, 64, 2, 1, 64, 1.0, 0.0, 0, 0, None]
    for i in range(7):
        assert L.fa_cache_decode_fwd(*at(d, i, None), ws, *tail) == inv
    assert L.fa_cache_decode_fwd(*at(d, 9, None), ws, *tail) == wsp
    assert L.fa_cache_decode_fwd(*d, ws - 1, *tail) == wsp
    assert L.fa_cache_decode_fwd(*at(d, 9, P + 16), ws, *tail) == inv
    for i, x, want in ((1, 17, uns), (1, 0, inv), (3, 3, None), (4, 4, inv), (5, 96, uns), (6, float("nan"), inv),
                       (7, -1.0, inv), (7, 1e-40, inv), (8, -1, inv), (9, 2, inv), (0, 65536, inv)):
        if want is not None:
            assert L.fa_cache_decode_fwd(*d, ws, *at(tail, i, x)) == want, (i, x)


# --------------------------------------------------------- GPU: append, read
@pytest.mark.gpu
@pytest.mark.parametrize("B,T,Nk,Hkv,d", [(1, 1, 1, 1, 64), (2, 3, 50, 2, 128), (3, 41, 77, 3, 64), (2, 70, 70, 1, 128),
                                          (1, 5, 9, 100, 64), (2, 2, 3, 600, 64)])
def test_append_matches_the_oracle_and_touches_nothing_else(B, T, Nk, Hkv, d):
    k, v = rows(B, T, Hkv, d, 1), rows(B, T, Hkv, d, 2)
    k[0, 0, 0] = 0.0                       # a row of zeros
    v[0, 0, 0, :4] = torch.tensor([float("inf"), -float("inf"), float("nan"), 3.0])
    v[-1, -1, -1] = float("inf")           # no finite value
    k[-1, -1, -1] = 2.0 ** -133            # bf16's smallest subnormal: e = 1
    k[0, -1, 0, 0] = 3.38e38               # its largest value
    c = empty_cache(B, Nk, Hkv, d)
    before = {n: t.view(torch.uint8).cpu().numpy().copy() for n, t in c.items()}
    start = torch.tensor([(7 * b) % (Nk - T + 1) for b in range(B)], dtype=torch.int32)
    count = torch.tensor([max(0, T - 5 * b) for b in range(B)], dtype=torch.int32)
    fa.cache_append(k.cuda(), v.cuda(), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], start.cuda(), count.cuda())
    fa.check_device_error()
    for n, x in (("k", k), ("v", v)):
        codes, exps = before[n + "_cache"], before[n + "_scale"]
        for b in range(B):
            for t in range(int(count[b])):
                for h in range(Hkv):
                    codes[b, start[b] + t, h], exps[b, h, start[b] + t] = om.quantise_row(x[b, t, h].double().numpy())
        got = np8(c[n + "_cache"])
        nan = (codes & 0x7f) == 0x7f  # either sign of NaN
        assert np.array_equal(nan, (got & 0x7f) == 0x7f) and np.array_equal(got[~nan], codes[~nan])
        assert np.array_equal(c[n + "_scale"].cpu().numpy(), exps)
        # read back: exact, zero behind the length
        lens = torch.tensor([min(Nk, int(start[b]) + int(count[b])) for b in range(B)], dtype=torch.int32)
        out = torch.full((B, Nk, Hkv, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        fa.cache_read(c[n + "_cache"], c[n + "_scale"], lens.cuda(), out=out)
        want = om.cache_values(codes, exps)
        for b in range(B):
            want[b, lens[b]:] = 0.0
        assert np.array_equal(f64(out), want, equal_nan=True)
        assert np.array_equal(f64(fa.cache_read(c[n + "_cache"], c[n + "_scale"])), om.cache_values(codes, exps), equal_nan=True)


@pytest.mark.gpu
def test_read_decodes_every_code_and_exponent():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(1, 4, 1, 64).repeat(1, 64, 1, 1).contiguous()
    exps = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(1, 1, 256).contiguous()
    out = fa.cache_read(codes.view(torch.float8_e4m3fn).cuda(), exps.cuda())
    with np.errstate(over="ignore", invalid="ignore"):
        want = torch.from_numpy(om.cache_values(codes.numpy(), exps.numpy())).float().bfloat16()
    assert torch.equal(torch.nan_to_num(out.cpu(), nan=7.0), torch.nan_to_num(want, nan=7.0))


@pytest.mark.gpu
def test_rows_that_do_not_fit_are_reported_and_left_out():
    B, T, Nk, Hkv, d = 6, 4, 10, 2, 64
    k = rows(B, T, Hkv, d, 3).cuda()
    start = torch.tensor([6, 7, -1, 0, 0, 2**31 - 2], dtype=torch.int32).cuda()
    count = torch.tensor([4, 4, 4, 5, -1, 4], dtype=torch.int32).cuda()
    c = empty_cache(B, Nk, Hkv, d)
    fa.cache_append(k, k, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], start, count)
    with pytest.raises(fa.FaError) as e:
        fa.check_device_error()
    assert e.value.status == fa.FA_ERR_INVALID_ARG
    fa.check_device_error()
    assert (np8(c["k_cache"])[1:] == 0x55).all() and (c["v_scale"][1:] == 0x77).all()
    assert (c["k_scale"][0, :, 6:] != 0x77).any() and (np8(c["k_cache"])[0, :6] == 0x55).all()
    out = torch.full((B, Nk, Hkv, d), 3.0, dtype=torch.bfloat16, device="cuda")
    fa.cache_read(c["k_cache"], c["k_scale"], torch.tensor([0, 11, -1, 10, 0, 0], dtype=torch.int32).cuda(), out=out)
    with pytest.raises(fa.FaError):
        fa.check_device_error()
    assert (out[1:3] == 3.0).all() and (out[0] == 0).all()


# ------------------------------------------------------------------ decoding
def filled(B, Nk, Hkv, d, seed, spread=1.0):
    c = empty_cache(B, Nk, Hkv, d)
    z = torch.zeros(B, dtype=torch.int32, device="cuda")
    fa.cache_append(rows(B, Nk, Hkv, d, seed, 0.3).cuda(), rows(B, Nk, Hkv, d, seed + 1, spread).cuda(), c["k_cache"],
                    c["v_cache"], c["k_scale"], c["v_scale"], z)
    return c


def values(c):
    return (om.cache_values(np8(c["k_cache"]), c["k_scale"].cpu().numpy()),
            om.cache_values(np8(c["v_cache"]), c["v_scale"].cpu().numpy()))


def check_decode(q, c, lens, causal=True, softcap=0.0, slopes=None, window=0):
    """Bounds: z is an fp32 sum of d exact products of fp16 numbers (q itself
    loses 2^-40 of its row's maximum), scaled, capped (a few fp32 operations:
    2^-21 of |z|) and biased; the weights are rounded to fp16, the sums kept in
    fp32, the output rounded to bf16."""
    B, Nq, H, d = q.shape
    scale = 1 / math.sqrt(d)
    k, v = values(c)
    for b in range(B):  # what no query may use
        k[b, int(lens[b]):] = 0.0
        v[b, int(lens[b]):] = 0.0
    sl = None if slopes is None else slopes.double().numpy()
    out = torch.full(q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H, Nq), float("nan"), device="cuda")
    fa.cache_decode_fwd(q.cuda(), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], lens.cuda(), causal=causal,
                        softcap=softcap, slopes=None if slopes is None else slopes.cuda(), window=window, out=out, lse=lse)
    fa.check_device_error()
    O, L = om.cache_decode_ref(f64(q), k, v, lens, scale, causal, softcap, sl, window)
    A, _ = om.cache_decode_ref(f64(q), k, np.abs(v), lens, scale, causal, softcap, sl, window)  # sum p |v|
    l64, o64 = lse.double().cpu().numpy(), f64(out)
    assert np.array_equal(np.isneginf(l64), np.isneginf(L)) and not np.isnan(l64).any()
    G = H // k.shape[2]
    away = float(max(1, int(lens.max())))
    dz = np.zeros((B, H, Nq))
    for b in range(B):
        for h in range(H):
            mag = np.abs(f64(q)[b, :, h]) @ np.abs(k[b, :max(1, int(lens[b])), h // G]).T * scale
            if window:  # keys far away do not count
                near = np.abs((int(lens[b]) - Nq + np.arange(Nq))[:, None] - np.arange(mag.shape[1])[None]) < window
                mag = np.where(near, mag, 0.0)
            m = mag.max(1)
            dz[b, h] = (d + 8) * 2.0 ** -24 * m + 2.0 ** -21 * (np.minimum(m, softcap or np.inf) + (0 if sl is None else abs(sl[h])) * away) + 2.0 ** -20
    fin = np.isfinite(L)
    assert np.all(np.abs(l64[fin] - L[fin]) <= (dz + 2.0 ** -21 * (1 + np.abs(np.where(fin, L, 0.0))))[fin])
    tol = (2 * dz.transpose(0, 2, 1)[..., None] + H16 + 2.0 ** -16) * A
    tol = tol + U * (np.abs(O) + tol)
    over = np.abs(o64 - O) - tol
    assert not np.isnan(o64).any() and over.max() <= 0, over.max()
    return out, lse


def query(B, Nq, H, d, seed, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(B, Nq, H, d, generator=g) * gain).bfloat16()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Nq,H,Hkv", [(1, 3, 3), (1, 8, 2), (3, 4, 2), (16, 2, 2), (5, 14, 2), (16, 6, 1)])
def test_decode_ragged(Nq, H, Hkv, d):
    lens = torch.tensor([700, 0, 1, 2, 64, 65, 513, 15], dtype=torch.int32)
    c = filled(8, 700, Hkv, d, 10)
    for causal in (True, False):
        check_decode(query(8, Nq, H, d, 11, 2.0), c, lens, causal)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap,bias,window,causal", [(20.0, False, 0, True), (2.0, True, 0, True), (0.0, True, 100, True),
                                                    (30.0, True, 7, False), (0.0, False, 1, True), (0.0, False, 64, True),
                                                    (0.0, False, 10**6, True), (0.0, False, 2**31 - 1, False)])
def test_decode_modifications(cap, bias, window, causal, d):
    lens = torch.tensor([400, 64, 3, 257], dtype=torch.int32)
    check_decode(query(4, 2, 4, d, 12, 3.0), filled(4, 401, 2, d, 13), lens, causal, cap,
                 torch.tensor([0.5, 0.01, 0.0, -0.02]) if bias else None, window)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Nk,Hkv,G", [(1, 20000, 1, 4), (2, 5000, 4, 1), (64, 130, 4, 2), (300, 40, 1, 1)])
def test_decode_splits(B, Nk, Hkv, G):
    g = torch.Generator().manual_seed(14)
    lens = torch.randint(0, Nk + 1, (B,), generator=g, dtype=torch.int32)
    lens[0] = Nk
    check_decode(query(B, 1, Hkv * G, 64, 15), filled(B, Nk, Hkv, 64, 16), lens)


@pytest.mark.gpu
@pytest.mark.parametrize("B,Hkv,Nq", [(1, 600, 1), (3, 500, 3), (1, 149, 9)])
def test_decode_many_key_heads(B, Hkv, Nq):
    """More key heads than a wave of thread blocks, and counts that leave part of one unused."""
    check_decode(query(B, Nq, Hkv, 64, 31), filled(B, 90, Hkv, 64, 32), torch.tensor([90, 0, 33][:B], dtype=torch.int32))


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """Caches of more than 2^31 bytes: rows appended, read and attended to at their end."""
    B, Nk, Hkv, d, T, W = 2, 600000, 16, 128, 40, 30
    assert Nk * Hkv * d * B > 2**31
    c = empty_cache(B, Nk, Hkv, d, fill=0x7f)  # NaN wherever nothing was written
    k, v = rows(B, T, Hkv, d, 33, 0.3).cuda(), rows(B, T, Hkv, d, 34, 0.3).cuda()
    start = torch.tensor([Nk - T, Nk - T - 5], dtype=torch.int32).cuda()
    fa.cache_append(k, v, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], start)
    lens = start + T
    q = query(B, 2, 32, d, 35)
    o, lse = fa.cache_decode_fwd(q.cuda(), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], lens, causal=True, window=W)
    fa.check_device_error()
    small = empty_cache(B, T, Hkv, d)
    fa.cache_append(k, v, small["k_cache"], small["v_cache"], small["k_scale"], small["v_scale"], torch.zeros_like(start))
    want = fa.cache_decode_fwd(q.cuda(), small["k_cache"], small["v_cache"], small["k_scale"], small["v_scale"], None, causal=True, window=W)
    check_decode(q, small, torch.tensor([T, T], dtype=torch.int32), True, window=W)
    # the same keys at other places of a tile: the sums are taken in another order
    assert (lse - want[1]).abs().max() <= 1e-5
    assert ((o - want[0]).float().abs() <= 2 * U * want[0].float().abs() + 2.0 ** -10).all()
    out = fa.cache_read(c["k_cache"][1:], c["k_scale"][1:], lens[1:])
    assert torch.equal(out[0, Nk - T - 5:Nk - 5], fa.cache_read(small["k_cache"], small["k_scale"])[1]) and (out[0, Nk - 5:] == 0).all()


@pytest.mark.gpu
def test_decode_spread_of_value_scales():
    """Value rows whose scales differ by tens of powers of two, zero rows, and the
    largest weight on a small row: the output keeps the precision of what it sums."""
    check_decode(query(2, 1, 2, 128, 17, 4.0), filled(2, 300, 1, 128, 18, spread=12.0), torch.tensor([300, 200], dtype=torch.int32))
    B, Nk, d = 1, 70, 64
    c = empty_cache(B, Nk, 1, d)
    k, v = torch.zeros(B, Nk, 1, d), torch.zeros(B, Nk, 1, d)
    k[0, 5, 0] = 1.0      # all weight on key 5 ...
    v[0, 5, 0] = 2.0 ** -30  # ... whose value is tiny next to the others
    v[0, 6:, 0] = 1000.0
    fa.cache_append(k.bfloat16().cuda(), v.bfloat16().cuda(), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"],
                    torch.zeros(1, dtype=torch.int32, device="cuda"))
    q = torch.full((1, 1, 1, d), 100.0).bfloat16()
    out, _ = check_decode(q, c, torch.tensor([Nk], dtype=torch.int32))
    assert (out == 2.0 ** -30).all()


@pytest.mark.gpu
def test_decode_query_range():
    """Queries near the ends of bf16's range."""
    c = filled(1, 100, 1, 64, 19)
    c["k_scale"].fill_(40)
    check_decode((query(1, 2, 2, 64, 20) * 2.0 ** 60).bfloat16(), c, torch.tensor([100], dtype=torch.int32))
    check_decode((query(1, 2, 2, 64, 21) * 2.0 ** -130).bfloat16(), c, torch.tensor([100], dtype=torch.int32))
    check_decode(torch.zeros(1, 2, 2, 64).bfloat16(), c, torch.tensor([100], dtype=torch.int32))


@pytest.mark.gpu
def test_decode_ignores_rows_no_query_sees():
    c = filled(3, 333, 2, 128, 22)
    lens = torch.tensor([333, 100, 7], dtype=torch.int32)
    q = query(3, 1, 4, 128, 23)
    for window in (0, 50):
        want = check_decode(q, c, lens, window=window)
        dirty = {n: t.clone() for n, t in c.items()}
        for b, L in enumerate(lens.tolist()):
            for n in ("k", "v"):
                dirty[n + "_cache"].view(torch.uint8)[b, L:] = 0x7f   # NaN codes
                dirty[n + "_scale"][b, :, L:] = 255
                if window:
                    dirty[n + "_cache"].view(torch.uint8)[b, :max(0, L - window)] = 0xff
                    dirty[n + "_scale"][b, :, :max(0, L - window)] = 255
        got = fa.cache_decode_fwd(q.cuda(), dirty["k_cache"], dirty["v_cache"], dirty["k_scale"], dirty["v_scale"],
                                  lens.cuda(), causal=True, window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.gpu
def test_decode_bad_length_is_reported_and_nothing_written():
    c = filled(3, 100, 1, 64, 24)
    q = query(3, 1, 1, 64, 25).cuda()
    out = torch.full(q.shape, 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((3, 1, 1), 3.0, device="cuda")
    for bad in (101, -1):
        fa.cache_decode_fwd(q, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"],
                            torch.tensor([100, bad, 5], dtype=torch.int32).cuda(), out=out, lse=lse)
        with pytest.raises(fa.FaError) as e:
            fa.check_device_error()
        assert e.value.status == fa.FA_ERR_INVALID_ARG
        assert (out == 3.0).all() and (lse == 3.0).all()
    fa.check_device_error()


@pytest.mark.gpu
def test_decode_nan_query_stays_in_its_row():
    c = filled(1, 200, 1, 64, 26)
    q = query(1, 2, 4, 64, 27)
    q[0, 1, 2, 5] = float("nan")
    o, lse = fa.cache_decode_fwd(q.cuda(), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"])
    assert torch.isnan(o[0, 1, 2]).all() and torch.isnan(lse[0, 2, 1])
    o[0, 1, 2], lse[0, 2, 1] = 0, 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.gpu
def test_decode_is_reproducible_captured_and_on_another_stream():
    c = filled(4, 900, 2, 128, 28)
    lens = torch.tensor([900, 17, 400, 0], dtype=torch.int32).cuda()
    q = query(4, 1, 8, 128, 29).cuda()
    call = lambda: fa.cache_decode_fwd(q, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], lens, causal=True, softcap=30.0)
    want = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    graph.replay()
    torch.cuda.synchronize()
    for got in (other, held, call()):
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    lens.copy_(torch.tensor([5, 900, 0, 64]))  # the captured call reads the lengths anew
    graph.replay()
    now = call()
    torch.cuda.synchronize()
    assert torch.equal(held[0], now[0]) and torch.equal(held[1], now[1])


@pytest.mark.gpu
@pytest.mark.parametrize("softcap,bias,window", [(0.0, False, 0), (30.0, True, 0), (0.0, True, 90)])
def test_prompt_then_tokens_equal_the_whole_sequence(softcap, bias, window):
    """A prompt and then single tokens go through the cache; each step's output is
    the last row of the modified-score attention over the cached values so far."""
    B, H, Hkv, d, P, steps = 2, 4, 2, 128, 150, 4
    c = empty_cache(B, 200, Hkv, d)
    sl = torch.tensor([0.25, 0.125, 0.0625, 0.03]).cuda() if bias else None
    g = torch.Generator().manual_seed(30)
    new = lambda T, h: torch.randn(B, T, h, d, generator=g).bfloat16().cuda()
    lens = torch.tensor([P, P - 37], dtype=torch.int32).cuda()
    fa.cache_append(new(P, Hkv), new(P, Hkv), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"],
                    torch.zeros_like(lens), lens)
    one = torch.ones_like(lens)
    for _ in range(steps):
        q = new(1, H)
        fa.cache_append(new(1, Hkv), new(1, Hkv), c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], lens, one)
        lens = lens + 1
        o, lse = fa.cache_decode_fwd(q, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], lens, causal=True,
                                     softcap=softcap, slopes=sl, window=window)
        kk, vv = fa.cache_read(c["k_cache"], c["k_scale"], lens), fa.cache_read(c["v_cache"], c["v_scale"], lens)
        for b in range(B):
            L = int(lens[b])
            qq = torch.zeros(1, L, H, d, dtype=torch.bfloat16, device="cuda")
            qq[0, -1] = q[b, 0]
            plan = fa.mask_plan(1, L, causal=True, window=window, device="cuda")
            o2, l2 = fa.mod_fwd(qq, kk[b:b + 1, :L].contiguous(), vv[b:b + 1, :L].contiguous(), plan, softcap=softcap, slopes=sl)
            # both round their weights (bf16: 2 U) and their output (U each)
            mag = vv[b, :L].float().abs().amax()
            assert (o[b, 0].float() - o2[0, -1].float()).abs().max() <= 4 * U * mag
            assert (lse[b, :, 0] - l2[0, :, -1]).abs().max() <= 1e-4
    fa.check_device_error()
