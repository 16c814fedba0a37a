"""Measured cases of the modified-score attention, the 8-bit key/value cache
and the decoding that reads it.

Four operators of exact_io_aware_95_b200, each with its plain form:

  train / prefill   exact attention whose scores are capped by a tanh, biased by
                    distance and masked by causality, a window, documents or a
                    prefix, with grouped heads; forward, and forward + backward
  append            new keys and values quantised into an 8-bit cache
  read              an 8-bit cache read back as bf16
  decode            a few new tokens against an 8-bit cache

``own`` selects the framework's calls (True) or the plain form (False):
elementary torch operations in 32 bits, rounded once at the end.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------------- cases
def listed():
    """The listed cases; the sizes follow the repository's own workloads
    (4 x 16 heads x 4096 tokens, 16384-token contexts and caches) or are generic."""
    return [
        # one short sequence, odd length: the smallest training step, launch latency counts
        _att("train_b1_h2_n130_d64_capped", "train", 1, 2, 1, 130, 64, causal=True, softcap=30.0),
        # the bench's training shape with grouped heads and capped scores
        _att("train_b4_h16_n4096_d128_capped", "train", 4, 16, 4, 4096, 128, causal=True, softcap=50.0),
        # packed documents of about a thousand tokens with a padded tail, distance bias
        _att("train_b2_h16_n8192_d64_documents", "train", 2, 16, 16, 8192, 64, causal=True, doc_len=1024, bias=True),
        # sliding window, one shared key head, odd length, scores that reach the cap
        _att("train_b2_h8_n2047_d64_window", "train", 2, 8, 1, 2047, 64, causal=True, window=512, softcap=20.0,
             bias=True, q_gain=8.0),
        # a long prompt whose first quarter sees itself in both directions, inference only
        _att("prefill_b1_h8_n16384_d128_prefix", "prefill", 1, 8, 2, 16384, 128, causal=True, prefix=4096, bias=True),
        # prompts of ragged lengths written to the cache
        _cache("append_b8_t2047_h8_d128_prompt", "append", 8, 8, 4096, 128, T=2047),
        # one token of each running sequence written to the cache: every decoding step
        _cache("append_b64_t1_h8_d128_token", "append", 64, 8, 2048, 128, T=1),
        # ragged caches read back, as before a bf16 prefill over cached tokens
        _cache("read_b8_n8191_h8_d128_ragged", "read", 8, 8, 8191, 128),
        # a short conversation: the smallest decoding step
        _dec("decode_b2_h4_nk100_d64", 2, 1, 4, 2, 100, 64, softcap=30.0),
        # the repository's serving workload, all caches full, one key head per query head
        _dec("decode_b16_h16_nk16384_d128_full", 16, 1, 16, 16, 16384, 128, full=True),
        # a large batch of ragged lengths with grouped heads and capped scores
        _dec("decode_b64_h32_kv8_nk8192_d128_ragged", 64, 1, 32, 8, 8192, 128, softcap=50.0),
        # one very long sequence, several tokens at once, one key head, distance bias
        _dec("decode_b1_h8_kv1_nk65536_d64_nq4", 1, 4, 8, 1, 65536, 64, bias=True, full=True),
    ]


def _att(name, op, B, H, Hkv, N, d, causal=True, window=0, doc_len=0, prefix=0, softcap=0.0, bias=False, q_gain=3.0):
    return {"name": name, "op": op, "B": B, "H": H, "Hkv": Hkv, "N": N, "d": d, "causal": causal, "window": window,
            "doc_len": doc_len, "prefix": prefix, "softcap": softcap, "bias": bias, "q_gain": q_gain}


def _cache(name, op, B, Hkv, Nk, d, T=0):
    return {"name": name, "op": op, "B": B, "Hkv": Hkv, "Nk": Nk, "d": d, "T": T}


def _dec(name, B, Nq, H, Hkv, Nk, d, softcap=0.0, bias=False, window=0, full=False):
    return {"name": name, "op": "decode", "B": B, "Nq": Nq, "H": H, "Hkv": Hkv, "Nk": Nk, "d": d, "softcap": softcap,
            "bias": bias, "window": window, "full": full}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("train", "train", "prefill", "append", "read", "decode", "decode"))
    d = rng.choice((64, 128))
    Hkv = rng.choice((1, 2, 3, 4, 8, 16))
    if op in ("train", "prefill"):
        H = Hkv * rng.choice((1, 2, 4))
        N = _log_int(rng, 16, 8192)  # a row with one key has no gradient but rounding to compare
        B = _log_int(rng, 1, 8)
        while B > 1 and B * H * N * N > 64 * 4096 * 4096:
            B -= 1
        while H * N * N > 64 * 4096 * 4096:
            N = N // 2 + 1
        kind = rng.choice(("plain", "window", "documents", "prefix"))
        c = _att("", op, B, H, Hkv, N, d, causal=kind == "prefix" or rng.random() < 0.75,
                 window=_log_int(rng, 8, N) if kind == "window" else 0,
                 doc_len=_log_int(rng, 8, N) if kind == "documents" else 0,
                 prefix=_log_int(rng, 1, N) if kind == "prefix" else 0,
                 softcap=rng.choice((0.0, 20.0, 30.0, 50.0)), bias=rng.random() < 0.5, q_gain=rng.choice((1.0, 3.0, 8.0)))
    elif op == "append":
        B = _log_int(rng, 1, 64)
        T = _log_int(rng, 1, max(1, 16384 // B))
        c = _cache("", op, B, Hkv, T + _log_int(rng, 1, 2048), d, T=T)
    elif op == "read":
        B = _log_int(rng, 1, 64)
        c = _cache("", op, B, Hkv, _log_int(rng, 1, max(1, 65536 // B)), d)
    else:
        B = _log_int(rng, 1, 64)
        Nk = _log_int(rng, 1, 16384)
        while B > 1 and B * Nk * Hkv > 16 * 16384 * 16:
            B = B // 2
        Nq = rng.choice((1, 1, 1, 2, 5, 16))
        c = _dec("", B, Nq, Hkv * rng.choice((1, 2, 4, 7, 8)), Hkv, Nk, d, softcap=rng.choice((0.0, 30.0, 50.0)),
                 bias=rng.random() < 0.5, window=_log_int(rng, 1, Nk) if rng.random() < 0.3 else 0,
                 full=rng.random() < 0.3)
    del c["name"]
    return c


# --------------------------------------------------------------------- inputs
def _normal(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _slopes(H):
    """The usual geometric slopes of a distance bias: 2^(-8 (h + 1) / H)."""
    return torch.pow(2.0, -8.0 * torch.arange(1, H + 1, device="cuda", dtype=torch.float32) / H)


def _quantise(x):
    """Rows of the last dimension in e4m3 with a power-of-two scale 2^(e - 127),
    the smallest that brings the row's largest magnitude to at most 448; e is 8 bits."""
    amax = x.abs().amax(-1)
    m, ex = torch.frexp(amax)  # amax = m 2^ex, m in [1/2, 1): 448 = (7/8) 2^9
    e = ex - 9 + (m > 0.875) + 127
    e = torch.where(amax > 0, e.clamp(min=1), torch.full_like(e, 127)).to(torch.int32)
    return torch.ldexp(x, (127 - e).unsqueeze(-1)).to(torch.float8_e4m3fn), e.to(torch.uint8)


def _dequantise(codes, e):
    """codes [B, N, Hkv, d], e [B, Hkv, N] -> float32 [B, N, Hkv, d]."""
    return torch.ldexp(codes.float(), (e.to(torch.int32) - 127).transpose(1, 2).unsqueeze(-1))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, d, B = case["op"], case["d"], case["B"]
    s = {"case": case, "op": op}
    if op in ("train", "prefill"):
        N, H, Hkv = case["N"], case["H"], case["Hkv"]
        s["q"] = (_normal(gen, B, N, H, d) * case["q_gain"]).bfloat16()
        s["k"] = _normal(gen, B, N, Hkv, d).bfloat16()
        s["v"] = _normal(gen, B, N, Hkv, d).bfloat16()
        if op == "train":
            s["do"] = _normal(gen, B, N, H, d).bfloat16()
        s["slopes"] = _slopes(H) if case["bias"] else None
        s["doc_ids"] = s["prefix"] = None
        if case["doc_len"]:  # documents of about doc_len tokens; the batch's tail is padding
            starts = torch.rand((B, N), generator=gen, device="cuda") < 1.0 / case["doc_len"]
            ids = torch.cumsum(starts, 1)
            tail = torch.randint(0, N // 16 + 1, (B, 1), generator=gen, device="cuda")
            ids = torch.where(torch.arange(N, device="cuda") >= N - tail, torch.full_like(ids, -1), ids)
            s["doc_ids"] = ids.to(torch.int32)
        if case["prefix"]:
            s["prefix"] = torch.full((B,), case["prefix"], dtype=torch.int32, device="cuda")
        return s
    Hkv, Nk = case["Hkv"], case["Nk"]
    if op == "append":
        T = case["T"]
        s["k"] = _normal(gen, B, T, Hkv, d).bfloat16()
        s["v"] = _normal(gen, B, T, Hkv, d).bfloat16()
        for n in ("k", "v"):
            s[n + "_cache"] = torch.zeros((B, Nk, Hkv, d), dtype=torch.float8_e4m3fn, device="cuda")
            s[n + "_scale"] = torch.full((B, Hkv, Nk), 127, dtype=torch.uint8, device="cuda")
        s["start"] = torch.randint(0, Nk - T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        s["count"] = torch.randint((T + 1) // 2, T + 1, (B,), generator=gen, device="cuda", dtype=torch.int32)
        return s
    channel = torch.exp2(_normal(gen, Hkv, d))  # channels of different size, as keys and values have
    for n in ("k", "v") if op == "decode" else ("k",):
        rows = _normal(gen, B, Nk, Hkv, d).mul_(channel if n == "k" else 1.0)
        s[n + "_cache"], e = _quantise(rows)
        s[n + "_scale"] = e.transpose(1, 2).contiguous()
        del rows
    if op == "decode":
        s["q"] = (_normal(gen, B, case["Nq"], case["H"], d) / channel.repeat_interleave(case["H"] // Hkv, 0)).bfloat16()
        s["slopes"] = _slopes(case["H"]) if case["bias"] else None
    s["lens"] = (torch.full((B,), Nk, dtype=torch.int32, device="cuda") if case.get("full") else
                 torch.randint(1, Nk + 1, (B,), generator=gen, device="cuda", dtype=torch.int32))
    return s


# ----------------------------------------------------------------- plain forms
def _visible(case, s):
    """[B, N, N] (or [1, N, N]) truth values: query i sees key j."""
    N = case["N"]
    i = torch.arange(N, device="cuda")[:, None]
    j = torch.arange(N, device="cuda")[None, :]
    see = (j <= i) if case["causal"] else torch.ones((N, N), dtype=torch.bool, device="cuda")
    see = see[None]
    if s["prefix"] is not None:
        see = see | (j[None] < s["prefix"][:, None, None])
    if case["window"]:
        see = see & ((i - j).abs() < case["window"])[None]
    if s["doc_ids"] is not None:
        ids = s["doc_ids"]
        run_of = torch.cumsum(torch.nn.functional.pad((ids[:, 1:] != ids[:, :-1]).int(), (1, 0)), 1)
        see = see & (run_of[:, :, None] == run_of[:, None, :]) & (ids >= 0)[:, :, None]
    return see


def _plain_attention(s):
    c = s["case"]
    B, N, H, Hkv, d = c["B"], c["N"], c["H"], c["Hkv"], c["d"]
    G = H // Hkv
    scale = 1.0 / math.sqrt(d)
    q = s["q"].float().view(B, N, Hkv, G, d).permute(0, 2, 3, 1, 4)  # [B, Hkv, G, N, d]
    k = s["k"].float().permute(0, 2, 1, 3)[:, :, None]               # [B, Hkv, 1, N, d]
    v = s["v"].float().permute(0, 2, 1, 3)[:, :, None]
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(scale)
    t = None
    if c["softcap"]:
        t = x.div_(c["softcap"]).tanh_()
        x = t * c["softcap"]
    if s["slopes"] is not None:
        pos = torch.arange(N, device="cuda", dtype=torch.float32)
        x -= s["slopes"].view(Hkv, G, 1, 1) * (pos[:, None] - pos[None, :]).abs()
    x.masked_fill_(~_visible(c, s)[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total == 0, torch.ones_like(total), total)
    o = torch.matmul(p, v)
    out = {"o": o.permute(0, 3, 1, 2, 4).reshape(B, N, H, d).bfloat16(), "lse": (m + total.log()).view(B, H, N)}
    if "do" not in s:
        return out
    do = s["do"].float().view(B, N, Hkv, G, d).permute(0, 2, 3, 1, 4)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2)
    ds = torch.matmul(do, v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    if t is not None:
        ds.mul_(t.square_().neg_().add_(1.0))
    dq = torch.matmul(ds, k).mul_(scale)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2).mul_(scale)
    out["dq"] = dq.permute(0, 3, 1, 2, 4).reshape(B, N, H, d).bfloat16()
    out["dk"] = dk.transpose(1, 2).bfloat16()
    out["dv"] = dv.transpose(1, 2).bfloat16()
    return out


def _plain_append(s):
    B, T = s["k"].shape[:2]
    j = torch.arange(T, device="cuda")
    b, j = torch.nonzero(j[None, :] < s["count"][:, None], as_tuple=True)
    row = s["start"][b] + j
    k, ke = _quantise(s["k"][b, j].float())
    v, ve = _quantise(s["v"][b, j].float())
    s["k_cache"].view(torch.uint8)[b, row] = k.view(torch.uint8)
    s["v_cache"].view(torch.uint8)[b, row] = v.view(torch.uint8)
    s["k_scale"][b, :, row] = ke
    s["v_scale"][b, :, row] = ve
    return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _plain_read(s):
    rows = torch.arange(s["k_cache"].shape[1], device="cuda")
    x = _dequantise(s["k_cache"], s["k_scale"])
    return x.masked_fill_((rows[None, :] >= s["lens"][:, None])[:, :, None, None], 0.0).bfloat16()


def _plain_decode(s):
    c = s["case"]
    B, Nq, H, Hkv, Nk, d = c["B"], c["Nq"], c["H"], c["Hkv"], c["Nk"], c["d"]
    G = H // Hkv
    q = s["q"].float().view(B, Nq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Nq, d)
    k = _dequantise(s["k_cache"], s["k_scale"]).permute(0, 2, 1, 3)
    x = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(B, Hkv, G, Nq, Nk)
    del k
    if c["softcap"]:
        x = x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    j = torch.arange(Nk, device="cuda")
    at = s["lens"][:, None] - Nq + torch.arange(Nq, device="cuda")  # [B, Nq]: the queries' positions
    away = at[:, :, None] - j[None, None, :]
    if s["slopes"] is not None:
        x -= s["slopes"].view(Hkv, G, 1, 1) * away[:, None, None].abs().float()
    see = away >= 0
    if c["window"]:
        see = see & (away < c["window"])
    x.masked_fill_(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    p /= torch.where(total == 0, torch.ones_like(total), total)
    v = _dequantise(s["v_cache"], s["v_scale"]).permute(0, 2, 1, 3)
    o = torch.matmul(p.view(B, Hkv, G * Nq, Nk), v)
    o = o.view(B, Hkv, G, Nq, d).permute(0, 3, 1, 2, 4).reshape(B, Nq, H, d)
    return {"o": o.bfloat16(), "lse": (m + total.log()).view(B, H, Nq)}


# ------------------------------------------------------------------- the calls
def _own(s):
    import exact_io_aware_95_b200 as fa
    c, op = s["case"], s["op"]
    if op in ("train", "prefill"):
        plan = fa.mask_plan(c["B"], c["N"], causal=c["causal"], window=c["window"], doc_ids=s["doc_ids"],
                            prefix=s["prefix"], device=s["q"].device)
        how = {"softcap": c["softcap"], "slopes": s["slopes"]}
        if op == "prefill":
            o, lse = fa.mod_fwd(s["q"], s["k"], s["v"], plan, **how)
            return {"o": o, "lse": lse}
        o, lse, o_low = fa.mod_fwd(s["q"], s["k"], s["v"], plan, low=True, **how)
        dq, dk, dv = fa.mod_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], plan, o_low=o_low, **how)
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    if op == "append":
        fa.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["start"], s["count"])
        return {n: s[n] for n in ("k_cache", "v_cache", "k_scale", "v_scale")}
    if op == "read":
        return fa.cache_read(s["k_cache"], s["k_scale"], s["lens"])
    o, lse = fa.cache_decode_fwd(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["lens"], causal=True,
                                 softcap=c["softcap"], slopes=s["slopes"], window=c["window"])
    return {"o": o, "lse": lse}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op in ("train", "prefill"):
        return _plain_attention(state)
    return {"append": _plain_append, "read": _plain_read, "decode": _plain_decode}[op](state)


# ------------------------------------------------------------------------ work
def _pairs(case):
    """(query, key) pairs of one head of the batch that the mask leaves, on average."""
    N = case["N"]
    if case["doc_len"]:
        n = min(N, 2.0 * case["doc_len"])  # a token's document is about this long, seen from inside it
    elif case["window"]:
        n = min(N, (1 if case["causal"] else 2) * case["window"])
        return case["B"] * (N * n - (n * n / 2 if case["causal"] else n * n / 4))
    else:
        n = N
    pairs = N * n * (0.5 if case["causal"] else 1.0)
    if case["prefix"]:
        pairs += 0.5 * min(N, case["prefix"]) ** 2
    return case["B"] * pairs


def work(case):
    op, B, Hkv, d = case["op"], case["B"], case["Hkv"], case["d"]
    if op in ("train", "prefill"):
        H, N = case["H"], case["N"]
        qo, kv = B * N * H * d * 2, B * N * Hkv * d * 2
        flops = 4.0 * _pairs(case) * H * d
        byts = 2 * qo + 2 * kv + B * H * N * 4  # q, k, v in; o, lse out
        if op == "train":
            flops *= 3.5                         # two products forward, five backward
            byts += 2 * qo + 2 * kv              # do in; dq, dk, dv out
        return {"bytes": byts, "flops": flops}
    if op == "append":
        rows = B * 0.75 * case["T"] * Hkv * 2
        return {"bytes": rows * (d * 3 + 1), "flops": rows * d * 2}
    keys = B * case["Nk"] * (1.0 if case.get("full") else 0.5) * Hkv
    if op == "read":
        return {"bytes": keys * (d + 1) + B * case["Nk"] * Hkv * d * 2, "flops": keys * d}
    if case["window"]:
        keys = min(keys, B * Hkv * (case["window"] + case["Nq"]))
    rows = case["Nq"] * case["H"] // Hkv
    return {"bytes": keys * 2 * (d + 1) + B * case["Nq"] * case["H"] * (d * 4 + 4), "flops": keys * rows * 4 * d}


# ----------------------------------------------------------------- in 64 bits
def _exact_head(q, k, v, see, scale, softcap, slope, away, do):
    """One head in float64 by the definition; gradients by differentiating it."""
    leaves = [t.double().requires_grad_(do is not None) for t in (q, k, v)]
    x = leaves[0] @ leaves[1].T * scale
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    if slope is not None:
        x = x - slope.double() * away
    some = see.any(-1)
    x = torch.where(see, x, torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
    x = torch.where(some[:, None], x, torch.zeros((), dtype=torch.float64, device="cuda"))
    o = torch.where(some[:, None], torch.softmax(x, -1) @ leaves[2], torch.zeros((), dtype=torch.float64, device="cuda"))
    lse = torch.where(some, torch.logsumexp(x, -1), torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
    grads = torch.autograd.grad(o, leaves, do.double()) if do is not None else None
    return o.detach(), lse.detach(), grads


def _exact_attention(s):
    c = s["case"]
    B, N, H, Hkv, d = c["B"], c["N"], c["H"], c["Hkv"], c["d"]
    f8 = {"dtype": torch.float64, "device": "cuda"}
    out = {"o": torch.zeros((B, N, H, d), **f8), "lse": torch.zeros((B, H, N), **f8)}
    if "do" in s:
        out |= {"dq": torch.zeros((B, N, H, d), **f8), "dk": torch.zeros((B, N, Hkv, d), **f8),
                "dv": torch.zeros((B, N, Hkv, d), **f8)}
    at = torch.arange(N, device="cuda")
    away = (at[:, None] - at[None, :]).abs().double()
    for b in range(B):
        lo, hi = torch.zeros_like(at), torch.full_like(at, N)  # query i sees keys lo[i] <= j < hi[i]
        if s["doc_ids"] is not None:
            ids = s["doc_ids"][b].tolist()
            first, a = [0] * N, 0
            for i in range(N):
                a = i if i and ids[i] != ids[i - 1] else a
                first[i] = a
            last, e = [N] * N, N
            for i in range(N - 1, -1, -1):
                e = i + 1 if i + 1 < N and ids[i + 1] != ids[i] else e
                last[i] = e
            lo = torch.tensor(first, device="cuda")
            hi = torch.where(s["doc_ids"][b] < 0, lo, torch.tensor(last, device="cuda"))
        if c["causal"]:
            ahead = at + 1
            if s["prefix"] is not None:
                ahead = torch.maximum(ahead, s["prefix"][b].long())
            hi = torch.minimum(hi, ahead)
        if c["window"]:
            lo, hi = torch.maximum(lo, at - c["window"] + 1), torch.minimum(hi, at + c["window"])
        see = (at[None, :] >= lo[:, None]) & (at[None, :] < hi[:, None])
        for h in range(H):
            g = h // (H // Hkv)
            o, lse, grads = _exact_head(s["q"][b, :, h], s["k"][b, :, g], s["v"][b, :, g], see, 1.0 / math.sqrt(d),
                                        c["softcap"], None if s["slopes"] is None else s["slopes"][h], away,
                                        s["do"][b, :, h] if "do" in s else None)
            out["o"][b, :, h], out["lse"][b, h] = o, lse
            if grads is not None:
                out["dq"][b, :, h] = grads[0]
                out["dk"][b, :, g] += grads[1]
                out["dv"][b, :, g] += grads[2]
    return out


def _value(codes, e):
    return codes.double() * torch.pow(torch.full((), 2.0, dtype=torch.float64, device="cuda"), e.double() - 127.0)


def _exact_decode(s):
    c = s["case"]
    B, Nq, H, Hkv, d = c["B"], c["Nq"], c["H"], c["Hkv"], c["d"]
    o = torch.zeros((B, Nq, H, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((B, H, Nq), dtype=torch.float64, device="cuda")
    for b in range(B):
        L = int(s["lens"][b])
        j = torch.arange(L, device="cuda")
        at = L - Nq + torch.arange(Nq, device="cuda")
        away = (at[:, None] - j[None, :])
        see = (away >= 0) & ((away < c["window"]) if c["window"] else True)
        for g in range(Hkv):
            k = _value(s["k_cache"][b, :L, g], s["k_scale"][b, g, :L, None])
            v = _value(s["v_cache"][b, :L, g], s["v_scale"][b, g, :L, None])
            for h in range(g * (H // Hkv), (g + 1) * (H // Hkv)):
                o[b, :, h], lse[b, h], _ = _exact_head(s["q"][b, :, h], k, v, see, 1.0 / math.sqrt(d), c["softcap"],
                                                       None if s["slopes"] is None else s["slopes"][h],
                                                       away.abs().double(), None)
    return {"o": o, "lse": lse}


def _exact_append(s):
    """Rows of the caches after the call, by the definition of the scale: the
    smallest power of two that brings the largest magnitude to 448 or less."""
    out = {}
    for n in ("k", "v"):
        x = s[n].double()
        top = x.abs().amax(-1)
        e = torch.ceil(torch.log2(torch.where(top > 0, top, torch.full_like(top, E4M3_MAX)) / E4M3_MAX)).clamp(min=-126.0)
        y = x / torch.exp2(e)[..., None]
        # round to e4m3 by hand: three bits behind the leading one, steps of 2^-9 at the least
        step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3.0)
        y = torch.round(y / step) * step
        cache = s[n + "_cache"].double()
        for b in range(x.shape[0]):
            m, r = int(s["count"][b]), int(s["start"][b])
            cache[b, r:r + m] = y[b, :m]
        out[n + "_cache"] = cache
        out[n + "_scale"] = None  # whole numbers: held equal by themselves
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("train", "prefill"):
        return _exact_attention(s)
    if op == "append":
        return _exact_append(s)
    if op == "read":
        x = _value(s["k_cache"], s["k_scale"].transpose(1, 2)[..., None])
        rows = torch.arange(x.shape[1], device="cuda")
        return torch.where((rows[None, :] < s["lens"][:, None])[..., None, None], x, torch.zeros_like(x))
    return _exact_decode(s)
