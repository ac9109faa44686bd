"""The measured cases of the operators around the attention: the rotary
embedding of queries and keys with its gradient, and the attention whose
scores are capped by a tanh, get a bias that depends on distance, or follow a
document or prefix mask, with its gradient.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from
a seed, ``run`` makes one pass: in plain fp32 torch operations, or with ``own``
through the library. ``exact`` is the same in 64 bits, written from the
formulas on its own.
"""
import math
import random

import torch

own = False  # the plain forms below, or (True) the library's kernels


def _rope(name, B, S, Hq, Hkv, D, rot, interleaved, dtype, scaling, start, packed, grad):
    return {"name": name, "op": "rope_grad" if grad else "rope", "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "D": D,
            "rot": rot, "interleaved": interleaved, "dtype": dtype, "scaling": scaling, "start": start,
            "packed": packed}


def _attn(name, B, S, Hq, Hkv, D, dtype, grad, softcap=0.0, slopes=False, docs=0, prefix=False, window=-1,
          padded=False, gain=1.0, det=False):
    return {"name": name, "op": "attn_grad" if grad else "attn", "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "D": D,
            "dtype": dtype, "softcap": softcap, "slopes": slopes, "docs": docs, "prefix": prefix,
            "window": window, "padded": padded, "gain": gain, "det": det}


def listed():
    return [
        # One new token for each of 16 running sequences, far into their contexts.
        _rope("rope_one_token", 16, 1, 32, 8, 128, 128, False, "bf16", "bands", 31000, False, False),
        # The queries and keys of a training batch, from the projection's (B, S, H, D) layout.
        _rope("rope_batch", 4, 4096, 32, 8, 128, 128, False, "bf16", "none", 0, False, False),
        # Packed documents of odd total length, 32 of 80 columns rotated in adjacent pairs.
        _rope("rope_packed_part", 3, 1531, 16, 16, 80, 32, True, "fp16", "linear", 0, True, False),
        # The gradients of a training batch back into the projection's layout.
        _rope("rope_grad_batch", 4, 4096, 32, 8, 128, 128, True, "bf16", "none", 0, False, True),
        # A short prompt: latency.
        _attn("fwd_short", 1, 77, 4, 4, 64, "bf16", False, softcap=30.0, gain=3.0),
        # The causal grouped-query shape of the benchmark with capped scores.
        _attn("fwd_capped_gqa", 1, 4096, 32, 8, 128, "bf16", False, softcap=50.0, gain=3.0),
        # A pretraining batch of packed documents, causal within each.
        _attn("fwd_packed_docs", 2, 4096, 16, 16, 128, "bf16", False, docs=9),
        # Distance-biased scores, a bidirectional prefix, ragged lengths, fp16.
        _attn("fwd_prefix_slopes", 2, 1777, 12, 4, 64, "fp16", False, slopes=True, prefix=True, padded=True),
        # The gradients of the same.
        _attn("bwd_short", 1, 77, 4, 4, 64, "bf16", True, softcap=30.0, gain=3.0),
        _attn("bwd_capped_gqa", 1, 4096, 32, 8, 128, "bf16", True, softcap=50.0, gain=3.0, det=True),
        _attn("bwd_packed_docs", 2, 4096, 16, 16, 128, "bf16", True, docs=9),
        _attn("bwd_prefix_slopes", 2, 1777, 12, 4, 64, "fp16", True, slopes=True, prefix=True, padded=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["rope", "rope_grad", "attn", "attn", "attn_grad", "attn_grad"])
    if kind.startswith("rope"):
        Hkv = rng.choice([1, 2, 4, 8, 16])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8] if Hkv <= 4 else [1, 2, 4])
        D = rng.choice([64, 80, 96, 128, 128, 256])
        rot = rng.choice([D, D, D // 2, D // 4])
        rot -= rot % 2
        S = _spread(rng, 1, 8192)
        # at most the elements of the largest listed batch
        B = max(1, min(_spread(rng, 1, 64), (4 * 4096 * 40 * 128) // (S * (Hq + Hkv) * D)))
        S = min(S, (4 * 4096 * 40 * 128) // (B * (Hq + Hkv) * D))
        c = _rope("", B, S, Hq, Hkv, D, rot, rng.random() < 0.5, rng.choice(["bf16", "fp16"]),
                  rng.choice(["none", "linear", "bands"]), rng.choice([0, 0, _spread(rng, 1, 1 << 20)]),
                  rng.random() < 0.4, kind == "rope_grad")
    else:
        D = rng.choice([64, 64, 128, 128, 32, 80, 96])
        Hkv = rng.choice([1, 2, 4, 8, 16])
        Hq = Hkv * rng.choice([1, 2, 3, 4, 8] if Hkv <= 4 else [1, 2])
        S = _spread(rng, 16, 4096)
        most = 32 * 4096 * 4096
        B = max(1, min(_spread(rng, 1, 16), most // (Hq * S * S)))
        docs = rng.choice([0, 0, _spread(rng, 1, max(1, min(40, S // 8)))])
        softcap = rng.choice([0.0, 15.0, 30.0, 50.0])
        slopes = rng.random() < 0.4
        prefix = rng.random() < 0.35
        if not (docs or softcap or slopes or prefix):
            softcap = 20.0
        c = _attn("", B, S, Hq, Hkv, D, rng.choice(["bf16", "bf16", "fp16"]), kind == "attn_grad",
                  softcap=softcap, slopes=slopes, docs=docs, prefix=prefix,
                  window=_spread(rng, 8, S) if rng.random() < 0.25 and not prefix else -1,
                  padded=rng.random() < 0.3, gain=rng.choice([1.0, 2.0, 4.0]),
                  det=D == 128 and rng.random() < 0.4)
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def _frequencies(c):
    """(rot / 2 angular frequencies in 64 bits, the factor on cos and sin)."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / c["rot"])
    if c["scaling"] == "linear":
        return f / 4.0, 1.0
    if c["scaling"] == "bands":  # low frequencies interpolated, high ones kept, by turns over 4096 positions
        turns = 4096.0 * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / 8.0), 0.1 * math.log(8.0) + 1.0
    return f, 1.0


def _cuts(c):
    """Per batch row the first positions of its documents, by the case alone."""
    r = random.Random(1000 * c["S"] + 10 * c["docs"] + c["B"])
    return [[0] + sorted(r.sample(range(1, c["S"]), min(c["docs"], c["S"]) - 1)) if c["docs"] > 1 else [0]
            for _ in range(c["B"])]


def _lengths(c):
    r = random.Random(77 * c["S"] + c["B"])
    return [r.randint(max(2, c["S"] // 2), c["S"]) if c["padded"] else c["S"] for _ in range(c["B"])]


def _doc_ids(c):
    ids = torch.zeros(c["B"], c["S"], dtype=torch.int32)
    for b, cuts in enumerate(_cuts(c)):
        for x in cuts[1:]:
            ids[b, x:] += 1
    return ids


def _prefix(c):
    """Positions at the start of each document (or of the row) that all its rows see."""
    r = random.Random(5 * c["S"] + c["docs"])
    span = max(1, c["S"] // max(1, c["docs"]))
    return [r.randint(0, max(1, span // 2)) if c["prefix"] else 0 for _ in range(c["B"])]


def _masked(c):
    return c["docs"] > 0 or c["prefix"]


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    t = _TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if c["op"].startswith("rope"):
        rows = (c["B"], c["S"]) if c["op"] == "rope" else (c["B"],)
        shape = (lambda H: rows + (H, c["D"])) if c["op"] == "rope" else (lambda H: rows + (H, c["S"], c["D"]))
        f, mult = _frequencies(c)
        s = {"case": c, "q": normal(*shape(c["Hq"])).to(t), "k": normal(*shape(c["Hkv"])).to(t),
             "freq": f.cuda(), "mult": mult, "positions": None}
        if c["packed"] or c["S"] == 1:  # positions that restart in the row, or a place of its own for each row
            at = torch.randint(0, max(1, c["S"]), (c["B"], 1), generator=g, device="cuda")
            s["positions"] = (c["start"] + (torch.arange(c["S"], device="cuda") + at) % max(c["S"], 2)).to(torch.int32)
        return s
    B, S, Hq, Hkv, D = c["B"], c["S"], c["Hq"], c["Hkv"], c["D"]
    s = {"case": c, "q": (normal(B, Hq, S, D) * c["gain"]).to(t), "k": normal(B, Hkv, S, D).to(t),
         "v": normal(B, Hkv, S, D).to(t), "slopes": None, "ids": None, "prefix": None, "lens": None, "plan": None}
    if c["slopes"]:
        s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, Hq + 1, device="cuda") / Hq)
    if c["padded"]:
        s["lens"] = torch.tensor(_lengths(c), dtype=torch.int32, device="cuda")
    if _masked(c):
        s["ids"] = _doc_ids(c).cuda()
        s["prefix"] = torch.tensor(_prefix(c), dtype=torch.int32, device="cuda")
    if c["op"] == "attn_grad":
        s["do"] = normal(B, Hq, S, D).to(t)
        o, s["lse"] = _attention(s)
        s["o"] = o.to(t)
    if own:
        import attention_backward_sdpa_gb300 as sdpa
        if _masked(c):  # one plan serves every layer and both directions of a batch
            s["plan"] = sdpa.mask_plan(B, S, S, doc_ids=s["ids"], prefix_lens=s["prefix"], causal=True)
    return s


# ------------------------------------------------------------------ plain forms
def _turn(x, cos, sin, rot, interleaved):
    """The first rot columns of x (fp32, (..., S, H, D)) rotated pair by pair."""
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : rot // 2], r[..., rot // 2:])
    u, w = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _plain_rope(s):
    c = s["case"]
    pos = s["positions"]
    pos = torch.arange(c["S"], device="cuda")[None] + c["start"] if pos is None else pos
    angle = pos.double()[..., None] * s["freq"]  # (1|B, S, rot / 2)
    cos, sin = (angle.cos() * s["mult"]).float(), (angle.sin() * s["mult"]).float()
    if c["op"] == "rope":  # (B, S, H, D) in, (B, H, S, D) out
        cos, sin = cos[:, :, None], sin[:, :, None]
        turn = lambda x: _turn(x.float(), cos, sin, c["rot"], c["interleaved"]).transpose(1, 2).to(x.dtype).contiguous()  # noqa: E731
    else:  # the gradient: the transposed rotation, (B, H, S, D) in, (B, S, H, D) out
        cos, sin = cos[:, None], -sin[:, None]
        turn = lambda x: _turn(x.float(), cos, sin, c["rot"], c["interleaved"]).transpose(1, 2).to(x.dtype).contiguous()  # noqa: E731
    return turn(s["q"]), turn(s["k"])


def _visible(s):
    """(B, S, S): which keys each row sees."""
    c = s["case"]
    n = torch.arange(c["S"], device="cuda")
    i, j = n[:, None], n[None, :]
    see = (j <= i)[None].expand(c["B"], -1, -1)
    if s["ids"] is not None:
        ids = s["ids"]
        same = ids[:, :, None] == ids[:, None, :]
        first = (ids[:, None, :] < ids[:, :, None]).sum(-1)  # positions before the row's document
        see = same & (see | (j[None] - first[:, :, None] < s["prefix"][:, None, None]))
    if c["window"] >= 0:
        see = see & (j >= i - c["window"])
    if s["lens"] is not None:
        inside = n[None] < s["lens"][:, None]
        see = see & inside[:, :, None] & inside[:, None, :]
    return see


def _scores(s):
    """(capped and biased scores (B, Hkv, G, S, S) with -inf where masked, tanh of the capped ones or None)."""
    c = s["case"]
    B, S, Hq, Hkv, D = c["B"], c["S"], c["Hq"], c["Hkv"], c["D"]
    q = s["q"].float().view(B, Hkv, -1, D)
    x = (q @ s["k"].float().transpose(2, 3)).view(B, Hkv, Hq // Hkv, S, S) * (1.0 / math.sqrt(D))
    t = None
    if c["softcap"]:
        t = torch.tanh(x / c["softcap"])
        x = t * c["softcap"]
    if s["slopes"] is not None:
        n = torch.arange(S, device="cuda")
        x = x - s["slopes"].view(1, Hkv, -1, 1, 1) * (n[:, None] - n[None, :]).abs()
    return x.masked_fill(~_visible(s)[:, None, None], -math.inf), t


def _attention(s):
    """O (fp32) and LSE."""
    c = s["case"]
    B, S, Hq, Hkv, D = c["B"], c["S"], c["Hq"], c["Hkv"], c["D"]
    x, _ = _scores(s)
    m = x.amax(-1, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = (p / total.masked_fill(total == 0, 1.0)).view(B, Hkv, -1, S) @ s["v"].float()
    return o.view(B, Hq, S, D), (m + total.log()).view(B, Hq, S)


def _plain_gradient(s):
    c = s["case"]
    B, S, Hq, Hkv, D = c["B"], c["S"], c["Hq"], c["Hkv"], c["D"]
    x, t = _scores(s)
    lse = s["lse"].view(B, Hkv, -1, S, 1)
    p = torch.exp(x - lse.masked_fill(lse == -math.inf, 0.0))
    do = s["do"].float().view(B, Hkv, -1, D)
    dv = p.view(B, Hkv, -1, S).transpose(2, 3) @ do
    delta = (s["do"].float() * s["o"].float()).sum(-1).view(B, Hkv, -1, S, 1)
    ds = p * ((do @ s["v"].float().transpose(2, 3)).view_as(p) - delta)
    if t is not None:
        ds = ds * (1.0 - t * t)
    ds = (ds * (1.0 / math.sqrt(D))).view(B, Hkv, -1, S)
    dq = ds @ s["k"].float()
    dk = ds.transpose(2, 3) @ s["q"].float().view(B, Hkv, -1, D)
    return dq.view(B, Hq, S, D).to(s["q"].dtype), dk.to(s["q"].dtype), dv.to(s["q"].dtype)


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if own:
        import attention_backward_sdpa_gb300 as sdpa
        if c["op"].startswith("rope"):
            kw = dict(mult=s["mult"], positions=s["positions"], offset=0 if s["positions"] is not None else c["start"],
                      interleaved=c["interleaved"])
            if c["op"] == "rope":
                return sdpa.rope_fwd(s["q"].transpose(1, 2), s["k"].transpose(1, 2), s["freq"], **kw)
            out = [torch.empty(c["B"], c["S"], H, c["D"], dtype=s["q"].dtype, device="cuda") for H in (c["Hq"], c["Hkv"])]
            sdpa.rope_bwd(s["q"], s["k"], s["freq"], q_out=out[0].transpose(1, 2), k_out=out[1].transpose(1, 2), **kw)
            return tuple(out)
        # The plan holds the causal side of the mask where there is one.
        kw = dict(causal=s["plan"] is None, window_left=c["window"], seq_q_lens=s["lens"], seq_kv_lens=s["lens"],
                  softcap=c["softcap"], alibi_slopes=s["slopes"], mask_plan=s["plan"])
        if c["op"] == "attn":
            return sdpa.sdpa_fwd(s["q"], s["k"], s["v"], **kw)
        return sdpa.sdpa_bwd(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], deterministic=c["det"], **kw)
    if c["op"].startswith("rope"):
        return _plain_rope(s)
    if c["op"] == "attn":
        o, lse = _attention(s)
        return o.to(s["q"].dtype), lse
    return _plain_gradient(s)


def _ranges(c):
    """Per batch row: the (first, end) keys of each of its rows, from the documents, prefixes, window and lengths."""
    got = []
    for b, cuts in enumerate(_cuts(c)):
        ends, L, pre = cuts[1:] + [c["S"]], _lengths(c)[b], _prefix(c)[b]
        rows, d = [], 0
        for i in range(c["S"]):
            while i >= ends[d]:
                d += 1
            lo, hi = cuts[d], min(ends[d], max(i + 1, cuts[d] + (pre if _masked(c) else 0)))
            if c["window"] >= 0:
                lo = max(lo, i - c["window"])
            hi = min(hi, L) if i < L else lo
            rows.append((lo, max(lo, hi)))
        got.append(rows)
    return got


def work(case):
    c = case
    tokens = c["B"] * c["S"]
    if c["op"].startswith("rope"):
        n = tokens * (c["Hq"] + c["Hkv"])
        return {"bytes": n * c["D"] * 2 * 2, "flops": n * c["rot"] * 3}
    pairs = c["Hq"] * sum(hi - lo for rows in _ranges(c) for lo, hi in rows)
    q, kv = tokens * c["Hq"] * c["D"] * 2, tokens * c["Hkv"] * c["D"] * 2
    lse = tokens * c["Hq"] * 4
    if c["op"] == "attn":  # Q, K, V in, O and LSE out
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * c["D"] * pairs}
    # Q, O, dO, K, V, LSE in, dQ, dK, dV out
    return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * c["D"] * pairs}


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    c = case
    s = prepare(dict(c), seed)
    if c["op"].startswith("rope"):
        pos = s["positions"]
        pos = torch.arange(c["start"], c["start"] + c["S"], device="cuda").expand(c["B"], -1) if pos is None else pos
        angle = pos.double()[:, :, None] * s["freq"]
        z = torch.polar(torch.full_like(angle, s["mult"]), angle if c["op"] == "rope" else -angle)  # (B, S, rot / 2)
        out = []
        for name in ("q", "k"):
            x = s[name].double()
            x = x if c["op"] == "rope" else x.transpose(1, 2)  # (B, S, H, D)
            y, half = x.clone(), c["rot"] // 2
            first = slice(0, c["rot"], 2) if c["interleaved"] else slice(0, half)
            second = slice(1, c["rot"], 2) if c["interleaved"] else slice(half, c["rot"])
            w = torch.complex(x[..., first], x[..., second]) * z[:, :, None]
            y[..., first], y[..., second] = w.real, w.imag
            out.append(y.transpose(1, 2).contiguous() if c["op"] == "rope" else y.contiguous())
        return tuple(out)
    B, S, Hq, Hkv, D = c["B"], c["S"], c["Hq"], c["Hkv"], c["D"]
    grad = c["op"] == "attn_grad"
    n = torch.arange(S, device="cuda")
    o, lse = torch.zeros(B, Hq, S, D, dtype=torch.float64, device="cuda"), torch.zeros(B, Hq, S, dtype=torch.float64, device="cuda")
    dq = torch.zeros_like(o)
    dk, dv = (torch.zeros(B, Hkv, S, D, dtype=torch.float64, device="cuda") for _ in range(2))
    for b, rows in enumerate(_ranges(c)):
        r = torch.tensor(rows, device="cuda")
        keep = (n[None] >= r[:, :1]) & (n[None] < r[:, 1:])
        for h in range(Hq):
            kh = h // (Hq // Hkv)
            q, k, v = s["q"][b, h].double(), s["k"][b, kh].double(), s["v"][b, kh].double()
            z = q @ k.T / math.sqrt(D)
            slope = torch.ones((), dtype=torch.float64, device="cuda")
            if c["softcap"]:
                th = torch.tanh(z / c["softcap"])
                z, slope = c["softcap"] * th, 1.0 - th * th
            if c["slopes"]:
                z = z - s["slopes"][h].double() * (n[:, None] - n[None]).abs()
            z = torch.where(keep, z, -math.inf)
            if not grad:
                lse[b, h] = torch.logsumexp(z, -1)
                o[b, h] = torch.nan_to_num(torch.softmax(z, -1)) @ v
                continue
            p = torch.where(keep, torch.exp(z - s["lse"][b, h].double()[:, None]), 0.0)
            do = s["do"][b, h].double()
            ds = p * (do @ v.T - (do * s["o"][b, h].double()).sum(-1, keepdim=True)) * slope / math.sqrt(D)
            dv[b, kh] += p.T @ do
            dq[b, h] = ds @ k
            dk[b, kh] += ds.T @ q
    return (dq, dk, dv) if grad else (o, lse)
