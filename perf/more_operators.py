"""The measured cases of the operators of serving: rotary positions with several
axes (time, height, width) and their gradient, appending keys and values to a
paged cache of 16 or 8 bits with the rotation on the way, and the attention that
reads such a cache, for single tokens, a few tokens and long chunks, under causal,
sliding-window and first-tokens masks.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from
a seed, ``run`` makes one pass: in plain fp32 torch operations, or with ``own``
through the library. ``exact`` is the same in 64 bits, written from the
formulas on its own.

The cache. Position j of a sequence is slot j % page of page table[j // page]; a
page holds the keys (or values) of all key/value heads, (pages, heads, page, D). In
8 bits (e4m3) each page and head has a scale, a power of two: a code stands for
code * scale. A call that writes a page takes the smallest power of two that brings
the largest new value within 448, or keeps the scale of the slots before them where that is
larger (the older slots are rounded anew where it is smaller).
"""
import math
import random

import torch

own = False  # the plain forms below, or (True) the library's kernels


def _rope(name, B, S, Hq, Hkv, D, sections, mixed, dtype, interleaved, grad):
    return {"name": name, "op": "rope_grad" if grad else "rope", "B": B, "S": S, "Hq": Hq, "Hkv": Hkv, "D": D,
            "sections": sections, "mixed": mixed, "dtype": dtype, "interleaved": interleaved}


def _append(name, B, T, context, Hq, Hkv, D, rot, page, cache, dtype, interleaved=False, ragged=False, axes=False):
    return {"name": name, "op": "append", "B": B, "T": T, "context": context, "Hq": Hq, "Hkv": Hkv, "D": D, "rot": rot,
            "page": page, "cache": cache, "dtype": dtype, "interleaved": interleaved, "ragged": ragged, "axes": axes}


def _attn(name, B, Sq, Skv, Hq, Hkv, D, page, cache, dtype, ragged=False, short_q=False, window=-1, first=0,
          softcap=0.0, slopes=False, sink=False, gain=1.0):
    return {"name": name, "op": "attn", "B": B, "Sq": Sq, "Skv": Skv, "Hq": Hq, "Hkv": Hkv, "D": D, "page": page,
            "cache": cache, "dtype": dtype, "ragged": ragged, "short_q": short_q, "window": window, "first": first,
            "softcap": softcap, "slopes": slopes, "sink": sink, "gain": gain}


def listed():
    return [
        # Video tokens: 16 + 24 + 24 pairs turn by time, height and width.
        _rope("rope_axes_video", 2, 4099, 32, 8, 128, "16,24,24", False, "bf16", False, False),
        # The gradients of an image encoder's batch, two axes that alternate from pair to pair.
        _rope("rope_axes_grad", 8, 1025, 16, 16, 80, "20,20", True, "fp16", True, True),
        # One new token for each of 64 running sequences, 16-bit pages.
        _append("append_step", 64, 1, 500, 32, 8, 128, 128, 16, "bf16", "bf16"),
        # The same into 8-bit pages, whose older slots may need a larger scale; and the cache read back.
        _append("append_step_8bit", 24, 1, 300, 32, 8, 128, 128, 64, "e4m3", "bf16"),
        # Ragged prompts with image positions behind what is cached already; and the cache read back.
        _append("append_prompts_8bit", 5, 1700, 333, 16, 4, 128, 128, 32, "e4m3", "bf16", ragged=True, axes=True),
        # One token over a short context: latency.
        _attn("decode_short", 1, 1, 500, 32, 8, 128, 16, "bf16", "bf16"),
        # One token for each of 64 sequences of very different lengths, 8-bit pages.
        _attn("decode_batch_8bit", 64, 1, 8192, 32, 8, 128, 64, "e4m3", "bf16", ragged=True, gain=2.0),
        # One token of a single long context.
        _attn("decode_long_8bit", 1, 1, 131072, 32, 8, 128, 64, "e4m3", "bf16", gain=2.0),
        # A window of the latest keys and the first few tokens of contexts much longer than both.
        _attn("decode_first_keys", 16, 1, 30000, 32, 8, 128, 32, "bf16", "bf16", ragged=True, window=4096, first=4),
        # Five proposed tokens to verify, capped scores and a sink logit, odd lengths.
        _attn("verify_capped", 8, 5, 1999, 16, 4, 64, 16, "fp16", "fp16", ragged=True, softcap=30.0, sink=True, gain=3.0),
        # A chunk of a long prompt over the chunks before it, 8-bit pages.
        _attn("chunk_8bit", 1, 2048, 10240, 32, 8, 128, 64, "e4m3", "bf16", gain=2.0),
        # Chunks of odd lengths, padded, distance-biased, one key head a query head.
        _attn("chunk_ragged", 3, 777, 3001, 16, 16, 80, 16, "fp16", "fp16", ragged=True, short_q=True, slopes=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def _heads(rng):
    Hkv = rng.choice([1, 2, 4, 8, 16])
    return Hkv * rng.choice([1, 2, 3, 4, 5, 8, 16] if Hkv <= 2 else [1, 2, 4, 8] if Hkv <= 4 else [1, 2, 4]), Hkv


def draw(rng):
    kind = rng.choice(["rope", "rope_grad", "append", "append", "attn", "attn", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    Hq, Hkv = _heads(rng)
    if kind.startswith("rope"):
        D = rng.choice([64, 80, 96, 128, 128])
        sections = rng.choice({64: ["16,16", "8,12,12", "10,22"], 80: ["20,20", "8,16,16"], 96: ["16,16,16", "24,24"],
                               128: ["16,24,24", "32,32", "8,28,28", "16,16,16,16"]}[D])
        S = _spread(rng, 1, 8192)
        B = max(1, min(_spread(rng, 1, 64), (2 * 4099 * 40 * 128) // (S * (Hq + Hkv) * D)))
        S = min(S, max(1, (2 * 4099 * 40 * 128) // (B * (Hq + Hkv) * D)))
        c = _rope("", B, S, Hq, Hkv, D, sections, rng.random() < 0.4, dtype, rng.random() < 0.5, kind == "rope_grad")
    elif kind == "append":
        D = rng.choice([64, 80, 96, 128, 128, 128])
        T = rng.choice([1, 1, rng.randint(2, 8), _spread(rng, 9, 4096)])
        context = rng.choice([0, _spread(rng, 1, 2000), _spread(rng, 1, 2000)])
        most = 5 * (1700 + 333) * 4 * 128 * 2
        B = max(1, min(_spread(rng, 1, 64), most // ((T + context) * Hkv * D), most * 3 // (T * (Hq + Hkv) * D)))
        T = min(T, max(1, most // (B * Hkv * D) - context), max(1, most * 3 // (B * (Hq + Hkv) * D)))
        rot = rng.choice([D, D, D // 2])
        c = _append("", B, T, context, Hq, Hkv, D, rot, rng.choice([16, 16, 32, 64, 128]),
                    rng.choice(["e4m3", "e4m3", dtype]), dtype, interleaved=rng.random() < 0.3,
                    ragged=T > 1 and rng.random() < 0.6, axes=rng.random() < 0.3)
    else:
        D = rng.choice([64, 128, 128, 128, 80, 96, 112])
        Sq = rng.choice([1, 1, 1, rng.randint(2, 8), _spread(rng, 9, 200), _spread(rng, 200, 2048)])
        Skv = Sq + _spread(rng, 1, 131072 if rng.random() < 0.3 else 16384) - 1
        Skv = min(Skv, max(Sq, (64 * 8192 * 8 * 128) // (Hkv * D)), max(Sq, (2048 * 10240 * 32) // (Sq * Hq)))
        B = max(1, min(_spread(rng, 1, 64), (64 * 8192 * 8 * 128) // (Skv * Hkv * D), (2048 * 10240 * 32) // (Sq * Skv * Hq)))
        window = _spread(rng, 16, max(17, Skv)) if rng.random() < 0.35 else -1
        c = _attn("", B, Sq, Skv, Hq, Hkv, D, rng.choice([16, 16, 32, 64, 128]), rng.choice(["e4m3", "e4m3", dtype]), dtype,
                  ragged=rng.random() < 0.6, short_q=Sq > 1 and rng.random() < 0.4, window=window,
                  first=rng.choice([0, 1, 4, 4, 37]) if window >= 0 else 0,
                  softcap=rng.choice([0.0, 0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.2, sink=rng.random() < 0.25,
                  gain=rng.choice([1.0, 2.0, 3.0]))
    del c["name"]
    return c


# ------------------------------------------------------------------ the inputs
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn}


def _lengths(c):
    """Per sequence the cached tokens with the new ones, and how many are new, by the case alone."""
    r = random.Random(31 * c["B"] + 7 * c["D"] + c.get("Skv", 0) + c.get("context", 0))
    T = c["Sq"] if c["op"] == "attn" else c["T"]
    got = []
    for _ in range(c["B"]):
        t = r.randint(max(1, T // 3), T) if c.get("short_q") or (c["op"] == "append" and c["ragged"]) else T
        if c["op"] == "attn":
            n = r.randint(t, c["Skv"]) if c["ragged"] else c["Skv"]
        else:
            n = t + (r.randint(c["context"] // 2, c["context"]) if c["context"] else 0)
        got.append((n, t))
    return got


def _pairs(c):
    if c["op"] == "append":
        return c["rot"] // 2
    return sum(int(x) for x in c["sections"].split(","))


def _axis_of_pair(c):
    """Which axis turns each pair: sections one after another, or in turn from pair to pair while an axis has any left."""
    if c["op"] == "append":
        n = c["rot"] // 2
        sizes = [n - 2 * (n // 3), n // 3, n // 3]
    else:
        sizes = [int(x) for x in c["sections"].split(",")]
    if not c.get("mixed"):
        return [a for a, n in enumerate(sizes) for _ in range(n)]
    left, out = list(sizes), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                out.append(a)
                left[a] -= 1
    return out


def _frequencies(c):
    n = _pairs(c)
    return 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)


def _grid(c, T):
    """(axes, T) positions of tokens of a picture 24 wide (and, with three axes, of many pictures)."""
    t = torch.arange(T, device="cuda")
    if c["op"] != "append" and len(c["sections"].split(",")) == 2:
        return torch.stack((t // 24, t % 24))
    rows = [t // 576, t // 24 % 24, t % 24]
    while c["op"] != "append" and len(rows) < len(c["sections"].split(",")):
        rows.append(t % 7)
    return torch.stack(rows)


def _scale_of(largest):
    """The smallest power of two that brings these values within 448 (at least 2^-64)."""
    m, x = torch.frexp(largest)
    e = torch.where(largest > 0, x - 9 + (m > 0.875).to(x.dtype), torch.full_like(x, -64)).clamp(min=-64)
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)  # (2^e by its bits: a power function may be a step off)


def _table(g, B, per_row, spare):
    """(B, per_row) pages in no order, of B * per_row + spare."""
    return torch.randperm(B * per_row + spare, generator=g, device="cuda")[: B * per_row].view(B, per_row).to(torch.int32)


def _pages(g, c, n):
    """Keys or values of n pages, all slots filled: (pages, scales or None)."""
    x = torch.randn(n, c["Hkv"], c["page"], c["D"], generator=g, device="cuda", dtype=torch.bfloat16)
    x *= torch.exp(0.4 * torch.randn(c["D"], generator=g, device="cuda")).to(torch.bfloat16)  # some columns are larger
    if c["cache"] != "e4m3":
        return x.to(_TYPES[c["cache"]]), None
    scale = _scale_of(x.abs().amax((2, 3)).float())
    return (x / scale[:, :, None, None].to(torch.bfloat16)).to(torch.float8_e4m3fn), scale


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda").manual_seed(seed)
    t = _TYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    s = {"case": c}
    if c["op"].startswith("rope"):
        rows = (lambda H: (c["B"], c["S"], H, c["D"])) if c["op"] == "rope" else (lambda H: (c["B"], H, c["S"], c["D"]))
        s["q"], s["k"] = normal(*rows(c["Hq"])).to(t), normal(*rows(c["Hkv"])).to(t)
        s["freq"] = _frequencies(c).cuda()
        s["axes"] = torch.tensor(_axis_of_pair(c), dtype=torch.int32, device="cuda")
        at = torch.randint(0, 50000, (c["B"], 1), generator=g, device="cuda")  # how far each row is into its stream
        s["positions"] = (_grid(c, c["S"])[:, None] + at[None]).to(torch.int32).contiguous()
        return s
    B, D, P = c["B"], c["D"], c["page"]
    lens = _lengths(c)
    s["lens"] = torch.tensor([n for n, _ in lens], dtype=torch.int32, device="cuda")
    per_row = -(-max(n for n, _ in lens) // P)
    s["table"] = _table(g, B, per_row, 8)
    s["kc"], s["ks"] = _pages(g, c, B * per_row + 8)
    s["vc"], s["vs"] = _pages(g, c, B * per_row + 8)
    T = c["Sq"] if c["op"] == "attn" else c["T"]
    s["new"] = torch.tensor([n for _, n in lens], dtype=torch.int32, device="cuda") if any(n < T for _, n in lens) else None
    if c["op"] == "append":
        s["q"], s["k"], s["v"] = (normal(B, T, H, D).to(t) for H in (c["Hq"], c["Hkv"], c["Hkv"]))
        s["k"] *= 1.5
        s["freq"] = _frequencies(c).cuda()
        s["axes"] = s["positions"] = None
        if c["axes"]:
            s["axes"] = torch.tensor(_axis_of_pair(c), dtype=torch.int32, device="cuda")
            at = torch.randint(0, 50000, (B, 1), generator=g, device="cuda")
            s["positions"] = (_grid(c, T)[:, None] + at[None]).to(torch.int32).contiguous()
        return s
    s["q"] = (normal(B, c["Hq"], T, D) * c["gain"]).to(t)
    s["sink"] = normal(c["Hq"]) if c["sink"] else None
    s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, c["Hq"] + 1, device="cuda") / c["Hq"]) if c["slopes"] else None
    return s


# ------------------------------------------------------------------ plain forms
def _turn(x, cos, sin, rot, interleaved):
    """The first rot columns of x (fp32, (..., D)) rotated pair by pair."""
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : rot // 2], r[..., rot // 2:])
    u, w = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((r, x[..., rot:]), -1)


def _cos_sin(s, T, start=None):
    """(B, T, pairs) cosines and sines, from angles in 64 bits."""
    if s["axes"] is not None:
        pos = s["positions"][s["axes"].long()].permute(1, 2, 0)
    else:
        pos = (start[:, None] + torch.arange(T, device="cuda"))[..., None]
    angle = pos.double() * s["freq"]
    return angle.cos().float(), angle.sin().float()


def _plain_rope(s):
    c = s["case"]
    rot = 2 * _pairs(c)
    cos, sin = _cos_sin(s, c["S"])
    if c["op"] == "rope":  # (B, S, H, D) in, (B, H, S, D) out
        cos, sin = cos[:, :, None], sin[:, :, None]
    else:  # the gradient: the transposed rotation, (B, H, S, D) in, (B, S, H, D) out
        cos, sin = cos[:, None], -sin[:, None]
    turn = lambda x: _turn(x.float(), cos, sin, rot, c["interleaved"]).transpose(1, 2).to(x.dtype).contiguous()  # noqa: E731
    return turn(s["q"]), turn(s["k"])


def _dense(pages, scale, table):
    """(B, heads, positions, D) values of the pages of a table, in fp32."""
    x = pages[table.long()].float()  # (B, pages, heads, page, D)
    if scale is not None:
        x = x * scale[table.long()][..., None, None]
    return x.transpose(1, 2).flatten(2, 3)


def _put(pages, scale, table, x, new):
    """Rows x (B, heads, positions, D; fp32) into the pages where new (B, positions)."""
    at = table.long()
    B, H, S, D = x.shape
    P = pages.shape[2]
    x = x.view(B, H, S // P, P, D).transpose(1, 2)  # (B, pages, heads, page, D)
    new = new.view(B, S // P, 1, P, 1)
    if scale is None:
        pages[at] = torch.where(new, x.to(pages.dtype), pages[at])
        return
    was = scale[at]
    need = _scale_of((x.abs() * new).amax((3, 4)))
    begun = new[:, :, 0, 0, 0][..., None]  # the page's first slot is new: nothing of it is kept
    now = torch.where(new.any(3)[..., 0], torch.where(begun, need, torch.maximum(was, need)), was)
    old = pages[at].float() * was[..., None, None]
    pages[at] = (torch.where(new, x, old) / now[..., None, None]).clamp(-448.0, 448.0).to(pages.dtype)
    scale[at] = now


def _plain_append(s):
    c = s["case"]
    lens, T = s["lens"].long(), c["T"]
    start = lens - (T if s["new"] is None else s["new"].long())
    cos, sin = _cos_sin(s, T, start)
    turn = lambda x: _turn(x.transpose(1, 2).float(), cos[:, None], sin[:, None], c["rot"], c["interleaved"])  # noqa: E731
    q, k, v = turn(s["q"]).to(s["q"].dtype), turn(s["k"]), s["v"].transpose(1, 2).float()
    j = torch.arange(s["table"].shape[1] * c["page"], device="cuda")[None]
    new = (j >= start[:, None]) & (j < lens[:, None])
    row = (j - start[:, None]).clamp(0, T - 1)[:, None, :, None]
    _put(s["kc"], s["ks"], s["table"], torch.take_along_dim(k, row, 2), new)
    _put(s["vc"], s["vs"], s["table"], torch.take_along_dim(v, row, 2), new)
    if s["ks"] is None:
        return q, s["kc"], s["vc"]
    in_use = (j < lens[:, None])[:, None, :, None]
    read = lambda x, scale: (_dense(x, scale, s["table"]) * in_use).to(q.dtype)  # noqa: E731
    return q, read(s["kc"], s["ks"]), read(s["vc"], s["vs"])


def _plain_attention(s):
    c = s["case"]
    B, Sq, Hq, Hkv, D = c["B"], c["Sq"], c["Hq"], c["Hkv"], c["D"]
    k, v = _dense(s["kc"], s["ks"], s["table"]), _dense(s["vc"], s["vs"], s["table"])
    S = k.shape[2]
    x = (s["q"].float().view(B, Hkv, -1, D) @ k.transpose(2, 3)).view(B, Hkv, Hq // Hkv, Sq, S) * (1.0 / math.sqrt(D))
    if c["softcap"]:
        x = torch.tanh(x / c["softcap"]) * c["softcap"]
    lens = s["lens"].long()
    n_q = torch.full_like(lens, Sq) if s["new"] is None else s["new"].long()
    i, j = torch.arange(Sq, device="cuda"), torch.arange(S, device="cuda")
    place = (lens - n_q)[:, None, None] + i[None, :, None]
    if s["slopes"] is not None:
        x = x - s["slopes"].view(1, Hkv, -1, 1, 1) * (place - j).abs()[:, None, None]
    see = (j <= place) & (i[None, :, None] < n_q[:, None, None])
    if c["window"] >= 0:
        see = see & ((j >= place - c["window"]) | (j < c["first"]))
    x = x.masked_fill(~see[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    sink = None if s["sink"] is None else s["sink"].view(1, Hkv, -1, 1, 1)
    m = m.masked_fill(m == -math.inf, 0.0) if sink is None else torch.maximum(m, sink)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    if sink is not None:
        total = total + torch.exp(sink - m)
    o = (p / total.masked_fill(total == 0, 1.0)).view(B, Hkv, -1, S) @ v
    return o.view(B, Hq, Sq, D).to(s["q"].dtype), (m + total.log()).view(B, Hq, Sq)


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if own:
        import attention_backward_sdpa_gb300 as sdpa
        if c["op"].startswith("rope"):
            kw = dict(positions=s["positions"], axes=s["axes"], interleaved=c["interleaved"])
            if c["op"] == "rope":
                return sdpa.rope_fwd(s["q"].transpose(1, 2), s["k"].transpose(1, 2), s["freq"], **kw)
            out = [torch.empty(c["B"], c["S"], H, c["D"], dtype=s["q"].dtype, device="cuda") for H in (c["Hq"], c["Hkv"])]
            sdpa.rope_bwd(s["q"], s["k"], s["freq"], q_out=out[0].transpose(1, 2), k_out=out[1].transpose(1, 2), **kw)
            return tuple(out)
        cache = sdpa.KVCache(s["kc"], s["vc"], s["ks"], s["vs"])
        if c["op"] == "append":
            q = sdpa.kv_append(s["k"].transpose(1, 2), s["v"].transpose(1, 2), cache, s["table"], s["lens"],
                               seq_q_lens=s["new"], q=s["q"].transpose(1, 2), inv_freq=s["freq"],
                               positions=s["positions"], axes=s["axes"], interleaved=c["interleaved"])
            if s["ks"] is None:
                return q, s["kc"], s["vc"]
            return (q, *sdpa.kv_gather(cache, s["table"], s["lens"], dtype=q.dtype))
        return sdpa.sdpa_fwd_cached(s["q"], cache, s["table"], s["lens"], causal=True, seq_q_lens=s["new"],
                                    window_left=c["window"], first_keys=c["first"], softcap=c["softcap"],
                                    alibi_slopes=s["slopes"], sink=s["sink"])
    if c["op"].startswith("rope"):
        return _plain_rope(s)
    return _plain_append(s) if c["op"] == "append" else _plain_attention(s)


def _visible(c):
    """Per sequence: (keys that some row reads, pairs of a row and a key it sees)."""
    got = []
    for n, t in _lengths(c):
        rows = [(min(c["first"], max(0, p - c["window"])) if c["window"] >= 0 else 0,
                 max(0, p - c["window"]) if c["window"] >= 0 else 0, p + 1) for p in range(n - t, n)]
        low = min(r[1] for r in rows)
        got.append((n - low + min(low, c["first"]), sum(f + hi - lo for f, lo, hi in rows)))
    return got


def work(case):
    c = case
    if c["op"].startswith("rope"):
        n = c["B"] * c["S"] * (c["Hq"] + c["Hkv"])
        return {"bytes": n * c["D"] * 2 * 2, "flops": n * _pairs(c) * 6}
    size = 1 if c["cache"] == "e4m3" else 2
    if c["op"] == "append":
        new, row = sum(t for _, t in _lengths(c)), c["D"]
        io = new * row * ((2 * c["Hq"] + 2 * c["Hkv"]) * 2 + 2 * c["Hkv"] * size)
        if c["cache"] == "e4m3":  # read back: the codes of the cached tokens, and 16-bit rows for every position
            per_row = -(-max(n for n, _ in _lengths(c)) // c["page"]) * c["page"]
            io += 2 * c["Hkv"] * row * (sum(n for n, _ in _lengths(c)) + 2 * c["B"] * per_row)
        return {"bytes": io, "flops": new * (c["Hq"] + c["Hkv"]) * c["rot"] * 3}
    seen = _visible(c)
    rows = c["B"] * c["Hq"] * c["Sq"]
    io = sum(n for n, _ in seen) * c["Hkv"] * c["D"] * 2 * size + rows * (c["D"] * 4 + 4)
    return {"bytes": io, "flops": 4 * c["D"] * c["Hq"] * sum(p for _, p in seen)}


# ------------------------------------------------------------------ in 64 bits
def _exact_turn(x, angle, interleaved):
    """x (..., D) in 64 bits with its first 2 * angle.shape[-1] columns as complex numbers turned by the angle."""
    n = angle.shape[-1]
    first = slice(0, 2 * n, 2) if interleaved else slice(0, n)
    second = slice(1, 2 * n, 2) if interleaved else slice(n, 2 * n)
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_angles(s, b, T, start):
    if s["positions"] is not None:
        which = _axis_of_pair(s["case"])
        pos = torch.stack([s["positions"][a, b] for a in which], -1).double()
    else:
        pos = torch.arange(start, start + T, device="cuda", dtype=torch.float64)[:, None]
    return pos * s["freq"]


def _power_of_two(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_code(x):
    """Values within 448 rounded to the nearest of 3 fraction bits, ties to even, multiples of 2^-9 at the low end."""
    size = x.abs().clamp(max=448.0)
    _, e = torch.frexp(size.clamp(min=2.0 ** -6))
    step = _power_of_two(e - 4)
    return torch.sign(x) * torch.round(size / step) * step


def _exact_page(old, was, x, lo, hi):
    """One page's (heads, page, D) values after rows [lo, hi) became x (heads, hi - lo, D)."""
    m, e = torch.frexp(x.abs().amax((1, 2)) / 448.0)  # the ratio's logarithm rounded up
    need = _power_of_two(torch.where(m == 0.5, e - 1, e).clamp(min=-64))
    unit = (need if lo == 0 else torch.maximum(need, was.double()))[:, None, None]
    return torch.cat((_exact_code(old[:, :lo] / unit) * unit, _exact_code(x / unit) * unit, _exact_code(old[:, hi:] / unit) * unit), 1)


def exact(case, seed):
    c = case
    s = prepare(dict(c), seed)
    if c["op"].startswith("rope"):
        out = []
        for name in ("q", "k"):
            x = s[name].double()
            x = x if c["op"] == "rope" else x.transpose(1, 2)  # (B, S, H, D)
            sign = 1.0 if c["op"] == "rope" else -1.0
            y = torch.stack([_exact_turn(x[b], sign * _exact_angles(s, b, c["S"], 0)[:, None], c["interleaved"])
                             for b in range(c["B"])])
            out.append(y.transpose(1, 2).contiguous() if c["op"] == "rope" else y)
        return tuple(out)
    B, D, P, Hkv = c["B"], c["D"], c["page"], c["Hkv"]
    table = s["table"].tolist()
    if c["op"] == "append":
        qs, dense, pages = [], {"k": [], "v": []}, {}
        for b, (n, t) in enumerate(_lengths(c)):
            start = n - t
            angle = _exact_angles(s, b, c["T"], start)[:, None]
            qs.append(_exact_turn(s["q"][b].double(), angle, c["interleaved"]).transpose(0, 1))
            new = {"k": _exact_turn(s["k"][b].double(), angle, c["interleaved"])[:t], "v": s["v"][b, :t].double()}
            for name in ("k", "v"):
                codes, scale = s[name + "c"], s[name + "s"]
                if scale is None:
                    at = torch.arange(start, n, device="cuda")
                    pages.setdefault(name, codes.double())
                    pages[name][s["table"][b].long()[at // P], :, at % P] = new[name]
                    continue
                got = torch.zeros(Hkv, len(table[b]) * P, D, dtype=torch.float64, device="cuda")
                for p in range(-(-n // P)):
                    was = scale[table[b][p]]
                    old = codes[table[b][p]].double() * was.double()[:, None, None]
                    lo, hi = max(0, start - p * P), min(P, n - p * P)
                    if lo < hi:
                        old = _exact_page(old, was, new[name][p * P + lo - start: p * P + hi - start].transpose(0, 1), lo, hi)
                    got[:, p * P: p * P + hi] = old[:, :hi]
                dense[name].append(got)
        q = torch.stack(qs)
        return (q, pages["k"], pages["v"]) if pages else (q, torch.stack(dense["k"]), torch.stack(dense["v"]))
    Hq, Sq = c["Hq"], c["Sq"]
    G = Hq // Hkv
    o = torch.zeros(B, Hq, Sq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Hq, Sq), -math.inf, dtype=torch.float64, device="cuda")
    if s["sink"] is not None:
        lse[:] = s["sink"].double()[None, :, None]
    for b, (n, t) in enumerate(_lengths(c)):
        j = torch.arange(n, device="cuda")
        place = torch.arange(n - t, n, device="cuda")[:, None]
        keep = j <= place
        if c["window"] >= 0:
            keep &= (j >= place - c["window"]) | (j < c["first"])
        at = s["table"][b].long()[j // P], j % P
        for h in range(Hkv):
            k, v = s["kc"][at[0], h, at[1]].double(), s["vc"][at[0], h, at[1]].double()
            if s["ks"] is not None:
                k, v = k * s["ks"][at[0], h].double()[:, None], v * s["vs"][at[0], h].double()[:, None]
            for g in range(G):
                head = h * G + g
                z = s["q"][b, head, :t].double() @ k.T / math.sqrt(D)
                if c["softcap"]:
                    z = c["softcap"] * torch.tanh(z / c["softcap"])
                if s["slopes"] is not None:
                    z = z - s["slopes"][head].double() * (place - j).abs()
                z = torch.where(keep, z, -math.inf)
                if s["sink"] is not None:
                    z = torch.cat((z, s["sink"][head].double().expand(t, 1)), 1)
                lse[b, head, :t] = torch.logsumexp(z, -1)
                o[b, head, :t] = torch.softmax(z, -1)[:, :n] @ v
    return o, lse
