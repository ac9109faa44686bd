"""Plain 64-bit attention with modified scores on the CPU (torch, one (batch, head)
at a time), and error bounds of the kernels derived from it.

The bounds are elementwise and count roundings: u is half a step of the io type
(finfo.eps / 2), the scores carry fp32 accumulation error. With A = P |V| and so on
(magnitude sums), for every element:

  |O_gpu - O|   <= u (P|V| [P is rounded for the PV product] + |O| [O is rounded])
                   + 2 e (P|V|)           e: error of a score, in the numerator and the sum
  |dV_gpu - dV| <= u (P^T|dO| [P rounded] + |dV|) + e P^T|dO|
  |dS_gpu - dS| <= E = u |dS| [rounded for dQ, dK] + e |dS| + P (e_d + e_f |dP - delta|)
  |dQ_gpu - dQ| <= scale E |K| + u |dQ|
  |dK_gpu - dK| <= scale E^T |Q| + u |dK|

e   = g (D + 16) max sum|q k| scale + g (|x| + |LSE|) + g |slope| distance (products and sums of D
      terms, the exponent's argument, the distance bias), g = 2^-23 (a unit of fp32: the tensor
      core's accumulation may truncate)
e_d = g (D + 16) (sum |dO V| + sum |dO O|),  e_f = 2^-20 (1 - tanh^2 from tanh to 2 units)
and sums over n terms add n g relative. fp16 weights below 2^-14 are subnormal:
each P and dS may be off by 2^-25 absolutely.
"""
from __future__ import annotations

import math

import torch

G23 = 2.0 ** -23


def doc_ranges(doc_ids, prefix_lens, causal, S):
    """Per row [lo, hi) of documents = runs of equal ids, from the definition (lists)."""
    B = len(doc_ids)
    out = []
    for b in range(B):
        ids, rows = doc_ids[b], []
        for i in range(S):
            lo = i
            while lo > 0 and ids[lo - 1] == ids[i]:
                lo -= 1
            hi = i + 1
            while hi < S and ids[hi] == ids[i]:
                hi += 1
            if causal:
                pre = 0
                if prefix_lens is not None:
                    pre = prefix_lens[b][i] if isinstance(prefix_lens[b], list) else prefix_lens[b]
                hi = min(hi, max(i + 1, lo + max(pre, 0)))
            rows.append((lo, hi))
        out.append(rows)
    return out


def visible(Sq, Skv, Lq, Lk, causal=False, bottom_right=False, window_left=-1, window_right=-1, rows=None):
    i, j = torch.arange(Sq)[:, None], torch.arange(Skv)[None]
    diag = Lk - Lq if bottom_right else 0
    see = (i < Lq) & (j < Lk)
    if causal:
        see = see & (j <= i + diag + max(window_right, 0))
    if window_left >= 0:
        see = see & (j >= i + diag - window_left)
    if rows is not None:
        r = torch.tensor(rows)
        see = see & (j >= r[:, :1]) & (j < r[:, 1:])
    return see, diag


class Case:
    """One problem: fp32-exact CPU tensors (already rounded to the io type) and options."""

    def __init__(self, B, Hq, Hkv, Sq, Skv, Dqk, Dv, io=torch.bfloat16, seed=0, gain=1.0, softcap=0.0,
                 slopes=None, rows=None, lens_q=None, lens_kv=None, sink=False, **mask):
        g = torch.Generator().manual_seed(seed)
        n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.q, self.k = (n(B, Hq, Sq, Dqk) * gain).to(io), n(B, Hkv, Skv, Dqk).to(io)
        self.v, self.do = n(B, Hkv, Skv, Dv).to(io), n(B, Hq, Sq, Dv).to(io)
        self.sink = n(Hq) if sink else None
        self.B, self.Hq, self.Hkv, self.Sq, self.Skv, self.Dqk, self.Dv, self.io = B, Hq, Hkv, Sq, Skv, Dqk, Dv, io
        self.softcap, self.rows, self.mask = softcap, rows, mask
        self.slopes = None if slopes is None else torch.tensor(slopes, dtype=torch.float32)
        self.lens_q, self.lens_kv = lens_q, lens_kv
        self.scale = float(torch.tensor(1.0 / math.sqrt(Dqk), dtype=torch.float32))  # as the library holds it
        self.u = torch.finfo(io).eps / 2

    def _lens(self, b):
        return (self.Sq if self.lens_q is None else self.lens_q[b],
                self.Skv if self.lens_kv is None else self.lens_kv[b])

    def head(self, b, h):
        """(q, k, v, x with -inf where masked, dx/dy, error of a score)."""
        kh = h // (self.Hq // self.Hkv)
        q, k, v = self.q[b, h].double(), self.k[b, kh].double(), self.v[b, kh].double()
        scale = self.scale
        y = q @ k.T * scale
        size = (q.abs() @ k.abs().T).max().item() * scale if self.Skv and self.Sq else 0.0
        f, x = torch.ones_like(y), y
        if self.softcap:
            t = torch.tanh(y / self.softcap)
            x, f = self.softcap * t, 1 - t * t
        see, diag = visible(self.Sq, self.Skv, *self._lens(b), rows=None if self.rows is None else self.rows[b],
                            **self.mask)
        e = G23 * (self.Dqk + 16) * size
        if self.slopes is not None:
            d = (torch.arange(self.Sq)[:, None] + diag - torch.arange(self.Skv)[None]).abs().double()
            x = x - self.slopes[h].double() * d
            e += G23 * (self.slopes[h].abs().item() * (d * see).max().item() if d.numel() else 0.0)
        big = x[see].abs().max().item() if see.any() else 0.0
        e += 2 * G23 * big
        return q, k, v, torch.where(see, x, -math.inf), f, e

    def forward(self):
        """O, LSE and the bounds of both."""
        o = torch.zeros(self.B, self.Hq, self.Sq, self.Dv, dtype=torch.float64)
        lse = torch.full((self.B, self.Hq, self.Sq), -math.inf, dtype=torch.float64)
        bo, bl = torch.zeros_like(o), torch.zeros_like(lse)
        sub = 2.0 ** -25 if self.io == torch.float16 else 0.0
        for b in range(self.B):
            for h in range(self.Hq):
                q, k, v, x, f, e = self.head(b, h)
                if self.sink is not None:
                    z = torch.cat((x, self.sink[h].double().expand(self.Sq, 1)), 1)
                else:
                    z = x
                if z.shape[1] == 0:
                    continue
                lse[b, h] = torch.logsumexp(z, 1)
                p = torch.nan_to_num(torch.exp(x - lse[b, h][:, None]), nan=0.0)
                Lq = self._lens(b)[0]
                if self.sink is not None:
                    lse[b, h, Lq:] = self.sink[h].double()
                o[b, h] = p @ v
                a = p @ v.abs()
                e = e + G23 * self.Skv
                bo[b, h] = self.u * 1.01 * (a + o[b, h].abs()) + 2 * e * a + 1e-30
                # an fp16 weight below 2^-14 relative to the running reference, which is at most
                # the row's maximum, so the sum that divides it is at least 1 (256: to spare)
                bo[b, h] += sub * 256 * v.abs().sum(0)
                # O itself below 2^-14 is rounded to multiples of 2^-24: half a step is 2^-25, for
                # O = 8.0993e-9 (0.136 steps) rounded to 0 more than the relative terms above allow
                bo[b, h] += sub
                fin = torch.nan_to_num(lse[b, h], neginf=0.0).abs()
                bl[b, h] = e + 4 * G23 * (1 + fin)
        return o, lse, bo, bl

    def backward(self, o, lse):
        """(dq, dk, dv) from the rounded o and fp32 lse that the library is given, with bounds."""
        z = lambda t: torch.zeros(t.shape, dtype=torch.float64)  # noqa: E731
        dq, dk, dv, bq, bk, bv = z(self.q), z(self.k), z(self.v), z(self.q), z(self.k), z(self.v)
        sub = 2.0 ** -25 if self.io == torch.float16 else 0.0
        G = self.Hq // self.Hkv
        for b in range(self.B):
            for h in range(self.Hq):
                kh = h // G
                q, k, v, x, f, e = self.head(b, h)
                do, oo, l = self.do[b, h].double(), o[b, h].double(), lse[b, h].double()
                alive = torch.isfinite(l)
                e = e + 2 * G23 * (l[alive].abs().max().item() if alive.any() else 0.0) + G23 * 4
                p = torch.where(alive[:, None], torch.exp(x - torch.nan_to_num(l, neginf=0.0)[:, None]), 0.0)
                dp, delta = do @ v.T, (do * oo).sum(1, keepdim=True)
                ds = p * (dp - delta) * f
                ed = G23 * (self.Dv + 16) * (do.abs() @ v.abs().T + (do * oo).abs().sum(1, keepdim=True))
                E = (self.u * 1.01 + e) * ds.abs() + p * (ed + 2.0 ** -20 * (dp - delta).abs()) + sub * (p > 0)
                n = G23 * max(self.Sq, self.Skv)
                pv = p.T @ do.abs()
                dv[b, kh] += p.T @ do
                bv[b, kh] += (self.u * 1.01 + e + n) * pv + sub * (p > 0).double().T @ do.abs()
                dq[b, h] = ds @ k * self.scale
                bq[b, h] = self.scale * ((E + n * ds.abs()) @ k.abs()) + self.u * 1.01 * dq[b, h].abs() + 1e-30
                dk[b, kh] += ds.T @ q * self.scale
                bk[b, kh] += self.scale * ((E + n * ds.abs()).T @ q.abs())
        bk += self.u * 1.01 * dk.abs() + 1e-30
        bv += self.u * 1.01 * dv.abs() + 1e-30
        if sub:  # rounding into fp16's subnormal range
            for t in (bq, bk, bv):
                t += 2 * sub
        return (dq, dk, dv), (bq, bk, bv)


def assert_within(name, got, ref, bound):
    got, ref = got.double().cpu(), ref.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    inf = torch.isinf(ref)
    assert torch.equal(torch.isinf(got) & (got == ref), inf), f"{name}: infinities differ"
    assert not torch.isnan(got).any(), f"{name}: NaN"
    over = ((got - ref).abs() - bound)[~inf]
    if over.numel():
        w = over.max().item()
        assert w <= 0, f"{name}: {w:.3e} over its bound (largest error {(got - ref)[~inf].abs().max().item():.3e})"
