"""The gated scan and a beam search's selection in 64 bits, for the tests.

The gated scan's results carry a bound on f32's error with them (`Ball`): every product and sum that the
definition writes adds 2 U of its result (one rounding where it is computed as written, one more where a
kernel groups three factors or terms otherwise, or joins spans of tokens), and the functions add theirs:

* exp(-|r|) by a power of two: log2(e) |r| has two roundings, which is 2 U |r| of the result, and the unit is
  good to 2^-22; a reciprocal to 2^-23. So sigma(r) = 1 / (1 + exp(-|r|)) or exp(-|r|) / (1 + exp(-|r|)) and
  1 - sigma(r) are each good to ((2 |r| + 8) U + 2^-21) of themselves (8 U for the sum, the products around
  the reciprocal, and a reciprocal shared by three gates; 2^-21 for the exponential, the reciprocal, and the other gates').
* 1 - exp(-u) below u = 1/4 by its series: 4 U of itself (one for the terms left out); above, from exp(-u), good to (2 u + 2) U + 2^-22 of
  itself. An error of u moves exp(-u) by u times its relative error, 1 - exp(-u) by at most that.
* 1 / sqrt(q): 2^-22, and half of q's error.

The recurrences' sums are made in spans (a warp's tokens, a CTA's, a cluster's), whose sums can be larger than
the states where terms of both signs meet: one token whose gradient all but cancels the one from behind it has a
span's sum a dh, rounded to U |a dh|, and only then a g added. So their roundings are counted against the
recurrence of absolute values, M' = |a| M + |b|, which no span's sum exceeds: for a token at most one for its term in the
span, one for the span's product of decays, and two where the span is joined to others, 4 U M' (and, for
the adjoint, one more addition of its own, 2 U (|dh| + M)). The terms' own errors go in as before: every
grouping is the same function of the computed a and b.
"""
import torch

import seq_ref as R

F64 = torch.float64
U = R.U


class Ball:
    """A value and a bound on f32's error in it."""

    def __init__(self, v, e=None):
        self.v, self.e = v, torch.zeros_like(v) if e is None else e

    def __mul__(self, o):
        v = self.v * o.v
        e = self.v.abs() * o.e + o.v.abs() * self.e + self.e * o.e
        return Ball(v, e + 2 * U * (v.abs() + e))

    def __add__(self, o):
        v, e = self.v + o.v, self.e + o.e
        return Ball(v, e + 2 * U * (v.abs() + e))

    def __sub__(self, o):
        return self + Ball(-o.v, o.e)

    def at(self, t):
        return Ball(self.v[:, t], self.e[:, t])

    def where(self, mask):
        z = torch.zeros((), dtype=F64)
        return Ball(torch.where(mask, self.v, z), torch.where(mask, self.e, z))


def sigmoid(x):
    """sigma(x) and 1 - sigma(x)."""
    rel = (2 * x.abs() + 8) * U + 2.0 ** -21
    s, c = torch.sigmoid(x), torch.sigmoid(-x)
    return Ball(s, s * rel), Ball(c, c * rel)


def step(a, h, b, m):
    """a h + b, made in spans; m and its next value are the recurrence of absolute values."""
    m = a.v.abs() * m + b.v.abs()
    e = a.v.abs() * h.e + h.v.abs() * a.e + a.e * h.e + b.e
    return Ball(a.v * h.v + b.v, e + 4 * U * (m + e)), m


def stack(balls):
    return Ball(torch.stack([b.v for b in balls], 1), torch.stack([b.e for b in balls], 1))


class GatedCase:
    """Inputs as the calls take them, on the CPU; h0 is None or the first states."""

    def __init__(self, x, r, i=None, z=None, rate=None, h0=None, lens=None):
        self.mask = R.live_mask(lens, x.shape[0], x.shape[1])[..., None]
        w = lambda t: None if t is None else R.zeroed(t, self.mask)  # noqa: E731
        self.x, self.r, self.i, self.z = w(x), w(r), w(i), w(z)
        self.rate = None if rate is None else rate.to("cpu", F64)
        b, length, d = x.shape
        self.h0 = torch.zeros(b, d, dtype=F64) if h0 is None else h0.to("cpu", F64)
        self.length = length

    def gates(self):
        self.s, self.c = s, c = sigmoid(self.r)
        self.rw = None
        if self.rate is None:
            a, w = c, s
        else:
            u = Ball(self.rate) * s
            a, d = torch.exp(-u.v), -torch.expm1(-u.v)
            low, high = u.v < 0.26, u.v > 0.24
            far = a * ((2 * u.v + 2) * U + 2.0 ** -22)
            ea = a * u.e + torch.where(low, 4 * U * d + U, 0.0) + torch.where(high, far, 0.0)
            rel = torch.where(u.v > 0, u.e / u.v.clamp(min=1e-300), torch.zeros((), dtype=F64))
            ed = d * rel + torch.where(low, 4 * U * d, 0.0) + torch.where(high, far + U, 0.0)
            a, d = Ball(a, ea), Ball(d, ed)
            two_less = Ball(2 - d.v, d.e + U * 2)
            q = d * two_less
            rw = 1 / torch.sqrt(q.v)
            self.rw = Ball(rw, rw * (q.e / q.v / 2 * 1.01 + 2.0 ** -22))
            w = q * self.rw
        self.a, self.w = a.where(self.mask), w.where(self.mask)
        self.a.v[~self.mask.expand_as(a.v)] = 1.0
        x = Ball(self.x)
        self.si = self.ci = None
        if self.i is not None:
            self.si, self.ci = sigmoid(self.i)
            x = x * self.si
        self.v = x
        self.b = (self.w * x).where(self.mask)

    def forward(self):
        self.gates()
        h, past = Ball(self.h0), []
        size = self.h0.abs()
        hs = []
        for t in range(self.length):
            past.append(h)
            m = self.mask[:, t]
            new, grown = step(self.a.at(t), h, self.b.at(t), size)
            h, size = Ball(torch.where(m, new.v, h.v), torch.where(m, new.e, h.e)), torch.where(m, grown, size)
            hs.append(h)
        self.final = h
        zero = Ball(torch.zeros_like(self.x))
        self.h, self.past = (stack(hs), stack(past)) if hs else (zero, zero)
        y = self.h
        if self.z is not None:
            self.sz, self.cz = sigmoid(self.z)
            y = self.h * (Ball(self.z) * self.sz)
        self.out = y.where(self.mask)
        return self.out, self.final

    def gradient(self, dout, dfinal=None):
        self.forward()
        dy = Ball(R.zeroed(dout, self.mask))
        got, dh = {}, dy
        if self.z is not None:
            z = Ball(self.z)
            dh = dy * (z * self.sz)
            one = Ball(torch.ones_like(self.z))
            got["dz"] = (dy * self.h * (self.sz * (z * self.cz + one))).where(self.mask)
        carry = Ball(torch.zeros_like(self.h0) if dfinal is None else dfinal.to("cpu", F64))
        gs, size = [], carry.v.abs()
        zero = Ball(torch.zeros_like(self.h0))
        for t in reversed(range(self.length)):
            g = dh.at(t) + carry
            grown = dh.at(t).v.abs() + size
            g = Ball(g.v, g.e + 2 * U * grown)
            m = self.mask[:, t]
            new, grown = step(self.a.at(t), g, zero, grown)
            gs.append(g.where(m))
            carry, size = Ball(torch.where(m, new.v, carry.v), torch.where(m, new.e, carry.e)), torch.where(m, grown, size)
        got["dinit"] = carry
        g = stack(gs[::-1]) if gs else Ball(torch.zeros_like(self.x))
        dv = g * self.w
        got["dx"] = dv if self.i is None else dv * self.si
        if self.i is not None:
            got["di"] = dv * self.v * self.ci
        if self.rate is None:
            got["dr"] = g * (self.v - self.past) * (self.s * self.c)
        else:
            e = (g * (self.v * (self.a * self.a) * (self.s * self.rw) - self.past * self.a * self.s)).where(self.mask)
            got["dr"] = (e * Ball(self.rate) * self.c).where(self.mask)
            n = e.v.shape[0] * e.v.shape[1]
            got["drate"] = Ball(e.v.sum((0, 1)), e.e.sum((0, 1)) + n * U * e.v.abs().sum((0, 1)))
        return got


def check(name, got, want):
    R.assert_within(name, got, want.v, want.e)


# ---- a beam search's selection ---------------------------------------------------------------------


def beam_select(logits, k_out, prior=None, finished=None, eos=-1, slots=None):
    """Sequence by sequence, over all continuations. Returns tokens, parents, scores (64 bits), finished, and
    with slots their new row and the copies."""
    b, k, v = logits.shape
    x = logits.detach().cpu().to(F64)
    x = torch.where(x.isnan(), float("-inf"), x).clamp(max=torch.finfo(logits.dtype).max)
    prior = torch.zeros(b, k, dtype=F64) if prior is None else prior.cpu().to(F64)
    prior = torch.where(prior.isnan(), float("-inf"), prior).clamp(max=torch.finfo(torch.float32).max)
    ended = torch.zeros(b, k, dtype=torch.bool) if finished is None else finished.cpu() != 0
    r = dict(tokens=[], parents=[], scores=[], finished=[], slots=[], src=[], dst=[])
    for n in range(b):
        rows = []
        for j in range(k):
            top = x[n, j].max()
            if ended[n, j]:
                row = torch.full((v,), float("-inf"), dtype=F64)
                row[eos] = prior[n, j]
            elif top == float("-inf") or prior[n, j] == float("-inf"):
                row = torch.full((v,), float("-inf"), dtype=F64)
            else:
                y = x[n, j] - top
                row = prior[n, j] + (y - torch.log(torch.exp(y).sum()))
            rows.append(row)
        score = torch.cat(rows)
        order = torch.sort(score, descending=True, stable=True).indices[:k_out].tolist()  # ties in order
        parents, tokens = [q // v for q in order], [q % v for q in order]
        r["parents"].append(parents)
        r["tokens"].append(tokens)
        r["scores"].append([score[q].item() for q in order])
        r["finished"].append([int(bool(ended[n, p]) or t == eos) for p, t in zip(parents, tokens)])
        if slots is None:
            continue
        old = slots[n].tolist()
        gone = [old[j] for j in range(len(old)) if j not in parents]
        now, src, dst = [], [], []
        for j, p in enumerate(parents):
            if p in parents[:j]:
                now.append(gone.pop(0))
                src.append(old[p])
                dst.append(now[-1])
            else:
                now.append(old[p])
                src.append(-1)
                dst.append(-1)
        r["slots"].append(now + gone)
        r["src"].append(src)
        r["dst"].append(dst)
    return {name: torch.tensor(rows, dtype=F64 if name == "scores" else torch.int64) for name, rows in r.items() if rows}
