"""The sequence-model operators in 64 bits, token by token, for the tests.

Each reference also runs on absolute values (`magnitude`), which gives for every
result the sum of the absolute values of its terms: rounding errors of sums are
measured against that. The bounds that the tests use:

* U = 2^-24 is f32's unit roundoff; a sum of k f32 terms in any fixed order is
  off by at most k U sum|terms| (to first order).
* EX = 2^-21 bounds the relative error of one evaluated exponential or
  reciprocal, rounding of its argument included, for the arguments used here
  (an argument x of exp is off by 2 U |x|, and |x| exp(-|x|) is below 0.4).
* a result stored as bf16 / f16 / f32 has one more rounding, EPS[dtype] relative
  (and f16's subnormal spacing).
"""
import torch

F64 = torch.float64
U = 2.0 ** -24
EX = 2.0 ** -21
EPS = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}  # unit roundoff: 24, 8, 11 bits
TINY = {torch.float32: 2.0 ** -126, torch.bfloat16: 2.0 ** -126, torch.float16: 2.0 ** -25}


def assert_within(name, got, want, slack):
    """|got - want| <= slack (the f32 part) + one rounding to got's type."""
    want = want.to("cpu", F64)
    got64 = got.detach().to("cpu").to(F64)
    assert got64.shape == want.shape, (name, got64.shape, want.shape)
    bound = slack.to("cpu", F64) * (1 + EPS[got.dtype]) + EPS[got.dtype] * want.abs() + TINY[got.dtype]
    err = (got64 - want).abs()
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(int(v[0]) for v in bad.nonzero(as_tuple=True))
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.numel()} out of bounds; first at {i}: got {got64[i]} "
                             f"want {want[i]} err {err[i]:.3g} bound {bound[i]:.3g}")


def sigmoid(x):
    return torch.sigmoid(x)


def softplus(x):
    return torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))


def live_mask(lens, batch, length):
    t = torch.arange(length)
    n = torch.full((batch,), length) if lens is None else lens.to("cpu").long().clamp(0, length)
    return t[None, :] < n[:, None]


def zeroed(x, mask):
    """x in 64 bits with what lies past a sequence's end replaced by zeros (never multiplied: it may be NaN)."""
    x = x.detach().to("cpu").to(F64)
    while mask.dim() < x.dim():
        mask = mask[..., None]
    return torch.where(mask, x, torch.zeros((), dtype=F64))


# ---- convolution ---------------------------------------------------------------------------------
def conv(x, w, bias, silu, before, mask):
    """out, the inputs with those before token 0, and p."""
    b, length, d = x.shape
    width = w.shape[1]
    px = torch.cat([before, x], 1)
    p = torch.zeros(b, length, d, dtype=F64) + (bias if bias is not None else 0.0)
    for k in range(width):
        p = p + w[:, k] * px[:, k:k + length]
    out = p * sigmoid(p) if silu else p
    return torch.where(mask[..., None], out, 0.0), px, p


def conv_grad(x, w, bias, silu, before, mask, dout, slope=None):
    """dx, dweight, dbias, dstate; `slope` replaces the activation's derivative."""
    width, length = w.shape[1], x.shape[1]
    _, px, p = conv(x, w, bias, silu, before, mask)
    if slope is None:
        s = sigmoid(p)
        slope = s * (1 + p * (1 - s)) if silu else torch.ones_like(p)
    g = torch.where(mask[..., None], dout * slope, 0.0)
    dpx = torch.zeros_like(px)
    dw = torch.zeros_like(w)
    for k in range(width):
        dpx[:, k:k + length] += w[:, k] * g
        dw[:, k] = (g * px[:, k:k + length]).sum((0, 1))
    return torch.where(mask[..., None], dpx[:, width - 1:], 0.0), dw, g.sum((0, 1)), dpx[:, :width - 1]


# ---- scan -------------------------------------------------------------------------------------------
def by_channel(x, dim):
    """[batch, len, groups, n] to [batch, len, dim, n]."""
    return x.repeat_interleave(dim // x.shape[2], 2)


def scan(u, step, a, B, C, D, gate, h0, mask):
    """out, y, the states after each token, from step sizes and decays; B and C by channel. Masked tokens have step 0, a 1."""
    b, length, d = u.shape
    h, hs, ys = h0, [], []
    for t in range(length):
        h = a[:, t] * h + (step[:, t] * u[:, t])[..., None] * B[:, t]
        hs.append(h)
        ys.append((C[:, t] * h).sum(-1) + D * u[:, t])
    hs = torch.stack(hs, 1) if length else torch.zeros(b, 0, *h0.shape[1:], dtype=F64)
    y = torch.stack(ys, 1) if length else torch.zeros(b, 0, d, dtype=F64)
    return torch.where(mask[..., None], y * gate, 0.0), y, hs


def scan_grad(u, step, a, A, B, C, D, gate, dgate, slope, h0, mask, dout, dfinal, groups):
    """Every gradient, by the adjoint recurrence."""
    b, length, d = u.shape
    n = A.shape[1]
    _, y, hs = scan(u, step, a, B, C, D, gate, h0, mask)
    dout = torch.where(mask[..., None], dout, 0.0)
    g = dout * gate
    got = {"dz": dout * y * dgate, "dD": (g * u).sum((0, 1))}
    du, dd = torch.zeros_like(u), torch.zeros_like(u)
    dB = torch.zeros(b, length, groups, n, dtype=F64)
    dC = torch.zeros_like(dB)
    dA = torch.zeros_like(A)
    r = dfinal
    for t in reversed(range(length)):
        dh = C[:, t] * g[:, t][..., None] + r
        r = a[:, t] * dh
        q = r * (hs[:, t - 1] if t > 0 else h0)
        hb = (dh * B[:, t]).sum(-1)
        on = mask[:, t][:, None]
        dd[:, t] = torch.where(on, ((q * A).sum(-1) + hb * u[:, t]) * slope[:, t], 0.0)
        du[:, t] = D * g[:, t] + step[:, t] * hb
        dA += (q * step[:, t][..., None]).sum(0)
        dB[:, t] = (dh * (step[:, t] * u[:, t])[..., None]).unflatten(1, (groups, d // groups)).sum(2)
        dC[:, t] = (hs[:, t] * g[:, t][..., None]).unflatten(1, (groups, d // groups)).sum(2)
    got.update(du=torch.where(mask[..., None], du, 0.0), ddelta=dd, dA=dA, dB=dB, dC=dC, ddelta_bias=dd.sum((0, 1)), dinit=r)
    return got


class ScanCase:
    """One case in 64 bits: its parts, results and their magnitudes."""

    def __init__(self, u, delta, A, B, C, D=None, z=None, delta_bias=None, use_softplus=True, h0=None, lens=None):
        b, length, d = u.shape
        n = A.shape[1]
        self.groups = B.shape[2]
        self.mask = mask = live_mask(lens, b, length)
        self.u = zeroed(u, mask)
        raw = zeroed(delta, mask) + (0.0 if delta_bias is None else delta_bias.to("cpu", F64))
        step = softplus(raw) if use_softplus else raw
        self.slope = sigmoid(raw) if use_softplus else torch.ones_like(raw)
        self.step = torch.where(mask[..., None], step, 0.0)
        self.A = A.to("cpu", F64)
        self.a = torch.exp(self.step[..., None] * self.A)
        self.B, self.C = by_channel(zeroed(B, mask), d), by_channel(zeroed(C, mask), d)
        self.D = torch.zeros(d, dtype=F64) if D is None else D.to("cpu", F64)
        if z is None:
            self.gate, self.dgate = torch.ones_like(self.u), torch.zeros_like(self.u)
        else:
            zz = zeroed(z, mask)
            s = sigmoid(zz)
            self.gate, self.dgate = zz * s, s * (1 + zz * (1 - s))
        self.h0 = torch.zeros(b, d, n, dtype=F64) if h0 is None else h0.to("cpu", F64)

    def forward(self):
        out, _, hs = scan(self.u, self.step, self.a, self.B, self.C, self.D, self.gate, self.h0, self.mask)
        return out, (hs[:, -1] if hs.shape[1] else self.h0)

    def grad(self, dout, dfinal=None):
        return scan_grad(self.u, self.step, self.a, self.A, self.B, self.C, self.D, self.gate, self.dgate, self.slope, self.h0,
                         self.mask, zeroed(dout, self.mask), self._final(dfinal), self.groups)

    def _final(self, dfinal):
        return torch.zeros_like(self.h0) if dfinal is None else dfinal.to("cpu", F64)

    def magnitude(self):
        m = object.__new__(ScanCase)
        m.__dict__.update(self.__dict__)
        for k in ("u", "step", "A", "B", "C", "D", "gate", "dgate", "slope", "h0"):
            setattr(m, k, getattr(self, k).abs())
        return m

    def rel(self):
        """Relative f32 error of a result against its magnitude. A term passes through at most len decays, each off by EX and a
        rounding, and len + nstate additions, on either side; step size, gate and skip add a few evaluations."""
        length, n = self.a.shape[1], self.A.shape[1]
        return (2 * length + 8) * (EX + 2 * U) + (length + n + 16) * U
