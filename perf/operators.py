"""The sequence-model operators as a user's program calls them, with plain forms to measure them against.

Three operators, each in the directions that a program has it: the embedding lookup (`embed`) and its table's
gradient (`embed_grad`), the short causal convolution (`conv`, `conv_grad`, and `conv_step` for one token a
sequence) and the selective state space scan (`scan`, `scan_train` for forward and gradients, `scan_step`).

`run` makes the framework's calls where `own` is true. Otherwise it computes the same in elementary torch
operations in 32 bits, rounded once at the end; the recurrence over tokens is a doubling scan.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}

# the most (token, channel, state) triples of a scan, and (token, channel) pairs of a convolution
MOST_TRIPLES = 4 * 2048 * 4096 * 16
MOST_PAIRS = 4 * 4096 * 4096


def listed():
    return [
        # the rows of a training batch's tokens: bandwidth both ways
        dict(name="lookup batch bf16", op="embed", dtype="bf16", tokens=8192, vocab=32768, dim=4096),
        # one token of each sequence that is being decoded: latency
        dict(name="lookup tokens f16", op="embed", dtype="f16", tokens=64, vocab=32768, dim=2048),
        # the table's gradient of a training batch: tokens fall as words do, few are frequent and most rows get none
        dict(name="table gradient bf16", op="embed_grad", dtype="bf16", grad="f32", tokens=16384, vocab=32768, dim=2048),
        # a small vocabulary with long runs, rows that no 16-byte load fits, and the gradient in the rows' own type
        dict(name="table gradient odd f32", op="embed_grad", dtype="f32", grad="f32", tokens=4099, vocab=5003, dim=1001),
        # a batch of prompts, x a half of a wider projection's rows
        dict(name="conv prompt bf16", op="conv", dtype="bf16", batch=4, length=4096, dim=4096, width=4, ragged=False),
        # the training direction at an odd length
        dict(name="conv gradient f16", op="conv_grad", dtype="f16", batch=2, length=4099, dim=2048, width=4, ragged=False),
        # one token of each sequence: latency
        dict(name="conv step bf16", op="conv_step", dtype="bf16", batch=64, dim=4096, width=4),
        # one long prompt: few channels, so the token axis has to be split
        dict(name="scan prompt bf16", op="scan", dtype="bf16", batch=1, length=16384, dim=2048, state=16, groups=1,
             ragged=False),
        # prompts of different lengths, one of them empty, that go on from states they have
        dict(name="scan ragged f16", op="scan", dtype="f16", batch=8, length=1027, dim=4096, state=16, groups=1, ragged=True),
        # a training step of a batch, forward and backward: the largest
        dict(name="scan train bf16", op="scan_train", dtype="bf16", batch=4, length=2048, dim=4096, state=16, groups=1,
             ragged=False),
        # odd sizes, channels in groups, states that are no multiple of a vector, gradients into the first state
        dict(name="scan train odd f32", op="scan_train", dtype="f32", batch=3, length=515, dim=1002, state=21, groups=2,
             ragged=True),
        # one token of each sequence: the states' bytes
        dict(name="scan step bf16", op="scan_step", dtype="bf16", batch=64, dim=4096, state=16, groups=1),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "conv", "conv_grad", "conv_step", "scan", "scan", "scan_train", "scan_train",
                     "scan_step"])
    case = dict(op=op, dtype=rng.choice(["f32", "bf16", "f16"]))
    if op in ("embed", "embed_grad"):
        case.update(tokens=_spread(rng, 1, 16384), vocab=_spread(rng, 64, 32768), dim=_spread(rng, 32, 2048))
        if op == "embed_grad":
            case["grad"] = rng.choice(["f32", case["dtype"]])
        return case
    if op in ("conv_step", "scan_step"):
        case.update(batch=_spread(rng, 1, 128), dim=_spread(rng, 64, 4096))
    else:
        case.update(batch=_spread(rng, 1, 8), dim=_spread(rng, 64, 4096), ragged=rng.random() < 0.5)
        case["length"] = min(_spread(rng, 1, 8192), MOST_PAIRS // 4 // (case["batch"] * case["dim"]))
    if op.startswith("conv"):
        case["width"] = rng.choice([2, 3, 4])
        return case
    case["groups"] = rng.choice([1, 1, 2])
    case["dim"] -= case["dim"] % case["groups"]
    case["state"] = rng.choice([4, 8, 16, 16, 16, 32, 64, 1 + rng.randrange(64)])
    if op != "scan_step":
        case["length"] = max(1, min(case["length"], MOST_TRIPLES // 4 // (case["batch"] * case["dim"] * case["state"])))
    return case


# --- inputs ---------------------------------------------------------------------------------------------------------


def _inputs(case, seed):
    """The inputs that plain form, kernels and exact form are given."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, by=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(by).to(dtype)

    def uniform(lo, hi, *shape):
        return torch.rand(shape, generator=g, device="cuda") * (hi - lo) + lo

    op, s = case["op"], {}
    if op in ("embed", "embed_grad"):
        n, v, h = case["tokens"], case["vocab"], case["dim"]
        # the rank of a word is spread over its logarithm, and words are numbered in no order of rank
        rank = torch.exp(uniform(0.0, math.log(v + 1.0), n)).long().sub_(1).clamp_(0, v - 1)
        s["tokens"] = torch.randperm(v, generator=g, device="cuda")[rank].to(torch.int32)
        if n > 16:
            s["tokens"][n - n // 16:] = -1  # padding: no row
        s["scale"] = math.sqrt(h)
        if op == "embed":
            s["table"] = normal(v, h, by=0.02)
        else:
            s["dout"] = normal(n, h)
        return s
    b, d = case["batch"], case["dim"]
    if "length" in case:
        t = case["length"]
        if case["ragged"]:
            s["lens"] = torch.randint(t // 4, t + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
            s["lens"][0] = t
            if b > 2:
                s["lens"][1] = 0
    if op.startswith("conv"):
        w = case["width"]
        s["weight"], s["bias"] = normal(d, w, by=0.5), normal(d, by=0.2)
        if op == "conv_step":
            s["x"], s["state"] = normal(b, d), normal(b, w - 1, d)
            return s
        s["x"] = normal(b, t, 2 * d)[:, :, :d]  # a half of a wider projection's output
        if op == "conv":
            if case["ragged"]:
                s["state"] = normal(b, w - 1, d)
        else:
            s["dout"] = normal(b, t, d)
        return s
    n, groups = case["state"], case["groups"]
    lead = (b,) if op == "scan_step" else (b, t)
    s["u"] = normal(*lead, d)
    s["delta"] = normal(*lead, d, by=0.5)
    # steps between 0.001 and 0.1 at delta = 0, decay rates from 1 to the number of states
    step = torch.exp(uniform(math.log(1e-3), math.log(1e-1), d))
    s["delta_bias"] = step + torch.log(-torch.expm1(-step))
    s["A"] = -torch.arange(1, n + 1, device="cuda", dtype=torch.float32) * uniform(0.8, 1.25, d, n)
    bc = normal(*lead, 2 * groups * n).unflatten(-1, (2 * groups, n))  # both come out of one projection
    s["B"], s["C"] = bc[..., :groups, :], bc[..., groups:, :]
    s["D"] = uniform(0.5, 1.5, d)
    s["z"] = normal(*lead, 2 * d)[..., d:]
    if op == "scan_step" or case["ragged"]:
        s["state"] = normal(b, d, n, dtype=torch.float32)
    if op == "scan_train":
        s["dout"] = normal(*lead, d)
        if case["ragged"]:
            s["dfinal"] = normal(b, d, n, dtype=torch.float32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    s["op"] = op
    dev = "cuda"
    if op == "embed":
        s["out"] = torch.empty(case["tokens"], case["dim"], dtype=s["table"].dtype, device=dev)
    elif op == "embed_grad":
        s["dtable"] = torch.empty(case["vocab"], case["dim"], dtype=DTYPES[case["grad"]], device=dev)
    elif op.startswith("conv"):
        if op == "conv_grad":
            s["dx"] = torch.empty(s["x"].shape, dtype=s["x"].dtype, device=dev)
            s["dweight"] = torch.empty(s["weight"].shape, dtype=torch.float32, device=dev)
            s["dbias"] = torch.empty(s["bias"].shape, dtype=torch.float32, device=dev)
        else:
            s["out"] = torch.empty(s["x"].shape, dtype=s["x"].dtype, device=dev)
            if "state" not in s:  # a prompt that starts a sequence: its state is written, not read
                s["state_out"] = torch.empty(case["batch"], case["width"] - 1, case["dim"], dtype=s["x"].dtype, device=dev)
    else:
        s["out"] = torch.empty(s["u"].shape, dtype=s["u"].dtype, device=dev)
        if op == "scan" and "state" not in s:
            s["state_out"] = torch.empty(case["batch"], case["dim"], case["state"], device=dev)
        if op == "scan_train":
            for k in ("u", "delta", "z", "B", "C"):
                s["d" + k] = torch.empty(s[k].shape, dtype=s[k].dtype, device=dev)
            for k in ("A", "D", "delta_bias"):
                s["d" + k] = torch.empty(s[k].shape, dtype=torch.float32, device=dev)
            if "dfinal" in s:
                s["dinit"] = torch.empty_like(s["dfinal"])
    return s


# --- the framework's calls ------------------------------------------------------------------------------------------


def _workspace(s, name, slots):
    if name not in s:  # kept from step to step, as a program keeps it
        s[name] = torch.empty(slots(), dtype=torch.int64, device="cuda")
    return s[name]


def _own_embed(s, mt):
    mt.mt_embed(s["tokens"], s["table"], s["out"], scale=s["scale"])
    return {"out": s["out"]}


def _own_embed_grad(s, mt):
    scratch = _workspace(s, "scratch", lambda: mt.mt_embed_grad_scratch_slots(s["tokens"].numel(), *s["dtable"].shape))
    mt.mt_embed_grad(s["tokens"], s["dout"], s["dtable"], scratch, scale=s["scale"])
    return {"dtable": s["dtable"]}


def _own_conv(s, mt):
    carry = "state" in s  # updated in place, so that the next pass goes on from it
    state = s["state"] if carry else s["state_out"]
    mt.mt_causal_conv(s["x"], s["weight"], s["out"], bias=s["bias"], state=state, carry_in=carry, lens=s.get("lens"))
    return {"out": s["out"], "state": state}


def _own_conv_grad(s, mt):
    b, t, d = s["x"].shape
    scratch = _workspace(s, "scratch", lambda: mt.mt_causal_conv_grad_scratch_slots(b, t, d, s["weight"].shape[1]))
    mt.mt_causal_conv_grad(s["x"], s["weight"], s["dout"], s["dx"], s["dweight"], scratch, bias=s["bias"], dbias=s["dbias"],
                           lens=s.get("lens"))
    return {"dx": s["dx"], "dweight": s["dweight"], "dbias": s["dbias"]}


def _own_conv_step(s, mt):
    mt.mt_causal_conv_step(s["x"], s["weight"], s["state"], s["out"], bias=s["bias"])
    return {"out": s["out"], "state": s["state"]}


def _scan_forward(s, mt, state, carry, checkpoints):
    b, t, d = s["u"].shape
    g, n = s["B"].shape[2:]
    scratch = _workspace(s, "scratch", lambda: mt.mt_selective_scan_scratch_slots(b, t, d, n, g))
    mt.mt_selective_scan(s["u"], s["delta"], s["A"], s["B"], s["C"], s["out"], scratch, D=s["D"], z=s["z"],
                         delta_bias=s["delta_bias"], state=state, carry_in=carry, lens=s.get("lens"), checkpoints=checkpoints)


def _own_scan(s, mt):
    carry = "state" in s  # updated in place, so that the next pass goes on from it
    state = s["state"] if carry else s["state_out"]
    _scan_forward(s, mt, state, carry, None)
    return {"out": s["out"], "state": state}


def _own_scan_train(s, mt):
    b, t, d = s["u"].shape
    g, n = s["B"].shape[2:]
    checkpoints = _workspace(s, "checkpoints", lambda: mt.mt_selective_scan_checkpoint_slots(b, t, d, n))
    _scan_forward(s, mt, s.get("state"), "state" in s, checkpoints)
    scratch = _workspace(s, "grad_scratch", lambda: mt.mt_selective_scan_scratch_slots(b, t, d, n, g, grad=True))
    mt.mt_selective_scan_grad(s["u"], s["delta"], s["A"], s["B"], s["C"], s["dout"], checkpoints, s["du"], s["ddelta"],
                              s["dA"], s["dB"], s["dC"], scratch, D=s["D"], dD=s["dD"], z=s["z"], dz=s["dz"],
                              delta_bias=s["delta_bias"], ddelta_bias=s["ddelta_bias"], dfinal=s.get("dfinal"),
                              dinit=s.get("dinit"), lens=s.get("lens"))
    got = {k: s[k] for k in ("out", "du", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias")}
    if "state" in s:
        got.update(state=s["state"], dinit=s["dinit"])
    return got


def _own_scan_step(s, mt):
    mt.mt_selective_scan_step(s["u"], s["delta"], s["A"], s["B"], s["C"], s["state"], s["out"], D=s["D"], z=s["z"],
                              delta_bias=s["delta_bias"])
    return {"out": s["out"], "state": s["state"]}


# --- the plain forms ------------------------------------------------------------------------------------------------


def _live(s, x):
    """True where token t of a sequence is one that it has; None where all are."""
    if "lens" not in s:
        return None
    t = torch.arange(x.shape[1], device=x.device)
    return (t[None, :] < s["lens"][:, None])[..., None]


def _keep(live, x):
    return x if live is None else torch.where(live, x, torch.zeros((), dtype=x.dtype, device=x.device))


def _advance(s, state):
    """The state after a pass: in place of the one it went on from, where it had one."""
    return s["state"].copy_(state) if "state" in s else state


def _plain_embed(s):
    tok = s["tokens"].long()
    rows = s["table"][tok.clamp(min=0)].float() * s["scale"]
    return {"out": torch.where((tok >= 0)[:, None], rows, 0.0).to(s["table"].dtype)}


def _plain_embed_grad(s):
    tok = s["tokens"].long()
    v, h = s["dtable"].shape
    sums = torch.zeros(v + 1, h, device=tok.device)  # the last row takes what belongs to none
    sums.index_add_(0, torch.where(tok >= 0, tok, v), s["dout"].float())
    return {"dtable": (sums[:v] * s["scale"]).to(s["dtable"].dtype)}


def _taps(s, x):
    """x with the W - 1 inputs before it."""
    w = s["weight"].shape[1]
    before = s["state"].float() if "state" in s else torch.zeros(x.shape[0], w - 1, x.shape[2], device=x.device)
    return torch.cat([before, x], 1)


def _conv_sum(s, padded, length):
    """sum_k w[:, k] x[t - W + 1 + k] + bias, through a view of W inputs a token."""
    windows = padded.unfold(1, s["weight"].shape[1], 1)[:, :length]  # [B, L, D, W]
    return (windows * s["weight"].float()).sum(-1) + s["bias"].float()


def _plain_conv(s):
    live = _live(s, s["x"])
    x = _keep(live, s["x"].float())
    padded = _taps(s, x)
    p = _conv_sum(s, padded, x.shape[1])
    out = _keep(live, p / (1 + torch.exp(-p))).to(s["x"].dtype)
    w, t = s["weight"].shape[1], x.shape[1]
    ends = s["lens"].long() if "lens" in s else torch.full((x.shape[0],), t, device=x.device)
    at = ends[:, None] + torch.arange(w - 1, device=x.device)
    state = torch.gather(padded, 1, at[..., None].expand(-1, -1, x.shape[2]))
    return {"out": out, "state": _advance(s, state.to(s["x"].dtype))}


def _plain_conv_grad(s):
    live = _live(s, s["x"])
    x = _keep(live, s["x"].float())
    w, t = s["weight"].shape[1], x.shape[1]
    padded = _taps(s, x)
    p = _conv_sum(s, padded, t)
    sig = 1 / (1 + torch.exp(-p))
    g = _keep(live, s["dout"].float()) * (sig * (1 + p * (1 - sig)))
    after = torch.cat([g, torch.zeros_like(g[:, :1]).expand(-1, w - 1, -1)], 1)
    dx = (after.unfold(1, w, 1) * s["weight"].float().flip(1)).sum(-1)
    dw = (padded.unfold(1, w, 1)[:, :t] * g[..., None]).sum((0, 1))
    return {"dx": _keep(live, dx).to(s["x"].dtype), "dweight": dw, "dbias": g.sum((0, 1))}


def _plain_conv_step(s):
    x = torch.cat([s["state"], s["x"][:, None]], 1).float()
    p = (x * s["weight"].float().t()).sum(1) + s["bias"].float()
    return {"out": (p / (1 + torch.exp(-p))).to(s["x"].dtype), "state": _advance(s, x[:, 1:].to(s["x"].dtype))}


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t over dimension 1 from h_{-1} = 0, in place of b, by doubling; a is used up."""
    step = 1
    while step < a.shape[1]:
        b[:, step:] += a[:, step:] * b[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    return b


def _softplus(x):
    return torch.where(x > 20, x, torch.log1p(torch.exp(x)))


def _heads(x, d):
    """[..., G, N] to one row for each channel, [..., D, N]."""
    return x.float().repeat_interleave(d // x.shape[-2], -2)


def _scan_parts(s):
    """Step sizes, decays and states of all tokens."""
    d = s["u"].shape[-1]
    live = _live(s, s["u"])
    raw = s["delta"].float() + s["delta_bias"]
    delta = _keep(live, _softplus(raw))
    u = _keep(live, s["u"].float())
    a = torch.exp(delta[..., None] * s["A"])
    b = (delta * u)[..., None] * _keep(None if live is None else live[..., None], _heads(s["B"], d))
    if "state" in s:
        b[:, 0] += a[:, 0] * s["state"]
    h = _recurrence(a.clone(), b)
    return live, raw, delta, u, a, h


def _gate(z):
    sig = 1 / (1 + torch.exp(-z))
    return z * sig, sig * (1 + z * (1 - sig))


def _plain_scan(s):
    d = s["u"].shape[-1]
    live, _, _, u, _, h = _scan_parts(s)
    y = (h * _heads(s["C"], d)).sum(-1) + s["D"] * u
    out = _keep(live, y * _gate(s["z"].float())[0]).to(s["u"].dtype)
    return {"out": out, "state": _advance(s, h[:, -1].contiguous())}


def _plain_scan_train(s):
    dt, (d, n) = s["u"].dtype, s["A"].shape
    groups = s["B"].shape[-2]
    live, raw, delta, u, a, h = _scan_parts(s)
    live4 = None if live is None else live[..., None]
    bm, cm = _keep(live4, _heads(s["B"], d)), _keep(live4, _heads(s["C"], d))
    y = (h * cm).sum(-1) + s["D"] * u
    gate, dgate = _gate(_keep(live, s["z"].float()))
    dout = _keep(live, s["dout"].float())
    g, dz = dout * gate, dout * y * dgate
    dh = g[..., None] * cm
    if "dfinal" in s:
        dh[:, -1] += s["dfinal"]
    ahead = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)  # a_{t+1}
    dh = _recurrence(ahead.flip(1), dh.flip(1)).flip(1)
    before = torch.cat([(s["state"] if "state" in s else torch.zeros_like(h[:, 0]))[:, None], h[:, :-1]], 1)
    q = dh * a * before
    hb = (dh * bm).sum(-1)
    ddelta = _keep(live, ((q * s["A"]).sum(-1) + hb * u) / (1 + torch.exp(-raw)))
    by_group = lambda x: x.unflatten(2, (groups, d // groups)).sum(3)  # noqa: E731
    got = {
        "out": _keep(live, y * gate).to(dt),
        "du": (s["D"] * g + hb * delta).to(dt),
        "ddelta": ddelta.to(dt),
        "dA": (q * delta[..., None]).sum((0, 1)),
        "dB": _keep(live4, by_group(dh * (delta * u)[..., None])).to(dt),
        "dC": _keep(live4, by_group(h * g[..., None])).to(dt),
        "dD": (g * u).sum((0, 1)),
        "dz": dz.to(dt),
        "ddelta_bias": ddelta.sum((0, 1)),
    }
    if "state" in s:
        got.update(state=_advance(s, h[:, -1]), dinit=dh[:, 0] * a[:, 0])
    return got


def _plain_scan_step(s):
    d = s["u"].shape[-1]
    u = s["u"].float()
    delta = _softplus(s["delta"].float() + s["delta_bias"])
    state = torch.exp(delta[..., None] * s["A"]) * s["state"] + (delta * u)[..., None] * _heads(s["B"], d)
    y = (state * _heads(s["C"], d)).sum(-1) + s["D"] * u
    return {"out": (y * _gate(s["z"].float())[0]).to(s["u"].dtype), "state": _advance(s, state)}


_PLAIN = {"embed": _plain_embed, "embed_grad": _plain_embed_grad, "conv": _plain_conv, "conv_grad": _plain_conv_grad,
          "conv_step": _plain_conv_step, "scan": _plain_scan, "scan_train": _plain_scan_train, "scan_step": _plain_scan_step}
_OWN = {"embed": _own_embed, "embed_grad": _own_embed_grad, "conv": _own_conv, "conv_grad": _own_conv_grad,
        "conv_step": _own_conv_step, "scan": _own_scan, "scan_train": _own_scan_train, "scan_step": _own_scan_step}


def run(state):
    if own:
        import prefix_scan_row_gb300 as mt
        return _OWN[state["op"]](state, mt)
    return _PLAIN[state["op"]](state)


# --- what a pass cannot do without ----------------------------------------------------------------------------------


def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op == "embed":
        n, h = case["tokens"], case["dim"]
        return {"bytes": 4 * n + (n + min(n, case["vocab"])) * h * e, "flops": n * h}
    if op == "embed_grad":
        n, v, h = case["tokens"], case["vocab"], case["dim"]
        return {"bytes": 4 * n + n * h * e + v * h * BYTES[case["grad"]], "flops": 2 * n * h}
    pairs = case["batch"] * case.get("length", 1) * case["dim"]
    if op.startswith("conv"):
        w, d = case["width"], case["dim"]
        state = case["batch"] * (w - 1) * d * e
        if op == "conv":
            return {"bytes": 2 * pairs * e + state + d * (w + 1) * e, "flops": pairs * (2 * w + 5)}
        if op == "conv_step":
            return {"bytes": 2 * pairs * e + 2 * state + d * (w + 1) * e, "flops": pairs * (2 * w + 5)}
        return {"bytes": 3 * pairs * e + d * (w + 1) * (e + 4), "flops": pairs * (6 * w + 10)}
    n, d = case["state"], case["dim"]
    tokens = case["batch"] * case.get("length", 1)
    shared = 2 * tokens * case["groups"] * n * e
    state = 4 * case["batch"] * d * n
    params = 4 * d * (n + 2)
    if op == "scan_step":
        return {"bytes": 4 * pairs * e + shared + 2 * state + params, "flops": pairs * (7 * n + 12)}
    if op == "scan":
        return {"bytes": 4 * pairs * e + shared + state + params, "flops": pairs * (7 * n + 12)}
    return {"bytes": 8 * pairs * e + 2 * shared + 2 * params, "flops": pairs * (24 * n + 40)}


# --- the definition in 64 bits --------------------------------------------------------------------------------------


def _sigmoid64(x):
    return 0.5 * (1 + torch.tanh(0.5 * x))


def _exact_conv(case, s):
    """Token by token: W products each, then the derivative of x * sigmoid(x) tap by tap."""
    b, t, d = s["x"].shape
    w = case["width"]
    x = torch.zeros(b, t + w - 1, d, dtype=torch.float64, device=s["x"].device)
    x[:, w - 1:] = s["x"].double()
    if "state" in s:
        x[:, :w - 1] = s["state"].double()
    mask = torch.ones(b, t, 1, dtype=torch.bool, device=x.device)
    ends = [t] * b
    if "lens" in s:
        ends = [int(v) for v in s["lens"].cpu()]
        for i, n in enumerate(ends):
            mask[i, n:] = False
            x[i, w - 1 + n:] = 0
    weight = s["weight"].double()
    p = s["bias"].double().expand(b, t, d).clone()
    for k in range(w):
        p += weight[:, k] * x[:, k:k + t]
    sig = _sigmoid64(p)
    if case["op"] == "conv":
        state = torch.stack([x[i, n:n + w - 1] for i, n in enumerate(ends)])
        return {"out": torch.where(mask, p * sig, 0.0), "state": state}
    g = torch.where(mask, s["dout"].double() * (sig + p * sig * (1 - sig)), 0.0)
    dx, dw = torch.zeros_like(x), torch.empty_like(weight)
    for k in range(w):
        dx[:, k:k + t] += weight[:, k] * g
        dw[:, k] = (g * x[:, k:k + t]).sum((0, 1))
    return {"dx": torch.where(mask, dx[:, w - 1:], 0.0), "dweight": dw, "dbias": g.sum((0, 1))}


def _exact_scan(case, s):
    """The recurrence one token after the other, and its adjoint one token before the other."""
    b, t, d = s["u"].shape
    n, groups, train = case["state"], case["groups"], case["op"] == "scan_train"
    f = torch.float64
    dev = s["u"].device
    ends = s["lens"].long() if "lens" in s else torch.full((b,), t, device=dev)
    A, D = s["A"].double(), s["D"].double()
    h = s["state"].double() if "state" in s else torch.zeros(b, d, n, dtype=f, device=dev)
    out = torch.zeros(b, t, d, dtype=f, device=dev)
    past = torch.empty(t, b, d, n, dtype=f, device=dev) if train else None
    per = d // groups
    channels = lambda x: x.double()[:, :, None].expand(b, groups, per, n).reshape(b, d, n)  # noqa: E731
    soft = lambda x: torch.clamp(x, min=0) + torch.log1p(torch.exp(-x.abs()))  # noqa: E731
    for i in range(t):
        on = (i < ends)[:, None]
        if train:
            past[i] = h
        step = soft(s["delta"][:, i].double() + s["delta_bias"].double())
        u = s["u"][:, i].double()
        new = torch.exp(step[..., None] * A) * h + (step * u)[..., None] * channels(s["B"][:, i])
        h = torch.where(on[..., None], new, h)
        z = s["z"][:, i].double()
        y = torch.einsum("bdn,bdn->bd", new, channels(s["C"][:, i])) + D * u
        out[:, i] = torch.where(on, y * z * _sigmoid64(z), 0.0)
    if not train:
        return {"out": out, "state": h}
    dh = s["dfinal"].double().clone() if "dfinal" in s else torch.zeros(b, d, n, dtype=f, device=dev)
    zero = lambda x: torch.zeros(x.shape, dtype=f, device=dev)  # noqa: E731
    r = {"out": out, **{"d" + k: zero(s[k]) for k in ("u", "delta", "A", "B", "C", "D", "z", "delta_bias")}}
    for i in reversed(range(t)):
        on = (i < ends)[:, None]
        raw = s["delta"][:, i].double() + s["delta_bias"].double()
        step, u, z = soft(raw), s["u"][:, i].double(), s["z"][:, i].double()
        bm, cm = channels(s["B"][:, i]), channels(s["C"][:, i])
        a = torch.exp(step[..., None] * A)
        now = a * past[i] + (step * u)[..., None] * bm
        sig = _sigmoid64(z)
        dout = torch.where(on, s["dout"][:, i].double(), 0.0)
        y = torch.einsum("bdn,bdn->bd", now, cm) + D * u
        g = dout * z * sig
        full = dh + g[..., None] * cm
        r["dz"][:, i] = torch.where(on, dout * y * (sig + z * sig * (1 - sig)), 0.0)
        q = full * a * past[i]
        hb = torch.einsum("bdn,bdn->bd", full, bm)
        raw_grad = (torch.einsum("bdn,dn->bd", q, A) + hb * u) * _sigmoid64(raw)
        r["ddelta"][:, i] = torch.where(on, raw_grad, 0.0)
        r["du"][:, i] = torch.where(on, D * g + step * hb, 0.0)
        r["dA"] += torch.where(on[..., None], q * step[..., None], 0.0).sum(0)
        r["dD"] += torch.where(on, g * u, 0.0).sum(0)
        db = torch.where(on[..., None], full * (step * u)[..., None], 0.0)
        dc = torch.where(on[..., None], now * g[..., None], 0.0)
        r["dB"][:, i] = db.reshape(b, groups, per, n).sum(2)
        r["dC"][:, i] = dc.reshape(b, groups, per, n).sum(2)
        dh = torch.where(on[..., None], full * a, dh)
    r["ddelta_bias"] = r["ddelta"].sum((0, 1))
    if "state" in s:
        r.update(state=h, dinit=dh)
    return r


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "embed":
        table = torch.cat([s["table"].double(), torch.zeros_like(s["table"][:1], dtype=torch.float64)])  # row -1: none
        return {"out": table[s["tokens"].long()] * s["scale"]}
    if op == "embed_grad":
        tok = s["tokens"].long()
        has = tok >= 0
        sums = torch.zeros(case["vocab"], case["dim"], dtype=torch.float64, device=tok.device)
        return {"dtable": sums.index_put_((tok[has],), s["dout"][has].double() * s["scale"], accumulate=True)}
    if op in ("conv", "conv_grad"):
        return _exact_conv(case, s)
    if op == "conv_step":
        x = torch.cat([s["state"].double(), s["x"].double()[:, None]], 1)
        p = torch.einsum("bwd,dw->bd", x, s["weight"].double()) + s["bias"].double()
        return {"out": p * _sigmoid64(p), "state": x[:, 1:]}
    if op == "scan_step":
        wide = {k: (v[:, None] if k in ("u", "delta", "B", "C", "z") else v) for k, v in s.items()}
        got = _exact_scan(dict(case, op="scan"), wide)
        return {"out": got["out"][:, 0], "state": got["state"]}
    return _exact_scan(case, s)
