"""A gated linear recurrence and beam search over pooled states, as a user's program calls them, with plain forms.

Three operators, each in the directions that a program has it: the gated linear recurrence (`gated` over prompts,
`gated_train` for forward and gradients, `gated_step` for one token a sequence), the selection of a beam search
over beams and vocabulary (`beam`), and the copying of rows of state pools between their slots (`copy`), with
which a beam search's states follow its beams.

`run` makes the framework's calls where `own` is true. Otherwise it computes the same in elementary torch
operations in 32 bits (scores of a beam search, whose order decides, in 64), rounded once at the end; the
recurrence over tokens is a doubling scan.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}

MOST_PAIRS = 4 * 2048 * 4096        # (token, channel) pairs of a drawn recurrence
MOST_LOGITS = 64 * 8 * 65536        # logits of a drawn selection
MOST_COPIED = 1 << 28               # bytes that a drawn copy writes


def listed():
    return [
        # a batch of prompts, gates and values parts of wider projections' rows: the largest, bandwidth
        dict(name="gated prompt bf16", op="gated", dtype="bf16", batch=4, length=4096, dim=4096, decay="rate", input_gate=True,
             z=False, ragged=False),
        # one long prompt: few channels, so the token axis has to be split
        dict(name="gated long prompt bf16", op="gated", dtype="bf16", batch=1, length=16384, dim=2048, decay="rate",
             input_gate=True, z=True, ragged=False),
        # prompts of different lengths, one of them empty, that go on from states they have
        dict(name="gated ragged f16", op="gated", dtype="f16", batch=8, length=1027, dim=4096, decay="blend", input_gate=False,
             z=True, ragged=True),
        # a training step of a batch, forward and backward, with every gate
        dict(name="gated train bf16", op="gated_train", dtype="bf16", batch=4, length=2048, dim=4096, decay="rate",
             input_gate=True, z=True, ragged=False),
        # odd sizes, gradients into the first state
        dict(name="gated train odd f32", op="gated_train", dtype="f32", batch=3, length=515, dim=1001, decay="rate",
             input_gate=True, z=False, ragged=True),
        # one token of each sequence: latency
        dict(name="gated step bf16", op="gated_step", dtype="bf16", batch=64, dim=4096, decay="rate", input_gate=True, z=True),
        # one sequence with a few beams: latency
        dict(name="beam single f32", op="beam", dtype="f32", batch=1, beams=4, vocab=32768, finished=0, slots=True),
        # a served batch, some of its beams finished
        dict(name="beam batch bf16", op="beam", dtype="bf16", batch=64, beams=8, vocab=32768, finished=1, slots=True),
        # a large vocabulary and many beams: bandwidth
        dict(name="beam large bf16", op="beam", dtype="bf16", batch=64, beams=16, vocab=131072, finished=0, slots=True),
        # rows that no 16-byte load fits
        dict(name="beam odd f16", op="beam", dtype="f16", batch=5, beams=7, vocab=100003, finished=2, slots=False),
        # the states of one small group of beams, a layer's: latency
        dict(name="copy group", op="copy", dtype="bf16", groups=1, beams=4, kept=2, layers=1, dim=4096, width=4, state=16),
        # the states of a served batch of beams, several layers at once
        dict(name="copy batch", op="copy", dtype="bf16", groups=64, beams=8, kept=5, layers=4, dim=4096, width=4, state=16),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_train", "gated_train", "gated_step", "beam", "beam", "beam", "copy", "copy"])
    case = dict(op=op, dtype=rng.choice(["f32", "bf16", "f16"]))
    if op.startswith("gated"):
        case.update(batch=_spread(rng, 1, 128 if op == "gated_step" else 8), dim=_spread(rng, 64, 4096),
                    decay=rng.choice(["rate", "blend"]), input_gate=rng.random() < 0.6, z=rng.random() < 0.5)
        if op != "gated_step":
            most = MOST_PAIRS // (2 if case["dtype"] == "f32" else 1) // (case["batch"] * case["dim"])
            case.update(length=max(1, min(_spread(rng, 1, 16384), most)), ragged=rng.random() < 0.5)
    elif op == "beam":
        case.update(batch=_spread(rng, 1, 64), beams=_spread(rng, 1, 32), vocab=_spread(rng, 500, 131072),
                    slots=rng.random() < 0.7)
        case["batch"] = max(1, min(case["batch"], MOST_LOGITS // (case["beams"] * case["vocab"])))
        case["finished"] = rng.randrange((case["beams"] + 1) // 2)
    else:
        case.update(groups=_spread(rng, 1, 64), beams=_spread(rng, 2, 16), layers=rng.choice([1, 1, 2, 4]),
                    dim=_spread(rng, 64, 4096), width=rng.choice([2, 3, 4]), state=rng.choice([1, 4, 16, 1 + rng.randrange(32)]))
        case["kept"] = 1 + rng.randrange(case["beams"] - 1)
        row = case["layers"] * _row_bytes(case)
        case["groups"] = max(1, min(case["groups"], MOST_COPIED // (row * case["beams"])))
    return case


def _row_bytes(case):
    """Bytes of one slot of a layer: the inputs that a short convolution keeps, and a recurrence's states."""
    return case["dim"] * ((case["width"] - 1) * BYTES[case["dtype"]] + case["state"] * 4)


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
    if op == "beam":
        b, k, v = case["batch"], case["beams"], case["vocab"]
        logits = normal(b, k, v, by=2.0)
        # each beam has a few likely tokens, and some that may not come next
        likely = torch.randint(0, v, (b, k, 8), generator=g, device="cuda")
        logits.scatter_(2, likely, normal(b, k, 8, by=1.5) + 9.0)
        banned = torch.randint(0, v, (b, k, 16), generator=g, device="cuda")
        logits.scatter_(2, banned, float("-inf"))
        s["logits"] = logits
        s["prior"] = torch.sort(uniform(-24.0, -20.0, b, k), descending=True).values
        if case["finished"]:
            s["finished"] = torch.zeros(b, k, dtype=torch.uint8, device="cuda")
            at = torch.rand(b, k, generator=g, device="cuda").argsort(1)[:, :case["finished"]]
            s["finished"].scatter_(1, at, 1)
        s["eos"] = 2
        if case["slots"]:
            s["slots"] = torch.randperm(b * k, generator=g, device="cuda").to(torch.int32).view(b, k)
        return s
    if op == "copy":
        n, k, layers, d = case["groups"], case["beams"], case["layers"], case["dim"]
        s["conv"] = normal(layers, n * k, case["width"] - 1, d)
        s["state"] = normal(layers, n * k, d, case["state"], dtype=torch.float32)
        # what a selection leaves: the first `kept` beams go on in their slots, the others follow one of them
        slots = torch.randperm(n * k, generator=g, device="cuda").to(torch.int32).view(n, k)
        j = torch.arange(k, device="cuda")
        follows = j % case["kept"]
        none = torch.full_like(slots, -1)
        s["src"] = torch.where(j < case["kept"], none, slots[:, follows]).contiguous()
        s["dst"] = torch.where(j < case["kept"], none, slots).contiguous()
        return s
    b, d = case["batch"], case["dim"]
    lead = (b,) if op == "gated_step" else (b, case["length"])
    if case.get("ragged"):
        t = case["length"]
        s["lens"] = torch.randint(t // 4, t + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
        s["lens"][0] = t
        if b > 2:
            s["lens"][1] = 0
    if case["z"]:  # halves of one projection's rows
        xz = normal(*lead, 2 * d)
        s["x"], s["z"] = xz[..., :d], xz[..., d:]
    else:
        s["x"] = normal(*lead, d)
    if case["input_gate"]:
        ri = normal(*lead, 2 * d)
        s["r"], s["i"] = ri[..., :d], ri[..., d:]
    else:
        s["r"] = normal(*lead, d)
    if case["decay"] == "rate":  # 0.9 to 0.999 an eighth of a token
        s["rate"] = -8.0 * torch.log(uniform(0.9, 0.999, d))
    if op == "gated_step" or case["ragged"]:
        s["state"] = normal(b, d, dtype=torch.float32)
    if op == "gated_train":
        s["dout"] = normal(*lead, d)
        if case["ragged"]:
            s["dfinal"] = normal(b, d, dtype=torch.float32)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    op, dev = case["op"], "cuda"
    s["op"] = op
    if op == "beam":
        shape = (case["batch"], case["beams"])
        for name in ("tokens", "parents"):
            s[name] = torch.empty(shape, dtype=torch.int32, device=dev)
        s["scores"] = torch.empty(shape, device=dev)
        s["finished_out"] = torch.empty(shape, dtype=torch.uint8, device=dev)
        if case["slots"]:
            s["src"], s["dst"] = (torch.empty(shape, dtype=torch.int32, device=dev) for _ in range(2))
    elif op != "copy":
        s["out"] = torch.empty(s["x"].shape, dtype=s["x"].dtype, device=dev)
        if op == "gated" and "state" not in s:
            s["state_out"] = torch.empty(case["batch"], case["dim"], device=dev)
        if op == "gated_train":
            for k in ("x", "r", "i", "z"):
                if k in s:
                    s["d" + k] = torch.empty(s[k].shape, dtype=s[k].dtype, device=dev)
            if "rate" in s:
                s["drate"] = torch.empty_like(s["rate"])
            if "dfinal" in s:
                s["dinit"] = torch.empty_like(s["dfinal"])
    return s


# --- the framework's calls ------------------------------------------------------------------------------------------


def _workspace(s, name, slots):
    if name not in s:  # kept from step to step, as a program keeps it
        s[name] = torch.empty(slots(), dtype=torch.int64, device="cuda")
    return s[name]


def _own_gated(s, mt):
    carry = "state" in s  # updated in place, so that the next pass goes on from it
    state = s["state"] if carry else s["state_out"]
    mt.mt_gated_scan(s["x"], s["r"], s["out"], i=s.get("i"), z=s.get("z"), rate=s.get("rate"), state=state, carry_in=carry,
                     lens=s.get("lens"))
    return {"out": s["out"], "state": state}


def _own_gated_train(s, mt):
    b, t, d = s["x"].shape
    checkpoints = _workspace(s, "checkpoints", lambda: mt.mt_gated_scan_checkpoint_slots(b, t, d))
    scratch = _workspace(s, "scratch", lambda: mt.mt_gated_scan_scratch_slots(b, t, d)) if "rate" in s else None
    gates = dict(i=s.get("i"), z=s.get("z"), rate=s.get("rate"), lens=s.get("lens"))
    mt.mt_gated_scan(s["x"], s["r"], s["out"], state=s.get("state"), carry_in="state" in s, checkpoints=checkpoints, **gates)
    mt.mt_gated_scan_grad(s["x"], s["r"], s["dout"], checkpoints, s["dx"], s["dr"], scratch, di=s.get("di"), dz=s.get("dz"),
                          drate=s.get("drate"), dfinal=s.get("dfinal"), dinit=s.get("dinit"), **gates)
    return {k: s[k] for k in ("out", "dx", "dr", "di", "dz", "drate", "state", "dinit") if k in s}


def _own_gated_step(s, mt):
    mt.mt_gated_scan_step(s["x"], s["r"], s["state"], s["out"], i=s.get("i"), z=s.get("z"), rate=s.get("rate"))
    return {"out": s["out"], "state": s["state"]}


def _own_beam(s, mt):
    b, k, v = s["logits"].shape
    scratch = _workspace(s, "scratch", lambda: mt.mt_beam_select_scratch_slots(b, k, k, v))
    mt.mt_beam_select(s["logits"], s["tokens"], s["parents"], s["scores"], scratch, prior=s["prior"],
                      finished=s.get("finished"), finished_out=s["finished_out"], eos=s["eos"], slots=s.get("slots"),
                      src=s.get("src"), dst=s.get("dst"))
    got = {"tokens": s["tokens"], "parents": s["parents"], "scores": s["scores"], "finished": s["finished_out"]}
    if "slots" in s:
        got.update(slots=s["slots"], src=s["src"], dst=s["dst"])
    return got


def _own_copy(s, mt):
    mt.mt_state_copy(s["src"], s["dst"], (s["conv"], s["state"]), axis=1)
    return {"conv": s["conv"], "state": s["state"]}


# --- the plain forms ------------------------------------------------------------------------------------------------


def _live(s):
    """True where token t of a sequence is one that it has; None where all are."""
    if "lens" not in s:
        return None
    t = torch.arange(s["x"].shape[1], device=s["x"].device)
    return (t[None, :] < s["lens"][:, None])[..., None]


def _keep(live, x):
    return x if live is None else torch.where(live, x, torch.zeros((), dtype=x.dtype, device=x.device))


def _advance(s, state):
    """The state after a pass: in place of the one it went on from, where it had one."""
    return s["state"].copy_(state) if "state" in s else state


def _recurrence(a, b):
    """h_t = a_t h_{t-1} + b_t over dimension 1 from h_{-1} = 0, in place of b, by doubling; a is used up."""
    step = 1
    while step < a.shape[1]:
        b[:, step:] += a[:, step:] * b[:, :-step]
        a[:, step:] = a[:, step:] * a[:, :-step]
        step *= 2
    return b


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _gates(s):
    """Decay, the weight of the input, and the input after its gate (with the gate)."""
    r = s["r"].float()
    open_ = _sigmoid(r)
    if "rate" in s:
        u = s["rate"] * open_
        a, w = torch.exp(-u), torch.sqrt(-torch.expm1(-2 * u))
    else:
        u, a, w = None, _sigmoid(-r), open_
    x = s["x"].float()
    gate = _sigmoid(s["i"].float()) if "i" in s else None
    return open_, u, a, w, x if gate is None else gate * x, gate


def _plain_gated(s):
    live = _live(s)
    _, _, a, w, v, _ = _gates(s)
    a, b = (a, w * v) if live is None else (torch.where(live, a, 1.0), _keep(live, w * v))
    if "state" in s:
        b[:, 0] += a[:, 0] * s["state"]
    h = _recurrence(a.clone(), b)
    y = h
    if "z" in s:
        z = s["z"].float()
        y = h * z * _sigmoid(z)
    return {"out": _keep(live, y).to(s["x"].dtype), "state": _advance(s, h[:, -1].contiguous())}


def _plain_gated_train(s):
    dt = s["x"].dtype
    live = _live(s)
    open_, u, a, w, v, gate = _gates(s)
    a, b = (a, w * v) if live is None else (torch.where(live, a, 1.0), _keep(live, w * v))
    first = s["state"] if "state" in s else torch.zeros_like(b[:, 0])
    b[:, 0] += a[:, 0] * first
    h = _recurrence(a.clone(), b)
    before = torch.cat([first[:, None], h[:, :-1]], 1)
    dout = _keep(live, s["dout"].float())
    got, y, dh = {}, h, dout.clone()
    if "z" in s:
        z = _keep(live, s["z"].float())
        sig = _sigmoid(z)
        y, dh = h * z * sig, dout * z * sig
        got["dz"] = (dout * h * sig * (1 + z * (1 - sig))).to(dt)
    got["out"] = _keep(live, y).to(dt)
    if "dfinal" in s:
        dh[:, -1] += s["dfinal"]
    ahead = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)  # a_{t+1}
    dh = _recurrence(ahead.flip(1), dh.flip(1)).flip(1)
    dv = _keep(live, dh * w)
    if gate is None:
        got["dx"] = dv.to(dt)
    else:
        got["dx"] = (dv * gate).to(dt)
        got["di"] = (dv * v * (1 - gate)).to(dt)
    da, dw = dh * before, dh * v
    if "rate" in s:
        du = _keep(live, dw * a * a / w - da * a)  # w = sqrt(1 - exp(-2 u))
        got["dr"] = (du * u * (1 - open_)).to(dt)
        got["drate"] = (du * open_).double().sum((0, 1)).float()
    else:
        got["dr"] = _keep(live, (dw - da) * open_ * _sigmoid(-s["r"].float())).to(dt)
    if "state" in s:
        got["dinit"] = dh[:, 0] * a[:, 0]
        got["state"] = _advance(s, h[:, -1])
    return got


def _plain_gated_step(s):
    _, _, a, w, v, _ = _gates(s)
    h = a * s["state"] + w * v
    y = h
    if "z" in s:
        z = s["z"].float()
        y = h * z * _sigmoid(z)
    return {"out": y.to(s["x"].dtype), "state": _advance(s, h)}


def _plain_beam(s):
    b, k, v = s["logits"].shape
    # the first k tokens of every beam, by value and then by place: one whole number for both
    x = s["logits"].float() + 0.0
    bits = x.view(torch.int32).long()
    place = torch.arange(v, device=x.device)
    keys = torch.where(bits >= 0, bits, -(bits & 0x7FFFFFFF)) * (1 << 32) + (v - 1 - place)
    del bits
    tokens = v - 1 - (torch.topk(keys, min(k, v), dim=2).values & 0xFFFFFFFF)
    del keys
    wide = x.double()
    top = wide.amax(2, keepdim=True)
    wide -= top
    total = torch.log(wide.exp_().sum(2, keepdim=True))
    score = s["prior"].double()[..., None] + ((torch.gather(x, 2, tokens).double() - top) - total)
    if "finished" in s:  # goes on with its end and nothing else
        j = torch.arange(tokens.shape[2], device=x.device)
        others = torch.where(j - 1 < s["eos"], j - 1, j)
        done = (s["finished"] != 0)[..., None]
        tokens = torch.where(done, torch.where(j == 0, s["eos"], others), tokens)
        score = torch.where(done, torch.where(j == 0, s["prior"].double()[..., None], float("-inf")), score)
    # all beams' candidates by their place, then by score: equal scores stay in order
    flat = (tokens + torch.arange(k, device=x.device)[:, None] * v).flatten(1)
    flat, order = torch.sort(flat, dim=1)
    score, order = torch.sort(torch.gather(score.flatten(1), 1, order), dim=1, descending=True, stable=True)
    flat, score = torch.gather(flat, 1, order)[:, :k], score[:, :k]
    parents = flat // v
    finished = flat % v == s["eos"]
    if "finished" in s:
        finished |= torch.gather(s["finished"], 1, parents) != 0
    got = {"tokens": (flat % v).to(torch.int32), "parents": parents.to(torch.int32), "scores": score.float(),
           "finished": finished.to(torch.uint8)}
    if "slots" in s:
        # a beam's first child goes on in its slot, the others take slots that no beam goes on in, in order
        first = (parents[:, :, None] == parents[:, None, :]).long().argmax(2) == torch.arange(k, device=x.device)
        used = torch.zeros(b, k, dtype=torch.bool, device=x.device).scatter_(1, parents, True)
        free = torch.gather(s["slots"], 1, torch.sort(used.long(), dim=1, stable=True).indices)
        rank = (torch.cumsum((~first).long(), 1) - 1).clamp(min=0)
        old = torch.gather(s["slots"], 1, parents)
        new = torch.where(first, old, torch.gather(free, 1, rank))
        none = torch.full_like(new, -1)
        got.update(slots=s["slots"].copy_(new), src=torch.where(first, none, old), dst=torch.where(first, none, new))
    return got


def _plain_copy(s):
    src, dst = s["src"].flatten().long(), s["dst"].flatten().long()
    # a pair that copies nothing copies a row that others copy from, which none copies to, to itself
    on, same = (src >= 0) & (dst >= 0), src.max().clamp(min=0)
    src, dst = torch.where(on, src, same), torch.where(on, dst, same)
    for pool in (s["conv"], s["state"]):
        pool[:, dst] = pool[:, src]
    return {"conv": s["conv"], "state": s["state"]}


_PLAIN = {"gated": _plain_gated, "gated_train": _plain_gated_train, "gated_step": _plain_gated_step, "beam": _plain_beam,
          "copy": _plain_copy}
_OWN = {"gated": _own_gated, "gated_train": _own_gated_train, "gated_step": _own_gated_step, "beam": _own_beam,
        "copy": _own_copy}


def run(state):
    if own:
        import prefix_scan_row_gb300 as mt
        return _OWN[state["op"]](state, mt)
    return _PLAIN[state["op"]](state)


# --- what a pass cannot do without ----------------------------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "beam":
        b, k, v = case["batch"], case["beams"], case["vocab"]
        rows = b * (k - case["finished"])  # a finished beam's logits decide nothing
        return {"bytes": rows * v * BYTES[case["dtype"]] + b * k * (4 + 14 + (16 if case["slots"] else 0)), "flops": 4 * rows * v}
    if op == "copy":
        row = case["layers"] * _row_bytes(case)
        made = case["beams"] - case["kept"]
        return {"bytes": case["groups"] * row * (made + min(made, case["kept"])), "flops": 0}
    e = BYTES[case["dtype"]]
    pairs = case["batch"] * case.get("length", 1) * case["dim"]
    inputs = 2 + case["input_gate"] + case["z"]
    rate = case["decay"] == "rate"
    params = 4 * case["dim"] * rate
    state = 4 * case["batch"] * case["dim"]
    flops = 10 + 12 * rate + 5 * case["input_gate"] + 6 * case["z"]
    if op == "gated_step":
        return {"bytes": pairs * e * (inputs + 1) + 2 * state + params, "flops": pairs * flops}
    if op == "gated":
        return {"bytes": pairs * e * (inputs + 1) + state * (1 + case["ragged"]) + params, "flops": pairs * flops}
    # inputs and dout read once, out and a gradient for each input written once
    return {"bytes": pairs * e * (2 * inputs + 2) + state * 4 * case["ragged"] + 2 * params, "flops": pairs * flops * 3}


# --- the definition in 64 bits --------------------------------------------------------------------------------------


def _sigmoid64(x):
    return 0.5 * (1 + torch.tanh(0.5 * x.double()))


def _exact_gated(case, s):
    """The recurrence one token after the other, and its adjoint one token before the other."""
    b, t, d = s["x"].shape
    f, dev, train = torch.float64, s["x"].device, case["op"] == "gated_train"
    ends = s["lens"].long() if "lens" in s else torch.full((b,), t, device=dev)
    h = s["state"].double() if "state" in s else torch.zeros(b, d, dtype=f, device=dev)
    out = torch.zeros(b, t, d, dtype=f, device=dev)
    past = torch.empty(t, b, d, dtype=f, device=dev) if train else None

    def token(n):
        opened = _sigmoid64(s["r"][:, n])
        if "rate" in s:
            log_decay = -s["rate"].double() * opened
            a = torch.exp(log_decay)
            w = torch.sqrt(-torch.expm1(2 * log_decay))
        else:
            log_decay, a, w = None, _sigmoid64(-s["r"][:, n].double()), opened
        i = _sigmoid64(s["i"][:, n]) if "i" in s else torch.ones_like(opened)
        return opened, log_decay, a, w, i, s["x"][:, n].double()

    for n in range(t):
        on = (n < ends)[:, None]
        if train:
            past[n] = h
        _, _, a, w, i, x = token(n)
        new = a * h + w * (i * x)
        h = torch.where(on, new, h)
        y = new
        if "z" in s:
            z = s["z"][:, n].double()
            y = new * (z * _sigmoid64(z))
        out[:, n] = torch.where(on, y, 0.0)
    if not train:
        return {"out": out, "state": h}
    got = {"out": out}
    for k in ("x", "r", "i", "z"):
        if k in s:
            got["d" + k] = torch.zeros(b, t, d, dtype=f, device=dev)
    if "rate" in s:
        got["drate"] = torch.zeros(d, dtype=f, device=dev)
    dh = s["dfinal"].double() if "dfinal" in s else torch.zeros(b, d, dtype=f, device=dev)
    for n in reversed(range(t)):
        on = (n < ends)[:, None]
        opened, log_decay, a, w, i, x = token(n)
        dy = s["dout"][:, n].double()
        full = dh + dy
        if "z" in s:
            z = s["z"][:, n].double()
            sig = _sigmoid64(z)
            now = a * past[n] + w * (i * x)
            got["dz"][:, n] = torch.where(on, dy * now * (sig + z * sig * (1 - sig)), 0.0)
            full = dh + dy * z * sig
        got["dx"][:, n] = torch.where(on, full * w * i, 0.0)
        if "i" in s:
            got["di"][:, n] = torch.where(on, full * w * x * i * (1 - i), 0.0)
        # by the decay and by the weight, which both follow the recurrence gate
        to_a, to_w = full * past[n], full * i * x
        if "rate" in s:
            to_log = to_a * a - to_w * torch.exp(2 * log_decay) / w
            got["dr"][:, n] = torch.where(on, to_log * log_decay * (1 - opened), 0.0)
            got["drate"] -= torch.where(on, to_log * opened, 0.0).sum(0)
        else:
            got["dr"][:, n] = torch.where(on, (to_w - to_a) * opened * (1 - opened), 0.0)
        dh = torch.where(on, full * a, dh)
    if "state" in s:
        got.update(state=h, dinit=dh)
    return got


def _exact_beam(case, s):
    """Every sequence by itself: all of its continuations in one row of 64-bit scores, sorted."""
    b, k, v = s["logits"].shape
    got = {name: [] for name in ("tokens", "parents", "scores", "finished", "slots", "src", "dst")}
    prior = s["prior"].double()
    done_all = s["finished"].tolist() if "finished" in s else [[0] * k] * b
    slots_all = s["slots"].tolist() if "slots" in s else None
    for n in range(b):
        x = s["logits"][n].double()
        score = prior[n][:, None] + (x - torch.logsumexp(x, 1, keepdim=True))
        for j in range(k):
            if done_all[n][j]:
                score[j] = float("-inf")
                score[j, s["eos"]] = prior[n, j]
        value, flat = torch.sort(score.flatten(), descending=True, stable=True)
        value, flat = value[:k], flat[:k].tolist()
        parents = [p // v for p in flat]
        got["tokens"].append([p % v for p in flat])
        got["parents"].append(parents)
        got["scores"].append(value)
        got["finished"].append([int(bool(done_all[n][p // v]) or p % v == s["eos"]) for p in flat])
        if slots_all is not None:
            old = slots_all[n]
            free = [old[j] for j in range(k) if j not in parents]
            taken, now, src, dst = set(), [], [], []
            for p in parents:
                if p in taken:
                    now.append(free.pop(0))
                    src.append(old[p])
                    dst.append(now[-1])
                else:
                    taken.add(p)
                    now.append(old[p])
                    src.append(-1)
                    dst.append(-1)
            for name, row in (("slots", now), ("src", src), ("dst", dst)):
                got[name].append(row)
    whole = lambda rows, dtype: torch.tensor(rows, dtype=dtype, device="cuda")  # noqa: E731
    r = {"tokens": whole(got["tokens"], torch.int32), "parents": whole(got["parents"], torch.int32),
         "scores": torch.stack(got["scores"]), "finished": whole(got["finished"], torch.uint8)}
    if slots_all is not None:
        r.update({name: whole(got[name], torch.int32) for name in ("slots", "src", "dst")})
    return r


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "beam":
        return _exact_beam(case, s)
    if op == "copy":
        pairs = [(p, q) for p, q in zip(s["src"].flatten().tolist(), s["dst"].flatten().tolist()) if p >= 0 and q >= 0]
        for p, q in pairs:
            for name in ("conv", "state"):
                s[name][:, q].copy_(s[name][:, p])
        return {"conv": s["conv"].double(), "state": s["state"].double()}
    if op == "gated_step":
        wide = {k: (v[:, None] if k in ("x", "r", "i", "z") else v) for k, v in s.items()}
        got = _exact_gated(dict(case, op="gated"), wide)
        return {"out": got["out"][:, 0], "state": got["state"]}
    return _exact_gated(case, s)
