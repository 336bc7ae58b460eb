"""A small language model made of the library's sequence operators: trained for
a few steps, then used as it would be served (prompts, then single tokens).

    tokens -> embedding -> x, z = projection -> short convolution + SiLU -> step sizes, B, C = projection
           -> selective scan with gate -> projection -> + -> logits (the embedding's table, transposed)

Forward and backward of the embedding, the convolution and the scan are the
library's calls; the projections are torch matrix products. Run it on a GB300:

    python examples/sequence_model.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import prefix_scan_row_gb300 as mt  # noqa: E402


class SequenceModel:
    def __init__(self, vocab=512, dim=256, inner=512, nstate=16, width=4, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s, by: torch.randn(*s, generator=g, device="cuda") * by  # noqa: E731
        self.vocab, self.dim, self.inner, self.nstate, self.width, self.dtype = vocab, dim, inner, nstate, width, dtype
        step = torch.exp(torch.rand(inner, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
        # master weights, f32
        self.w = dict(
            table=r(vocab, dim, by=dim ** -0.5), into=r(dim, 2 * inner, by=dim ** -0.5), conv=r(inner, width, by=width ** -0.5),
            conv_bias=torch.zeros(inner, device="cuda"), select=r(inner, inner + 2 * nstate, by=inner ** -0.5),
            delta_bias=step + torch.log(-torch.expm1(-step)),
            A_log=torch.log(torch.arange(1, nstate + 1, device="cuda").float()).repeat(inner, 1), D=torch.ones(inner, device="cuda"),
            out=r(inner, dim, by=inner ** -0.5))
        self.moments, self.steps = {k: (torch.zeros_like(v), torch.zeros_like(v)) for k, v in self.w.items()}, 0
        self.scratch = {}

    def _slots(self, name, n):
        """Workspace kept from call to call."""
        t = self.scratch.get(name)
        if t is None or t.numel() < n:
            t = self.scratch[name] = torch.empty(n, dtype=torch.int64, device="cuda")
        return t

    def _cast(self):
        return {k: v.to(self.dtype) if k in ("table", "into", "select", "out") else v for k, v in self.w.items()}

    def _mix(self, c, e, conv_state=None, scan_state=None, carry=False, lens=None, checkpoints=None):
        """The token mixer on embedded prompts [batch, len, dim]; everything the backward pass needs."""
        b, t, _ = e.shape
        d, n = self.inner, self.nstate
        xz = e @ c["into"]
        x, z = xz[..., :d], xz[..., d:]  # halves of one projection's rows, used where they lie
        v = torch.empty(b, t, d, dtype=self.dtype, device="cuda")
        mt.mt_causal_conv(x, c["conv"], v, bias=c["conv_bias"], state=conv_state, carry_in=carry, lens=lens)
        p = v @ c["select"]
        delta, B, C = p[..., :d], p[..., d:d + n].unsqueeze(2), p[..., d + n:].unsqueeze(2)
        A = -torch.exp(c["A_log"])
        y = torch.empty(b, t, d, dtype=self.dtype, device="cuda")
        slots = mt.mt_selective_scan_scratch_slots(b, t, d, n)
        mt.mt_selective_scan(v, delta, A, B, C, y, self._slots("scan", slots) if slots else None, D=c["D"], z=z,
                             delta_bias=c["delta_bias"], state=scan_state, carry_in=carry, lens=lens, checkpoints=checkpoints)
        return dict(x=x, z=z, v=v, delta=delta, B=B, C=C, A=A, y=y)

    def train_step(self, tokens, lr=0.003):
        """One step on next-token prediction; returns the loss."""
        c, b, t = self._cast(), tokens.shape[0], tokens.shape[1] - 1
        d, n, dt = self.inner, self.nstate, self.dtype
        inputs, targets = tokens[:, :-1].contiguous(), tokens[:, 1:].long()
        e = torch.empty(b, t, self.dim, dtype=dt, device="cuda")
        scale = math.sqrt(self.dim)
        mt.mt_embed(inputs, c["table"], e, scale=scale)
        checkpoints = self._slots("checkpoints", mt.mt_selective_scan_checkpoint_slots(b, t, d, n))
        m = self._mix(c, e, checkpoints=checkpoints)
        hidden = e + m["y"] @ c["out"]
        logits = (hidden @ c["table"].t()).float()
        logp = torch.log_softmax(logits, -1)
        loss = -logp.gather(-1, targets[..., None]).mean()
        # backward
        g = {}
        dlogits = torch.exp(logp)
        dlogits.scatter_add_(-1, targets[..., None], torch.full_like(targets[..., None], -1, dtype=torch.float32))
        dlogits = (dlogits / (b * t)).to(dt)
        flat = lambda v: v.reshape(-1, v.shape[-1])  # noqa: E731
        dhidden = dlogits @ c["table"]
        g["table"] = (flat(dlogits).t() @ flat(hidden)).float()
        g["out"] = (flat(m["y"]).t() @ flat(dhidden)).float()
        dy = dhidden @ c["out"].t()
        new = lambda *s, dtype=dt: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        dv, dxz, dp = new(b, t, d), new(b, t, 2 * d), new(b, t, d + 2 * n)
        dA, g["D"], g["delta_bias"] = (new(*s, dtype=torch.float32) for s in ((d, n), (d,), (d,)))
        mt.mt_selective_scan_grad(
            m["v"], m["delta"], m["A"], m["B"], m["C"], dy, checkpoints, dv, dp[..., :d], dA, dp[..., d:d + n].unsqueeze(2),
            dp[..., d + n:].unsqueeze(2), self._slots("scan_grad", mt.mt_selective_scan_scratch_slots(b, t, d, n, grad=True)),
            D=c["D"], dD=g["D"], z=m["z"], dz=dxz[..., d:], delta_bias=c["delta_bias"], ddelta_bias=g["delta_bias"])
        g["A_log"] = dA * m["A"]  # A = -exp(A_log)
        g["select"] = (flat(m["v"]).t() @ flat(dp)).float()
        dv = dv + dp @ c["select"].t()
        g["conv"], g["conv_bias"] = new(d, self.width, dtype=torch.float32), new(d, dtype=torch.float32)
        mt.mt_causal_conv_grad(m["x"], c["conv"], dv, dxz[..., :d], g["conv"],
                               self._slots("conv_grad", mt.mt_causal_conv_grad_scratch_slots(b, t, d, self.width)),
                               bias=c["conv_bias"], dbias=g["conv_bias"])
        g["into"] = (flat(e).t() @ flat(dxz)).float()
        de = dhidden + dxz @ c["into"].t()
        # the table is used twice: the lookup's gradient is added to the logits'
        mt.mt_embed_grad(inputs, de, g["table"], self._slots("embed", mt.mt_embed_grad_scratch_slots(b * t, self.vocab, self.dim)),
                         scale=scale, accumulate=True)
        self.grads = g
        self.steps += 1
        for k, v in g.items():  # Adam
            m1, m2 = self.moments[k]
            m1.lerp_(v, 0.1)
            m2.lerp_(v * v, 0.01)
            self.w[k] = self.w[k] - lr * (m1 / (1 - 0.9 ** self.steps)) / ((m2 / (1 - 0.99 ** self.steps)).sqrt() + 1e-8)
        return float(loss)

    def prompt(self, tokens, lens, states):
        """Logits after the last live token of each prompt [batch, len]; `states` are left at it."""
        c = self._cast()
        e = torch.empty(*tokens.shape, self.dim, dtype=self.dtype, device="cuda")
        mt.mt_embed(tokens, c["table"], e, scale=math.sqrt(self.dim))
        m = self._mix(c, e, states[0], states[1], lens=lens)
        hidden = e + m["y"] @ c["out"]
        last = hidden[torch.arange(len(tokens), device="cuda"), lens.long() - 1]
        return (last @ c["table"].t()).float()

    def token(self, tokens, states):
        """Logits after one more token [batch] of each sequence."""
        c, b, d, n = self._cast(), len(tokens), self.inner, self.nstate
        new = lambda *s: torch.empty(*s, dtype=self.dtype, device="cuda")  # noqa: E731
        e, v, y = new(b, self.dim), new(b, d), new(b, d)
        mt.mt_embed(tokens, c["table"], e, scale=math.sqrt(self.dim))
        xz = e @ c["into"]
        mt.mt_causal_conv_step(xz[:, :d], c["conv"], states[0], v, bias=c["conv_bias"])
        p = v @ c["select"]
        mt.mt_selective_scan_step(v, p[:, :d], -torch.exp(c["A_log"]), p[:, d:d + n].unsqueeze(1), p[:, d + n:].unsqueeze(1),
                                  states[1], y, D=c["D"], z=xz[:, d:], delta_bias=c["delta_bias"])
        return ((e + y @ c["out"]) @ c["table"].t()).float()

    def new_states(self, batch):
        return (torch.empty(batch, self.width - 1, self.inner, dtype=self.dtype, device="cuda"),
                torch.empty(batch, self.inner, self.nstate, device="cuda"))


def counting(batch, length, vocab, seed):
    """Sequences that count up by a step of their own: each next token follows from the two before it."""
    g = torch.Generator().manual_seed(seed)
    start, by = torch.randint(0, vocab, (batch, 1), generator=g), torch.randint(1, 4, (batch, 1), generator=g)
    return ((start + by * torch.arange(length)) % vocab).to(torch.int32).cuda()


def main(steps=60, vocab=64, batch=16, length=65):
    model = SequenceModel(vocab=vocab)
    losses = [model.train_step(counting(batch, length, vocab, s)) for s in range(steps)]
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f} over {steps} steps")
    prompts = counting(3, 24, vocab, 999)
    lens = torch.tensor([24, 9, 17], dtype=torch.int32, device="cuda")
    states = model.new_states(3)
    logits = model.prompt(prompts, lens, states)
    for _ in range(8):
        tokens = logits.argmax(-1).to(torch.int32)
        logits = model.token(tokens, states)
    print("next tokens after 8 more:", logits.argmax(-1).tolist())
    return losses


if __name__ == "__main__":
    main()
