"""The gated scan, the beam selection and the state copies together and as parts of larger programs: a search of the example
model against whole prompts, a recurrent model's search step in a CUDA graph, several host threads, memory the kernels
cannot reach, offsets past 32 bits."""
import os
import subprocess
import sys
import threading

import pytest
import torch

import gated_ref as G

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.fixture(scope="module")
def mt():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import prefix_scan_row_gb300 as m
    return m


@pytest.fixture(scope="module")
def example(mt):
    import sequence_model
    return sequence_model


@pytest.mark.parametrize("beams,eos", [(1, -1), (3, -1), (4, 5), (8, 0)])
def test_search_agrees_with_whole_prompts(example, beams, eos):
    """Every hypothesis run from its first token, without states, and all continuations of a prompt's sorted in 64 bits. Scores
    are sums of `steps` log-probabilities of f32 logits, which differ by the order of f32 sums between a prompt and its
    tokens: 1e-4 of their size, as for the example's other test of that."""
    m = example.SequenceModel(vocab=12, dim=32, inner=48, nstate=8, dtype=torch.float32, seed=2)
    m.w["table"] *= 3.0  # distributions with some shape
    steps, prompts = 5, example.counting(3, 9, 12, 4)
    lens = torch.tensor([9, 4, 7], dtype=torch.int32, device="cuda")
    tokens, scores = m.search(prompts, lens, beams, steps, eos)
    for n in range(3):
        head = prompts[n, :int(lens[n])].tolist()
        hyps = [([], 0.0)]
        for _ in range(steps):
            rows = []
            for words, score in hyps:
                if eos >= 0 and eos in words:
                    row = torch.full((12,), float("-inf"), dtype=torch.float64)
                    row[eos] = score
                else:
                    t = torch.tensor([head + words], dtype=torch.int32, device="cuda")
                    logits = m.prompt(t, torch.tensor([t.shape[1]], dtype=torch.int32, device="cuda"), m.new_states(1))[0]
                    row = score + torch.log_softmax(logits.double().cpu(), 0)
                rows.append(row)
            order = torch.sort(torch.cat(rows), descending=True, stable=True)
            hyps = [(hyps[i // 12][0] + [i % 12], float(v)) for v, i in zip(order.values[:beams], order.indices[:beams].tolist())]
        assert tokens[n].tolist() == [w for w, _ in hyps]
        assert all(abs(float(a) - b) <= 1e-4 * (1 + abs(b)) for a, (_, b) in zip(scores[n], hyps))


class Search:
    """Beam search with a gated recurrence: the lookup of the last tokens, one step of every beam's state in a pool of two layers,
    logits, selection in place, copies of states."""

    def __init__(self, mt, seed=0, batch=3, beams=4, vocab=50, d=64, layers=2, length=21):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, by=1.0: (torch.randn(*s, generator=g) * by).cuda()  # noqa: E731
        self.mt, self.b, self.k, self.v, self.d, self.layers = mt, batch, beams, vocab, d, layers
        self.table, self.gate, self.head = r(vocab, d), r(layers, d, 3 * d, by=d ** -0.5), r(d, vocab, by=2 * d ** -0.5)
        self.rate = torch.rand(layers, d, generator=g).cuda()
        self.prompts = torch.randint(0, vocab, (batch, length), generator=g).to(torch.int32).cuda()
        self.lens = torch.tensor([length, 5, 14][:batch], dtype=torch.int32, device="cuda")
        self.pool = torch.full((layers, batch * beams + 1, d), float("nan"), device="cuda")
        new = lambda dtype: torch.zeros(batch, beams, dtype=dtype, device="cuda")  # noqa: E731
        self.tokens, self.parents, self.src, self.dst = (new(torch.int32) for _ in range(4))
        self.scores, self.finished = new(torch.float32), new(torch.uint8)
        self.first = torch.randperm(batch * beams, generator=g).to(torch.int32).cuda().view(batch, beams)
        self.slots = self.first.clone()
        self.scratch = torch.empty(max(mt.mt_beam_select_scratch_slots(batch, k, beams, vocab) for k in (1, beams)), dtype=torch.int64,
                                   device="cuda")
        n = batch * beams
        self.e, self.h, self.y = torch.empty(n, d, device="cuda"), torch.empty(n, d, device="cuda"), torch.empty(n, d, device="cuda")

    def begin(self):
        mt, b, t = self.mt, self.b, self.prompts.shape[1]
        x = torch.empty(b, t, self.d, device="cuda")
        mt.mt_embed(self.prompts, self.table, x)
        slots = self.slots[:, 0].contiguous()
        for n in range(self.layers):
            p = x @ self.gate[n]
            out = torch.empty_like(x)
            mt.mt_gated_scan(x, p[..., :self.d], out, i=p[..., self.d:2 * self.d], z=p[..., 2 * self.d:], rate=self.rate[n],
                             state=self.pool[n], slots=slots, lens=self.lens)
            x = x + out
        last = x[torch.arange(b, device="cuda"), self.lens.long() - 1]
        self.select((last @ self.head).view(b, 1, self.v))

    def select(self, logits, **more):
        mt = self.mt
        mt.mt_beam_select(logits, self.tokens, self.parents, self.scores, self.scratch, finished_out=self.finished, eos=3, slots=self.slots,
                          src=self.src, dst=self.dst, **more)
        mt.mt_state_copy(self.src, self.dst, self.pool, axis=1)

    def step(self):
        mt, d = self.mt, self.d
        mt.mt_embed(self.tokens.view(-1), self.table, self.e)
        self.h.copy_(self.e)
        for n in range(self.layers):
            p = self.h @ self.gate[n]
            mt.mt_gated_scan_step(self.h, p[:, :d], self.pool[n], self.y, i=p[:, d:2 * d], z=p[:, 2 * d:], rate=self.rate[n],
                                  slots=self.slots.view(-1))
            self.h.add_(self.y)
        self.select((self.h @ self.head).view(self.b, self.k, self.v), prior=self.scores, finished=self.finished)

    def results(self):
        return [t.clone() for t in (self.tokens, self.parents, self.scores, self.finished, self.slots, self.pool[:, :-1])]


def reference(s, steps):
    """The same search in 64 bits, with a list of hypotheses that each keep their own states."""
    f = torch.float64
    w = {n: getattr(s, n).detach().cpu().to(f) for n in ("table", "gate", "head", "rate")}

    def token(states, t):
        x = w["table"][t]
        new = []
        for n in range(s.layers):
            p = x @ w["gate"][n]
            r, i, z = p[:s.d], p[s.d:2 * s.d], p[2 * s.d:]
            u = w["rate"][n] * torch.sigmoid(r)
            h = torch.exp(-u) * states[n] + torch.sqrt(-torch.expm1(-2 * u)) * torch.sigmoid(i) * x
            new.append(h)
            x = x + h * z * torch.sigmoid(z)
        return new, torch.log_softmax(x @ w["head"], 0)

    out = []
    for b in range(s.b):
        states = [torch.zeros(s.d, dtype=f)] * s.layers
        for t in s.prompts[b, :int(s.lens[b])].tolist():
            states, logp = token(states, t)
        beams = [(states, logp, 0.0, False, [])]
        for step in range(steps):
            rows = []
            for _, logp, score, done, _ in beams:
                row = torch.full((s.v,), float("-inf"), dtype=f)
                if done:
                    row[3] = score
                else:
                    row = score + logp
                rows.append(row)
            top = torch.sort(torch.cat(rows), descending=True, stable=True)
            gap = (top.values[:s.k] - top.values[1:s.k + 1]).min()
            assert gap > 1e-4, "the inputs leave the order open"  # far above the f32 run's rounding
            new = []
            for value, i in zip(top.values[:s.k].tolist(), top.indices[:s.k].tolist()):
                states, _, _, done, words = beams[i // s.v]
                t = i % s.v
                nstates, logp = token(states, t)
                new.append((nstates, logp, value, done or t == 3, words + [t], states))
            last, beams = new, [n[:5] for n in new]
        out.append([(words, value, done, states) for _, _, value, done, words, states in last])
    return out


@pytest.mark.parametrize("beams", [2, 4])
def test_a_search_with_the_gated_scan(mt, beams):
    """Tokens, marks and scores after every step, and at the end each beam's states where its slot says. The states are those before
    the last tokens; f32 against 64 bits over 21 + 6 tokens of 64 channels."""
    steps = 6
    s = Search(mt, seed=5, beams=beams)
    path = []
    s.begin()
    path.append((s.tokens.cpu(), s.parents.cpu()))
    for _ in range(steps - 1):
        s.step()
        path.append((s.tokens.cpu(), s.parents.cpu()))
    want = reference(s, steps)
    pool, slots = s.pool.cpu(), s.slots.cpu()
    for b in range(s.b):
        assert sorted(slots[b].tolist()) == sorted(s.first[b].tolist())
        for k in range(s.k):
            words, at = [], k
            for tokens, parents in reversed(path):
                words.append(int(tokens[b, at]))
                at = int(parents[b, at])
            want_words, score, done, states = want[b][k]
            assert words[::-1] == want_words and bool(s.finished[b, k]) == done
            assert abs(float(s.scores[b, k]) - score) < 1e-4
            for n in range(s.layers):
                assert (pool[n, int(slots[b, k])].double() - states[n]).abs().max() < 1e-4
    assert pool[:, -1].isnan().all()  # a row that no beam has


def test_the_search_step_replays_in_a_cuda_graph(mt):
    a, b = Search(mt, seed=7), Search(mt, seed=7)
    a.begin()
    a.step()
    b.begin()
    b.step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for _ in range(5):
        a.step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.results(), b.results()))
    assert mt.mt_scan_status() == 0


def test_first_calls_inside_a_capture(mt):
    """A process whose first launches of each call are captured: nothing that a first call does disturbs a capture."""
    code = """
import torch, prefix_scan_row_gb300 as mt
dev = dict(device="cuda")
x = torch.randn(2, 300, 96, **dev).half()
out, st, rate = torch.empty_like(x), torch.zeros(2, 96, **dev), torch.rand(96, **dev)
ck = torch.empty(mt.mt_gated_scan_checkpoint_slots(2, 300, 96), dtype=torch.int64, **dev)
sc = torch.empty(mt.mt_gated_scan_scratch_slots(2, 300, 96), dtype=torch.int64, **dev)
g = [torch.empty_like(x) for _ in range(4)]
dr = torch.empty_like(rate)
lg = torch.randn(2, 3, 40000, **dev)
i = lambda: torch.empty(2, 3, dtype=torch.int32, **dev)
tok, par, src, dst, sl = i(), i(), i(), i(), torch.arange(6, dtype=torch.int32, **dev).view(2, 3)
sco = torch.empty(2, 3, **dev)
bs = torch.empty(mt.mt_beam_select_scratch_slots(2, 3, 3, 40000), dtype=torch.int64, **dev)
pool = torch.randn(6, 1000, **dev)
def run():
    mt.mt_gated_scan(x, x, out, i=x, z=x, rate=rate, state=st, checkpoints=ck)
    mt.mt_gated_scan_grad(x, x, x, ck, g[0], g[1], sc, i=x, di=g[2], z=x, dz=g[3], rate=rate, drate=dr)
    mt.mt_gated_scan_step(x[:, 0], x[:, 1], st, out[:, 0], rate=rate)
    mt.mt_beam_select(lg, tok, par, sco, bs, slots=sl, src=src, dst=dst)
    mt.mt_state_copy(src, dst, pool)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    run()
keep = pool.clone(), sl.clone()
graph.replay()
torch.cuda.synchronize()
first = [t.clone() for t in (out, st, dr, *g, tok, par, sco, pool, sl)]
pool.copy_(keep[0]); sl.copy_(keep[1])
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, (out, st, dr, *g, tok, par, sco, pool, sl)))
assert mt.mt_scan_status() == 0
"""
    subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, timeout=300)


def test_searches_from_many_threads(mt):
    want = []
    for n in range(4):
        s = Search(mt, seed=20 + n)
        s.begin()
        for _ in range(4):
            s.step()
        want.append(s.results())
    runs = [Search(mt, seed=20 + n) for n in range(4)]
    torch.cuda.synchronize()

    def work(s):
        with torch.cuda.stream(torch.cuda.Stream()):
            s.begin()
            for _ in range(4):
                s.step()
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(s,)) for s in runs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for w, s in zip(want, runs):
        assert all(torch.equal(a, b) for a, b in zip(w, s.results()))


def test_an_explicit_stream_and_the_launch_counter(mt):
    x = torch.randn(2, 70, 64, device="cuda")
    out, other = torch.empty_like(x), torch.empty_like(x)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    before = mt.mt_scan_launches()
    mt.mt_gated_scan(x, x, out, stream=side)
    side.synchronize()
    assert mt.mt_scan_launches() == before + 1
    mt.mt_gated_scan(x, x, other)
    assert torch.equal(out, other)


def test_host_memory_is_refused(mt):
    x = torch.randn(2, 8, 16, device="cuda")
    pinned = lambda t: t.cpu().pin_memory()  # noqa: E731
    t = torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    o = lambda: torch.zeros_like(t)  # noqa: E731
    logits, scores = torch.randn(2, 3, 40, device="cuda"), torch.zeros(2, 3, device="cuda")
    scratch = torch.empty(mt.mt_beam_select_scratch_slots(2, 3, 3, 40), dtype=torch.int64, device="cuda")
    calls = [lambda: mt.mt_gated_scan(pinned(x), x, torch.empty_like(x)),
             lambda: mt.mt_gated_scan(x, x, torch.empty_like(x), state=pinned(x[:, 0])),
             lambda: mt.mt_gated_scan_step(x[:, 0], x[:, 0], pinned(x[:, 0]), torch.empty(2, 16, device="cuda")),
             lambda: mt.mt_beam_select(pinned(logits), o(), o(), scores, scratch),
             lambda: mt.mt_beam_select(logits, o(), o(), scores, scratch, prior=pinned(scores)),
             lambda: mt.mt_state_copy(t, o(), pinned(x)),
             lambda: mt.mt_state_copy(pinned(t), o(), x)]
    for call in calls:
        with pytest.raises(mt.ScanError) as e:
            call()
        assert e.value.code == mt.MT_ERR_MEMORY


def test_offsets_past_32_bits(mt):
    """Rows 60,000 values apart, 40,000 of them (2.4e9 values), a state in row 3e7 of a pool, and logits of beams 2^31 + 8 values
    apart: the same bits as of contiguous ones."""
    g = torch.Generator(device="cuda").manual_seed(3)
    length, d, gap = 40_000, 64, 60_000
    x = torch.randn(1, length, d, generator=g, device="cuda").to(torch.bfloat16)
    far = lambda: torch.empty(length * gap, dtype=torch.bfloat16, device="cuda").view(1, length, gap)[:, :, 8:8 + d]  # noqa: E731
    xs, out_s = far(), far()
    xs.copy_(x)
    rate = torch.rand(d, generator=g, device="cuda")
    out = torch.empty_like(x)
    ck = torch.empty(mt.mt_gated_scan_checkpoint_slots(1, length, d), dtype=torch.int64, device="cuda")
    pool = torch.empty(34_000_000, d, device="cuda")
    at = torch.tensor([33_999_999], dtype=torch.int32, device="cuda")
    state = torch.randn(1, d, generator=g, device="cuda")
    pool[33_999_999] = state[0]
    mt.mt_gated_scan(x, x, out, rate=rate, state=state, carry_in=True)
    mt.mt_gated_scan(xs, xs, out_s, rate=rate, state=pool, carry_in=True, slots=at)
    assert torch.equal(out, out_s) and torch.equal(pool[33_999_999], state[0])
    one = torch.empty(1, d, dtype=torch.bfloat16, device="cuda")
    mt.mt_gated_scan_step(x[:, 0], x[:, 1], pool, one, rate=rate, slots=at)
    two = torch.empty_like(one)
    mt.mt_gated_scan_step(x[:, 0], x[:, 1], state, two, rate=rate)
    assert torch.equal(one, two) and torch.equal(pool[33_999_999], state[0])
    del pool
    mt.mt_gated_scan(x, x, out, rate=rate, checkpoints=ck)
    scratch = torch.empty(mt.mt_gated_scan_scratch_slots(1, length, d), dtype=torch.int64, device="cuda")
    near = [torch.empty_like(x), torch.empty_like(x), torch.empty_like(rate)]
    mt.mt_gated_scan_grad(x, x, x, ck, near[0], near[1], scratch, rate=rate, drate=near[2])
    dr_s, drate = far(), torch.empty_like(rate)
    mt.mt_gated_scan_grad(xs, xs, xs, ck, out_s, dr_s, scratch, rate=rate, drate=drate)
    assert torch.equal(near[0], out_s) and torch.equal(near[1], dr_s) and torch.equal(near[2], drate)
    del xs, out_s, dr_s

    step = (1 << 31) + 8
    logits = torch.randn(1, 2, 5000, generator=g, device="cuda").half()
    wide = torch.empty(step + 5000, dtype=torch.float16, device="cuda").as_strided((1, 2, 5000), (step, step, 1))
    wide.copy_(logits)
    results = []
    for lg in (logits, wide):
        tokens, parents = (torch.empty(1, 2, dtype=torch.int32, device="cuda") for _ in range(2))
        scores = torch.empty(1, 2, device="cuda")
        mt.mt_beam_select(lg, tokens, parents, scores, torch.empty(mt.mt_beam_select_scratch_slots(1, 2, 2, 5000), dtype=torch.int64, device="cuda"))
        results.append((tokens, parents, scores))
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rate,i,z", [(True, True, True), (False, False, False)])
def test_many_sequences(mt, dtype, rate, i, z):
    """More CTAs than three an SM, whose prompts and gradients smaller CTAs take."""
    from test_gpu_gated_scan import Inputs, check_forward, check_gradient
    lens = torch.arange(60, dtype=torch.int32) + 11
    p = Inputs(dtype, 60, 70, 512, rate, i, z, lens=lens)
    check_forward(mt, p)
    check_gradient(mt, p)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_logits_far_out(mt, dtype):
    """Largest values above 2^22, where sums are made another way, in some spans of a row or in all, and next to that border."""
    from test_gpu_beam_select import check, rows
    x, prior, _, g = rows(dtype, 2, 3, 20000, 9)
    if dtype == torch.float32:
        x[0, 0] = 4194304.0 + torch.randint(-40, 40, (20000,), generator=g) * 0.5
        x[0, 1, 7000:] += 4.19e6
        x[1, 2] = -5e6 - torch.rand(20000, generator=g) * 20
    elif dtype == torch.bfloat16:
        x[0, 0] = 2.0 ** 23
        x[0, 1, 5::7] = 2.0 ** 22
    x[1, 0] = torch.finfo(dtype).min
    x[1, 0, 11], x[1, 1, 1::2] = -3.0, torch.finfo(dtype).max
    check(mt, x, 3, prior)
    check(mt, x, 9, prior - 1e4)


def test_more_equal_groups_and_vectors_than_there_is_place_for(mt):
    """The selection's last resort. 35,200 groups of logits, of which every 32nd part's 1,100 are high and the rest low; and 31 of
    32 parts of a beam's vectors equal: more than reach any threshold that the parts give."""
    beams, per_beam, group = 32, 1100, 1024
    x = torch.full((1, beams, per_beam, group), -8.0, dtype=torch.bfloat16, device="cuda")
    i = torch.arange(beams * per_beam, device="cuda").view(beams, per_beam)
    x[0][i % 512 < 16] = 2.0
    x[0, 3, 500, 77] = 3.0
    x = x.view(1, beams, per_beam * group)
    out = lambda dtype: torch.empty(1, beams, dtype=dtype, device="cuda")  # noqa: E731
    tokens, parents, scores = out(torch.int32), out(torch.int32), out(torch.float32)
    scratch = torch.empty(mt.mt_beam_select_scratch_slots(1, beams, beams, per_beam * group), dtype=torch.int64, device="cuda")
    mt.mt_beam_select(x, tokens, parents, scores, scratch)
    lse = torch.logsumexp(x[0].double(), 1)
    cands = []  # every beam's first tokens, with their scores
    for b in range(beams):
        for t in torch.sort(x[0, b].float(), descending=True, stable=True).indices[:beams].tolist():
            cands.append((-float(x[0, b, t].double() - lse[b]), b, t))
    want = sorted(cands)[:beams]
    assert tokens[0].tolist() == [t for _, _, t in want] and parents[0].tolist() == [b for _, b, _ in want]

    y = torch.ones(1, 1, 32 * group, dtype=torch.bfloat16)
    v = torch.arange(32 * group) // 8
    y[0, 0, v % 512 < 16] = 0.0
    from test_gpu_beam_select import check
    check(mt, y, 32)
    assert G.beam_select(y, 32)["tokens"][0, 0] == 128
