"""The sequence-model calls as parts of larger programs: captured in a CUDA graph, from several host threads on their own
streams, on pools and tables whose offsets pass 32 bits, on memory the kernels cannot reach, and with the launch counter."""
import threading

import pytest
import torch

import seq_ref as R
from test_gpu_selective_scan import Inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import prefix_scan_row_gb300 as m
    return m


class Layer:
    """Every call once, on buffers of its own."""

    def __init__(self, mt, seed, b=2, t=70, d=40, n=16, vocab=30):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
        z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
        self.mt = mt
        self.tok = torch.randint(0, vocab, (b, t), generator=g).to(torch.int32).cuda()
        self.table, self.e, self.dtable = r(vocab, d), z(b, t, d), z(vocab, d)
        self.w, self.v, self.cs = r(d, 4), z(b, t, d), z(b, 3, d)
        self.delta, self.B, self.C, self.z, self.A, self.D = r(b, t, d), r(b, t, 1, n), r(b, t, 1, n), r(b, t, d), -r(d, n).abs(), r(d)
        self.y, self.ss, self.one, self.oy = z(b, t, d), z(b, d, n), z(b, d), z(b, d)
        self.g = [z(b, t, d), z(b, t, d), z(d, n), z(b, t, 1, n), z(b, t, 1, n), z(b, t, d), z(d), z(b, t, d), z(d, 4)]
        s = lambda k: torch.empty(max(1, k), dtype=torch.int64, device="cuda")  # noqa: E731
        self.ck = s(mt.mt_selective_scan_checkpoint_slots(b, t, d, n))
        self.s1 = s(mt.mt_selective_scan_scratch_slots(b, t, d, n))
        self.s2 = s(mt.mt_selective_scan_scratch_slots(b, t, d, n, grad=True))
        self.s3 = s(mt.mt_causal_conv_grad_scratch_slots(b, t, d, 4))
        self.s4 = s(mt.mt_embed_grad_scratch_slots(b * t, vocab, d))

    def run(self):
        mt, g = self.mt, self.g
        mt.mt_embed(self.tok, self.table, self.e, scale=0.5)
        mt.mt_causal_conv(self.e, self.w, self.v, state=self.cs)
        mt.mt_selective_scan(self.v, self.delta, self.A, self.B, self.C, self.y, self.s1, D=self.D, z=self.z, state=self.ss,
                             checkpoints=self.ck)
        mt.mt_selective_scan_grad(self.v, self.delta, self.A, self.B, self.C, self.y, self.ck, g[0], g[1], g[2], g[3], g[4], self.s2,
                                  D=self.D, dD=g[6], z=self.z, dz=g[5])
        mt.mt_causal_conv_grad(self.e, self.w, g[0], g[7], g[8], self.s3)
        mt.mt_embed_grad(self.tok, g[7], self.dtable, self.s4, scale=0.5)
        mt.mt_causal_conv_step(self.e[:, 0], self.w, self.cs, self.one)
        mt.mt_selective_scan_step(self.one, self.delta[:, 0], self.A, self.B[:, 0], self.C[:, 0], self.ss, self.oy, D=self.D)

    def results(self):
        return [t.clone() for t in (self.e, self.v, self.cs, self.y, self.ss, self.dtable, self.one, self.oy, *self.g)]


def test_calls_replay_in_a_cuda_graph(mt):
    x = Layer(mt, 1)
    x.run()
    want = x.results()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.run()
    for t in (x.e, x.v, x.cs, x.y, x.ss, x.dtable, x.one, x.oy, *x.g):
        t.fill_(9)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, x.results()))
    assert mt.mt_scan_status() == 0


def test_calls_from_many_threads(mt):
    alone = []
    for i in range(4):
        x = Layer(mt, i)
        x.run()
        alone.append(x.results())
    layers = [Layer(mt, i) for i in range(4)]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(5):
                layers[i].run()
            torch.cuda.current_stream().synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for want, x in zip(alone, layers):
        assert all(torch.equal(a, b) for a, b in zip(want, x.results()))


def test_an_explicit_stream_and_the_launch_counter(mt):
    x, y = Layer(mt, 7), torch.empty(2, 70, 40, device="cuda")
    before = mt.mt_scan_launches()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    mt.mt_embed(x.tok, x.table, y, scale=0.5, stream=side)
    side.synchronize()
    assert mt.mt_scan_launches() == before + 1
    x.run()
    assert torch.equal(x.e, y)


def test_host_memory_is_refused(mt):
    x = Layer(mt, 2)
    with pytest.raises(mt.ScanError) as e:
        mt.mt_embed(x.tok, x.table.cpu().pin_memory(), x.e)
    assert e.value.code == mt.MT_ERR_MEMORY
    with pytest.raises(mt.ScanError) as e:
        mt.mt_causal_conv(x.e, x.w, x.v, state=x.cs.cpu().pin_memory())
    assert e.value.code == mt.MT_ERR_MEMORY
    with pytest.raises(mt.ScanError) as e:
        mt.mt_selective_scan(x.v, x.delta, x.A, x.B, x.C, x.y, x.s1, state=x.ss.cpu().pin_memory())
    assert e.value.code == mt.MT_ERR_MEMORY


def test_several_sequences_a_lane(mt):
    """The single-token form with enough channels that a lane takes several sequences; their number is odd."""
    b, d, n = 5, 32768, 16
    x = Inputs(torch.bfloat16, b, 1, d, n)
    slots = torch.tensor([3, -1, 0, 4, 9], dtype=torch.int32)
    pool = torch.randn(6, d, n, generator=torch.Generator().manual_seed(2))
    state, out = pool.cuda(), torch.full((b, d), 5.0, dtype=torch.bfloat16, device="cuda")
    at = lambda v: v.cuda()[:, 0]  # noqa: E731
    mt.mt_selective_scan_step(at(x.u), at(x.delta), x.A.cuda(), at(x.B), at(x.C), state, out, D=x.D.cuda(), z=at(x.z),
                              delta_bias=x.bias.cuda(), slots=slots.cuda())
    x.h0 = pool[[3, 0, 0, 4, 0]]
    want, last = x.case().forward()
    mag, lmag = x.case().magnitude().forward()
    on = [0, 2, 3]
    R.assert_within("out", out[on], want[on, 0], x.case().rel() * mag[on, 0])
    R.assert_within("state", state[[3, 0, 4]], last[on], x.case().rel() * lmag[on])
    assert (out[[1, 4]] == 0).all()
    assert torch.equal(state.cpu()[[1, 2, 5]], pool[[1, 2, 5]])


def test_offsets_past_32_bits(mt):
    """A pool of 40,000 states of 4096 x 16 (2.6e9 values), and a table of 600,000 rows of 4096 (2.5e9 values)."""
    d, n, last = 4096, 16, 39_999
    x = Inputs(torch.bfloat16, 1, 3, d, n)
    c = lambda v: v.cuda()  # noqa: E731
    outs, states = [], []
    for rows, slot in ((1, 0), (40_000, last)):
        pool = torch.empty(rows, d, n, device="cuda")
        pool[slot].copy_(x.h0[0])
        out, one = torch.empty(1, 3, d, dtype=torch.bfloat16, device="cuda"), torch.empty(1, d, dtype=torch.bfloat16, device="cuda")
        slots = torch.tensor([slot], dtype=torch.int32, device="cuda")
        need = mt.mt_selective_scan_scratch_slots(1, 3, d, n)
        scratch = torch.empty(need, dtype=torch.int64, device="cuda") if need else None
        mt.mt_selective_scan(c(x.u), c(x.delta), c(x.A), c(x.B), c(x.C), out, scratch, z=c(x.z), state=pool, carry_in=True, slots=slots)
        mt.mt_selective_scan_step(c(x.u)[:, 0], c(x.delta)[:, 0], c(x.A), c(x.B)[:, 0], c(x.C)[:, 0], pool, one, slots=slots)
        outs.append((out, one))
        states.append(pool[slot].clone())
        del pool
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1]) and torch.equal(*states)

    vocab, dim = 600_000, 4096
    table = torch.empty(vocab, dim, dtype=torch.bfloat16, device="cuda")
    tokens = torch.tensor([vocab - 1, 3, vocab - 2, vocab - 1], dtype=torch.int32, device="cuda")
    rows = torch.randn(4, dim, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    table[tokens.long()] = rows
    out = torch.empty(4, dim, dtype=torch.bfloat16, device="cuda")
    mt.mt_embed(tokens, table, out)
    assert torch.equal(out, table[tokens.long()])
    scratch = torch.empty(mt.mt_embed_grad_scratch_slots(4, vocab, dim), dtype=torch.int64, device="cuda")
    mt.mt_embed_grad(tokens, rows, table, scratch)
    want = torch.zeros(3, dim, device="cuda")
    want[0], want[1], want[2] = rows[1].float(), rows[2].float(), rows[0].float() + rows[3].float()
    assert torch.equal(table[[3, vocab - 2, vocab - 1]], want.to(torch.bfloat16))
    assert (table[4:vocab - 2].view(-1)[::4099] == 0).all() and (table[:3] == 0).all()
