"""Scratch memory of the calls: CUDA graphs have their own, whatever the stream's later calls need."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def nv():
    import __graft_entry__
    __graft_entry__.build()
    import nvfp4_bit_quantized_gb300 as nv
    nv.reset_status()
    return nv


class Calls:
    """Every kind of call with scratch memory: partial maxima (quantizers), column sums (layer norm backward), parts of few tiles with
    many steps (attention forward), delta and parts (attention backward)."""

    def __init__(self, nv, tokens, keys, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def rnd(*s):
            return torch.randn(*s, generator=g, device="cuda").to(BF16)
        self.nv = nv
        self.x, self.dy, self.w = rnd(tokens, 1024), rnd(tokens, 1024), torch.ones(1024, device="cuda")
        _, self.mean, self.rstd, _ = nv.layer_norm_forward(self.x, self.w)
        self.q, self.k, self.v, self.dout = rnd(tokens, 4, 64), rnd(keys, 2, 64), rnd(keys, 2, 64), rnd(tokens, 4, 64)
        self.out, self.lse = nv.attention_forward(self.q, self.k, self.v)

    def __call__(self):
        nv = self.nv
        a, b = nv.quantize_dual(self.x, nv.RNE, nv.SR, sr_seed=3, rht_seed=4)
        return [a.codes, a.scales, a.s_dec[:1], b.codes, b.scales, b.s_dec[:1],      # the one element that is written
                *nv.layer_norm_backward(self.dy, self.x, self.w, self.mean, self.rstd),
                *nv.attention_forward(self.q, self.k, self.v),
                *nv.attention_backward(self.dout, self.q, self.k, self.v, self.out, self.lse)]


def captured(calls, stream):
    with torch.cuda.stream(stream):
        want = [t.clone() for t in calls()]                # loads the kernels, and the stream has its buffer
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        got = calls()
    return graph, want, got


def test_a_graph_is_replayed_after_larger_calls_on_its_stream(nv):
    stream = torch.cuda.Stream()
    small, large = Calls(nv, 128, 3000, 1), Calls(nv, 4096, 9000, 2)
    torch.cuda.synchronize()
    graph, want, got = captured(small, stream)
    with torch.cuda.stream(stream):
        large()                                            # outgrows the stream's buffer
        others = [torch.full((n,), 77, dtype=torch.uint8, device="cuda")       # and the memory goes round
                  for n in [1 << k for k in range(12, 25)] * 3]
        for _ in range(3):
            for t in got:
                t.zero_()
            graph.replay()
    stream.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert all((t == 77).all() for t in others)
    assert nv.status_query() == 0


def test_graphs_of_one_stream_are_replayed_on_two(nv):
    """Two graphs captured on one stream, replayed beside each other and beside eager calls on the stream of their capture."""
    home, streams = torch.cuda.Stream(), [torch.cuda.Stream() for _ in range(2)]
    calls = [Calls(nv, 256, 3000, 3), Calls(nv, 384, 2000, 4), Calls(nv, 512, 2500, 5)]
    torch.cuda.synchronize()
    graphs = [captured(c, home) for c in calls[:2]]
    with torch.cuda.stream(home):
        eager = [t.clone() for t in calls[2]()]
    home.synchronize()
    for _ in range(20):
        for (graph, _, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                graph.replay()
        with torch.cuda.stream(home):
            again = calls[2]()
        torch.cuda.synchronize()
        for _, want, got in graphs + [(None, eager, again)]:
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_threads_on_one_stream(nv):
    import threading
    stream = torch.cuda.Stream()
    calls = [Calls(nv, 256 + 128 * i, 2000 + 300 * i, 20 + i) for i in range(4)]
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        want = [[t.clone() for t in c()] for c in calls]
    stream.synchronize()
    bad = []

    def work(i):
        with torch.cuda.stream(stream):
            for _ in range(40):
                got = calls[i]()
                bad.extend((i, n) for n, (a, b) in enumerate(zip(got, want[i])) if not torch.equal(a, b))
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:10]
    assert nv.status_query() == 0
