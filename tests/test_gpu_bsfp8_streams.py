"""The scored routing's three launches, rows packed once and copied, grouped products and the gradient as one chain: each
launch set up while the one before it ends, captured in two graphs that replay at once, and called from two host threads,
against the same calls with a wait after each."""

import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import precision_integer_gemm_gb300 as pig  # noqa: E402

T, E, K, N, k = 6000, 256, 1024, 256, 8
I32 = dict(dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pig.build_library()
    yield pig.load()
    assert pig.igemm_last_status() == pig.IGEMM_OK


class Chain:
    """One user's buffers; run() makes the calls and leaves its results in self.out."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
        self.logits = torch.randn((T, E), generator=g, device="cuda")
        self.bias = 0.1 * torch.randn((E,), generator=g, device="cuda")
        self.B = torch.randint(0, 120, (E, N, K), generator=g, dtype=torch.uint8, device="cuda")
        self.SFB = torch.rand((E, N // 128, pig.bsfp8_scale_pitch(K)), generator=g, device="cuda")
        self.dw = torch.randn((T, k), generator=g, device="cuda")
        self.codes = torch.empty((T * k, K), dtype=torch.uint8, device="cuda")
        self.scales = torch.empty((T * k, pig.bsfp8_scale_pitch(K)), device="cuda")
        self.out = [torch.empty((T, k), **I32), torch.empty((T, k), device="cuda"), torch.empty((E + 1,), **I32),
                    torch.empty((T * k,), **I32), torch.empty((T, k), **I32),
                    torch.empty((T * k, N), dtype=torch.bfloat16, device="cuda"), torch.empty((T, E), device="cuda"),
                    torch.empty((T, N), dtype=torch.bfloat16, device="cuda")]

    def run(self, wait=lambda: None, stream=None):
        experts, weights, offsets, tokens, slots, y, dlogits, sums = self.out
        pig.igemm_moe_route_scored(self.logits, self.bias, experts, weights, offsets, tokens, slots, T, E, k, score="sigmoid",
                                   groups=8, group_k=4, group_top=2, stream=stream)
        wait()
        pig.pack_bsfp8(self.x, self.codes, self.scales, T * k, K, index=tokens, stream=stream)
        wait()
        pig.igemm_bsfp8_grouped(self.codes, self.B, self.scales, self.SFB, offsets, y, T * k, E, N, K, stream=stream)
        wait()
        pig.igemm_moe_combine(y, slots, weights, sums, T, k, N, stream=stream)
        wait()
        pig.igemm_moe_route_scored_grad(self.logits, experts, self.dw, dlogits, T, E, k, score="sigmoid", stream=stream)
        wait()

    def expected(self):
        self.run(torch.cuda.synchronize)
        want = [o.clone() for o in self.out]
        self.clear()
        return want

    def clear(self):
        for o in self.out:
            o.fill_(-3)
        self.codes.fill_(0x7F)
        torch.cuda.synchronize()

    def new_inputs(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x.copy_(torch.randn((T, K), generator=g, device="cuda"))
        self.logits.copy_(torch.randn((T, E), generator=g, device="cuda"))
        torch.cuda.synchronize()

    def same(self, want):
        return all(torch.equal(a, b) for a, b in zip(self.out, want))


def test_launches_of_the_chain():
    c = Chain(1)
    before = pig.igemm_kernels_launched()
    c.run()
    # routing three, packing two (once, then copies), one each for the rest
    assert pig.igemm_kernels_launched() - before == 8


def test_chain_without_waits():
    c = Chain(2)
    want = c.expected()
    for _ in range(5):
        c.clear()
        for _ in range(3):
            c.run()
        torch.cuda.synchronize()
        assert c.same(want)


def test_two_graphs_at_once():
    chains, graphs = [Chain(3), Chain(4)], []
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for c in chains:
            c.run()
    side.synchronize()
    for c in chains:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in chains]
    for turn in range(4):
        wants = []
        for i, c in enumerate(chains):
            c.new_inputs(10 * turn + i)
            wants.append(c.expected())
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert all(c.same(w) for c, w in zip(chains, wants))


def test_two_threads_on_their_own_streams():
    chains = [Chain(5), Chain(6)]
    wants = [c.expected() for c in chains]
    streams, errors = [torch.cuda.Stream() for _ in chains], []

    def work(c, s):
        try:
            for _ in range(10):
                c.run(stream=s)
            s.synchronize()
        except Exception as e:  # (a thread's exception ends nothing by itself)
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(chains, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors and all(c.same(w) for c, w in zip(chains, wants))
