"""The block-scaled fp8 operators run together: the example layer stage by stage against 64 bits, its gradients, the
products of the backward pass on transposed packing, captured graphs, streams and launch counts.

A stage is compared with the same stage in 64 bits on the values that it was given, so its tolerance is its own: the
products' as in test_gpu_bsfp8 (one rounding to the output type and (128 + KB + 4) 2^-23 of the sum of magnitudes).
"""

import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")

import precision_integer_gemm_gb300 as pig  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pig.build_library()
    yield pig.load()
    assert pig.igemm_last_status() == pig.IGEMM_OK


def values(packed, tile_rows, K):
    codes, scales = packed
    row = torch.arange(codes.shape[0], device="cuda") // tile_rows
    return codes.view(torch.float8_e4m3fn).double()[:, :K] * scales[row].double().repeat_interleave(128, dim=1)[:, :K]


def near(C, a, b, K):
    want, size = a @ b.t(), a.abs() @ b.abs().t()
    bound = torch.finfo(C.dtype).eps / 2 * want.abs() + (128 + -(-K // 128) + 4) * 2.0 ** -23 * size
    assert bool(((C.double() - want).abs() <= bound).all())


def make(E, D, F, k, dtype=torch.bfloat16, **kw):
    from moe_fp8 import MoeFp8

    g = torch.Generator(device="cuda").manual_seed(E + D)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    router, gate_up, down = rand(E, D) / D ** 0.5, (rand(E, 2 * F, D) / D ** 0.5).to(dtype), (rand(E, D, F) / F ** 0.5).to(dtype)
    return MoeFp8(router, gate_up, down, k, **kw), router, gate_up, down


@pytest.mark.parametrize("T,E,D,F,k,kw", [(1, 4, 128, 96, 2, {}), (37, 8, 200, 136, 3, dict(groups=4, group_k=2, scale=2.5)),
                                          (600, 16, 256, 320, 4, dict(groups=4, group_k=2)), (1300, 4, 384, 130, 2, {})])
def test_layer_stage_by_stage(T, E, D, F, k, kw):
    from moe_fp8 import pack

    layer, router, gate_up, down = make(E, D, F, k, **kw)
    layer.bias.copy_(0.1 * torch.randn((E,), device="cuda"))
    x = torch.randn((T, D), device="cuda").to(torch.bfloat16)
    out = layer(x)
    _, logits, experts, weights, offsets, tokens, slots, h, act, y = layer.saved
    ends = offsets.tolist()
    assert ends[-1] == T * k and bool((experts >= 0).all())
    a, ap = values(pack(x, index=tokens), 1, D), values(pack(act), 1, F)
    for e, (i, j) in enumerate(zip(ends, ends[1:])):
        near(h[i:j], a[i:j], values((layer.gate_up[0][e], layer.gate_up[1][e]), 128, D), D)
        near(y[i:j], ap[i:j], values((layer.down[0][e], layer.down[1][e]), 128, F), F)
    want = (weights.double().unsqueeze(-1) * y[slots.long()].double()).sum(1)
    size = (weights.double().unsqueeze(-1) * y[slots.long()].double()).abs().sum(1)
    assert bool(((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (k + 1) * 2.0 ** -24 * size + 1e-30).all())
    # quantisation: an e4m3 value is off by at most 2^-4 of itself or 2^-10 of its block's largest, so packed rows differ
    # from their source by at most that
    src = x[tokens.long()].double()
    block = torch.nn.functional.pad(src, (0, -D % 128)).view(T * k, -1, 128).abs().amax(-1).repeat_interleave(128, 1)[:, :D]
    assert bool(((a - src).abs() <= torch.maximum(2.0 ** -4 * src.abs(), 2.0 ** -9 / 448 * block) * (1 + 2.0 ** -20)).all())


@pytest.mark.parametrize("T,E,D,F,k", [(50, 4, 128, 96, 2), (700, 8, 256, 160, 3)])
def test_layer_gradients(T, E, D, F, k):
    from moe_fp8 import pack

    layer, router, gate_up, down = make(E, D, F, k, scale=1.5)
    x = torch.randn((T, D), device="cuda").to(torch.bfloat16)
    out = layer(x)
    dout = torch.randn_like(out)
    dx, d_router, d_gate_up, d_down = layer.backward(dout)
    _, logits, experts, weights, offsets, tokens, slots, h, act, y = layer.saved
    assert dx.shape == x.shape and d_router.shape == router.shape and d_gate_up.shape == gate_up.shape
    assert d_down.shape == down.shape
    # a product of the backward pass on its own operands: dact = dy . down (packed transposed)
    ends = offsets.tolist()
    w = torch.zeros((T * k,), device="cuda")
    w[slots.view(-1).long()] = weights.view(-1)
    dy = (dout[tokens.long()].float() * w.unsqueeze(1)).to(torch.bfloat16)
    dact = layer.grouped(pack(dy), layer.down_t, offsets, F, D, torch.float32)
    d = values(pack(dy), 1, D)
    for e, (i, j) in enumerate(zip(ends, ends[1:])):
        near(dact[i:j], d[i:j], values((layer.down_t[0][e], layer.down_t[1][e]), 128, D), D)
        # a weight matrix's gradient from packed operands: both quantised along the tokens
        if j > i:
            n = j - i
            p = values(pack(torch.nn.functional.pad(dy[i:j], (0, 0, 0, -n % 512)).t()), 1, n + -n % 512)
            q = values(pack(torch.nn.functional.pad(act[i:j], (0, 0, 0, -n % 512)).t()), 1, n + -n % 512)
            near(d_down[e], p, q, n + -n % 512)
        else:
            assert bool((d_down[e] == 0).all())
    # the layer's derivative in float64 on unquantised weights: quantisation moves a value by at most 2^-4 of itself
    # either way, at random, and no gradient here is a product of more than five such values
    xx = x.double().requires_grad_(True)
    rr, gg, dd = router.double().requires_grad_(True), gate_up.double().requires_grad_(True), down.double().requires_grad_(True)
    s = torch.sigmoid(xx @ rr.t()).gather(1, experts.long())
    ww = 1.5 * s / s.sum(-1, keepdim=True)
    ref = torch.zeros_like(xx)
    for e in range(E):
        t, j = torch.nonzero(experts == e, as_tuple=True)
        hh = xx[t] @ gg[e].t()
        yy = (torch.nn.functional.silu(hh[:, :F]) * hh[:, F:]) @ dd[e].t()
        ref = ref.index_add(0, t, yy * ww[t, j].unsqueeze(1))
    (ref * dout.double()).sum().backward()
    for got, want in ((out, ref), (dx, xx.grad), (d_router, rr.grad), (d_gate_up, gg.grad), (d_down, dd.grad)):
        assert ((got.double() - want).norm() / want.norm()).item() <= 5 * 2.0 ** -4


def test_layer_of_no_tokens():
    layer, *_ = make(4, 128, 96, 2)
    assert layer(torch.empty((0, 128), device="cuda", dtype=torch.bfloat16)).shape == (0, 128)


def test_layer_captured_and_replayed():
    # two graphs captured one after the other share the library's pool; each replays its own inputs' results
    layer, *_ = make(8, 256, 320, 3, groups=4, group_k=2)
    xs = [torch.randn((n, 256), device="cuda").to(torch.bfloat16) for n in (700, 40)]
    side = torch.cuda.Stream()
    graphs, outs = [], []
    with torch.cuda.stream(side):
        for x in xs:
            layer(x)
    side.synchronize()
    for x in xs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(layer(x))
        graphs.append(g)
    for round_ in range(3):
        for x in xs:
            x.normal_()
        for g in graphs if round_ != 1 else reversed(graphs):
            g.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for x, o in zip(xs, got):
            assert torch.equal(layer(x), o)


def test_two_streams_at_once():
    layer, *_ = make(8, 256, 320, 3)
    xs = [torch.randn((900, 256), device="cuda").to(torch.bfloat16) for _ in range(2)]
    want = [layer(x).clone() for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = []
        for s, x in zip(streams, xs):
            with torch.cuda.stream(s):
                got.append(layer(x))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_explicit_stream_and_raw_addresses():
    M, N, K = 40, 256, 384
    from moe_fp8 import pack

    A, SFA = pack(torch.randn((M, K), device="cuda"))
    B, SFB = pack(torch.randn((N, K), device="cuda"), tile_rows=128)
    want = torch.empty((M, N), device="cuda")
    pig.igemm_bsfp8(A, B, SFA, SFB, want, M, N, K)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    C = torch.zeros((M, N), device="cuda")
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        C.zero_()
        torch.cuda.synchronize()
        pig.igemm_bsfp8(A.data_ptr(), B.data_ptr(), SFA.data_ptr(), SFB.data_ptr(), C, M, N, K, stream=stream)
        s.synchronize()
        assert torch.equal(C, want)


def test_launches():
    from moe_fp8 import pack

    def launched(f):
        n = pig.igemm_kernels_launched()
        f()
        return pig.igemm_kernels_launched() - n

    x = torch.randn((64, 256), device="cuda")
    a, b = pack(x), pack(torch.randn((512, 256), device="cuda"), tile_rows=128)
    C = torch.empty((64, 512), device="cuda")
    assert launched(lambda: pack(x)) == 1 and launched(lambda: pack(x, tile_rows=128)) == 1
    assert launched(lambda: pig.igemm_bsfp8(a[0], b[0], a[1], b[1], C, 64, 512, 256)) == 1
    logits = torch.randn((600, 64), device="cuda")
    layer, *_ = make(64, 64, 64, 2)
    layer.router = torch.randn((64, 64), device="cuda")
    assert launched(lambda: layer.route(logits)) == 2 and launched(lambda: layer.route(logits[:500])) == 1
    dw = torch.randn((600, 2), device="cuda")
    e = torch.zeros((600, 2), dtype=torch.int32, device="cuda")
    assert launched(lambda: pig.igemm_moe_route_scored_grad(logits, e, dw, torch.empty_like(logits), 600, 64, 2)) == 1


def test_chain_without_synchronisation():
    # routing, packing and products back to back, each launched while the one before ends: the same bits every time
    layer, *_ = make(16, 512, 256, 4, groups=4, group_k=2)
    x = torch.randn((2000, 512), device="cuda").to(torch.bfloat16)
    want = layer(x).clone()
    for _ in range(20):
        assert torch.equal(layer(x), want)


def test_example_runs():
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "examples", "moe_fp8.py"), "--tokens", "100", "--steps", "2"],
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "gradients of" in r.stdout


def test_large_offsets():
    # rows and codes past 2^31 bytes: the last rows of a tall product
    M, N, K = (1 << 31) // 2048 + 300, 128, 2048
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    A = torch.full((M, K), 0x38, dtype=torch.uint8, device="cuda")  # ones
    A[M - 1] = 0x40                                                  # twos
    SFA = torch.ones((M, 16), device="cuda")
    B = torch.full((N, K), 0x38, dtype=torch.uint8, device="cuda")
    SFB = torch.full((1, 16), 0.5, device="cuda")
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    pig.igemm_bsfp8(A, B, SFA, SFB, C, M, N, K)
    assert bool((C[:M - 1] == K / 2).all()) and bool((C[M - 1] == K).all())
    del C
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    x.fill_(448.0)
    x[M - 1, :128] = 896.0
    codes = torch.empty((M, K), dtype=torch.uint8, device="cuda")
    pig.pack_bsfp8(x, codes, SFA, M, K)
    assert bool((codes == 0x7E).all()) and bool((SFA[:M - 1] == 1).all())
    assert SFA[M - 1].tolist() == [2.0] + [1.0] * 15
    assert math.isclose(SFA[M - 1, 0].item(), 2.0)
