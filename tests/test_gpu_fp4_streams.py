"""GPU tests of what one call of the 4-bit and mixture-of-experts operators sees of another's memory: chains in which
each kernel is set up while the one before it still writes, against the same calls with a wait after each."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import precision_integer_gemm_gb300 as pig  # noqa: E402

I32 = dict(dtype=torch.int32, device="cuda")
U8 = dict(dtype=torch.uint8, device="cuda")


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pig.build_library()
    return pig.load()


def packed(fmt, x):
    """Codes and scales of the rows of x."""
    rows, K = x.shape
    codes = torch.empty((rows, pig.fp4_code_bytes(K)), **U8)
    scales = torch.empty((rows, (pig.mxfp4_scale_pitch if fmt == "mx" else pig.nvfp4_scale_pitch)(K)), **U8)
    pack(fmt, x, codes, scales, rows, K)
    return codes, scales


def pack(fmt, x, codes, scales, rows, K, index=None):
    if fmt == "mx":
        pig.pack_mxfp4(x, codes, scales, rows, K, index=index)
    else:
        pig.pack_nvfp4(x, None, codes, scales, rows, K, index=index)


def same_with_waits(chain):
    """chain(wait) gives the tensors of its steps; wait() stands between any two of its calls."""
    free = chain(lambda: None)
    torch.cuda.synchronize()
    waited = chain(torch.cuda.synchronize)
    assert pig.igemm_last_status() == 0
    for a, b in zip(free, waited):
        assert bool(torch.isfinite(a).all()) and torch.equal(a, b)


@pytest.mark.parametrize("M", [3, 48, 300])
def test_tensor_scale_and_alpha_written_by_the_call_before(M):
    gen = torch.Generator(device="cuda").manual_seed(M)
    N = K = 512
    steps = 40
    B, SB = packed("nv", torch.randn((N, K), generator=gen, device="cuda") * 0.05)
    x0 = torch.randn((M, K), generator=gen, device="cuda")
    one, first = torch.ones((1, 1), device="cuda"), torch.zeros((1, 1), **I32)
    # another scale and factor every step, each the sum of one row of one value
    scale = (0.01 * (1 + torch.arange(steps, device="cuda") % 5)).view(steps, 1, 1)
    codes = torch.empty((M, pig.fp4_code_bytes(K)), **U8)
    scales = torch.empty((M, pig.nvfp4_scale_pitch(K)), **U8)
    g, alpha = torch.ones((1, 1), device="cuda"), torch.ones((1, 1), device="cuda")

    def chain(wait):
        x, out = x0.clone(), []
        for s in range(steps):
            pig.igemm_moe_combine(one, first, scale[s], g, 1, 1, 1)
            wait()
            pig.pack_nvfp4(x, g, codes, scales, M, K)
            wait()
            pig.igemm_moe_combine(one, first, scale[(s + 2) % steps], alpha, 1, 1, 1)
            wait()
            pig.igemm_nvfp4(codes, B, scales, SB, alpha, x, M, N, K)
            wait()
            out.append(x.clone())
            wait()
        return out

    same_with_waits(chain)


# one routing launch, two and three; the last gathers its rows through a workspace
@pytest.mark.parametrize("fmt,T,E,k,steps", [("mx", 12, 16, 4, 30), ("nv", 300, 16, 4, 30), ("mx", 600, 40, 4, 20),
                                             ("nv", 16384, 68, 4, 6)])
def test_layer_after_layer(fmt, T, E, k, steps):
    # router's product, routing, gathered packing, grouped product and sum: every buffer is written again each time
    gen = torch.Generator(device="cuda").manual_seed(T)
    D = 256
    R, SR = packed(fmt, torch.randn((E, D), generator=gen, device="cuda") * 0.1)
    B, SB = packed(fmt, torch.randn((E * D, D), generator=gen, device="cuda") * 0.13)
    x0 = torch.randn((T, D), generator=gen, device="cuda")
    ones = None if fmt == "mx" else torch.ones((E,), device="cuda")
    logits = torch.empty((T, E), device="cuda")
    experts, weights, slots = torch.empty((T, k), **I32), torch.empty((T, k), device="cuda"), torch.empty((T, k), **I32)
    offsets, tokens = torch.empty((E + 1,), **I32), torch.empty((T * k,), **I32)
    a, sa = packed(fmt, x0)
    h, sh = packed(fmt, torch.zeros((T * k, D), device="cuda"))
    y = torch.empty((T * k, D), device="cuda")

    def chain(wait):
        x, out = x0.clone(), []
        for _ in range(steps):
            pack(fmt, x, a, sa, T, D)
            wait()
            if fmt == "mx":
                pig.igemm_mxfp4(a, R, sa, SR, logits, T, E, D)
            else:
                pig.igemm_nvfp4(a, R, sa, SR, None, logits, T, E, D)
            wait()
            pig.igemm_moe_route(logits, experts, weights, offsets, tokens, slots, T, E, k)
            wait()
            pack(fmt, x, h, sh, T * k, D, index=tokens)
            wait()
            if fmt == "mx":
                pig.igemm_mxfp4_grouped(h, B, sh, SB, offsets, y, T * k, E, D, D)
            else:
                pig.igemm_nvfp4_grouped(h, B, sh, SB, offsets, ones, y, T * k, E, D, D)
            wait()
            pig.igemm_moe_combine(y, slots, weights, x, T, k, D)
            wait()
            out.append(x.clone())
            wait()
        return out

    same_with_waits(chain)


def route_buffers(T, E, k):
    return (torch.empty((T, k), **I32), torch.empty((T, k), device="cuda"), torch.empty((E + 1,), **I32),
            torch.empty((T * k,), **I32), torch.empty((T, k), **I32))


def test_kernels_launched_by_each_operator():
    def launched(call):
        before = pig.igemm_kernels_launched()
        call()
        return pig.igemm_kernels_launched() - before

    # routing: one up to 512 tokens, two while 4 ceil(T / 64)^2 ceil(E / 4) bytes are at most 4 MB, three above
    for T, E, want in [(0, 8, 0), (1, 8, 1), (65, 8, 1), (512, 8, 1), (513, 8, 2), (16384, 64, 2), (16384, 65, 3),
                       (16385, 64, 3), (4096, 1024, 2), (4097, 1024, 3)]:
        logits = torch.zeros((T, E), dtype=torch.bfloat16, device="cuda")
        assert launched(lambda: pig.igemm_moe_route(logits, *route_buffers(T, E, 2), T, E, 2)) == want, (T, E)
    # packing: two where rows are gathered twice or more on average and that saves reading 32 MB
    for rows, source, K, want in [(4, 4, 64, 1), (8192, 4096, 4096, 2), (8192, 4096, 4095, 1), (8193, 4096, 4096, 2),
                                  (16384, 8192, 2048, 2), (16383, 8192, 4096, 1), (0, 4, 64, 0)]:
        x = torch.zeros((source, K), dtype=torch.bfloat16, device="cuda")
        codes = torch.empty((rows, pig.fp4_code_bytes(K)), **U8)
        scales = torch.empty((rows, pig.mxfp4_scale_pitch(K)), **U8)
        index = torch.zeros((rows,), **I32)
        assert launched(lambda: pig.pack_mxfp4(x, codes, scales, rows, K, index=index)) == want, (rows, source, K)
    # a product one, whatever its kernel, and so the sum
    for M in (1, 40, 300):
        A, SA = packed("mx", torch.zeros((M, 1024), device="cuda"))
        C = torch.empty((M, M), device="cuda")
        off = torch.tensor([0, M], **I32)
        assert launched(lambda: pig.igemm_mxfp4(A, A, SA, SA, C, M, M, 1024)) == 1
        assert launched(lambda: pig.igemm_mxfp4_grouped(A, A, SA, SA, off, C, M, 1, M, 1024)) == 1
        slots = torch.zeros((M, 1), **I32)
        assert launched(lambda: pig.igemm_moe_combine(C, slots, torch.ones((M, 1), device="cuda"), torch.empty_like(C), M,
                                                      1, M)) == 1
    torch.cuda.synchronize()
    assert pig.igemm_last_status() == 0


# routing in two launches and in three, and gathered packing through its workspace: every call that allocates
@pytest.mark.parametrize("fmt,T,E,k,K", [("mx", 600, 40, 8, 256), ("nv", 8192, 64, 4, 1024), ("mx", 16400, 68, 3, 768)])
def test_workspaces_in_a_graph(fmt, T, E, k, K):
    gen = torch.Generator(device="cuda").manual_seed(T)
    logits, x = torch.empty((T, E), device="cuda"), torch.empty((T, K), device="cuda")
    route = route_buffers(T, E, k)
    tokens, slots, weights = route[3], route[4], route[1]
    a = torch.empty((T * k, pig.fp4_code_bytes(K)), **U8)
    sa = torch.empty((T * k, (pig.mxfp4_scale_pitch if fmt == "mx" else pig.nvfp4_scale_pitch)(K)), **U8)
    N = 64
    B, SB = packed(fmt, torch.randn((E * N, K), generator=gen, device="cuda") * 0.1)
    y, out = torch.empty((T * k, N), device="cuda"), torch.empty((T, N), device="cuda")

    def layer():
        pig.igemm_moe_route(logits, *route, T, E, k)
        pack(fmt, x, a, sa, T * k, K, index=tokens)
        if fmt == "mx":
            pig.igemm_mxfp4_grouped(a, B, sa, SB, route[2], y, T * k, E, N, K)
        else:
            pig.igemm_nvfp4_grouped(a, B, sa, SB, route[2], None, y, T * k, E, N, K)
        pig.igemm_moe_combine(y, slots, weights, out, T, k, N)

    before = pig.igemm_kernels_launched()
    logits.normal_(generator=gen), x.normal_(generator=gen)
    layer()
    assert pig.igemm_kernels_launched() - before == 2 + (2 if T * E < 16400 * 68 else 3) + (2 if T > 600 else 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for _ in range(4):
        logits.normal_(generator=gen), x.normal_(generator=gen)
        out.fill_(float("nan"))
        graph.replay()
        graph.replay()  # right behind itself, on the same workspaces
        got = [t.clone() for t in (out, a, sa, *route)]
        layer()  # and a call of its own right behind the graph
        assert bool(torch.isfinite(got[0]).all())
        for g, w in zip(got, (out, a, sa, *route)):
            assert torch.equal(g, w)
    assert pig.igemm_last_status() == 0


def test_calls_on_two_streams():
    # routing and gathered packing through the pool's workspaces, products and sums, on two streams at once
    fmt, T, E, k, K, N, steps = "mx", 16384, 68, 3, 1024, 128, 12
    gen = torch.Generator(device="cuda").manual_seed(1)
    B, SB = packed(fmt, torch.randn((E * N, K), generator=gen, device="cuda") * 0.1)
    logits = torch.randn((2, steps, T, E), generator=gen, device="cuda")
    x = torch.randn((2, T, K), generator=gen, device="cuda")
    work = [(route_buffers(T, E, k), packed(fmt, torch.zeros((T * k, K), device="cuda")),
             torch.empty((T * k, N), device="cuda")) for _ in range(2)]
    out = torch.empty((2, steps, T, N), device="cuda")

    def step(i, s):
        route, (a, sa), y = work[i]
        pig.igemm_moe_route(logits[i, s], *route, T, E, k)
        pack(fmt, x[i], a, sa, T * k, K, index=route[3])
        pig.igemm_mxfp4_grouped(a, B, sa, SB, route[2], y, T * k, E, N, K)
        pig.igemm_moe_combine(y, route[4], route[1], out[i, s], T, k, N)

    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s in range(steps):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                step(i, s)
    torch.cuda.synchronize()
    together = out.clone()
    out.fill_(float("nan"))
    for s in range(steps):
        for i in range(2):
            step(i, s)
            torch.cuda.synchronize()
    assert bool(torch.isfinite(together).all()) and torch.equal(together, out)
    assert pig.igemm_last_status() == 0
