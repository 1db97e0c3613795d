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
