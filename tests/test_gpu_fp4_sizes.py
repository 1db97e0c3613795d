"""GPU tests of the 4-bit and mixture-of-experts operators at sizes where a count or an index passes 2^31."""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import precision_integer_gemm_gb300 as pig  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pig.build_library()
    return pig.load()


@pytest.fixture(autouse=True)
def memory():
    yield
    torch.cuda.empty_cache()


def needs(gigabytes):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gigabytes * 10 ** 9:
        pytest.skip(f"needs {gigabytes} GB of free device memory")


def some_rows(M):
    """The first and last rows of M, and rows all over."""
    gen = torch.Generator(device="cuda").manual_seed(7)
    return torch.cat([torch.arange(1000, device="cuda"), torch.arange(M - 3000, M, device="cuda"),
                      torch.randint(0, M, (200000,), generator=gen, device="cuda")])


def mx_values(codes, scales):
    """float64 values of rows of 32 mxfp4 codes with one scale each."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device="cuda").double()
    v = table[torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1).long()]
    return v * torch.exp2(scales[:, :1].double() - 127)


@pytest.mark.parametrize("groups", [None, [2 ** 31 - 4000, 0, 3000]])
def test_product_of_nearly_2_to_31_rows(groups):
    needs(110)
    M, N, K = (2 ** 31 - 600 if groups is None else sum(groups)), 2, 32
    E = 1 if groups is None else len(groups)
    gen = torch.Generator(device="cuda").manual_seed(1)
    A = torch.randint(0, 256, (M, 16), generator=gen, dtype=torch.uint8, device="cuda")
    SA = torch.randint(125, 130, (M, 16), generator=gen, dtype=torch.uint8, device="cuda")
    B = torch.randint(0, 256, (E * N, 16), generator=gen, dtype=torch.uint8, device="cuda")
    SB = torch.randint(125, 130, (E * N, 16), generator=gen, dtype=torch.uint8, device="cuda")
    buf = torch.full((M * N + 4096,), -777.0, device="cuda")
    C = buf[:M * N].view(M, N)
    b = mx_values(B, SB)
    rows = some_rows(M)
    if groups is None:
        pig.igemm_mxfp4(A, B, SA, SB, C, M, N, K)
        b = b.expand(rows.numel(), N, 32)
    else:
        ends = torch.tensor([0, *groups], device="cuda").cumsum(0)
        pig.igemm_mxfp4_grouped(A, B, SA, SB, ends.int(), C, M, E, N, K)
        b = b.view(E, N, 32)[torch.searchsorted(ends[1:], rows, right=True)]
    assert pig.igemm_last_status() == 0
    # 32 products of eighths of integers and powers of two: exact in float32
    want = torch.einsum("rk,rnk->rn", mx_values(A[rows], SA[rows]), b)
    assert torch.equal(C[rows].double(), want)
    assert bool((buf[M * N:] == -777).all())


@pytest.mark.parametrize("N,start", [(2 ** 31 - 101, 0), (2 ** 31 - 2, 0), (2 ** 31 - 2, 1)])
def test_combine_of_rows_of_nearly_2_to_31(N, start):
    # two tokens of two rows, neither a multiple of a wide load; `start`: off 4 bytes
    needs(30)
    T, k = 2, 2
    gen = torch.Generator(device="cuda").manual_seed(2)
    Y = torch.empty((T * k * N + start,), dtype=torch.bfloat16, device="cuda")
    Y.random_(-64, 64, generator=gen)
    Y = Y[start:].view(T * k, N)
    slots = torch.tensor([[3, 0], [1, 2]], dtype=torch.int32, device="cuda")
    weights = torch.tensor([[0.5, -2.0], [1.0, 0.25]], device="cuda")
    buf = torch.full((T * N + 4096,), -777.0, dtype=torch.bfloat16, device="cuda")
    pig.igemm_moe_combine(Y, slots, weights, buf[:T * N].view(T, N), T, k, N)
    for t in range(T):
        for at in range(0, N, 1 << 28):
            part = slice(at, min(at + (1 << 28), N))
            # small integers times powers of two: the float32 sum is exact, one rounding to bfloat16
            want = Y[slots[t, 0], part].float() * weights[t, 0] + Y[slots[t, 1], part].float() * weights[t, 1]
            assert torch.equal(buf[t * N + part.start:t * N + part.stop], want.bfloat16())
    assert bool((buf[T * N:] == -777).all())


@pytest.mark.parametrize("typ", [torch.bfloat16, torch.float32])
def test_route_of_2_to_31_tokens_but_one(typ):
    needs(90)
    T, E, k = 2 ** 31 - 1, 2, 1
    gen = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.empty((T, E), dtype=typ, device="cuda")
    logits.random_(-8, 8, generator=gen)  # ties too
    i32 = dict(dtype=torch.int32, device="cuda")
    experts, slots, weights = torch.empty((T, k), **i32), torch.empty((T, k), **i32), torch.empty((T, k), device="cuda")
    offsets, tokens = torch.empty((E + 1,), **i32), torch.empty((T * k,), **i32)
    pig.igemm_moe_route(logits, experts, weights, offsets, tokens, slots, T, E, k)
    second = 0
    for at in range(0, T, 1 << 27):
        part = slice(at, min(at + (1 << 27), T))
        want = (logits[part, 1] > logits[part, 0]).int()  # a tie: the lower expert
        assert torch.equal(experts[part, 0], want) and bool((weights[part] == 1).all())
        # the place holds the token, and lies behind the places of the same expert's earlier tokens
        place = slots[part, 0].long()
        assert torch.equal(tokens[place].long(), torch.arange(part.start, part.stop, device="cuda"))
        mask = want.bool()
        assert bool((place[mask].diff() == 1).all()) and bool((place[~mask].diff() == 1).all())
        second += int(want.sum())
    assert offsets.tolist() == [0, T - second, T]


def test_gathered_packing_without_room_for_its_workspace():
    needs(8)
    source, rows, K = 1 << 18, 1 << 19, 4096  # a workspace of 570 MB
    x = torch.randint(-8, 8, (source, K), device="cuda", dtype=torch.int8).to(torch.bfloat16)
    index = torch.randint(0, source, (rows,), device="cuda", dtype=torch.int32)
    codes = torch.full((2, rows, K // 2), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((2, rows, pig.mxfp4_scale_pitch(K)), 0xA5, dtype=torch.uint8, device="cuda")
    # the reference: fewer rows a call, which never takes a workspace
    for at in range(0, rows, source // 2):
        part = slice(at, at + source // 2)
        pig.pack_mxfp4(x, codes[0, part], scales[0, part], source // 2, K, index=index[part])
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    rest = torch.cuda.mem_get_info()[0] - (256 << 20)
    filler = torch.empty((rest,), dtype=torch.uint8, device="cuda")
    try:
        pig.pack_mxfp4(x, codes[1], scales[1], rows, K, index=index)
        torch.cuda.synchronize()
    finally:
        del filler
    assert torch.equal(codes[0], codes[1]) and torch.equal(scales[0], scales[1])
