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
