"""Block-scaled fp8 packing and products on the GPU against plain forms in 64 bits.

Tolerances.  Packing is defined bit for bit.  A product's value is off by one rounding to the output type (half a
step, relative) and by the float32 sums before it: a block's 128 products are summed in the tensor core (each addition
may truncate, at most 2^-23 of the largest partial sum), the scale is a rounded product, then one fused step a block:
at most (128 + KB + 4) 2^-23 of sum |a b| of the output.
"""

import math

import pytest

torch = pytest.importorskip("torch")

import precision_integer_gemm_gb300 as pig  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pig.build_library()
    yield pig.load()
    assert pig.igemm_last_status() == pig.IGEMM_OK


def plain_pack(x, tile_rows, fmt):
    """(codes uint8, scales float32) of the rows of x; the definition's float32 roundings from float64."""
    rows, K = x.shape
    cb, pitch = pig.bsfp8_code_bytes(K), pig.bsfp8_scale_pitch(K)
    codes = torch.zeros((rows, cb), dtype=torch.uint8, device=x.device)
    scales = torch.zeros((-(-rows // tile_rows), pitch), device=x.device)
    for b in range(-(-K // 128)):
        part = x[:, 128 * b:128 * b + 128].float()
        for r in range(0, rows, tile_rows) if tile_rows > 1 else [None]:
            p = part if r is None else part[r:r + tile_rows]
            amax = p.abs().amax(1, keepdim=True) if r is None else p.abs().amax().view(1, 1)
            fine = torch.isfinite(amax)
            s = (amax.double() / LARGEST[fmt]).float().clamp(min=2.0 ** -126)
            f = (1.0 / s.double()).float()
            y = (p.double() * f.double()).float().clamp(-LARGEST[fmt], LARGEST[fmt])
            q = torch.where(fine, y, 0.0).to(FP8[fmt]).view(torch.uint8)
            s = torch.where(fine, s, math.nan)
            if r is None:
                codes[:, 128 * b:128 * b + p.shape[1]] = q
                scales[:, b] = s[:, 0]
            else:
                codes[r:r + tile_rows, 128 * b:128 * b + p.shape[1]] = q
                scales[r // tile_rows, b] = s[0, 0]
    return codes, scales


def pack(x, tile_rows=1, fmt="e4m3", index=None):
    rows, K = (x.shape[0] if index is None else index.numel()), x.shape[1]
    codes = torch.full((rows, pig.bsfp8_code_bytes(K)), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-rows // tile_rows), pig.bsfp8_scale_pitch(K)), 7.0, device="cuda")
    pig.pack_bsfp8(x, codes, scales, rows, K, tile_rows=tile_rows, format=fmt, index=index)
    return codes, scales


def same(got, want):
    (c, s), (wc, ws) = got, want
    assert torch.equal(torch.isnan(s), torch.isnan(ws))
    assert torch.equal(torch.nan_to_num(s, nan=-1.0), torch.nan_to_num(ws, nan=-1.0))
    assert torch.equal(c, wc)


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("rows,K", [(1, 1), (3, 100), (16, 128), (7, 129), (130, 513), (257, 1000), (33, 4160), (5, 9000)])
def test_pack_rows_and_tiles(rows, K, fmt, typ):
    g = torch.Generator(device="cuda").manual_seed(rows * K)
    x = (torch.randn((rows, K), generator=g, device="cuda") * torch.exp(2 * torch.randn((rows, 1), generator=g,
                                                                                         device="cuda"))).to(TYPES[typ])
    for tile_rows in (1, 128):
        want = plain_pack(x, tile_rows, fmt)
        same(pack(x, tile_rows, fmt), want)
        same(pack(x.t().contiguous().t(), tile_rows, fmt), want)  # transposed: unit stride along the rows


@pytest.mark.parametrize("typ", ["f32", "bf16"])
@pytest.mark.parametrize("offset,ld", [(0, 208), (1, 201), (3, 200), (8, 333)])
def test_pack_strides(offset, ld, typ):
    # rows that start anywhere: views into a larger matrix
    rows, K = 70, 190
    base = torch.randn((max(rows, K) * ld + offset,), device="cuda").to(TYPES[typ])
    x = base.as_strided((rows, K), (ld, 1), offset)
    xt = base.as_strided((rows, K), (1, ld), offset)
    for tile_rows in (1, 128):
        same(pack(x, tile_rows), plain_pack(x, tile_rows, "e4m3"))
        same(pack(xt, tile_rows), plain_pack(xt.contiguous(), tile_rows, "e4m3"))


def test_pack_special_values():
    # zeros, -0, subnormals, the largest float32, infinities and NaN, each in blocks of their own
    x = torch.randn((8, 700), device="cuda")
    x[0, :128] = 0.0
    x[1, 128:256] = -0.0
    x[2, 256:384] = 1e-42
    x[3, 5] = math.inf
    x[4, 200] = -math.inf
    x[5, 699] = math.nan
    x[6, 0] = torch.finfo(torch.float32).max
    x[7, 300:310] = torch.finfo(torch.float32).tiny
    for fmt in ("e4m3", "e5m2"):
        for tile_rows in (1, 128):
            same(pack(x, tile_rows, fmt), plain_pack(x, tile_rows, fmt))
            same(pack(x.t().contiguous().t(), tile_rows, fmt), plain_pack(x, tile_rows, fmt))
    h = x.half()  # (many infinities)
    same(pack(h), plain_pack(h, 1, "e4m3"))


@pytest.mark.parametrize("rows,source,K", [(1, 1, 64), (100, 30, 300), (64, 500, 1024), (9000, 300, 4096)])
def test_pack_gathered(rows, source, K):
    x = torch.randn((source, K), device="cuda").to(torch.bfloat16)
    index = torch.randint(-2, source + 2, (rows,), device="cuda", dtype=torch.int32)
    keep = (index >= 0) & (index < source)
    want = torch.where(keep.unsqueeze(1), x[index.clamp(0, source - 1).long()], torch.zeros((), dtype=x.dtype, device="cuda"))
    same(pack(x, index=index), plain_pack(want, 1, "e4m3"))


def values(codes, scales, tile_rows, fmt, K):
    v = codes.view(FP8[fmt]).double()[:, :K]
    row = torch.arange(codes.shape[0], device="cuda") // tile_rows
    return v * scales[row].double().repeat_interleave(128, dim=1)[:, :K]


def operands(M, N, K, fmt="e4m3", seed=0, experts=1):
    g = torch.Generator(device="cuda").manual_seed(seed + M + 3 * N + 7 * K)
    a = torch.randn((M, K), generator=g, device="cuda")
    A, SFA = plain_pack(a, 1, fmt)
    B = torch.zeros((experts, N, pig.bsfp8_code_bytes(K)), dtype=torch.uint8, device="cuda")
    SFB = torch.zeros((experts, -(-N // 128), pig.bsfp8_scale_pitch(K)), device="cuda")
    for e in range(experts):
        scale = torch.exp(torch.randn((N, 1), generator=g, device="cuda"))
        B[e], SFB[e] = plain_pack(torch.randn((N, K), generator=g, device="cuda") * scale, 128, fmt)
    # what lies past K and past the last block is not looked at
    A[:, K:] = 0x7F
    B[:, :, K:] = 0x7F
    SFA[:, -(-K // 128):] = math.nan
    SFB[:, :, -(-K // 128):] = math.nan
    return A, SFA, B, SFB


def near(C, a, b, K):
    want = a @ b.t()
    size = a.abs() @ b.abs().t()
    bound = torch.finfo(C.dtype).eps / 2 * want.abs() + (128 + -(-K // 128) + 4) * 2.0 ** -23 * size
    if C.dtype == torch.float16:
        bound += 2.0 ** -25  # subnormal results
    bad = (C.double() - want).abs() > bound
    assert not bool(bad.any()), (int(bad.sum()), (C.double() - want).abs().max().item())


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 128, 128), (3, 130, 200), (16, 256, 512), (17, 100, 640), (32, 1000, 384), (33, 512, 1024),
    (64, 300, 1111), (65, 257, 512), (100, 128, 4160), (128, 640, 256), (129, 1000, 130), (200, 512, 2048),
    (256, 256, 128), (257, 520, 1024), (300, 129, 513), (512, 512, 512), (600, 1002, 416), (1000, 384, 4100)])
@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
def test_product(M, N, K, typ):
    A, SFA, B, SFB = operands(M, N, K)
    C = torch.full((M, N), math.nan, dtype=TYPES[typ], device="cuda")
    pig.igemm_bsfp8(A, B[0], SFA, SFB[0], C, M, N, K)
    assert pig.igemm_last_status() == pig.IGEMM_OK
    near(C, values(A, SFA, 1, "e4m3", K), values(B[0], SFB[0], 128, "e4m3", K), K)


@pytest.mark.parametrize("M,N,K", [(8, 2048, 8192), (24, 1024, 5000), (48, 640, 16384), (70, 256, 40000), (128, 384, 9000),
                                   (16, 28672, 512), (500, 4096, 700), (2100, 700, 300)])
def test_product_split_and_wide(M, N, K):
    # few tiles and a long k (split over a cluster), and many tiles per CTA
    A, SFA, B, SFB = operands(M, N, K, seed=1)
    C = [torch.full((M, N), math.nan, device="cuda") for _ in range(2)]
    for c in C:
        pig.igemm_bsfp8(A, B[0], SFA, SFB[0], c, M, N, K)
    near(C[0], values(A, SFA, 1, "e4m3", K), values(B[0], SFB[0], 128, "e4m3", K), K)
    assert torch.equal(C[0], C[1])  # the order of the sums is fixed


@pytest.mark.parametrize("M,N,K", [(5, 300, 700), (90, 512, 1024), (520, 300, 640)])
def test_product_e5m2(M, N, K):
    A, SFA, B, SFB = operands(M, N, K, "e5m2")
    C = torch.empty((M, N), device="cuda")
    pig.igemm_bsfp8(A, B[0], SFA, SFB[0], C, M, N, K, format="e5m2")
    near(C, values(A, SFA, 1, "e5m2", K), values(B[0], SFB[0], 128, "e5m2", K), K)


@pytest.mark.parametrize("M", [20, 300])
@pytest.mark.parametrize("typ,offset", [("f32", 1), ("bf16", 1), ("bf16", 2), ("f16", 8)])
def test_product_rows_of_c_off_16_bytes(M, typ, offset):
    N, K = 264, 300
    A, SFA, B, SFB = operands(M, N, K)
    whole = torch.full((M * N + offset + 1,), math.nan, dtype=TYPES[typ], device="cuda")
    C = whole[offset:offset + M * N].view(M, N)
    pig.igemm_bsfp8(A, B[0], SFA, SFB[0], C, M, N, K)
    near(C, values(A, SFA, 1, "e4m3", K), values(B[0], SFB[0], 128, "e4m3", K), K)
    assert bool(torch.isnan(whole[:offset]).all()) and bool(torch.isnan(whole[offset + M * N:]).all())


@pytest.mark.parametrize("M", [4, 300])
def test_product_nan_scales(M):
    N, K = 400, 600
    A, SFA, B, SFB = operands(M, N, K)
    SFA[1, 2] = math.nan
    SFB[0, 1, 4] = math.nan
    C = torch.empty((M, N), device="cuda")
    pig.igemm_bsfp8(A, B[0], SFA, SFB[0], C, M, N, K)
    nan = torch.isnan(C)
    assert bool(nan[1].all()) and bool(nan[:, 128:256].all())
    nan[1], nan[:, 128:256] = False, False
    assert not bool(nan.any())


def test_product_empty():
    C = torch.full((3, 5), 7.0, device="cuda")
    e = torch.empty((0,), dtype=torch.uint8, device="cuda")
    f = torch.empty((0,), device="cuda")
    pig.igemm_bsfp8(e, e, f, f, C, 3, 5, 0)
    assert bool((C == 0).all())
    B, SFB = torch.zeros((5, 64), dtype=torch.uint8, device="cuda"), torch.ones((1, 4), device="cuda")
    pig.igemm_bsfp8(e, B, f, SFB, C[:0], 0, 5, 64)


@pytest.mark.parametrize("counts", [[1], [0, 3, 0, 0, 1], [5, 0, 40, 1], [0, 0], [130, 3, 260, 0, 17], [700, 1, 0, 300],
                                    [16] * 40])
@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_grouped(counts, typ):
    E, N, K = len(counts), 300, 700
    start, after = 2, 5  # rows of no group before and behind
    rows = start + sum(counts) + after
    A, SFA, B, SFB = operands(rows, N, K, experts=E)
    ends = [start]
    for n in counts:
        ends.append(ends[-1] + n)
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    C = torch.full((rows, N), 3.0, dtype=TYPES[typ], device="cuda")
    pig.igemm_bsfp8_grouped(A, B, SFA, SFB, offsets, C, rows, E, N, K)
    a = values(A, SFA, 1, "e4m3", K)
    for e in range(E):
        if counts[e]:
            near(C[ends[e]:ends[e + 1]], a[ends[e]:ends[e + 1]], values(B[e], SFB[e], 128, "e4m3", K), K)
    assert bool((C[:start] == 3).all()) and bool((C[ends[-1]:] == 3).all())


@pytest.mark.parametrize("E,each,N,K", [(1024, 70, 256, 640), (700, 20, 384, 1152), (1000, 140, 128, 896)])
def test_grouped_many_experts(E, each, N, K):
    # the largest tables of groups (few slots of codes), an odd number of blocks a tile, several tiles a CTA
    g = torch.Generator(device="cuda").manual_seed(E)
    counts = torch.randint(0, 2 * each, (E,), generator=g, device="cuda")
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    rows = int(offsets[-1])
    A, SFA, B, SFB = operands(rows, N, K, experts=E)
    a, at = values(A, SFA, 1, "e4m3", K), offsets.tolist()
    C = torch.empty((rows, N), dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        C.fill_(math.nan)
        pig.igemm_bsfp8_grouped(A, B, SFA, SFB, offsets, C, rows, E, N, K)
        for e in range(0, E, 37):
            near(C[at[e]:at[e + 1]], a[at[e]:at[e + 1]], values(B[e], SFB[e], 128, "e4m3", K), K)


@pytest.mark.parametrize("M,N,K", [(96, 4096, 640), (128, 20000, 4992), (100, 24000, 384), (16, 60000, 896)])
def test_product_many_tiles_of_odd_blocks(M, N, K):
    A, SFA, B, SFB = operands(M, N, K)
    a, b = values(A, SFA, 1, "e4m3", K), values(B[0], SFB[0], 128, "e4m3", K)
    C = torch.empty((M, N), device="cuda")
    for _ in range(3):
        C.fill_(math.nan)
        pig.igemm_bsfp8(A, B[0], SFA, SFB[0], C, M, N, K)
        near(C, a, b, K)


def test_grouped_offsets_out_of_range():
    # clamped to the rows there are; a group whose end is not past its start is empty
    E, N, K, rows = 4, 128, 256, 50
    A, SFA, B, SFB = operands(rows, N, K, experts=E)
    offsets = torch.tensor([-5, 10, 4, 40, 99], dtype=torch.int32, device="cuda")
    C = torch.full((rows, N), 3.0, device="cuda")
    pig.igemm_bsfp8_grouped(A, B, SFA, SFB, offsets, C, rows, E, N, K)
    a = values(A, SFA, 1, "e4m3", K)
    near(C[40:50], a[40:50], values(B[3], SFB[3], 128, "e4m3", K), K)
    near(C[:4], a[:4], values(B[0], SFB[0], 128, "e4m3", K), K)
