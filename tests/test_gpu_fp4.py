"""GPU tests of the 4-bit floating-point and mixture-of-experts operators against plain implementations in 64 bits.

Packing is defined bit for bit, so its bytes are compared exactly.  Products: the tensor core's products of codes and
scales are exact, and each of the at most K + 64 float32 additions of a sum (k steps, slices of a split k) is off by at
most 2^-23 of the sum of magnitudes (truncation included), so |C - exact| <= (K + 64) 2^-23 sum |a b|, plus half a unit
in the last place of a 16-bit C.
"""

import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
np = pytest.importorskip("numpy")
pytestmark = pytest.mark.gpu

import precision_integer_gemm_gb300 as pig  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_ULP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # of a significand of 24, 8 and 11 bits
TINY = {"f32": 2.0 ** -149, "bf16": 2.0 ** -134, "f16": 2.0 ** -25}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6])
BLOCK = {"mx": 32, "nv": 16}
PITCH = {"mx": pig.mxfp4_scale_pitch, "nv": pig.nvfp4_scale_pitch}


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pig.build_library()
    return pig.load()


def e4m3_values():
    s = np.arange(127)
    return np.where(s >= 8, 2.0 ** (s // 8 - 7) * (1 + s % 8 / 8), s % 8 * 2.0 ** -9)


def nearest_even(v, steps):
    """Index of the nearest of `steps` (ascending); between two, the even index."""
    mids = (steps[1:] + steps[:-1]) / 2
    lo, hi = np.searchsorted(mids, v, side="left"), np.searchsorted(mids, v, side="right")
    return np.where(lo % 2 == 0, lo, hi)


def plain_pack(x, fmt, g=1.0):
    """Codes and scales of a float64 matrix, from the definition (nv: quotient, products and reciprocal in float32)."""
    with np.errstate(over="ignore", invalid="ignore"):
        return _plain_pack(x, fmt, g)


def _plain_pack(x, fmt, g):
    rows, K = x.shape
    Kp, bs = -(-K // 32) * 32, BLOCK[fmt]
    v = np.zeros((rows, Kp))
    v[:, :K] = x
    v = v.reshape(rows, -1, bs)
    fine = np.isfinite(v).all(-1)
    amax = np.where(fine, np.abs(np.where(np.isfinite(v), v, 0)).max(-1), 0)
    if fmt == "mx":
        e = np.maximum(np.frexp(amax)[1] - 3, -127)
        e = np.where(amax > 0, e, -127)
        y = v * 2.0 ** -e[..., None].astype(np.float64)
        s = np.where(fine, e + 127, 255)
    else:
        g = np.float32(g)
        q = np.minimum(amax.astype(np.float32) / (np.float32(6) * g), np.float32(448))
        s8 = nearest_even(q.astype(np.float64), e4m3_values())
        t = e4m3_values()[s8].astype(np.float32) * g
        live = t >= np.float32(2.0 ** -126)
        inv = np.where(live, np.float32(1) / np.where(live, t, np.float32(1)), np.float32(0)).astype(np.float32)
        y = np.where(live[..., None], v.astype(np.float32) * inv[..., None], np.float32(0)).astype(np.float64)
        s = np.where(fine, s8, 0x7F)
    y = np.where(fine[..., None], y, 0)  # (a product that overflows saturates like any other)
    q = nearest_even(np.abs(y), E2M1[:8]) + 8 * np.signbit(y)
    q = np.where(fine[..., None], q, 0).reshape(rows, Kp).astype(np.uint8)
    scales = np.zeros((rows, PITCH[fmt](K)), np.uint8)
    n = -(-K // bs)
    scales[:, :n] = s[:, :n]
    return q[:, 0::2] | (q[:, 1::2] << 4), scales


def gpu_pack(x, fmt, rows=None, index=None, g=None):
    rows, K = (x.shape[0] if rows is None else rows), x.shape[1]
    codes = torch.full((rows, pig.fp4_code_bytes(K)), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((rows, PITCH[fmt](K)), 0xA5, dtype=torch.uint8, device="cuda")
    if fmt == "mx":
        pig.pack_mxfp4(x, codes, scales, rows, K, index=index)
    else:
        pig.pack_nvfp4(x, g, codes, scales, rows, K, index=index)
    return codes, scales


def same_bytes(got, want):
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a.cpu().numpy(), b)


def values(codes, scales, fmt, K):
    """float64 values of packed operands (on the GPU)."""
    q = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1).long()
    s = scales[:, : q.shape[1] // BLOCK[fmt]].long()
    table = torch.tensor(E2M1, device="cuda")
    if fmt == "mx":
        s = torch.where(s == 255, math.nan, torch.exp2(s.double() - 127))
    else:
        steps = torch.tensor(np.concatenate([e4m3_values(), [math.nan]]), device="cuda")
        s = steps[s]
    return (table[q].view(codes.shape[0], -1, BLOCK[fmt]) * s.unsqueeze(-1)).view(codes.shape[0], -1)


def operand(fmt, rows, K, seed, std=1.0):
    """Packed normal values, with every code and rather different scales; padding bytes that have to be ignored."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, K), generator=gen, device="cuda") * std
    x *= torch.exp2(torch.randint(-3, 4, (rows, 1), generator=gen, device="cuda").float())
    codes, scales = gpu_pack(x, fmt)
    scales[:, -(-K // BLOCK[fmt]):] = 0xFF if fmt == "mx" else 0x7F  # NaN: past the last block
    clean = scales.clone()
    clean[:, -(-K // BLOCK[fmt]):] = 0
    return codes, scales, values(codes, clean, fmt, K)


def check_product(C, a, b, K, typ, alpha=1.0):
    exact = alpha * (a @ b.t())
    mag = abs(alpha) * (a.abs() @ b.abs().t())
    bound = (K + 64) * 2.0 ** -23 * mag
    bound = bound + HALF_ULP[typ] * (exact.abs() + bound) * 1.01 + TINY[typ]
    bad = (C.double() - exact).abs() > bound
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} beyond the bound"


# ---------------------------------------------------------------- packing

@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,K", [(1, 1), (1, 32), (3, 31), (5, 33), (2, 48), (17, 256), (9, 500), (130, 544),
                                    (33, 1000), (7, 4160), (3, 8224), (4, 16640)])
def test_pack_rows(fmt, typ, rows, K):
    gen = torch.Generator(device="cuda").manual_seed(rows * 7 + K)
    x = torch.randn((rows, K), generator=gen, device="cuda").to(TYPES[typ])
    g = torch.tensor([0.0029], device="cuda") if fmt == "nv" else None
    same_bytes(gpu_pack(x, fmt, g=g), plain_pack(x.double().cpu().numpy(), fmt, 0.0029))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,K", [(1, 1), (31, 40), (32, 256), (33, 257), (100, 520), (700, 1000)])
def test_pack_transposed(fmt, typ, rows, K):
    gen = torch.Generator(device="cuda").manual_seed(rows + K)
    x = torch.randn((K, rows), generator=gen, device="cuda").to(TYPES[typ])
    same_bytes(gpu_pack(x.t(), fmt), plain_pack(x.t().double().cpu().numpy(), fmt))
    # a part of a wider matrix: rows further apart than their length
    wide = torch.randn((K, rows + 5), generator=gen, device="cuda").to(TYPES[typ])
    part = wide[:, 2:2 + rows].t()
    same_bytes(gpu_pack(part, fmt), plain_pack(part.double().cpu().numpy(), fmt))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
def test_pack_strided_and_unaligned_rows(fmt, typ):
    gen = torch.Generator(device="cuda").manual_seed(3)
    wide = torch.randn((40, 203), generator=gen, device="cuda").to(TYPES[typ])
    for x in (wide[:, 1:129], wide[3:20, :96], wide[::2, 5:105]):
        same_bytes(gpu_pack(x, fmt), plain_pack(x.double().cpu().numpy(), fmt))


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("transposed", [False, True])
def test_pack_from_every_start(typ, transposed):
    gen = torch.Generator(device="cuda").manual_seed(11)
    buf = torch.randn(4096, generator=gen, device="cuda").to(TYPES[typ])
    buf[0] = buf[-1] = math.nan  # (outside of what the views hold)
    for start in range(1, 10):
        for rows, K, ld in ((1, 47, 47), (5, 96, 96), (5, 100, 101), (7, 129, 130), (3, 260, 263)):
            shape, strides = ((rows, K), (ld, 1)) if not transposed else ((K // 8, rows), (1, ld))
            x = buf.as_strided(shape, strides, start)
            same_bytes(gpu_pack(x, "mx"), plain_pack(x.double().cpu().numpy(), "mx"))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_pack_special_values(fmt):
    x = np.zeros((16, 64), np.float32)
    x[0] = -0.0
    x[1, 5], x[2, 40], x[3, 3] = np.nan, np.inf, -np.inf
    x[4] = np.float32(2.0 ** -149)                      # smallest subnormal
    x[5] = np.linspace(-2.0 ** -127, 2.0 ** -127, 64)   # subnormals
    x[6] = np.finfo(np.float32).max
    x[7] = np.tile(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], np.float32), 8)  # ties (mx: scale 1)
    x[8] = -x[7]
    x[9] = 7.99                                         # saturates at 6
    x[10, 0] = 1e-30                                    # the rest of its block is zero
    x[11] = np.float32(2.0 ** 120) * x[7]
    x[12] = np.float32(2.0 ** -126)
    x[13, ::2] = 1e38
    x[13, 1::2] = -1e-38
    x[14] = np.nan
    same_bytes(gpu_pack(torch.from_numpy(x).cuda(), fmt), plain_pack(x.astype(np.float64), fmt))
    same_bytes(gpu_pack(torch.from_numpy(x.T.copy()).cuda().t(), fmt), plain_pack(x.astype(np.float64), fmt))
    for g in (1e-3, 2.0 ** -20, 1e20, 1e-38):
        if fmt == "nv":
            same_bytes(gpu_pack(torch.from_numpy(x).cuda(), fmt, g=torch.tensor([g], device="cuda")),
                       plain_pack(x.astype(np.float64), fmt, g))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
def test_pack_gathers_rows(fmt, typ):
    gen = torch.Generator(device="cuda").manual_seed(11)
    x = torch.randn((20, 300), generator=gen, device="cuda").to(TYPES[typ])
    index = torch.tensor([5, -1, 19, 0, 0, 20, 7, -2147483648, 2147483647, 3], dtype=torch.int32, device="cuda")
    want = x.double().cpu().numpy()[np.clip(index.cpu().numpy(), 0, 19)]
    want[(index.cpu().numpy() < 0) | (index.cpu().numpy() > 19)] = 0
    same_bytes(gpu_pack(x, fmt, rows=10, index=index), plain_pack(want, fmt))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("typ,rows,source,K", [("f32", 17000, 100, 515), ("bf16", 8400, 4200, 4096),
                                               ("f16", 140001, 7, 130)])
def test_pack_gathers_rows_many_times(fmt, typ, rows, source, K):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn((source, K + 3), generator=gen, device="cuda").to(TYPES[typ])[:, :K]
    x[source // 2, 5] = math.nan
    index = torch.randint(-2, source + 2, (rows,), generator=gen, device="cuda").int()  # some out of range
    index[:3] = torch.tensor([-2 ** 31, 2 ** 31 - 1, source], dtype=torch.int32)
    g = torch.tensor([0.0031], device="cuda") if fmt == "nv" else None
    codes, scales = plain_pack(x.double().cpu().numpy(), fmt, 0.0031)
    at = index.cpu().numpy()
    out = (at < 0) | (at >= source)
    at = np.where(out, 0, at)
    want = [np.where(out[:, None], 0, a[at]) for a in (codes, scales)]
    same_bytes(gpu_pack(x, fmt, rows=rows, index=index, g=g), want)


def test_pack_refuses_what_it_cannot_read():
    x = torch.zeros((8, 64), device="cuda")
    c = torch.zeros((8, 32), dtype=torch.uint8, device="cuda")
    s = torch.zeros((8, 16), dtype=torch.uint8, device="cuda")
    with pytest.raises(ValueError, match="packs"):
        pig.pack_mxfp4(x, c, s, 8, 32)
    with pytest.raises(ValueError, match="packs"):
        pig.pack_mxfp4(x, c, s, 7, 64)
    with pytest.raises(ValueError, match="unit stride"):
        pig.pack_mxfp4(torch.zeros((8, 128), device="cuda")[:, ::2], c, s, 8, 64)
    with pytest.raises(ValueError, match="overlapping"):
        pig.pack_mxfp4(x[0].expand(8, 64), c, s, 8, 64)
    with pytest.raises(ValueError, match="bytes"):
        pig.pack_mxfp4(x, c[:7], s, 8, 64)
    with pytest.raises(ValueError, match="gathered"):
        pig.pack_mxfp4(torch.zeros((64, 8), device="cuda").t(), c, s, 8, 64,
                       index=torch.zeros(8, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="int32"):
        pig.pack_mxfp4(x, c, s, 8, 64, index=torch.zeros(8, dtype=torch.int64, device="cuda"))


# ---------------------------------------------------------------- products

def product(fmt, A, B, SFA, SFB, C, M, N, K, alpha=None):
    if fmt == "mx":
        pig.igemm_mxfp4(A, B, SFA, SFB, C, M, N, K)
    else:
        pig.igemm_nvfp4(A, B, SFA, SFB, alpha, C, M, N, K)


# every kernel width (M up to 16, 32, 64, 128 and the CTA pairs), one and several k slices, ragged N and K, one value
SHAPES = [(1, 1, 1), (1, 128, 32), (2, 7, 33), (16, 130, 512), (16, 4096, 4096), (5, 300, 1000), (17, 640, 2080),
          (32, 1000, 520), (33, 257, 4160), (64, 2048, 8192), (65, 129, 640), (100, 500, 96), (128, 1200, 3000),
          (129, 512, 1056), (200, 10002, 416), (300, 5000, 2080), (512, 4096, 544), (600, 10002, 4160), (777, 3001, 260)]


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(fmt, M, N, K):
    A, SFA, a = operand(fmt, M, K, M + N)
    B, SFB, b = operand(fmt, N, K, N + K, 0.05)
    typ = ("f32", "bf16", "f16")[(M + N + K) % 3]
    C = torch.full((M, N), 777.0, dtype=TYPES[typ], device="cuda")
    product(fmt, A, B, SFA, SFB, C, M, N, K)
    assert pig.igemm_last_status() == 0
    check_product(C, a, b, K, typ)
    again = torch.full_like(C, -1.0)
    product(fmt, A, B, SFA, SFB, again, M, N, K)
    assert torch.equal(C, again)


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N", [512, 516, 515, 1026])
def test_product_output_types_and_row_alignments(typ, N):
    A, SFA, a = operand("nv", 300, 320, 1)
    B, SFB, b = operand("nv", N, 320, 2, 0.05)
    alpha = torch.tensor([0.37], device="cuda")
    buf = torch.zeros((300 * N + 16,), dtype=TYPES[typ], device="cuda")
    for shift in (0, 1, 2):  # rows that start off a 16-byte boundary
        C = buf[shift:shift + 300 * N].view(300, N)
        buf.fill_(5.0)
        pig.igemm_nvfp4(A, B, SFA, SFB, alpha, C, 300, N, 320)
        check_product(C, a, b, 320, typ, alpha.double())
        assert bool((buf[:shift] == 5).all()) and bool((buf[shift + 300 * N:] == 5).all())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M", [3, 40, 300])
def test_product_exact_integers(fmt, M):
    # codes times unit scales: every sum is an integer or a quarter below 2^22, exact in float32
    gen = torch.Generator(device="cuda").manual_seed(M)
    N, K = 384, 1536
    A = torch.randint(0, 256, (M, K // 2), generator=gen, dtype=torch.uint8, device="cuda")
    B = torch.randint(0, 256, (N, K // 2), generator=gen, dtype=torch.uint8, device="cuda")
    one = 127 if fmt == "mx" else 0x38
    SFA, SFB = (torch.full((r, PITCH[fmt](K)), one, dtype=torch.uint8, device="cuda") for r in (M, N))
    C = torch.empty((M, N), device="cuda")
    product(fmt, A, B, SFA, SFB, C, M, N, K)
    assert torch.equal(C.double(), values(A, SFA, fmt, K) @ values(B, SFB, fmt, K).t())


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("M", [4, 300])
def test_product_extreme_and_nan_scales(fmt, M):
    N, K = 300, 640
    A, SFA, _ = operand(fmt, M, K, 5)
    B, SFB, _ = operand(fmt, N, K, 6)
    lo, hi = (60, 190) if fmt == "mx" else (0, 126)
    gen = torch.Generator(device="cuda").manual_seed(9)
    blocks = -(-K // BLOCK[fmt])
    SFA[:, :blocks] = torch.randint(lo, hi + 1, (M, blocks), generator=gen, device="cuda").to(torch.uint8)
    clean = SFA.clone()
    clean[:, blocks:] = 0
    cleanb = SFB.clone()
    cleanb[:, blocks:] = 0
    C = torch.empty((M, N), device="cuda")
    product(fmt, A, B, SFA, SFB, C, M, N, K)
    check_product(C, values(A, clean, fmt, K), values(B, cleanb, fmt, K), K, "f32")
    # a NaN scale makes its row (of B: its column) NaN and nothing else
    SFA[1, 3] = SFB[7, blocks - 1] = 0xFF if fmt == "mx" else 0x7F
    product(fmt, A, B, SFA, SFB, C, M, N, K)
    nan = torch.isnan(C)
    want = torch.zeros_like(nan)
    want[1] = want[:, 7] = True
    assert torch.equal(nan, want)


def test_product_of_nothing():
    C = torch.full((4, 8), 3.0, device="cuda")
    u8 = torch.zeros((256,), dtype=torch.uint8, device="cuda")
    pig.igemm_mxfp4(u8, u8, u8, u8, C, 4, 8, 0)
    assert bool((C == 0).all())
    pig.igemm_mxfp4(u8, u8, u8, u8, C, 0, 8, 32)


def test_operators_on_another_stream():
    side = torch.cuda.Stream()
    x = torch.randn((64, 1024), device="cuda")
    B, SFB, b = operand("mx", 256, 1024, 4, 0.05)
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x2 = x * 2
        codes, scales = gpu_pack(x2, "mx")
        C = torch.empty((64, 256), device="cuda")
        pig.igemm_mxfp4(codes, B, scales, SFB, C, 64, 256, 1024)
    side.synchronize()
    check_product(C, values(codes, scales, "mx", 1024), b, 1024, "f32")


def test_calls_back_to_back_see_each_other():
    # each call reads what the call before it wrote and overwrites what the one before that read; nothing waits between
    gen = torch.Generator(device="cuda").manual_seed(2)
    N = K = 512
    B, SFB, _ = operand("mx", N, K, 3, 0.05)
    for M in (4, 48, 300):
        x0 = torch.randn((M, K), generator=gen, device="cuda")
        codes = torch.empty((M, pig.fp4_code_bytes(K)), dtype=torch.uint8, device="cuda")
        scales = torch.empty((M, pig.mxfp4_scale_pitch(K)), dtype=torch.uint8, device="cuda")

        def chain(wait):
            x, out = x0.clone(), []
            for _ in range(40):
                pig.pack_mxfp4(x, codes, scales, M, K)
                wait()
                pig.igemm_mxfp4(codes, B, scales, SFB, x, M, N, K)
                wait()
                out.append(x.clone())
                wait()
            torch.cuda.synchronize()
            return out

        for a, b in zip(chain(lambda: None), chain(torch.cuda.synchronize)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T", [7, 200])
def test_layer_in_a_graph(T):
    # routing, gathered packing, a grouped product and the sum, captured once and replayed on new values
    E, k, N, K = 16, 4, 256, 512
    gen = torch.Generator(device="cuda").manual_seed(T)
    logits, x = torch.empty((T, E), device="cuda"), torch.empty((T, K), device="cuda")
    b, sb, _ = operand("mx", E * N, K, 3)
    i32 = dict(dtype=torch.int32, device="cuda")
    experts, weights, slots = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda"), torch.empty((T, k), **i32)
    offsets, tokens = torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
    a = torch.empty((T * k, pig.fp4_code_bytes(K)), dtype=torch.uint8, device="cuda")
    sa = torch.empty((T * k, pig.mxfp4_scale_pitch(K)), dtype=torch.uint8, device="cuda")
    y, out = torch.empty((T * k, N), device="cuda"), torch.empty((T, N), device="cuda")

    def layer():
        pig.igemm_moe_route(logits, experts, weights, offsets, tokens, slots, T, E, k)
        pig.pack_mxfp4(x, a, sa, T * k, K, index=tokens)
        pig.igemm_mxfp4_grouped(a, b, sa, sb, offsets, y, T * k, E, N, K)
        pig.igemm_moe_combine(y, slots, weights, out, T, k, N)

    logits.normal_(generator=gen), x.normal_(generator=gen)
    layer()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer()
    for _ in range(3):
        logits.normal_(generator=gen), x.normal_(generator=gen)
        out.fill_(math.nan)
        graph.replay()
        got = out.clone()
        layer()
        assert bool(torch.isfinite(got).all()) and torch.equal(got, out)
    assert pig.igemm_last_status() == 0


def test_timing_events_around_a_product():
    A, SFA, a = operand("nv", 8, 256, 1)
    B, SFB, b = operand("nv", 64, 256, 2)
    C = torch.empty((8, 64), device="cuda")
    start, stop = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    start.record(), stop.record()
    before = pig.igemm_kernels_launched()
    pig.igemm_time_next_gemm(start, stop)
    pig.igemm_nvfp4(A, B, SFA, SFB, None, C, 8, 64, 256)
    torch.cuda.synchronize()
    assert pig.igemm_kernels_launched() == before + 1 and start.elapsed_time(stop) > 0
    check_product(C, a, b, 256, "f32")


# ---------------------------------------------------------------- grouped products

def grouped(fmt, counts, N, K, typ, seed=0, alpha=None, rows=None, offsets=None):
    E, total = len(counts), sum(counts)
    rows = total if rows is None else rows
    A, SFA, a = operand(fmt, max(rows, 1), K, seed + 1)
    B, SFB, b = operand(fmt, E * N, K, seed + 2, 0.05)
    if offsets is None:
        offsets = np.concatenate([[0], np.cumsum(counts)])
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    C = torch.full((rows, N), 777.0, dtype=TYPES[typ], device="cuda")
    if fmt == "mx":
        pig.igemm_mxfp4_grouped(A, B, SFA, SFB, off, C, rows, E, N, K)
    else:
        pig.igemm_nvfp4_grouped(A, B, SFA, SFB, off, alpha, C, rows, E, N, K)
    assert pig.igemm_last_status() == 0
    return C, a, b.view(E, N, -1)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("counts,N,K,typ", [
    ([1], 130, 64, "f32"), ([0, 3, 0, 1, 0], 257, 1000, "bf16"), ([4, 2, 1] * 20, 512, 544, "f16"),
    ([20, 0, 31, 17, 5], 640, 2080, "f32"), ([70, 1, 128, 0, 64], 384, 4128, "bf16"),
    ([128, 129, 300, 0, 65, 1], 1000, 416, "f32"), ([1000, 7, 513], 515, 288, "bf16"),
    (list(range(1, 258)) + [300] * 40, 256, 288, "bf16")])  # tiles of every number of rows, on CTA pairs
def test_grouped_product(fmt, counts, N, K, typ):
    C, a, b = grouped(fmt, counts, N, K, typ)
    at = 0
    for e, n in enumerate(counts):
        if n:
            check_product(C[at:at + n], a[at:at + n], b[e], K, typ)
        at += n


@pytest.mark.parametrize("n", list(range(1, 129, 9)) + [127, 128])
def test_grouped_product_narrow_tiles(n):
    # every number of rows on the single-CTA kernels, next to an empty and a one-row group
    C, a, b = grouped("mx", [n, 0, 1], 200, 544, "f32", seed=n)
    check_product(C[:n], a[:n], b[0], 544, "f32")
    check_product(C[n:], a[n:], b[2], 544, "f32")


# weights of more than 32 MB, asked for ahead of the kernel's turn
@pytest.mark.parametrize("fmt,M,N,K", [("mx", 5, 16500, 4196), ("nv", 40, 9001, 8256), ("mx", 100, 66001, 1090)])
def test_product_of_large_ragged_weights(fmt, M, N, K):
    A, SA, a = operand(fmt, M, K, 21)
    B, SB, b = operand(fmt, N, K, 22)
    for _ in range(2):
        C = torch.full((M, N), math.nan, device="cuda")
        product(fmt, A, B, SA, SB, C, M, N, K)
        check_product(C, a, b, K, "f32")


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_grouped_product_of_large_weights_right_after_routing(fmt):
    # the kernel that writes the offsets is the one before; they hold anything until then
    T, E, k, N, K = 12, 8, 2, 8200, 1100
    gen = torch.Generator(device="cuda").manual_seed(5)
    B, SB, b = operand(fmt, E * N, K, 23)
    b = b.view(E, N, -1)
    i32 = dict(dtype=torch.int32, device="cuda")
    experts, weights, slots = torch.empty((T, k), **i32), torch.empty((T, k), device="cuda"), torch.empty((T, k), **i32)
    offsets, tokens = torch.empty(E + 1, **i32), torch.empty(T * k, **i32)
    A, SA, a = operand(fmt, T * k, K, 24)
    for fill in (0, -5, 2 ** 31 - 1, -2 ** 31, 11):
        logits = torch.randn((T, E), generator=gen, device="cuda")
        C = torch.full((T * k, N), math.nan, device="cuda")
        offsets.fill_(fill)
        pig.igemm_moe_route(logits, experts, weights, offsets, tokens, slots, T, E, k)
        if fmt == "mx":
            pig.igemm_mxfp4_grouped(A, B, SA, SB, offsets, C, T * k, E, N, K)
        else:
            pig.igemm_nvfp4_grouped(A, B, SA, SB, offsets, None, C, T * k, E, N, K)
        ends = offsets.tolist()
        assert ends == sorted(ends) and ends[-1] == T * k
        for e in range(E):
            if ends[e] < ends[e + 1]:
                check_product(C[ends[e]:ends[e + 1]], a[ends[e]:ends[e + 1]], b[e], K, "f32")


def test_grouped_product_alpha_per_expert():
    alpha = torch.tensor([0.5, -2.0, 3e-3], device="cuda")
    C, a, b = grouped("nv", [40, 9, 100], 300, 320, "f32", alpha=alpha)
    for e, (i, j) in enumerate([(0, 40), (40, 49), (49, 149)]):
        check_product(C[i:j], a[i:j], b[e], 320, "f32", alpha[e].double())


def test_grouped_product_rows_of_no_group_stay():
    C, a, b = grouped("mx", [5, 6], 256, 96, "f32", rows=40, offsets=[8, 13, 19])
    assert bool((C[:8] == 777).all()) and bool((C[19:] == 777).all())
    check_product(C[8:13], a[8:13], b[0], 96, "f32")
    check_product(C[13:19], a[13:19], b[1], 96, "f32")


def test_grouped_product_clamps_offsets():
    # offsets out of range or out of order name fewer rows, never others than C's
    for offsets, groups in [([-5, 10, 60], [(0, 10), (10, 40)]), ([30, 20, 25], [(30, 30), (20, 25)]),
                            ([50, 60, 70], []), ([2147483647, -2147483648, 12], [(0, 0), (0, 12)])]:
        C, a, b = grouped("mx", [1, 1], 200, 160, "f32", rows=40, offsets=offsets)
        touched = torch.zeros(40, dtype=torch.bool, device="cuda")
        for e, (i, j) in enumerate(groups):
            if j > i:
                check_product(C[i:j], a[i:j], b[e], 160, "f32")
                touched[i:j] = True
        assert bool((C[~touched] == 777).all())


def test_grouped_product_most_experts():
    counts = [(7 * e) % 5 for e in range(1024)]
    C, a, b = grouped("nv", counts, 128, 64, "f32")
    b_of_row = torch.repeat_interleave(torch.arange(1024, device="cuda"), torch.tensor(counts, device="cuda"))
    exact = torch.einsum("rk,rnk->rn", a, b[b_of_row])
    assert (C.double() - exact).abs().max() <= 1e-5 * exact.abs().max()


# ---------------------------------------------------------------- routing and combining

def plain_route(x, k, normalize):
    """From float64 logits [T, E], by sorting."""
    T, E = x.shape
    x = np.where(np.isnan(x), -np.inf, x)
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -x), axis=-1)[:, :k]
    top = np.take_along_axis(x, order, -1)
    there = top > -np.inf
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        m = np.where(there[:, :1], top[:, :1], 0.0)
        total = np.exp((top if normalize else x) - m).sum(-1, keepdims=True)
        weights = np.where(there, np.exp(top - m) / total, 0.0)
    experts = np.where(there, order, -1)
    t, j = np.nonzero(there)
    by = np.lexsort((t, experts[t, j]))
    tokens, slots = np.full(T * k, -1), np.full((T, k), -1)
    tokens[:by.size] = t[by]
    slots[t[by], j[by]] = np.arange(by.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(experts[t, j], minlength=E))])
    return experts, weights, offsets, tokens, slots


def gpu_route(logits, k, normalize):
    T, E = logits.shape
    out = [torch.full(s, 99, dtype=d, device="cuda") for s, d in
           (((T, k), torch.int32), ((T, k), torch.float32), ((E + 1,), torch.int32), ((T * k,), torch.int32),
            ((T, k), torch.int32))]
    pig.igemm_moe_route(logits, *out, T, E, k, normalize=normalize)
    return out


def check_route(logits, k, normalize):
    got = gpu_route(logits, k, normalize)
    want = plain_route(logits.double().cpu().numpy(), k, normalize)
    for i in (0, 2, 3, 4):
        np.testing.assert_array_equal(got[i].cpu().numpy(), want[i])
    # a logit's difference is exact or rounded once (2^-24 of it, at most 2^-17 here), exp and sum a few units more
    np.testing.assert_allclose(got[1].cpu().numpy(), want[1], rtol=2e-5, atol=1e-38)


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 8), (3, 60, 4), (64, 64, 6), (65, 65, 8), (100, 128, 1),
                                   (130, 200, 32), (257, 256, 8), (1000, 257, 3), (70, 512, 16), (300, 1024, 8),
                                   (33, 1000, 10)])
def test_route(typ, T, E, k):
    gen = torch.Generator(device="cuda").manual_seed(T + E)
    x = (torch.randn((T, E), generator=gen, device="cuda") * 2).to(TYPES[typ])
    for normalize in (True, False):
        check_route(x, k, normalize)


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E", [(20, 40), (200, 96), (90, 700)])
def test_route_ties_masks_and_specials(typ, T, E):
    gen = torch.Generator(device="cuda").manual_seed(E)
    x = torch.randint(-2, 3, (T, E), generator=gen, device="cuda").to(TYPES[typ])  # ties everywhere
    x[0] = 0.0
    x[1, ::2] = -0.0                               # equal to +0
    x[2] = -math.inf                               # nothing to choose
    x[3] = -math.inf
    x[3, E - 1] = -3.0                             # one expert only
    x[4, ::3] = math.nan
    x[5] = math.nan
    x[6] = torch.finfo(TYPES[typ]).min             # the type's lowest value is not a mask
    x[7, 5] = torch.finfo(TYPES[typ]).min
    x[8] = torch.finfo(TYPES[typ]).max
    x[torch.rand((T, E), generator=gen, device="cuda") < 0.3] = -math.inf
    for k in (1, 5, 8):
        for normalize in (True, False):
            check_route(x, k, normalize)


@pytest.mark.parametrize("typ", ["bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(65, 5, 3), (127, 40, 8), (67, 64, 1), (66, 66, 7), (129, 128, 2), (190, 201, 8),
                                   (259, 256, 5), (512, 30, 8), (513, 5, 3), (600, 40, 8), (530, 64, 1), (1025, 66, 7),
                                   (700, 128, 2), (514, 201, 8), (777, 256, 5)])
def test_route_of_several_blocks(typ, T, E, k):
    gen = torch.Generator(device="cuda").manual_seed(T * E)
    for scale in (1, 200):                         # ties everywhere, and hardly any
        x = (torch.randint(-2 * scale, 2 * scale + 1, (T, E), generator=gen, device="cuda") / scale).to(TYPES[typ])
        x[torch.rand((T, E), generator=gen, device="cuda") < 0.2] = -math.inf
        x[torch.rand((T, E), generator=gen, device="cuda") < 0.05] = math.nan
        x[-1] = -math.inf
        x[-2] = math.nan
        x[-3, 1:] = -math.inf
        x[-3, 0] = torch.finfo(TYPES[typ]).min
        for normalize in (True, False):
            check_route(x, k, normalize)


@pytest.mark.parametrize("typ,T,E,k", [("bf16", 32769, 256, 2), ("f32", 16500, 1000, 3), ("f16", 20000, 3, 2)])
def test_route_of_many_tokens(typ, T, E, k):
    gen = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, E), generator=gen, device="cuda").to(TYPES[typ])
    x[torch.rand(T, generator=gen, device="cuda") < 0.1] = -math.inf
    check_route(x, k, True)


def test_route_infinite_logit_gives_nan_weights():
    x = torch.zeros((2, 8), device="cuda")
    x[0, 3] = math.inf
    experts, weights, offsets, *_ = gpu_route(x, 2, True)
    assert experts[0].tolist() == [3, 0] and bool(torch.isnan(weights[0]).all())
    assert not bool(torch.isnan(weights[1]).any()) and int(offsets[-1]) == 4


def test_route_of_nothing():
    off = torch.full((9,), 7, dtype=torch.int32, device="cuda")
    e = torch.empty((0,), dtype=torch.int32, device="cuda")
    pig.igemm_moe_route(torch.empty((0, 8), device="cuda"), e, e.float(), off, e, e, 0, 8, 2)
    assert bool((off == 0).all())


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 4, 7), (5, 8, 64), (100, 2, 1000), (33, 32, 520), (64, 5, 4096)])
def test_combine(typ, T, k, N):
    gen = torch.Generator(device="cuda").manual_seed(T * k + N)
    Y = torch.randn((T * k, N), generator=gen, device="cuda").to(TYPES[typ])
    slots = torch.randperm(T * k, generator=gen, device="cuda").int().view(T, k)
    slots[torch.rand((T, k), generator=gen, device="cuda") < 0.2] = -1
    if T > 2:
        slots[1] = -1              # a token none of whose pairs were routed
        slots[2, 0] = T * k        # out of range
        Y[int(slots[0].clamp(min=0)[0])] = 2.0
    w = torch.rand((T, k), generator=gen, device="cuda")
    out = torch.full((T, N), 9.0, dtype=TYPES[typ], device="cuda")
    pig.igemm_moe_combine(Y, slots, w, out, T, k, N)
    live = (slots >= 0) & (slots < T * k)
    rows = Y.double()[slots.clamp(0, T * k - 1).long()] * live.unsqueeze(-1)
    exact, mag = (rows * w.double().unsqueeze(-1)).sum(1), (rows.abs() * w.double().unsqueeze(-1)).sum(1)
    bound = k * 2.0 ** -24 * mag  # one rounding an addition
    bound = bound + HALF_ULP[typ] * (exact.abs() + bound) * 1.01 + TINY[typ]
    assert bool(((out.double() - exact).abs() <= bound).all())


def test_combine_ignores_rows_it_does_not_take():
    Y = torch.full((6, 64), math.nan, device="cuda")
    Y[2], Y[4] = 1.0, 3.0
    slots = torch.tensor([[2, -1], [4, 2], [-1, -1]], dtype=torch.int32, device="cuda")
    out = torch.empty((3, 64), device="cuda")
    pig.igemm_moe_combine(Y, slots, torch.full((3, 2), 0.5, device="cuda"), out, 3, 2, 64)
    assert out[:, 0].tolist() == [0.5, 2.0, 0.0] and not bool(torch.isnan(out).any())


# ---------------------------------------------------------------- together

def test_linear_layer_gradients_from_transposed_packing():
    # dX = dY W and dW = dY^T X on 4-bit operands: the blocks run along the summed axis, so each operand is
    # packed the other way round than for the forward product
    gen = torch.Generator(device="cuda").manual_seed(1)
    T, D, N = 200, 320, 416
    x, dy, w = (torch.randn(s, generator=gen, device="cuda") for s in ((T, D), (T, N), (N, D)))
    for a, b, rows, cols, K in ((dy, w.t(), T, D, N), (dy.t(), x.t(), N, D, T)):
        pa, pb = gpu_pack(a, "mx"), gpu_pack(b, "mx")
        C = torch.empty((rows, cols), device="cuda")
        pig.igemm_mxfp4(pa[0], pb[0], pa[1], pb[1], C, rows, cols, K)
        check_product(C, values(*pa, "mx", K), values(*pb, "mx", K), K, "f32")
        exact = a.double() @ b.double().t()
        assert (C.double() - exact).norm() < 0.25 * exact.norm()  # two operands of e2m1, about 0.11 each


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("T", [1, 9, 300])
def test_moe_layer(fmt, T):
    """examples/moe_fp4.py against the same layer in float64 on the operands that it packed."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import moe_fp4
    finally:
        sys.path.pop(0)
    gen = torch.Generator(device="cuda").manual_seed(T)
    E, D, F, k = 12, 256, 160, 3
    router, gate_up, down = (torch.randn(s, generator=gen, device="cuda") / s[-1] ** 0.5
                             for s in ((E, D), (E, 2 * F, D), (E, D, F)))
    layer = moe_fp4.MoeFp4(router, gate_up, down, k, fmt)
    x = torch.randn((T, D), generator=gen, device="cuda")
    out = layer(x)
    assert pig.igemm_last_status() == 0

    def unpacked(p, g, K):
        return values(*p, fmt, K)[:, :K] * (1.0 if g is None else g.double())

    w1 = unpacked(layer.gate_up, layer.g1, D).view(E, 2 * F, D)
    w2 = unpacked(layer.down, layer.g2, F).view(E, D, F)
    gx = layer._tensor_scale(x)
    xq = unpacked(layer.pack(x, gx), gx, D)
    top, ids = torch.topk((x @ router.t()), k, dim=-1)
    weights = torch.softmax(top.double(), -1)
    h = torch.einsum("td,tkfd->tkf", xq, w1[ids])
    act = (torch.nn.functional.silu(h[..., :F]) * h[..., F:]).float().view(-1, F)
    ga = layer._tensor_scale(act)
    aq = unpacked(layer.pack(act, ga), ga, F).view(T, k, F)
    exact = (torch.einsum("tkf,tkdf->tkd", aq, w2[ids]) * weights.unsqueeze(-1)).sum(1)
    # (an activation on the edge between two codes may fall the other way in float32)
    assert (out.double() - exact).norm() <= 0.01 * exact.norm()
