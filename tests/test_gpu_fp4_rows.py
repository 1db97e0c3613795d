"""GPU tests of the sum of the experts' rows at every width of a load and store, against float64.

Each of the k products of a sum is added with one rounding, so |out - exact| <= k 2^-24 sum |w y|, plus half a unit in the
last place of a 16-bit output (significands of 8 and 11 bits) and half the smallest subnormal.
"""

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import precision_integer_gemm_gb300 as pig  # noqa: E402

TYPES = {"f32": (torch.float32, 2.0 ** -24, 2.0 ** -149), "bf16": (torch.bfloat16, 2.0 ** -8, 2.0 ** -134),
         "f16": (torch.float16, 2.0 ** -11, 2.0 ** -25)}


@pytest.fixture(scope="module", autouse=True)
def lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    pig.build_library()
    return pig.load()


# columns: multiples of 16 bytes, of 8, of 4 and of 2, of a few, of one and of several blocks of threads, whole and not
WIDTHS = [1, 2, 3, 4, 6, 12, 127, 128, 130, 254, 510, 511, 512, 513, 514, 516, 1022, 1024, 1025, 1026, 1028, 1030, 1540,
          2047, 2050, 4100]


@pytest.mark.parametrize("typ", list(TYPES))
@pytest.mark.parametrize("shift", [(0, 0), (1, 0), (0, 1), (2, 2), (4, 4), (3, 6)])
def test_combine_rows_of_every_width_and_start(typ, shift):
    dtype, half, tiny = TYPES[typ]
    gen = torch.Generator(device="cuda").manual_seed(sum(shift))
    for T, k in ((1, 1), (3, 5), (7, 8)):
        for N in WIDTHS:
            # Y and out start `shift` elements after a 16-byte boundary; nothing around out may be written
            Y = torch.randn((T * k * N + 8,), generator=gen, device="cuda").to(dtype)[shift[0]:shift[0] + T * k * N]
            Y = Y.view(T * k, N)
            slots = torch.randint(-1, T * k + 1, (T, k), generator=gen, device="cuda", dtype=torch.int32)  # some none
            w = torch.randn((T, k), generator=gen, device="cuda")
            buf = torch.full((T * N + 16,), -777.0, dtype=dtype, device="cuda")
            out = buf[shift[1]:shift[1] + T * N].view(T, N)
            pig.igemm_moe_combine(Y, slots, w, out, T, k, N)
            live = (slots >= 0) & (slots < T * k)
            rows = Y.double()[slots.clamp(0, T * k - 1).long()] * (w.double() * live).unsqueeze(-1)
            exact, bound = rows.sum(1), k * 2.0 ** -24 * rows.abs().sum(1)
            bound = bound + half * (exact.abs() + bound) * 1.01 + tiny
            assert bool(((out.double() - exact).abs() <= bound).all()), (T, k, N)
            assert bool((buf[:shift[1]] == -777).all()) and bool((buf[shift[1] + T * N:] == -777).all()), (T, k, N)


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_moe_layer_of_no_tokens(fmt):
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import moe_fp4
    finally:
        sys.path.pop(0)
    router, gate_up, down = (torch.randn(s, device="cuda") for s in ((4, 64), (4, 2 * 96, 64), (4, 64, 96)))
    layer = moe_fp4.MoeFp4(router, gate_up, down, 2, fmt)
    out = layer(torch.empty((0, 64), device="cuda"))
    assert out.shape == (0, 64) and out.dtype == torch.float32
    assert pig.igemm_last_status() == 0
