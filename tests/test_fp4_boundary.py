"""Host-side checks of the 4-bit floating-point and mixture-of-experts entry points: argument errors come back
before anything is launched, so no GPU is needed.  (No call here passes FAKE with valid arguments.)"""

import pytest

import precision_integer_gemm_gb300 as pig

FAKE = 0x10000  # a 16-byte-aligned address that the rejected calls never touch


@pytest.fixture(scope="module")
def lib():
    pig.build_library()
    return pig.load()


def test_sizes_of_rows():
    for K, code, mx, nv in [(1, 16, 16, 16), (32, 16, 16, 16), (33, 32, 16, 16), (256, 128, 16, 16), (257, 144, 16, 32),
                            (512, 256, 16, 32), (513, 272, 32, 48), (4160, 2080, 144, 272), (8192, 4096, 256, 512)]:
        assert (pig.fp4_code_bytes(K), pig.mxfp4_scale_pitch(K), pig.nvfp4_scale_pitch(K)) == (code, mx, nv)


@pytest.mark.parametrize("nv", [False, True])
def test_pack_refusals(lib, nv):
    fn = lib.pack_nvfp4 if nv else lib.pack_mxfp4

    def call(x=FAKE, typ=1, ld=64, transposed=0, index=None, x_rows=8, g=None, codes=FAKE, scales=FAKE, rows=8, K=64):
        extra = (g,) if nv else ()
        return fn(x, typ, ld, transposed, index, x_rows, *extra, codes, scales, rows, K, None)

    assert call(rows=0, x=None) == pig.IGEMM_OK and call(K=0, x=None) == pig.IGEMM_OK
    for bad in (dict(rows=-1), dict(K=-1), dict(x_rows=-1), dict(ld=-1), dict(typ=3), dict(typ=-1), dict(codes=None),
                dict(scales=None), dict(x=None), dict(x_rows=7), dict(ld=63), dict(transposed=1, ld=7)):
        assert call(**bad) == pig.IGEMM_INVALID_ARGUMENT, bad
    assert call(transposed=1, index=FAKE) == pig.IGEMM_UNSUPPORTED_SHAPE
    assert call(K=(1 << 22) + 1, ld=1 << 23) == pig.IGEMM_OVERFLOW_BOUND
    for bad in (dict(codes=FAKE + 8), dict(scales=FAKE + 4), dict(x=FAKE + 1), dict(index=FAKE + 2)):
        assert call(**bad) == pig.IGEMM_MISALIGNED, bad
    if nv:
        assert call(g=FAKE + 2) == pig.IGEMM_MISALIGNED


@pytest.mark.parametrize("name", ["igemm_mxfp4", "igemm_nvfp4", "igemm_mxfp4_grouped", "igemm_nvfp4_grouped"])
def test_gemm_refusals(lib, name):
    fn, grouped, nv = getattr(lib, name), name.endswith("grouped"), "nv" in name

    def call(A=FAKE, B=FAKE, SFA=FAKE, SFB=FAKE, offsets=FAKE, alpha=None, C=FAKE, typ=0, M=8, E=4, N=8, K=64):
        args = [A, B, SFA, SFB] + ([offsets] if grouped else []) + ([alpha] if nv else []) + [C, typ, M]
        return fn(*args, *([E] if grouped else []), N, K, None)

    assert call(M=0, A=None, C=None) == pig.IGEMM_OK and call(N=0, B=None, C=None) == pig.IGEMM_OK
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(typ=3), dict(C=None), dict(A=None), dict(B=None),
                dict(SFA=None), dict(SFB=None)):
        assert call(**bad) == pig.IGEMM_INVALID_ARGUMENT, bad
    assert call(K=(1 << 22) + 1) == pig.IGEMM_OVERFLOW_BOUND
    for bad in (dict(A=FAKE + 8), dict(B=FAKE + 1), dict(SFA=FAKE + 4), dict(SFB=FAKE + 2), dict(C=FAKE + 2),
                dict(C=FAKE + 1, typ=1)):
        assert call(**bad) == pig.IGEMM_MISALIGNED, bad
    if grouped:
        assert call(E=-1) == pig.IGEMM_INVALID_ARGUMENT and call(offsets=None) == pig.IGEMM_INVALID_ARGUMENT
        assert call(E=0) == pig.IGEMM_OK
        assert call(E=1025) == pig.IGEMM_UNSUPPORTED_SHAPE and call(K=0) == pig.IGEMM_UNSUPPORTED_SHAPE
        assert call(E=1024, N=1 << 21) == pig.IGEMM_UNSUPPORTED_SHAPE
        assert call(offsets=FAKE + 2) == pig.IGEMM_MISALIGNED
    if nv:
        assert call(alpha=FAKE + 2) == pig.IGEMM_MISALIGNED
    assert call(M=(1 << 31) - 1, N=(1 << 31) - 600) == pig.IGEMM_UNSUPPORTED_SHAPE


def test_route_and_combine_refusals(lib):
    def route(logits=FAKE, typ=0, experts=FAKE, weights=FAKE, offsets=FAKE, tokens=FAKE, slots=FAKE, T=4, E=8, k=2):
        return lib.igemm_moe_route(logits, typ, experts, weights, offsets, tokens, slots, T, E, k, 1, None)

    for bad in (dict(T=-1), dict(E=-1), dict(k=-1), dict(typ=3), dict(offsets=None), dict(logits=None),
                dict(experts=None), dict(weights=None), dict(tokens=None), dict(slots=None)):
        assert route(**bad) == pig.IGEMM_INVALID_ARGUMENT, bad
    for bad in (dict(E=1025), dict(k=33, E=64), dict(k=9), dict(T=1 << 30, k=4)):
        assert route(**bad) == pig.IGEMM_UNSUPPORTED_SHAPE, bad
    for bad in (dict(logits=FAKE + 2), dict(logits=FAKE + 1, typ=1), dict(experts=FAKE + 1), dict(offsets=FAKE + 2)):
        assert route(**bad) == pig.IGEMM_MISALIGNED, bad

    def combine(Y=FAKE, slots=FAKE, weights=FAKE, out=FAKE, typ=1, T=4, k=2, N=8):
        return lib.igemm_moe_combine(Y, slots, weights, out, typ, T, k, N, None)

    assert combine(T=0, out=None) == pig.IGEMM_OK and combine(N=0, out=None) == pig.IGEMM_OK
    for bad in (dict(T=-1), dict(k=-1), dict(N=-1), dict(typ=4), dict(Y=None), dict(slots=None), dict(weights=None),
                dict(out=None)):
        assert combine(**bad) == pig.IGEMM_INVALID_ARGUMENT, bad
    assert combine(k=33) == pig.IGEMM_UNSUPPORTED_SHAPE
    assert combine(out=FAKE + 1) == pig.IGEMM_MISALIGNED and combine(Y=FAKE + 2, typ=0) == pig.IGEMM_MISALIGNED


def test_binding_checks_tensors(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 64))
    u8 = torch.zeros((4, 64), dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        pig.pack_mxfp4(x, u8, u8, 4, 64, stream=0)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        pig.pack_mxfp4(x.double(), u8, u8, 4, 64, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        pig.igemm_mxfp4(u8, u8, u8, u8, x, 4, 4, 64, stream=0)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        pig.igemm_nvfp4(u8, u8, u8, u8, None, u8, 4, 4, 64, stream=0)
    with pytest.raises(ValueError, match="int32"):
        pig.igemm_moe_route(FakeLogits(torch), FAKE, FAKE, torch.zeros(9, dtype=torch.int64), FAKE, FAKE, 4, 8, 2,
                            stream=0)
    with pytest.raises(ValueError, match="Y's type"):
        pig.igemm_moe_combine(x, FAKE, FAKE, x.half(), 2, 2, 64, stream=0)
    with pytest.raises(pig.IgemmError) as e:
        pig.igemm_mxfp4_grouped(FAKE, FAKE, FAKE, FAKE, FAKE, FakeLogits(torch), 4, 1025, 4, 64, stream=0)
    assert e.value.code == pig.IGEMM_UNSUPPORTED_SHAPE


class FakeLogits:
    """A float32 tensor as far as the binding looks, on no device."""

    def __init__(self, torch):
        self.dtype, self.is_cuda, self.nbytes = torch.float32, True, 1 << 40

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


def test_plan_without_the_clusters_that_do_not_fit(tmp_path):
    import os
    import shutil
    import subprocess

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    csrc, cuda = os.path.join(root, "precision_integer_gemm_gb300", "csrc"), "/usr/local/cuda/include"
    if not shutil.which("g++") or not os.path.isdir(cuda):
        pytest.skip("g++ or the CUDA headers are missing")
    exe = str(tmp_path / "fp4_plan_check")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", csrc, "-I", cuda, "-x", "c++",
                        os.path.join(root, "tests", "c", "fp4_plan_check.cpp"), os.path.join(csrc, "fp4_plan.cu"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout[:2000]
    assert r.stdout.startswith("fp4 plan ok")
