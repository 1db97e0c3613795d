"""Host-side checks of the block-scaled fp8 entry points: argument errors come back before anything is launched, so no
GPU is needed.  (No call here passes FAKE with valid arguments.)"""

import os
import re

import pytest

import precision_integer_gemm_gb300 as pig

FAKE = 0x10000  # a 16-byte-aligned address that the rejected calls never touch
CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "precision_integer_gemm_gb300", "csrc")


@pytest.fixture(scope="module")
def lib():
    pig.build_library()
    return pig.load()


def test_sizes_of_rows():
    for K, code, scales in [(1, 16, 4), (16, 16, 4), (17, 32, 4), (128, 128, 4), (512, 512, 4), (513, 528, 8),
                            (4160, 4160, 36), (8192, 8192, 64)]:
        assert (pig.bsfp8_code_bytes(K), pig.bsfp8_scale_pitch(K)) == (code, scales)


def test_pack_refusals(lib):
    def call(x=FAKE, typ=1, ld=64, transposed=0, index=None, x_rows=8, tile=1, fmt=0, codes=FAKE, scales=FAKE, rows=8,
             K=64):
        return lib.pack_bsfp8(x, typ, ld, transposed, index, x_rows, tile, fmt, codes, scales, rows, K, None)

    assert call(rows=0, x=None) == pig.IGEMM_OK and call(K=0, x=None) == pig.IGEMM_OK
    for bad in (dict(rows=-1), dict(K=-1), dict(x_rows=-1), dict(ld=-1), dict(typ=3), dict(typ=-1), dict(fmt=2),
                dict(fmt=-1), dict(codes=None), dict(scales=None), dict(x=None), dict(x_rows=7), dict(ld=63),
                dict(transposed=1, ld=7)):
        assert call(**bad) == pig.IGEMM_INVALID_ARGUMENT, bad
    for bad in (dict(tile=0), dict(tile=64), dict(transposed=1, index=FAKE), dict(tile=128, index=FAKE)):
        assert call(**bad) == pig.IGEMM_UNSUPPORTED_SHAPE, bad
    assert call(K=(1 << 22) + 1, ld=1 << 23) == pig.IGEMM_OVERFLOW_BOUND
    for bad in (dict(codes=FAKE + 8), dict(scales=FAKE + 4), dict(x=FAKE + 1), dict(index=FAKE + 2)):
        assert call(**bad) == pig.IGEMM_MISALIGNED, bad


@pytest.mark.parametrize("grouped", [False, True])
def test_product_refusals(lib, grouped):
    def call(A=FAKE, B=FAKE, SFA=FAKE, SFB=FAKE, offsets=FAKE, C=FAKE, typ=0, fmt=0, M=8, E=4, N=8, K=64):
        if grouped:
            return lib.igemm_bsfp8_grouped(A, B, SFA, SFB, offsets, C, typ, fmt, M, E, N, K, None)
        return lib.igemm_bsfp8(A, B, SFA, SFB, C, typ, fmt, M, N, K, None)

    assert call(M=0, A=None, C=None) == pig.IGEMM_OK and call(N=0, B=None, C=None) == pig.IGEMM_OK
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(typ=3), dict(fmt=2), dict(C=None), dict(A=None), dict(B=None),
                dict(SFA=None), dict(SFB=None)):
        assert call(**bad) == pig.IGEMM_INVALID_ARGUMENT, bad
    assert call(K=(1 << 22) + 1) == pig.IGEMM_OVERFLOW_BOUND
    for bad in (dict(A=FAKE + 8), dict(B=FAKE + 1), dict(SFA=FAKE + 4), dict(SFB=FAKE + 8), dict(C=FAKE + 2),
                dict(C=FAKE + 1, typ=1)):
        assert call(**bad) == pig.IGEMM_MISALIGNED, bad
    assert call(M=(1 << 31) - 1, N=(1 << 31) - 600) == pig.IGEMM_UNSUPPORTED_SHAPE
    if grouped:
        assert call(E=-1) == pig.IGEMM_INVALID_ARGUMENT and call(offsets=None) == pig.IGEMM_INVALID_ARGUMENT
        assert call(E=0) == pig.IGEMM_OK
        assert call(E=1025) == pig.IGEMM_UNSUPPORTED_SHAPE and call(K=0) == pig.IGEMM_UNSUPPORTED_SHAPE
        assert call(E=1024, N=1 << 21) == pig.IGEMM_UNSUPPORTED_SHAPE
        assert call(offsets=FAKE + 2) == pig.IGEMM_MISALIGNED


def test_binding_checks_tensors(lib):
    torch = pytest.importorskip("torch")
    x, u8, s = torch.zeros((4, 64)), torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 4))
    with pytest.raises(ValueError, match="CUDA"):
        pig.pack_bsfp8(x, u8, s, 4, 64, stream=0)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        pig.pack_bsfp8(x.double(), u8, s, 4, 64, stream=0)
    with pytest.raises(ValueError, match="format"):
        pig.igemm_bsfp8(FAKE, FAKE, FAKE, FAKE, Fake(torch), 4, 4, 64, format="e4m3fn", stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        pig.igemm_bsfp8(u8, u8, s, s, x, 4, 4, 64, stream=0)
    with pytest.raises(ValueError, match="SFA must be torch.float32"):
        pig.igemm_bsfp8(FAKE, FAKE, s.half(), FAKE, Fake(torch), 4, 4, 64, stream=0)
    with pytest.raises(ValueError, match="int32"):
        pig.igemm_bsfp8_grouped(FAKE, FAKE, FAKE, FAKE, torch.zeros(5, dtype=torch.int64), Fake(torch), 4, 4, 4, 64,
                                stream=0)
    with pytest.raises(pig.IgemmError) as e:
        pig.igemm_bsfp8_grouped(FAKE, FAKE, FAKE, FAKE, FAKE, Fake(torch), 4, 1025, 4, 64, stream=0)
    assert e.value.code == pig.IGEMM_UNSUPPORTED_SHAPE


class Fake:
    """A float32 tensor as far as the binding looks, on no device."""

    def __init__(self, torch):
        self.dtype, self.is_cuda, self.nbytes = torch.float32, True, 1 << 40

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


def code_of(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["pack_bsfp8.cu", "pack_values.cuh", "gemm_bsfp8_kernel.cuh"])
def test_kernels_set_up_early_make_no_read_only_loads(name):
    # such a load promises memory that nobody writes during the kernel's life, which begins while the kernel before runs
    code = code_of(name)
    for word in ("__ldg", "__ldcg", "__ldcs", "__restrict__", "ld.global.nc"):
        assert word not in code, word


def test_hand_overs_between_the_ctas_of_a_product():
    # what threads wrote or read goes to another CTA with a release at cluster scope, never by mbar_arrive_peer
    code = code_of("gemm_bsfp8_kernel.cuh")
    targets = re.findall(r"mbar_arrive_peer\(([^;]*)\);", code)
    assert targets and all(t.startswith("empty_leader") for t in targets), targets  # (tensor memory that was read)
    assert re.search(r"bulk_copy_to_cta\([^;]*smem_u32\(&red_empty", code)
    waits = re.findall(r"(\w+)\(&red_(?:empty|full)\[warp\], ph", code)
    assert len(waits) == 2 and set(waits) == {"fp4_warp_wait_cluster"}


def test_register_shares_of_the_pair_kernel():
    # setmaxnreg deals out what the block was launched with, no more: a larger sum would wait for ever
    code = code_of("gemm_bsfp8_kernel.cuh")
    inc, dec = re.findall(r"bsfp8_regs_inc<(\d+)>\(\)", code), re.findall(r"bsfp8_regs_dec<(\d+)>\(\)", code)
    assert len(inc) == 1 and len(dec) == 1
    launched = re.search(r"attr\.numRegs != (\d+)\) return 0", code_of("gemm_bsfp8.cu"))
    assert 256 * int(inc[0]) + 128 * int(dec[0]) <= 384 * int(launched.group(1))


def test_both_issuing_warps_see_every_use_of_a_slot_of_codes():
    # a wait by parity that skips uses of a slot may be passed by an earlier one
    code = code_of("gemm_bsfp8_kernel.cuh")
    assert re.search(r"mbar_init\(&empty\[lane\], 2\);", code)
    skipped = re.search(r"if \(!mine\) \{(.*?)__syncwarp\(\);", code, flags=re.S).group(1)
    assert "fp4_warp_wait(&full[cr.slot], cr.phase, wd)" in skipped
    assert "mma_commit_pair_multicast(&empty[cr.slot], 0x3)" in skipped and "mbar_arrive(&empty[cr.slot])" in skipped


def test_plan_without_the_clusters_that_do_not_fit(tmp_path):
    import shutil
    import subprocess

    root, cuda = os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "/usr/local/cuda/include"
    if not shutil.which("g++") or not os.path.isdir(cuda):
        pytest.skip("g++ or the CUDA headers are missing")
    exe = str(tmp_path / "bsfp8_plan_check")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, "-I", cuda, "-x", "c++",
                        os.path.join(root, "tests", "c", "bsfp8_plan_check.cpp"), os.path.join(CSRC, "bsfp8_plan.cu"),
                        "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout[:2000]
    assert r.stdout.startswith("bsfp8 plan ok")
