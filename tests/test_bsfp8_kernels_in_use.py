"""Which kernels the block-scaled fp8 products run on: the CTA pairs leave without an error where the compiler gave them
another number of registers than their shares were dealt from, so that their use is checked here."""

import os
import shutil
import subprocess

import pytest

import precision_integer_gemm_gb300 as pig

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "precision_integer_gemm_gb300", "csrc")


def test_answers_are_kept(tmp_path):
    cuda = "/usr/local/cuda/include"
    if not shutil.which("g++") or not os.path.isdir(cuda):
        pytest.skip("g++ or the CUDA headers are missing")
    exe = str(tmp_path / "ask_once")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, "-I", cuda, "-x", "c++",
                        os.path.join(ROOT, "tests", "c", "bsfp8_ask_once_check.cpp"), "-o", exe, "-pthread"],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
    assert r.stdout.startswith("ask once ok")


def test_weights_that_leave_l2_first(tmp_path):
    cuda = "/usr/local/cuda/include"
    if not shutil.which("g++") or not os.path.isdir(cuda):
        pytest.skip("g++ or the CUDA headers are missing")
    exe = str(tmp_path / "stream")
    r = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", CSRC, "-I", cuda, "-x", "c++",
                        os.path.join(ROOT, "tests", "c", "bsfp8_stream_check.cpp"), os.path.join(CSRC, "bsfp8_plan.cu"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
    assert r.stdout.startswith("bsfp8 stream ok")


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K,grouped,kernel", [(4096, 4096, 1024, False, "<256, true>"), (2048, 4096, 512, True, "<256, true>"),
                                                  (16, 512, 1024, False, "<16, false>")])
def test_kernel_of_a_product(M, N, K, grouped, kernel):
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from torch.profiler import ProfilerActivity, profile

    E = 2 if grouped else 1
    A, B = torch.zeros((M, K), dtype=torch.uint8, device="cuda"), torch.zeros((E, N, K), dtype=torch.uint8, device="cuda")
    SFA, SFB = torch.ones((M, pig.bsfp8_scale_pitch(K)), device="cuda"), torch.ones((E, N // 128, pig.bsfp8_scale_pitch(K)), device="cuda")
    offsets = torch.tensor([0, M // 2, M], dtype=torch.int32, device="cuda")
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")

    def run():
        if grouped:
            pig.igemm_bsfp8_grouped(A, B, SFA, SFB, offsets, C, M, E, N, K)
        else:
            pig.igemm_bsfp8(A, B, SFA, SFB, C, M, N, K)

    names = []
    for _ in range(3):  # (the first recording of a process may be empty)
        with profile(activities=[ProfilerActivity.CUDA]) as p:
            run()
            torch.cuda.synchronize()
        names = [e.name for e in p.events() if "igemm_bsfp8_kernel" in e.name]
        if names:
            break
    if not names:
        pytest.skip("kernels are not recorded here")
    assert names and all(kernel in n for n in names), names
    assert pig.igemm_last_status() == pig.IGEMM_OK
