"""Host-side checks of routing by scores: argument errors come back before anything is launched, so no GPU is needed.
(No call here passes FAKE with valid arguments.)"""

import os
import re

import pytest

import precision_integer_gemm_gb300 as pig

FAKE = 0x10000  # a 16-byte-aligned address that the rejected calls never touch


@pytest.fixture(scope="module")
def lib():
    pig.build_library()
    return pig.load()


def test_route_refusals(lib):
    def call(logits=FAKE, typ=0, bias=None, experts=FAKE, weights=FAKE, offsets=FAKE, tokens=FAKE, slots=FAKE, T=4, E=8,
             k=2, score=1, groups=4, group_k=2, top=2):
        return lib.igemm_moe_route_scored(logits, typ, bias, experts, weights, offsets, tokens, slots, T, E, k, score,
                                          groups, group_k, top, 1, 1.0, None)

    for bad in (dict(T=-1), dict(E=-1), dict(k=-1), dict(typ=3), dict(score=2), dict(score=-1), dict(offsets=None),
                dict(logits=None), dict(experts=None), dict(weights=None), dict(tokens=None), dict(slots=None)):
        assert call(**bad) == pig.IGEMM_INVALID_ARGUMENT, bad
    for bad in (dict(E=1028), dict(k=33, E=64, group_k=4), dict(k=9), dict(T=1 << 30, k=4), dict(groups=0),
                dict(groups=3), dict(groups=33, E=66), dict(group_k=0), dict(group_k=5), dict(top=0), dict(top=3),
                dict(k=5), dict(E=0, k=0, groups=0)):
        assert call(**bad) == pig.IGEMM_UNSUPPORTED_SHAPE, bad
    for bad in (dict(logits=FAKE + 2), dict(logits=FAKE + 1, typ=1), dict(bias=FAKE + 2), dict(experts=FAKE + 1),
                dict(offsets=FAKE + 2)):
        assert call(**bad) == pig.IGEMM_MISALIGNED, bad


def test_gradient_refusals(lib):
    def call(logits=FAKE, typ=0, experts=FAKE, dw=FAKE, out=FAKE, T=4, E=8, k=2, score=1):
        return lib.igemm_moe_route_scored_grad(logits, typ, experts, dw, out, T, E, k, score, 1, 1.0, None)

    assert call(T=0, out=None) == pig.IGEMM_OK and call(E=0, out=None) == pig.IGEMM_OK
    for bad in (dict(T=-1), dict(E=-1), dict(k=-1), dict(typ=3), dict(score=2), dict(logits=None), dict(experts=None),
                dict(dw=None), dict(out=None)):
        assert call(**bad) == pig.IGEMM_INVALID_ARGUMENT, bad
    for bad in (dict(E=1025), dict(k=33), dict(T=1 << 30, k=4)):
        assert call(**bad) == pig.IGEMM_UNSUPPORTED_SHAPE, bad
    for bad in (dict(logits=FAKE + 2), dict(out=FAKE + 1, typ=1), dict(experts=FAKE + 2), dict(dw=FAKE + 1)):
        assert call(**bad) == pig.IGEMM_MISALIGNED, bad


def test_binding_checks_tensors(lib):
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 8))
    with pytest.raises(ValueError, match="score"):
        pig.igemm_moe_route_scored(Fake(torch), None, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 8, 2, score="relu", stream=0)
    with pytest.raises(ValueError, match="bias must be torch.float32"):
        pig.igemm_moe_route_scored(Fake(torch), x[0].half(), FAKE, FAKE, FAKE, FAKE, FAKE, 4, 8, 2, stream=0)
    with pytest.raises(ValueError, match="CUDA"):
        pig.igemm_moe_route_scored(x, None, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 8, 2, stream=0)
    with pytest.raises(ValueError, match="logits' type"):
        pig.igemm_moe_route_scored_grad(x, FAKE, FAKE, x.half(), 4, 8, 2, stream=0)
    with pytest.raises(pig.IgemmError) as e:
        pig.igemm_moe_route_scored(Fake(torch), None, FAKE, FAKE, FAKE, FAKE, FAKE, 4, 8, 2, groups=3, stream=0)
    assert e.value.code == pig.IGEMM_UNSUPPORTED_SHAPE


class Fake:
    """A float32 tensor as far as the binding looks, on no device."""

    def __init__(self, torch):
        self.dtype, self.is_cuda, self.nbytes = torch.float32, True, 1 << 40

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return FAKE


@pytest.mark.parametrize("name", ["moe_scored.cu", "moe_route.cuh"])
def test_kernels_set_up_early_make_no_read_only_loads(name):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "precision_integer_gemm_gb300", "csrc", name)) as f:
        code = re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)
    for word in ("__ldg", "__ldcg", "__ldcs", "__restrict__", "ld.global.nc"):
        assert word not in code, word
