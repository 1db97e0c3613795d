"""The scored routing where float32 cannot tell: equal choices at the border of the k-th with a better one behind them.
The choice is compared exactly with that of the scores in 64 bits.
"""

import pytest

torch = pytest.importorskip("torch")

import precision_integer_gemm_gb300 as pig  # noqa: E402
from test_gpu_moe_scored import check, plain_choice  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pig.build_library()
    yield pig.load()
    assert pig.igemm_last_status() == pig.IGEMM_OK


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("k", [1, 2, 8, 16, 17, 31, 32])
@pytest.mark.parametrize("equal,better", [((0, 1), 2), ((0, 1), 63), ((4, 5), 6), ((3, 40), 41), ((10, 20, 30, 31), 50),
                                          ((7, 9), 8), ((50, 60), 3)])
@pytest.mark.parametrize("E", [64, 256])
def test_a_better_one_behind_equal_ones_at_the_border(E, equal, better, k, score):
    # k - 1 sure choices, then experts of equal logit and bias on the places k - 1, k, ..., and one whose score is larger
    # by far less than the float32 sum with its bias of 1000 can hold
    logits = torch.full((3, E), -3.0, device="cuda")
    bias = torch.zeros((E,), device="cuda")
    at = list(equal) + [better]
    sure = [e for e in range(E) if e not in at][: k - 1]
    bias[sure] = 2000.0 + 8 * torch.arange(len(sure), device="cuda").float()
    bias[at] = 1000.0
    logits[:, at] = 0.0
    logits[0, better], logits[1, better], logits[2, better] = 1e-5, 1e-7, -1e-5
    check(logits, bias, k, score)
    # (the inputs are what they are said to be)
    chosen = plain_choice(logits, bias, k, score, 1, 1, 1)
    assert better in chosen[0].tolist() and better in chosen[1].tolist() and better not in chosen[2].tolist()


def test_a_better_one_behind_equal_ones_with_ordinary_biases():
    E = 64
    logits = torch.full((1, E), -3.0, device="cuda")
    bias = torch.zeros((E,), device="cuda")
    logits[0, 0] = logits[0, 1] = 0.12573022
    bias[0] = bias[1] = 0.497
    logits[0, 2], bias[2] = 0.061584298, 0.513
    check(logits, bias, 1, "sigmoid")
    # the same three among bfloat16 logits and stepped biases, many times over
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randn((4000, 256), generator=g, device="cuda").to(torch.bfloat16)
    logits[:, 1::2] = logits[:, ::2]
    bias = (torch.randint(-8, 9, (128,), generator=g, device="cuda") / 1024).repeat_interleave(2).float()
    for k in (1, 3, 8, 17):
        check(logits, bias, k, "sigmoid")
        check(logits, bias, k, "softmax")
