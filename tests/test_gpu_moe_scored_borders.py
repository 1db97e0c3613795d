"""The scored routing where float32 cannot tell: equal choices at the border of the k-th with a better one behind them,
group scores whose parts cancel, biases at the ends of float32's range; its launches for long prompts; its
gradient on rows without scores.  The choice is compared exactly with that of the scores in 64 bits.
"""

import math

import pytest

torch = pytest.importorskip("torch")

import precision_integer_gemm_gb300 as pig  # noqa: E402
from test_gpu_moe_scored import check, grad, plain_choice, route, scores_of  # noqa: E402

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


def cancelling(T, E, groups, size, seed, step):
    """Logits and a bias of +-size whose two largest of a group cancel: one expert of a group at +size, the others at
    -size, the groups' logits `step` apart."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = E // groups
    one = torch.randn((T, 1, per), generator=g, device="cuda")
    logits = one + step * torch.randn((T, groups, per), generator=g, device="cuda")
    sign = torch.full((groups, per), -1.0, device="cuda")
    sign[torch.arange(groups), torch.randint(0, per, (groups,), generator=g, device="cuda").cpu()] = 1.0
    return logits.view(T, E).contiguous(), (size * sign).view(E).contiguous()


def decided(logits, bias, score, groups, group_k, group_top):
    """Tokens whose border between groups taken and left 64 bits can tell.  A score's relative error is at most (E + 8)
    2^-53 (an exponential, a sum over the experts in some order, a quotient), that of c = s + bias 2^-53 of |c|, that of
    a group's sum 2^-53 of it; two groups of equal experts with the signs of the biases swapped are equal by the formula
    and differ by such errors alone (token 2361 of 3000 x 64, softmax, size 0.5: 0 apart in 128 bits)."""
    T, E = logits.shape
    s = scores_of(logits.double(), score)[0]
    v = torch.sort((s + bias.double()).view(T, groups, -1), dim=-1, descending=True)[0][..., :group_top]
    slip = 2.0 ** -53 * ((E + 8) * group_top * s.amax(-1, keepdim=True) + v.abs().sum(-1) + v.sum(-1).abs())
    best, at = torch.sort(v.sum(-1), dim=-1, descending=True, stable=True)
    slip = slip.gather(1, at)
    low = (best - slip)[:, :group_k].amin(-1)
    return low > (best + slip)[:, group_k:].amax(-1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [0.5, 4.0, 16.0, 64.0, 100.0, 1000.0])
@pytest.mark.parametrize("T,E,k,groups,group_k", [(3000, 256, 8, 8, 4), (3000, 64, 4, 32, 5), (1000, 160, 6, 20, 7),
                                                  (500, 96, 3, 2, 1), (600, 1024, 8, 16, 3)])
def test_group_scores_of_parts_that_cancel(T, E, k, groups, group_k, size, score):
    # c is rounded at the size of the bias, the sum of the two is as small as the scores
    for step in (1e-6, 1e-5, 1e-4):
        logits, bias = cancelling(T, E, groups, size, E + groups, step)
        for group_top in (1, 2):
            sure = decided(logits, bias, score, groups, group_k, group_top)
            # (32 groups 1e-6 apart, float32 logits 2^-23 apart: one border in seven is between equal groups)
            assert sure.float().mean().item() > 0.5
            check(logits[sure], bias, k, score, groups, group_k, group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("low", [torch.finfo(torch.float32).min, -1e38, -3e38])
def test_groups_switched_off_by_the_lowest_bias(low, group_top, score):
    # only -inf and NaN are never chosen: with more groups to take than are left, those of the lowest finite bias follow
    g = torch.Generator(device="cuda").manual_seed(11)
    for T, E, k, groups, group_k, on in ((200, 64, 32, 8, 5, 3), (50, 256, 8, 8, 4, 2), (40, 256, 32, 32, 8, 1),
                                         (30, 60, 12, 20, 4, 0)):
        logits = torch.randn((T, E), generator=g, device="cuda")
        bias = 0.1 * torch.randn((E,), generator=g, device="cuda")
        bias.view(groups, -1)[on:] = low
        check(logits, bias, k, score, groups, group_k, group_top)
        bias.view(groups, -1)[on:, 1:] = 0.0  # one expert of a group off
        check(logits, bias, k, score, groups, group_k, group_top)
        bias.view(groups, -1)[-1] = -math.inf
        check(logits, bias, k, score, groups, group_k, group_top)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
def test_groups_of_the_largest_bias(group_top, score):
    g = torch.Generator(device="cuda").manual_seed(12)
    T, E, k, groups = 100, 64, 8, 8
    logits = torch.randn((T, E), generator=g, device="cuda")
    for high in (torch.finfo(torch.float32).max, math.inf, 2e38):
        bias = 0.1 * torch.randn((E,), generator=g, device="cuda")
        bias[8:16] = bias[40:48] = high
        bias[56] = high
        for group_k in (1, 2, 4):
            check(logits, bias, k, score, groups, group_k, group_top)


@pytest.mark.parametrize("T,E,launches", [(4864, 256, 3), (4865, 256, 3), (16384, 256, 3), (19456, 256, 3), (20000, 256, 3),
                                          (1025, 1024, 3), (9000, 64, 3), (9000, 16, 2)])
@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16])
def test_long_prompts(T, E, launches, typ):
    # blocks of more than 16 tokens and of more than 32 (a mask's second word), more than one wave of them, the scan
    g = torch.Generator(device="cuda").manual_seed(T)
    logits = torch.randn((T, E), generator=g, device="cuda")
    logits[torch.rand((T, E), generator=g, device="cuda") < 0.1] = -math.inf
    logits[T - T // 20:] = -math.inf
    logits = logits.to(typ)
    bias = 0.1 * torch.randn((E,), generator=g, device="cuda")
    before = pig.igemm_kernels_launched()
    route(logits, bias, 4, "sigmoid", 8, 4, 2)
    assert pig.igemm_kernels_launched() - before == launches
    check(logits, bias, 4, "sigmoid", 8, 4, 2, scale=2.5)
    check(logits, None, 4, "softmax", 8, 3, 1, normalize=False)


@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_of_a_named_expert_without_scores(normalize, typ):
    # a softmax row with +inf has no scores, also where its experts are named; a sigmoid of +inf is 1 and flat
    T, E, k = 6, 40, 3
    g = torch.Generator(device="cuda").manual_seed(2)
    logits = torch.randn((T, E), generator=g, device="cuda").to(typ)
    experts = torch.tensor([[3, 1, 2]] * T, device="cuda")
    dw = torch.randn((T, k), generator=g, device="cuda")
    logits[0, 3] = math.inf
    logits[1, 2] = math.inf
    logits[2, 1:4] = math.inf
    rest = grad(logits, experts, dw, "softmax", normalize, 1.0)
    assert bool(torch.isfinite(rest).all()) and bool((rest[:3] == 0).all()) and bool((rest[3:] != 0).any(-1).all())
    alone = grad(logits[3:].contiguous(), experts[3:].contiguous(), dw[3:].contiguous(), "softmax", normalize, 1.0)
    assert torch.equal(alone, rest[3:])
    flat = grad(logits, experts, dw, "sigmoid", normalize, 1.0)
    assert bool(torch.isfinite(flat).all()) and flat[0, 3] == 0 and flat[1, 2] == 0 and bool((flat[2, 1:4] == 0).all())


@pytest.mark.parametrize("typ", [torch.float32, torch.bfloat16])
def test_sigmoids_below_the_smallest_normal_number(typ):
    # e^-88.8 .. e^-103: float32 holds them to fewer and fewer bits, the weights and the gradients that are made of them
    # to half of its smallest step, 2^-150, and the rounding of a product or two
    T, E, k = 40, 64, 8
    logits = torch.linspace(-104.0, -86.0, T * E, device="cuda").view(T, E).to(typ).contiguous()
    got = route(logits, None, k, "sigmoid", normalize=False, scale=1.0)
    want = torch.sigmoid(logits.double().gather(1, got["experts"].long()))
    tol = 250 * 2.0 ** -24 * want + 2.0 ** -149  # (spread 104: as in test_gpu_moe_scored)
    assert bool(((got["weights"].double() - want).abs() <= tol).all()) and bool((got["weights"][:-1] > 0).any())
    # above: s (1 - s) of logits whose 1 - s is as small
    dw = torch.ones((T, k), device="cuda")
    for x in (logits, -logits):
        d = grad(x.contiguous(), got["experts"].long(), dw, "sigmoid", False, 1.0).gather(1, got["experts"].long())
        s = torch.sigmoid(-x.double().abs()).gather(1, got["experts"].long())
        rounded = torch.finfo(typ).eps / 2 * s + (2.0 ** -134 if typ == torch.bfloat16 else 0.0)  # (half bfloat16's smallest)
        assert bool(((d.double() - s * (1 - s)).abs() <= 250 * 2.0 ** -24 * s + 2.0 ** -148 + rounded).all())
