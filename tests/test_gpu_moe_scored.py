"""Routing by scores and its gradient on the GPU against plain forms in 64 bits.

Tolerances.  The choice is that of the scores in 64 bits and compared exactly.  A weight is a few float32 exponentials
(2 ulp each; the argument x - m is rounded, |x - m| 2^-24 of the result), a sum over at most E of them (E / 32 + 6
roundings), a quotient and a product: relative (2 |x - m| + E / 32 + 24) 2^-24 with the spread of the logits for |x -
m|.  A gradient is a product of such weights with g - mean, whose sum of k terms has k + 2 more roundings, relative to
scale u (|g| + sum |g u|).
"""

import math

import pytest

torch = pytest.importorskip("torch")

import precision_integer_gemm_gb300 as pig  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pig.build_library()
    yield pig.load()
    assert pig.igemm_last_status() == pig.IGEMM_OK


def scores_of(x, score):
    """float64 scores; a softmax row with +inf has none (zeros)."""
    x = torch.where(torch.isnan(x), -math.inf, x)
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x)), x > -math.inf
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
    there = (x > -math.inf) & (m < math.inf)
    return torch.where(m < math.inf, e / e.sum(-1, keepdim=True).clamp(min=1e-300), 0.0), there


def plain_choice(logits, bias, k, score, groups, group_k, group_top):
    x = logits.double()
    s, there = scores_of(x, score)
    c = x if bias is None else s + bias.double()
    there = there & (c > -math.inf)
    c = torch.where(there, c, -math.inf)
    T, E = x.shape
    if groups > 1:
        v = torch.where(there, s if bias is None and group_top == 2 else c, -math.inf).view(T, groups, -1)
        v = torch.sort(v, dim=-1, descending=True)[0][..., :group_top]
        g = torch.where(v > -math.inf, v, 0.0).sum(-1)
        g = torch.where(v[..., 0] > -math.inf, g, -math.inf)
        best = torch.sort(g, dim=-1, descending=True, stable=True)[1][:, :group_k]
        keep = torch.zeros((T, groups), dtype=torch.bool, device=x.device).scatter_(1, best, True)
        c = torch.where(keep.repeat_interleave(E // groups, 1), c, -math.inf)
    v, ids = torch.sort(c, dim=-1, descending=True, stable=True)
    return torch.where(v[:, :k] > -math.inf, ids[:, :k], -1)


def plain_weights(x, experts, score, normalize, scale):
    """Weights of the chosen, differentiable in x (float64)."""
    there = experts >= 0
    at = experts.clamp(min=0).long()
    if normalize:
        top = torch.where(there, x.gather(1, at), -math.inf)
        if score == "sigmoid":
            # log sigmoid, so that small scores do not underflow
            top = torch.where(there, torch.nn.functional.logsigmoid(torch.where(there, top, 0.0)), -math.inf)
        some = there.any(-1, keepdim=True)
        w = torch.softmax(torch.where(some, top, 0.0), -1)
    elif score == "sigmoid":
        w = torch.sigmoid(x.gather(1, at))
    else:
        w = torch.softmax(x, -1).gather(1, at)
    return scale * torch.where(there, w, 0.0)


def route(logits, bias, k, score, groups=1, group_k=1, group_top=1, normalize=True, scale=1.0):
    T, E = logits.shape
    out = {"experts": torch.full((T, k), 99999, dtype=torch.int32, device="cuda"), "weights": torch.full((T, k), -7.0, device="cuda"),
           "offsets": torch.full((E + 1,), -9, dtype=torch.int32, device="cuda"),
           "tokens": torch.full((T * k,), -9, dtype=torch.int32, device="cuda"),
           "slots": torch.full((T, k), -9, dtype=torch.int32, device="cuda")}
    pig.igemm_moe_route_scored(logits, bias, *out.values(), T, E, k, score=score, groups=groups, group_k=group_k,
                               group_top=group_top, normalize=normalize, scale=scale)
    return out


def check(logits, bias, k, score, groups=1, group_k=1, group_top=1, normalize=True, scale=1.0):
    T, E = logits.shape
    got = route(logits, bias, k, score, groups, group_k, group_top, normalize, scale)
    experts = plain_choice(logits, bias, k, score, groups, group_k, group_top)
    assert torch.equal(got["experts"].long(), experts)
    x = torch.where(torch.isnan(logits), -math.inf, logits.float()).double()
    w = plain_weights(x, experts, score, normalize, scale)
    finite = x[torch.isfinite(x)]
    spread = (finite.max() - finite.min()).item() if finite.numel() else 0.0
    tol = (2 * min(spread, 120.0) + E / 32 + 24) * 2.0 ** -24
    assert bool(((got["weights"].double() - w).abs() <= tol * w.abs() + 1e-44).all())
    # the sorted pairs
    key, order = torch.sort(torch.where(experts >= 0, experts, E).view(-1), stable=True)
    assert torch.equal(got["offsets"].long(), torch.searchsorted(key, torch.arange(E + 1, device="cuda")))
    assert torch.equal(got["tokens"].long(), torch.where(key < E, order // k, -1))
    slots = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device="cuda")).view(T, k)
    assert torch.equal(got["slots"].long(), torch.where(experts >= 0, slots, -1))


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,group_k,group_top", [
    (1, 4, 1, 1, 1, 1), (3, 8, 8, 2, 2, 2), (17, 60, 6, 4, 2, 1), (100, 64, 6, 8, 3, 1), (513, 128, 8, 1, 1, 1),
    (700, 256, 8, 8, 4, 2), (1000, 162, 6, 9, 3, 2), (600, 512, 32, 16, 5, 2), (80, 1000, 10, 25, 4, 1),
    (2000, 96, 4, 32, 3, 2), (520, 1024, 8, 32, 32, 2), (64, 31, 5, 31, 6, 1)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route(T, E, k, groups, group_k, group_top, score, with_bias, typ):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    logits = (2 * torch.randn((T, E), generator=g, device="cuda")).to(TYPES[typ])
    bias = 0.05 * torch.randn((E,), generator=g, device="cuda") if with_bias else None
    for normalize, scale in ((True, 1.0), (False, 2.5)):
        check(logits, bias, k, score, groups, group_k, group_top, normalize, scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("group_top", [1, 2])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masks_and_special_values(score, group_top, with_bias):
    T, E, k = 300, 64, 6
    logits = 3 * torch.randn((T, E), device="cuda")
    logits[torch.rand((T, E), device="cuda") < 0.5] = -math.inf
    logits[0] = -math.inf                  # nothing to choose
    logits[1] = math.nan
    logits[2, 5:] = -math.inf              # fewer than k
    logits[3, 7] = math.inf
    logits[4] = torch.finfo(torch.float32).min
    logits[5] = -300.0                     # scores that underflow float32
    logits[6] = 0.0
    logits[7, ::2] = math.nan
    logits[8] = 60.0                       # sigmoids that round to 1
    logits[8, 40:] = 80.0
    logits[9, :8] = -math.inf              # a whole group masked
    logits[10, 1:] = -math.inf
    bias = None
    if with_bias:
        bias = 0.1 * torch.randn((E,), device="cuda")
        bias[3], bias[9], bias[17] = -math.inf, math.nan, math.inf
    for normalize in (True, False):
        check(logits, bias, k, score, 8, 3, group_top, normalize)
        check(logits, bias, k, score, 1, 1, group_top, normalize)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_and_equal_scores(score):
    # neighbours far nearer than float32 can tell once the bias is added, and many equal ones
    T, E, k = 2000, 256, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn((T, E), generator=g, device="cuda")
    logits[:, 1::2] = logits[:, ::2] * (1 + 2.0 ** -22)  # one or two steps apart
    bias = 0.01 * torch.randn((E,), generator=g, device="cuda")
    bias[1::2] = bias[::2]
    check(logits, bias, k, score)
    check(logits, bias, k, score, 8, 4, 2)
    s = scores_of(logits.double(), score)[0]
    bias = (0.5 - s[0]).float()  # every expert of token 0 within a rounding of the others
    check(logits[:1].contiguous(), bias, k, score, 8, 4, 2)
    coarse = (2 * logits).round() / 2
    for b in (torch.zeros((E,), device="cuda"), None):
        check(coarse, b, k, score, 8, 4, 2)
        check(coarse.to(torch.bfloat16), b, k, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,groups,group_k", [(200, 256, 8, 8, 4), (90, 160, 6, 20, 7), (70, 64, 4, 32, 9), (40, 1024, 8, 8, 2)])
@pytest.mark.parametrize("spread", [0.0, 4.0, 16.0, 60.0])
@pytest.mark.parametrize("typ", ["f32", "bf16"])
def test_scores_of_very_different_size(T, E, k, groups, group_k, score, spread, typ):
    # scores that float32 holds to few bits, not at all (60: e^-300), or as 1, and all equal ones
    g = torch.Generator(device="cuda").manual_seed(T)
    logits = (spread * torch.randn((T, E), generator=g, device="cuda")).to(TYPES[typ])
    for group_top in (1, 2):
        check(logits, None, k, score, groups, group_k, group_top)
        with_zeros = route(logits, torch.zeros((E,), device="cuda"), k, score, groups, group_k, group_top)
        without = route(logits, None, k, score, groups, group_k, group_top)
        for name in without:
            assert torch.equal(with_zeros[name], without[name])
    bias = 0.02 * torch.randn((E,), generator=g, device="cuda")
    check(logits, bias, k, score, groups, group_k, 2)
    bias[1:] = 0.0  # one that is not zero: sums as they round
    check(logits, bias, k, score, groups, group_k, 2)


@pytest.mark.parametrize("k", [1, 2, 7, 8, 15, 16, 17, 31, 32])
@pytest.mark.parametrize("T,E", [(70, 40), (300, 256), (40, 512)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_numbers_of_choices_and_of_candidates(T, E, k, with_bias):
    # logits of a few values, so that from k to E experts are as large as the last choice, all of it in one lane's
    # experts or one in each
    g = torch.Generator(device="cuda").manual_seed(E + k)
    bias = (torch.randint(0, 3, (E,), generator=g, device="cuda") / 64).float() if with_bias else None
    for values in (2, 9, 60):
        logits = torch.randint(0, values, (T, E), generator=g, device="cuda").float() / 8
        logits[0], logits[1, 1:] = 0.5, -math.inf
        logits[2] = torch.arange(E, 0, -1, device="cuda") / 16
        logits[3] = torch.arange(E, device="cuda") % 32
        for typ in ("f32", "bf16"):
            check(logits.to(TYPES[typ]), bias, k, "sigmoid", normalize=False)
            check(logits.to(TYPES[typ]), bias, k, "softmax")


@pytest.mark.parametrize("E,one", [(64, 512), (128, 512), (256, 256), (1024, 64)])
def test_launches(E, one):
    # one cluster up to 2^16 scores or 512 tokens; above, the choices and the places
    g = torch.Generator(device="cuda").manual_seed(E)
    bias = 0.1 * torch.randn((E,), generator=g, device="cuda")
    for T, launches in ((one - 1, 1), (one, 1), (one + 1, 2)):
        logits = torch.randn((T, E), generator=g, device="cuda")
        before = pig.igemm_kernels_launched()
        route(logits, bias, 8, "sigmoid", 8, 4, 2)
        assert pig.igemm_kernels_launched() - before == launches
        check(logits, bias, 8, "sigmoid", 8, 4, 2)


@pytest.mark.parametrize("offset", [1, 3])
def test_logits_off_16_bytes(offset):
    T, E = 600, 128
    for typ in TYPES.values():
        whole = torch.randn((T * E + offset,), device="cuda").to(typ)
        check(whole[offset:].view(T, E), None, 4, "sigmoid", 4, 2, 2)


def test_empty():
    E = 8
    offsets = torch.full((E + 1,), 5, dtype=torch.int32, device="cuda")
    none = torch.empty((0,), dtype=torch.int32, device="cuda")
    pig.igemm_moe_route_scored(torch.empty((0, E), device="cuda"), None, none, torch.empty((0,), device="cuda"), offsets,
                               none, none, 0, E, 2)
    assert bool((offsets == 0).all())


def grad(logits, experts, dweights, score, normalize, scale):
    T, E = logits.shape
    out = torch.full_like(logits, 7.0)
    pig.igemm_moe_route_scored_grad(logits, experts.int(), dweights, out, T, E, experts.shape[1], score=score,
                                    normalize=normalize, scale=scale)
    return out


@pytest.mark.parametrize("typ", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 2), (700, 64, 6), (300, 162, 8), (90, 1024, 32), (5000, 256, 8),
                                   (64, 333, 4)])
def test_gradient(T, E, k, normalize, score, typ):
    g = torch.Generator(device="cuda").manual_seed(T + E + k)
    logits = (2 * torch.randn((T, E), generator=g, device="cuda"))
    logits[torch.rand((T, E), generator=g, device="cuda") < 0.1] = -math.inf
    logits[T // 2] = -math.inf
    logits = logits.to(TYPES[typ])
    dw = torch.randn((T, k), generator=g, device="cuda")
    experts = plain_choice(logits, None, k, score, 1, 1, 1)
    scale = 2.5
    got = grad(logits, experts, dw, score, normalize, scale)
    # torch's own derivative of the weights in float64
    x = logits.double()
    live = torch.where(torch.isinf(x), -1e4, x).requires_grad_(True)
    (plain_weights(live, experts, score, normalize, scale) * dw.double()).sum().backward()
    want = torch.where(torch.isinf(x), 0.0, live.grad)
    with torch.no_grad():
        u = plain_weights(live, experts, score, normalize, 1.0)
        gu = (dw.double().abs() * u).sum(-1, keepdim=True)
        size = torch.zeros((T, E + 1), dtype=torch.float64, device="cuda").scatter_add_(
            1, torch.where(experts >= 0, experts, E), scale * u * (dw.double().abs() + gu))[:, :E]
        if score == "softmax" and not normalize:
            size = size + scale * torch.softmax(live, -1) * gu
    spread = 20.0
    tol = (2 * spread + E / 32 + k + 40) * 2.0 ** -24 * size + torch.finfo(logits.dtype).eps / 2 * want.abs() + \
        (2.0 ** -25 if typ == "f16" else 1e-44)
    assert bool(((got.double() - want).abs() <= tol).all()), (got.double() - want).abs().max().item()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_against_differences(score, normalize):
    # central differences of the routing's own weights: error h^2 / 6 |f'''| <= h^2, rounding of the weights 2^-22 / h
    T, E, k, h = 40, 12, 3, 2.0 ** -7
    logits = torch.randn((T, E), device="cuda")
    dw = torch.randn((T, k), device="cuda")
    base = route(logits, None, k, score, normalize=normalize)
    got = grad(logits, base["experts"], dw, score, normalize, 1.0)
    for e in range(E):
        f = []
        for sign in (1, -1):
            moved = logits.clone()
            moved[:, e] += sign * h
            x = moved.double()
            f.append((plain_weights(x, base["experts"].long(), score, normalize, 1.0) * dw.double()).sum(-1))
        diff = (f[0] - f[1]) / (2 * h)
        assert bool(((got[:, e].double() - diff).abs() <= 2 * h * h * (1 + dw.abs().sum(-1))).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_gradient_of_experts_named_twice_or_out_of_range(score, normalize):
    T, E, k = 50, 20, 4
    logits = torch.randn((T, E), device="cuda")
    experts = torch.randint(0, E, (T, k), device="cuda")
    experts[:, 1] = experts[:, 0]
    experts[::3, 2] = -1
    experts[1::3, 3] = E + 5
    dw = torch.randn((T, k), device="cuda")
    got = grad(logits, experts, dw, score, normalize, 1.0)
    x = logits.double().requires_grad_(True)
    named = torch.where((experts >= 0) & (experts < E), experts, -1)
    (plain_weights(x, named, score, normalize, 1.0) * dw.double()).sum().backward()
    assert bool(((got.double() - x.grad).abs() <= 200 * 2.0 ** -24 * (1 + dw.abs().sum(-1, keepdim=True))).all())


def test_gradient_without_scores():
    # a softmax row with +inf chose nothing; NaN logits have no part
    logits = torch.randn((4, 8), device="cuda")
    logits[0, 3] = math.inf
    logits[1, 2] = math.nan
    experts = torch.tensor([[-1, -1], [0, 1], [2, -1], [-1, -1]], device="cuda")
    dw = torch.randn((4, 2), device="cuda")
    for normalize in (True, False):
        for score in ("softmax", "sigmoid"):
            got = grad(logits, experts, dw, score, normalize, 1.0)
            assert bool(torch.isfinite(got).all()) and bool((got[0] == 0).all()) and bool((got[3] == 0).all())
            assert got[1, 2].item() == 0.0
    out = torch.full((4, 8), 7.0, device="cuda")
    pig.igemm_moe_route_scored_grad(logits, experts[:, :0].int().contiguous(), dw[:, :0].contiguous(), out, 4, 8, 0)
    assert bool((out == 0).all())
