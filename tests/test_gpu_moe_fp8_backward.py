"""The backward pass of the block-scaled fp8 example layer stage by stage, each against 64 bits on the values that it was
given.

Tolerances.  A product's: one rounding to its type and (128 + KB + 4) 2^-23 of the sum of magnitudes (test_gpu_bsfp8).  An
elementwise stage in float32: n roundings of 2^-24 relative to its terms' magnitudes.  Sums of float32 terms: their
number times 2^-24 of the sum of magnitudes, in whatever order.
"""

import os
import sys

import pytest

torch = pytest.importorskip("torch")

import precision_integer_gemm_gb300 as pig  # noqa: E402
from test_gpu_moe_fp8_layer import make, near, values  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    pig.build_library()
    yield pig.load()
    assert pig.igemm_last_status() == pig.IGEMM_OK


@pytest.mark.parametrize("T,E,D,F,k,kw", [(1, 4, 128, 96, 2, {}), (50, 4, 128, 96, 2, dict(scale=1.5)),
                                          (700, 8, 256, 160, 3, dict(scale=2.5)), (600, 16, 384, 136, 4, dict(groups=4, group_k=2))])
def test_backward_stage_by_stage(T, E, D, F, k, kw, monkeypatch):
    import moe_fp8
    from moe_fp8 import pack

    layer, router, _, _ = make(E, D, F, k, **kw)
    layer.bias.copy_(0.1 * torch.randn((E,), device="cuda"))
    x = torch.randn((T, D), device="cuda").to(torch.bfloat16)
    out = layer(x)
    dout = torch.randn_like(out)
    # what the pass makes on its way
    products, grads, matrices = [], [], []
    grouped, weight_gradient, route_grad = layer.grouped, moe_fp8.MoeFp8.weight_gradient, pig.igemm_moe_route_scored_grad

    def grouped_seen(a, b, offsets, N, K, dtype):
        products.append((a, grouped(a, b, offsets, N, K, dtype)))
        return products[-1][1]

    def matrix_seen(d, a):
        matrices.append((d, a, weight_gradient(d, a)))
        return matrices[-1][2]

    def grad_seen(logits, experts, dweights, dlogits, *args, **kwargs):
        route_grad(logits, experts, dweights, dlogits, *args, **kwargs)
        grads.append((dweights, dlogits))

    layer.grouped, layer.weight_gradient = grouped_seen, matrix_seen
    monkeypatch.setattr(pig, "igemm_moe_route_scored_grad", grad_seen)
    dx, d_router, d_gate_up, d_down = layer.backward(dout)
    _, logits, experts, weights, offsets, tokens, slots, h, act, y = layer.saved
    ends = offsets.tolist()
    assert ends[-1] == T * k and len(products) == 2 and len(matrices) == 2 * E and len(grads) == 1
    (dy_packed, dact), (dh_packed, dx_rows) = products
    dweights, dlogits = grads[0]
    u = 2.0 ** -24

    # the experts' rows: dy = w dout, rounded once to bfloat16 after one float32 product
    w = torch.zeros((T * k,), dtype=torch.float64, device="cuda")
    w[slots.view(-1).long()] = weights.double().view(-1)
    dy = torch.cat([m[0] for m in matrices[E:]])
    want = dout[tokens.long()].double() * w.unsqueeze(1)
    assert bool(((dy.double() - want).abs() <= (2.0 ** -8 + 2 * u) * want.abs() + 1e-38).all())
    for got, ref in zip(dy_packed, pack(dy)):
        assert torch.equal(got, ref)
    # ... and the weights: D products and their sum
    rows = y[slots.long()].double()
    terms = rows * dout.double().unsqueeze(1)
    assert bool(((dweights.double() - terms.sum(-1)).abs() <= (D + 1) * u * terms.abs().sum(-1)).all())

    # products of the tokens' rows with the transposed matrices
    a, b = values(dy_packed, 1, D), values(dh_packed, 1, 2 * F)
    for e, (i, j) in enumerate(zip(ends, ends[1:])):
        near(dact[i:j], a[i:j], values((layer.down_t[0][e], layer.down_t[1][e]), 128, D), D)
        near(dx_rows[i:j], b[i:j], values((layer.gate_up_t[0][e], layer.gate_up_t[1][e]), 128, 2 * F), 2 * F)

    # SwiGLU's gradient: h, dact bfloat16, in float32, rounded once (up to eight float32 roundings, of which those of
    # 1 - sigmoid and of 1 + gate (1 - sigmoid) are relative to their terms)
    dh = torch.cat([m[0] for m in matrices[:E]])
    gate, up, d = h[:, :F].double(), h[:, F:].double(), dact.double()
    sig = torch.sigmoid(gate)
    wants = torch.cat([d * up * sig * (1 + gate * (1 - sig)), d * gate * sig], 1)
    sizes = torch.cat([(d * up * sig).abs() * (1 + 2 * gate.abs()), (d * gate * sig).abs()], 1)
    assert bool(((dh.double() - wants).abs() <= 2.0 ** -8 * wants.abs() + 12 * u * sizes + 1e-38).all())
    for got, ref in zip(dh_packed, pack(dh)):
        assert torch.equal(got, ref)

    # the matrices' gradients, from both operands quantised along the tokens
    src = x[tokens.long()]
    for n, (N, K, a_rows, whole) in enumerate(((2 * F, D, src, d_gate_up), (D, F, act, d_down))):
        for e, (i, j) in enumerate(zip(ends, ends[1:])):
            d_rows, a_part, got = matrices[n * E + e]
            assert torch.equal(a_part, a_rows[i:j]) and torch.equal(got, whole[e]) and got.shape == (N, K)
            if j == i:
                assert bool((got == 0).all())
                continue
            pad = -(j - i) % 512
            p = values(pack(torch.nn.functional.pad(d_rows, (0, 0, 0, pad)).t()), 1, j - i + pad)
            q = values(pack(torch.nn.functional.pad(a_part, (0, 0, 0, pad)).t()), 1, j - i + pad)
            near(got, p, q, j - i + pad)

    # routing: the gradient of renormalised sigmoid scores
    scale = kw.get("scale", 1.0)
    s = torch.sigmoid(logits.double()).gather(1, experts.long())
    share, g = s / s.sum(-1, keepdim=True), dweights.double()
    mean = (g * share).sum(-1, keepdim=True)
    want = torch.zeros((T, E), dtype=torch.float64, device="cuda")
    want.scatter_(1, experts.long(), scale * share * (1 - s) * (g - mean))
    size = torch.zeros_like(want).scatter_(1, experts.long(), scale * share * (g.abs() + (g * share).abs().sum(-1, keepdim=True)))
    spread = 2 * logits.abs().max().item()
    assert bool(((dlogits.double() - want).abs() <= (2 * spread + k + 40) * u * size).all())

    # the sums into the tokens: k rows, and E products of the router
    want = dx_rows.double()[slots.long()].sum(1) + dlogits.double() @ router.double()
    size = dx_rows.double()[slots.long()].abs().sum(1) + dlogits.double().abs() @ router.double().abs()
    assert bool(((dx.double() - want).abs() <= 2.0 ** -8 * want.abs() + (k + E + 2) * u * size).all())
    want, size = dlogits.double().t() @ x.double(), dlogits.double().abs().t() @ x.double().abs()
    assert bool(((d_router.double() - want).abs() <= (T + 1) * u * size).all())
