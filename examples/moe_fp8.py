"""A mixture-of-experts feed-forward layer in block-scaled fp8, with scored routing, forward and backward.

    python examples/moe_fp8.py [--tokens T] [--steps N]

Experts are chosen by sigmoid scores with a balance bias within the best groups; the weights are the renormalised
scores.  Weights are packed once per optimiser step with one scale per 128 x 128, and once more transposed for the
backward pass; activations and gradients get one scale per 128 values of a row.  A pass routes the tokens, packs each
token's row at the sorted places of its experts, runs the two grouped products with SwiGLU between them, and sums the
experts' rows back to the tokens.  The backward pass runs the transposed products and the routing's gradient; the
gradients of the expert matrices are fp8 products of the tokens' transposed rows.  No step of the forward pass reads
anything on the host.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import precision_integer_gemm_gb300 as pig  # noqa: E402


def pack(x, tile_rows=1, index=None):
    """(codes, scales) of the rows of x (any matrix with a unit stride), or of x[index]."""
    rows, K = (x.shape[0] if index is None else index.numel()), x.shape[1]
    codes = torch.empty((rows, pig.bsfp8_code_bytes(K)), dtype=torch.uint8, device=x.device)
    scales = torch.empty((-(-rows // tile_rows), pig.bsfp8_scale_pitch(K)), device=x.device)
    pig.pack_bsfp8(x, codes, scales, rows, K, tile_rows=tile_rows, index=index)
    return codes, scales


class MoeFp8:
    """Experts' weights: gate_up [E, 2 F, D] and down [E, D, F] (float32, bfloat16 or float16); router [E, D]."""

    def __init__(self, router, gate_up, down, k: int, groups: int = 1, group_k: int = 1, scale: float = 1.0):
        self.router, self.k, self.groups, self.group_k, self.scale = router, k, groups, group_k, scale
        self.E, f2, self.D = gate_up.shape
        self.F = f2 // 2
        self.bias = torch.zeros((self.E,), device=gate_up.device)
        self.set_weights(gate_up, down)

    def set_weights(self, gate_up, down):
        self.gate_up, self.down = self._pack_experts(gate_up), self._pack_experts(down)
        self.gate_up_t = self._pack_experts(gate_up.transpose(1, 2))
        self.down_t = self._pack_experts(down.transpose(1, 2))

    def _pack_experts(self, w):
        parts = [pack(m, tile_rows=128) for m in w]
        return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])

    def grouped(self, a, b, offsets, N, K, dtype):
        rows = a[0].shape[0]
        # (rows of no group are left as they are: pairs that were not routed read zeros)
        out = torch.zeros((rows, N), dtype=dtype, device=a[0].device)
        pig.igemm_bsfp8_grouped(a[0], b[0], a[1], b[1], offsets, out, rows, self.E, N, K)
        return out

    def route(self, x):
        T, E, k, dev = x.shape[0], self.E, self.k, x.device
        logits = (x.float() @ self.router.float().t()).contiguous()
        experts = torch.empty((T, k), dtype=torch.int32, device=dev)
        weights = torch.empty((T, k), device=dev)
        offsets = torch.empty((E + 1,), dtype=torch.int32, device=dev)
        tokens = torch.empty((T * k,), dtype=torch.int32, device=dev)
        slots = torch.empty_like(experts)
        pig.igemm_moe_route_scored(logits, self.bias, experts, weights, offsets, tokens, slots, T, E, k, score="sigmoid",
                                   groups=self.groups, group_k=self.group_k, group_top=2 if self.groups > 1 else 1,
                                   scale=self.scale)
        return logits, experts, weights, offsets, tokens, slots

    def __call__(self, x):
        """x [T, D] -> [T, D] of the same type; what backward() needs stays in self.saved."""
        T = x.shape[0]
        logits, experts, weights, offsets, tokens, slots = self.route(x)
        a = pack(x, index=tokens)
        h = self.grouped(a, self.gate_up, offsets, 2 * self.F, self.D, x.dtype)
        act = torch.nn.functional.silu(h[:, :self.F]) * h[:, self.F:]
        y = self.grouped(pack(act), self.down, offsets, self.D, self.F, x.dtype)
        out = torch.empty_like(x)
        pig.igemm_moe_combine(y, slots, weights, out, T, self.k, self.D)
        self.saved = (x, logits, experts, weights, offsets, tokens, slots, h, act, y)
        return out

    def backward(self, dout):
        """Gradients of x, the router and the experts' matrices (gate_up, down; float32) for that of the output."""
        x, logits, experts, weights, offsets, tokens, slots, h, act, y = self.saved
        T, k, F, D = x.shape[0], self.k, self.F, self.D
        at = tokens.clamp(min=0).long()
        live = (tokens >= 0).unsqueeze(1)
        pair = slots.clamp(min=0).long()
        # combine: of the experts' rows and of the weights
        w_sorted = torch.zeros((T * k,), device=x.device)
        w_sorted[slots[slots >= 0].long()] = weights[slots >= 0]
        dy = torch.where(live, dout[at].float() * w_sorted.unsqueeze(1), 0.0).to(x.dtype)
        dweights = torch.where(slots >= 0, (y[pair].float() * dout.float().unsqueeze(1)).sum(-1), 0.0)
        # the products, and SwiGLU between them
        dact = self.grouped(pack(dy), self.down_t, offsets, F, D, x.dtype).float()
        gate, up = h[:, :F].float(), h[:, F:].float()
        sig = torch.sigmoid(gate)
        dh = torch.cat([dact * up * sig * (1 + gate * (1 - sig)), dact * gate * sig], 1).to(x.dtype)
        dx_rows = self.grouped(pack(dh), self.gate_up_t, offsets, D, 2 * F, x.dtype)
        dx = torch.zeros((T, D), device=x.device)
        dx.index_add_(0, at, torch.where(live, dx_rows.float(), 0.0))
        # routing
        dlogits = torch.empty_like(logits)
        pig.igemm_moe_route_scored_grad(logits, experts, dweights, dlogits, T, self.E, k, score="sigmoid",
                                        scale=self.scale)
        dx += dlogits @ self.router.float()
        ends = offsets.tolist()
        xs = torch.where(live, x[at], 0.0).to(x.dtype)
        d_gate_up = torch.stack([self.weight_gradient(dh[i:j], xs[i:j]) for i, j in zip(ends, ends[1:])])
        d_down = torch.stack([self.weight_gradient(dy[i:j], act[i:j]) for i, j in zip(ends, ends[1:])])
        return dx.to(x.dtype), dlogits.t() @ x.float(), d_gate_up, d_down

    @staticmethod
    def weight_gradient(d, a):
        """d [n, N], a [n, K] -> d^T a [N, K]: both packed along the n tokens, one scale per 128 of them."""
        n, N, K = d.shape[0], d.shape[1], a.shape[1]
        out = torch.zeros((N, K), device=d.device)
        if n == 0:
            return out
        full = -(-n // 512) * 512  # whole groups of four scales
        pad = torch.nn.functional.pad
        p, q = pack(pad(d, (0, 0, 0, full - n)).t()), pack(pad(a, (0, 0, 0, full - n)).t())
        pig.fp8_blockscaled_gemm(p[0], q[0], p[1], q[1], out, N, K, full)
        return out


def main() -> None:
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--steps", type=int, default=20)
    a = p.parse_args()
    E, D, F, k = 16, 1024, 1280, 4
    torch.manual_seed(0)
    router = torch.randn((E, D), device="cuda") / D ** 0.5
    gate_up = torch.randn((E, 2 * F, D), device="cuda", dtype=torch.bfloat16) / D ** 0.5
    down = torch.randn((E, D, F), device="cuda", dtype=torch.bfloat16) / F ** 0.5
    layer = MoeFp8(router, gate_up, down, k, groups=4, group_k=2, scale=2.5)
    x = torch.randn((a.tokens, D), device="cuda", dtype=torch.bfloat16)
    out = layer(x)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        out = layer(x)
    stop.record()
    torch.cuda.synchronize()
    grads = layer.backward(torch.randn_like(out))
    print(f"fp8: {a.tokens} tokens, {E} experts, top {k}: {start.elapsed_time(stop) / a.steps:.3f} ms a pass; gradients of "
          f"{', '.join(str(tuple(g.shape)) for g in grads)}")
    if pig.igemm_last_status() != 0:
        raise SystemExit("device status not 0")


if __name__ == "__main__":
    main()
