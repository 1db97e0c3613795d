"""A mixture-of-experts feed-forward layer in 4-bit floating point, from router logits to token rows.

    python examples/moe_fp4.py [--format mx|nv] [--tokens T]

Weights are packed once (gate and up projections of an expert stacked as one matrix).  A pass routes the tokens,
packs each token's row at the sorted places of its experts, runs the two grouped products with SwiGLU between them,
and sums the experts' rows back to the tokens.  No step reads anything on the host.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import precision_integer_gemm_gb300 as pig  # noqa: E402


class MoeFp4:
    """Experts' weights: gate_up [E, 2 F, D] and down [E, D, F] (float32, bfloat16 or float16); router [E, D]."""

    def __init__(self, router, gate_up, down, k: int, fmt: str = "mx"):
        self.router, self.k, self.fmt = router, k, fmt
        self.E, f2, self.D = gate_up.shape
        self.F = f2 // 2
        # nv: block scales are e4m3 relative to one scale per tensor (here 6 * 448 at the largest value)
        self.gate_up, self.g1 = self._pack_weights(gate_up)
        self.down, self.g2 = self._pack_weights(down)

    def _tensor_scale(self, x):
        if self.fmt != "nv":
            return None
        if x.numel() == 0:
            return torch.ones((1,), device=x.device)
        return (x.abs().amax().float() / (6 * 448)).clamp(min=1e-30).view(1)

    def _pack_weights(self, w):
        g = self._tensor_scale(w)
        return self.pack(w.reshape(-1, w.shape[-1]), g), g

    def pack(self, x, tensor_scale=None, index=None):
        """(codes, scales) of the rows of x, or of x[index]."""
        rows, K = (x.shape[0] if index is None else index.numel()), x.shape[1]
        pitch = pig.mxfp4_scale_pitch(K) if self.fmt == "mx" else pig.nvfp4_scale_pitch(K)
        codes = torch.empty((rows, pig.fp4_code_bytes(K)), dtype=torch.uint8, device=x.device)
        scales = torch.empty((rows, pitch), dtype=torch.uint8, device=x.device)
        if self.fmt == "mx":
            pig.pack_mxfp4(x, codes, scales, rows, K, index=index)
        else:
            pig.pack_nvfp4(x, tensor_scale, codes, scales, rows, K, index=index)
        return codes, scales

    def grouped(self, a, g_a, b, g_b, offsets, rows, N, K, out):
        if self.fmt == "mx":
            pig.igemm_mxfp4_grouped(a[0], b[0], a[1], b[1], offsets, out, rows, self.E, N, K)
        else:
            pig.igemm_nvfp4_grouped(a[0], b[0], a[1], b[1], offsets, (g_a * g_b).expand(self.E).contiguous(), out,
                                    rows, self.E, N, K)
        return out

    def __call__(self, x):
        """x [T, D] -> [T, D] of the same type."""
        T, rows, dev = x.shape[0], x.shape[0] * self.k, x.device
        logits = (x.float() @ self.router.float().t()).contiguous()
        experts = torch.empty((T, self.k), dtype=torch.int32, device=dev)
        weights = torch.empty((T, self.k), dtype=torch.float32, device=dev)
        offsets = torch.empty((self.E + 1,), dtype=torch.int32, device=dev)
        tokens = torch.empty((rows,), dtype=torch.int32, device=dev)
        slots = torch.empty_like(experts)
        pig.igemm_moe_route(logits, experts, weights, offsets, tokens, slots, T, self.E, self.k)

        g_x = self._tensor_scale(x)
        a = self.pack(x, g_x, index=tokens)
        # (rows of no group are left as they are: pairs that were not routed read zeros)
        h = torch.zeros((rows, 2 * self.F), dtype=x.dtype, device=dev)
        self.grouped(a, g_x, self.gate_up, self.g1, offsets, rows, 2 * self.F, self.D, h)
        act = torch.nn.functional.silu(h[:, :self.F]) * h[:, self.F:]
        g_act = self._tensor_scale(act)
        y = torch.zeros((rows, self.D), dtype=x.dtype, device=dev)
        self.grouped(self.pack(act, g_act), g_act, self.down, self.g2, offsets, rows, self.D, self.F, y)
        out = torch.empty_like(x)
        pig.igemm_moe_combine(y, slots, weights, out, T, self.k, self.D)
        return out


def main() -> None:
    p = argparse.ArgumentParser()
    p.add_argument("--format", choices=("mx", "nv"), default="mx")
    p.add_argument("--tokens", type=int, default=512)
    a = p.parse_args()
    E, D, F, k = 16, 1024, 1280, 4
    torch.manual_seed(0)
    router = torch.randn((E, D), device="cuda") / D ** 0.5
    gate_up = torch.randn((E, 2 * F, D), device="cuda", dtype=torch.bfloat16) / D ** 0.5
    down = torch.randn((E, D, F), device="cuda", dtype=torch.bfloat16) / F ** 0.5
    layer = MoeFp4(router, gate_up, down, k, a.format)
    x = torch.randn((a.tokens, D), device="cuda", dtype=torch.bfloat16)
    out = layer(x)
    start, stop = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(20):
        out = layer(x)
    stop.record()
    torch.cuda.synchronize()
    # the same layer in float32 on the unpacked weights
    top, ids = torch.topk(x.float() @ router.t(), k, dim=-1)
    w = torch.softmax(top, -1)
    ref = torch.zeros((a.tokens, D), device="cuda")
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        h = x[t].float() @ gate_up[e].float().t()
        y = (torch.nn.functional.silu(h[:, :F]) * h[:, F:]) @ down[e].float().t()
        ref.index_add_(0, t, y * w[t, j].unsqueeze(1))
    err = ((out.float() - ref).norm() / ref.norm()).item()
    print(f"{a.format}fp4: {a.tokens} tokens, {E} experts, top {k}: {start.elapsed_time(stop) / 20:.3f} ms a pass, "
          f"relative distance to float32 weights and activations {err:.3f}")
    if pig.igemm_last_status() != 0:
        raise SystemExit("device status not 0")


if __name__ == "__main__":
    main()
