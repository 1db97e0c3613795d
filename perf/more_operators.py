"""The measured operators of the block-scaled fp8 mixture-of-experts path: their cases, inputs, plain forms and exact
values.

`run` makes the library's calls where `own` is true, else computes the plain form: elementary torch operations in
float32, rounded once at the end.  The choice of experts is one between neighbouring values, so its plain form ranks
the scores in float64.
"""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}
BLOCK = 128


def _up(a: int, b: int) -> int:
    return -(-a // b) * b


def _code_bytes(K: int) -> int:
    return _up(K, 16)


def _scale_pitch(K: int) -> int:
    return _up(-(-K // BLOCK), 4)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decode batch's tokens to 6 of 64 experts in at most 3 of 8 groups, softmax scores: latency
        {"name": "route_decode", "op": "route", "type": "f32", "T": 8, "E": 64, "k": 6, "score": "softmax", "bias": False,
         "groups": 8, "group_k": 3, "group_top": 1, "normalize": False, "scale": 16.0, "masked": 0.0},
        # a long prompt's tokens to 8 of 256 experts in 4 of 8 groups, sigmoid scores with a balance bias, padding
        # tokens (rows of -inf) and experts masked out
        {"name": "route_prompt", "op": "route", "type": "f32", "T": 16384, "E": 256, "k": 8, "score": "sigmoid",
         "bias": True, "groups": 8, "group_k": 4, "group_top": 2, "normalize": True, "scale": 2.5, "masked": 0.1},
        # gradient of that routing in a training step: zeros but for the chosen logits
        {"name": "route_grad_sigmoid", "op": "route_grad", "type": "f32", "T": 16384, "E": 256, "k": 8,
         "score": "sigmoid", "bias": True, "groups": 8, "group_k": 4, "group_top": 2, "normalize": True, "scale": 2.5,
         "masked": 0.0},
        # gradient of softmax scores that are not renormalised: every logit has one; sizes that fit nothing
        {"name": "route_grad_softmax", "op": "route_grad", "type": "bf16", "T": 4097, "E": 162, "k": 6,
         "score": "softmax", "bias": False, "groups": 1, "group_k": 1, "group_top": 1, "normalize": False, "scale": 16.0,
         "masked": 0.05},
        # a decode batch's activations before a linear layer: latency
        {"name": "pack_decode", "op": "pack", "format": "e4m3", "type": "bf16", "rows": 16, "K": 8192, "form": "rows",
         "tile_rows": 1},
        # a prompt's tokens, each copied to its eight experts in sorted order
        {"name": "pack_gather", "op": "pack", "format": "e4m3", "type": "bf16", "rows": 32768, "K": 4096,
         "form": "gather", "source": 4096, "tile_rows": 1},
        # a float32 weight matrix stored [K, N], packed along K in tiles of 128 x 128
        {"name": "pack_tiles_transposed", "op": "pack", "format": "e4m3", "type": "f32", "rows": 28672, "K": 8192,
         "form": "transposed", "tile_rows": 128},
        # decode: 16 tokens through the widest weight matrix, the weights' bytes set the time
        {"name": "gemm_decode", "op": "gemm", "format": "e4m3", "type": "bf16", "M": 16, "N": 28672, "K": 8192},
        # a short prompt on ragged sizes: no dimension a multiple of a tile
        {"name": "gemm_ragged", "op": "gemm", "format": "e4m3", "type": "f32", "M": 600, "N": 10002, "K": 4160},
        # a long prompt: the tensor cores set the time
        {"name": "gemm_8192", "op": "gemm", "format": "e4m3", "type": "bf16", "M": 8192, "N": 8192, "K": 8192},
        # decode of 8 tokens, 4 of 64 experts each: most groups empty, the rest a row or two
        {"name": "grouped_decode", "op": "grouped", "format": "e4m3", "type": "bf16", "T": 8, "E": 64, "k": 4, "N": 4096,
         "K": 4096, "skew": 0.5},
        # a prompt of 4096 tokens, 8 of 64 experts each, some experts far more popular than others
        {"name": "grouped_prompt", "op": "grouped", "format": "e4m3", "type": "bf16", "T": 4096, "E": 64, "k": 8,
         "N": 4096, "K": 4096, "skew": 0.5},
    ]


def _log_int(rng, lo: int, hi: int) -> int:
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _depth(rng, lo: int, hi: int) -> int:
    """A length of the k axis: half of them whole blocks of 32, the others any."""
    K = _log_int(rng, lo, hi)
    return max(lo, K // 32 * 32) if rng.random() < 0.5 else K


def draw(rng):
    op = rng.choice(["route", "route_grad", "pack", "gemm", "gemm", "grouped", "grouped"])
    typ, fmt = rng.choice(["f32", "bf16", "f16"]), rng.choice(["e4m3", "e4m3", "e5m2"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 2, 4, 8, 16])
        per = _log_int(rng, max(2, 4 // groups), 512 // groups)
        group_k = rng.randint(1, groups)
        return {"op": op, "type": typ, "T": _log_int(rng, 1, 16384), "E": groups * per,
                "k": rng.randint(1, min(8, group_k * per)), "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "group_k": group_k, "group_top": rng.choice([1, 2]),
                "normalize": rng.random() < 0.5, "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0.0, 0.1, 0.5])}
    if op == "pack":
        form = rng.choice(["rows", "gather", "transposed"])
        c = {"op": op, "format": fmt, "type": typ, "rows": _log_int(rng, 1, 28672), "K": _depth(rng, 32, 8192),
             "form": form, "tile_rows": 1 if form == "gather" else rng.choice([1, 128])}
        if form == "gather":
            c["source"] = max(1, c["rows"] // rng.choice([1, 2, 4, 8]))
        return c
    if op == "gemm":
        return {"op": op, "format": fmt, "type": typ, "M": _log_int(rng, 1, 8192), "N": _log_int(rng, 64, 8192),
                "K": _depth(rng, 32, 8192)}
    E = _log_int(rng, 2, 128)
    return {"op": op, "format": fmt, "type": typ, "T": _log_int(rng, 1, 4096), "E": E, "k": rng.randint(1, min(8, E)),
            "N": _log_int(rng, 64, 4096), "K": _depth(rng, 64, 2048), "skew": rng.choice([0.0, 0.5, 1.0])}


# ------------------------------------------------------------------ plain forms

def _plain_pack(x, fmt: str, tile_rows: int):
    """Codes and scales of the rows of x (float32 [rows, K]), one scale per tile_rows x 128."""
    rows, K = x.shape
    Kp, Rp = _up(K, BLOCK), _up(rows, tile_rows)
    y = torch.nn.functional.pad(x, (0, Kp - K, 0, Rp - rows)).reshape(Rp // tile_rows, tile_rows, Kp // BLOCK, BLOCK)
    amax = y.abs().amax(dim=(1, 3), keepdim=True)
    # (by a tensor: division by a number is a product with its rounded reciprocal)
    s = (amax / torch.full_like(amax, LARGEST[fmt])).clamp(min=2.0 ** -126)
    fine = torch.isfinite(amax)
    y = torch.where(fine, y * (1.0 / s), 0.0).clamp(-LARGEST[fmt], LARGEST[fmt])
    codes = y.reshape(Rp, Kp)[:rows, : min(Kp, _code_bytes(K))].to(FP8[fmt])
    s = torch.where(fine, s, math.nan).view(Rp // tile_rows, Kp // BLOCK)
    return codes.contiguous(), torch.nn.functional.pad(s, (0, _scale_pitch(K) - Kp // BLOCK))


def _pack_by_rows(x, fmt, tile_rows, step=4096):
    parts = [_plain_pack(x[i:i + step].float(), fmt, tile_rows) for i in range(0, x.shape[0], step)]
    return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])


def _values(codes, scales, tile_rows: int, K: int):
    """[rows, K] values that codes and scales stand for."""
    v = codes.float()[:, :K]
    s = scales.repeat_interleave(BLOCK, dim=1)[:, :K]
    return v * (s if tile_rows == 1 else s.repeat_interleave(tile_rows, dim=0)[: codes.shape[0]])


def _plain_choice(c, logits, bias):
    """The chosen experts [T, k] by falling score, -1 where none is left; scores in float64."""
    T, E, G = c["T"], c["E"], c["groups"]
    x = logits.double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
        there = x > -math.inf
    else:
        m = x.amax(-1, keepdim=True)
        s = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
        s = s / s.sum(-1, keepdim=True)
        there = (x > -math.inf) & (m < math.inf)
    # without a bias the scores are in the order of the logits
    key = x if bias is None else s + bias.double()
    there = there & (key > -math.inf)  # (not NaN)
    key = torch.where(there, key, -math.inf)
    if G > 1:
        if c["group_top"] == 1:
            group = key.view(T, G, -1).amax(-1)
        else:
            best = torch.where(there, s if bias is None else key, -math.inf).view(T, G, -1)
            best = torch.sort(best, dim=-1, descending=True)[0][..., :2]
            group = torch.where(best > -math.inf, best, 0.0).sum(-1)
            group = torch.where(best[..., 0] > -math.inf, group, -math.inf)
        chosen = torch.sort(group, dim=-1, descending=True, stable=True)[1][:, : c["group_k"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=x.device).scatter_(1, chosen, True)
        key = torch.where(keep.repeat_interleave(E // G, dim=1), key, -math.inf)
    top, ids = torch.sort(key, dim=-1, descending=True, stable=True)
    return torch.where(top[:, : c["k"]] > -math.inf, ids[:, : c["k"]], -1)


def _plain_weights(c, logits, experts):
    """Weights [T, k] without the scale, and the scores [T, E] (softmax) that they come from."""
    x = logits.float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    there = experts >= 0
    top = torch.where(there, x.gather(1, experts.clamp(min=0).long()), -math.inf)
    if c["normalize"]:
        m = top.amax(-1, keepdim=True)
        m = torch.where(torch.isinf(m), 0.0, m)
        if c["score"] == "sigmoid":
            m = m.clamp(max=0.0)
            w = torch.where(top > 0, 1.0 / (1.0 + torch.exp(-top)), torch.exp(top - m) / (1.0 + torch.exp(top)))
        else:
            w = torch.exp(top - m)
        return torch.where(there, w / w.sum(-1, keepdim=True), 0.0), None
    if c["score"] == "sigmoid":
        return torch.where(there, 1.0 / (1.0 + torch.exp(-top)), 0.0), None
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - torch.where(torch.isinf(m), 0.0, m))
    p = torch.where(there[:, :1], p / p.sum(-1, keepdim=True), 0.0)
    return torch.where(there, p.gather(1, experts.clamp(min=0).long()), 0.0), p


def _run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "pack":
        x = s["x"]
        if s["index"] is not None:
            x = torch.where(s["index"].unsqueeze(1) >= 0, x[s["index"].clamp(min=0)], 0.0)
        codes, scales = _pack_by_rows(x, c["format"], c["tile_rows"])
        return {"codes": codes, "scales": scales}
    if op == "gemm":
        return (_values(s["A"], s["SFA"], 1, c["K"]) @ _values(s["B"], s["SFB"], BLOCK, c["K"]).t()).to(TYPES[c["type"]])
    if op == "grouped":
        a = _values(s["A"], s["SFA"], 1, c["K"])
        out = torch.empty((a.shape[0], c["N"]), dtype=torch.float32, device="cuda")
        at = 0
        for e, n in enumerate(s["counts"]):
            if n:
                out[at:at + n] = a[at:at + n] @ _values(s["B"][e], s["SFB"][e], BLOCK, c["K"]).t()
                at += n
        return out.to(TYPES[c["type"]])
    T, E, k = c["T"], c["E"], c["k"]
    if op == "route":
        experts = _plain_choice(c, s["logits"], s["bias"])
        weights, _ = _plain_weights(c, s["logits"], experts)
        there = experts >= 0
        key, order = torch.sort(torch.where(there, experts, E).view(-1), stable=True)
        offsets = torch.searchsorted(key, torch.arange(E + 1, device="cuda"))
        slots = torch.empty_like(order).scatter_(0, order, torch.arange(T * k, device="cuda"))
        tokens = torch.where(key < E, order // k, -1)
        return {"experts": experts.int(), "weights": c["scale"] * weights, "offsets": offsets.int(),
                "tokens": tokens.int(), "slots": torch.where(there, slots.view(T, k), -1).int()}
    # gradient of the logits for the weights' gradient g
    experts, g = s["experts"], s["dweights"]
    u, p = _plain_weights(c, s["logits"], experts)
    g = torch.where(experts >= 0, g, 0.0)
    mean = (g * u).sum(-1, keepdim=True)
    at = torch.where(experts >= 0, experts, E).long()
    x = s["logits"].float().gather(1, experts.clamp(min=0).long())
    if c["score"] == "sigmoid":
        d = u * (g - mean if c["normalize"] else g) / (1.0 + torch.exp(x))
    elif c["normalize"]:
        d = u * (g - mean)
    else:
        d = u * g
    out = torch.zeros((T, E + 1), device="cuda").scatter_add_(1, at, torch.where(experts >= 0, d, 0.0))[:, :E]
    if p is not None:
        out = out - p * mean
    return (c["scale"] * out).to(TYPES[c["type"]])


# ------------------------------------------------------------------ inputs

def _logits(gen, T: int, E: int, skew: float):
    """Router logits, an expert's popularity falling by exp(-skew i / 8)."""
    logits = torch.randn((T, E), generator=gen, device="cuda")
    return logits - skew / 8 * torch.randperm(E, generator=gen, device="cuda") * min(1.0, 64 / E)


def _operand(gen, fmt, rows, K, std, tile_rows):
    """A packed matrix of normal values (a few columns larger, as activations have)."""
    codes, scales = [], []
    gain = 1 + 4 * (torch.rand((K,), generator=gen, device="cuda") < 0.01).float()
    for i in range(0, rows, 16384):
        x = torch.randn((min(16384, rows - i), K), generator=gen, device="cuda") * std * gain
        q, s = _plain_pack(x, fmt, tile_rows)
        codes.append(q)
        scales.append(s)
    return torch.cat(codes), torch.cat(scales)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = c["op"]
    s = {"case": c}
    if op == "pack":
        rows, K = c["rows"], c["K"]
        shape = (K, rows) if c["form"] == "transposed" else (c.get("source", rows), K)
        x = torch.randn(shape, generator=gen, device="cuda").to(TYPES[c["type"]])
        s["x"] = x.t() if c["form"] == "transposed" else x
        s["index"] = None
        if c["form"] == "gather":
            s["index"] = torch.randint(0, shape[0], (rows,), generator=gen, device="cuda", dtype=torch.int32)
            s["index"][rows - rows // 64:] = -1  # pairs that were dropped
        s["codes"] = torch.empty((rows, _code_bytes(K)), dtype=FP8[c["format"]], device="cuda")
        s["scales"] = torch.empty((-(-rows // c["tile_rows"]), _scale_pitch(K)), device="cuda")
    elif op == "gemm":
        s["A"], s["SFA"] = _operand(gen, c["format"], c["M"], c["K"], 1.0, 1)
        s["B"], s["SFB"] = _operand(gen, c["format"], c["N"], c["K"], 0.02, BLOCK)
        s["C"] = torch.empty((c["M"], c["N"]), dtype=TYPES[c["type"]], device="cuda")
    elif op == "grouped":
        T, E, k, N, K = c["T"], c["E"], c["k"], c["N"], c["K"]
        ids = torch.topk(_logits(gen, T, E, c["skew"]), k, dim=-1)[1]
        counts = torch.bincount(ids.view(-1), minlength=E)
        s["counts"] = counts.tolist()
        s["offsets"] = torch.nn.functional.pad(counts.cumsum(0), (1, 0)).int()
        s["A"], s["SFA"] = _operand(gen, c["format"], T * k, K, 1.0, 1)
        parts = [_operand(gen, c["format"], N, K, 0.02, BLOCK) for _ in range(E)]
        s["B"], s["SFB"] = torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
        s["C"] = torch.empty((T * k, N), dtype=TYPES[c["type"]], device="cuda")
    else:
        T, E, k = c["T"], c["E"], c["k"]
        x = _logits(gen, T, E, 0.5)
        if c["masked"]:
            x[torch.rand((T, E), generator=gen, device="cuda") < c["masked"]] = -math.inf
            x[T - int(T * c["masked"] / 2):] = -math.inf  # padding tokens
        s["logits"] = x.to(TYPES[c["type"]])
        spread = 0.1 if c["score"] == "sigmoid" else 0.5 / E
        s["bias"] = spread * torch.randn((E,), generator=gen, device="cuda") if c["bias"] else None
        if op == "route":
            s["experts"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty((T, k), device="cuda")
            s["offsets"] = torch.empty((E + 1,), dtype=torch.int32, device="cuda")
            s["tokens"] = torch.empty((T * k,), dtype=torch.int32, device="cuda")
            s["slots"] = torch.empty((T, k), dtype=torch.int32, device="cuda")
        else:
            s["experts"] = _plain_choice(c, s["logits"], s["bias"]).int()
            s["dweights"] = torch.randn((T, k), generator=gen, device="cuda")
            s["dlogits"] = torch.empty((T, E), dtype=TYPES[c["type"]], device="cuda")
    return s


def run(state):
    if not own:
        return _run_plain(state)
    import precision_integer_gemm_gb300 as pig

    s, c = state, state["case"]
    op = c["op"]
    if op == "pack":
        pig.pack_bsfp8(s["x"], s["codes"], s["scales"], c["rows"], c["K"], tile_rows=c["tile_rows"], format=c["format"],
                       index=s["index"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if op == "gemm":
        pig.igemm_bsfp8(s["A"], s["B"], s["SFA"], s["SFB"], s["C"], c["M"], c["N"], c["K"], format=c["format"])
        return s["C"]
    if op == "grouped":
        pig.igemm_bsfp8_grouped(s["A"], s["B"], s["SFA"], s["SFB"], s["offsets"], s["C"], c["T"] * c["k"], c["E"],
                                c["N"], c["K"], format=c["format"])
        return s["C"]
    if op == "route":
        pig.igemm_moe_route_scored(s["logits"], s["bias"], s["experts"], s["weights"], s["offsets"], s["tokens"],
                                   s["slots"], c["T"], c["E"], c["k"], score=c["score"], groups=c["groups"],
                                   group_k=c["group_k"], group_top=c["group_top"], normalize=c["normalize"],
                                   scale=c["scale"])
        return {n: s[n] for n in ("experts", "weights", "offsets", "tokens", "slots")}
    pig.igemm_moe_route_scored_grad(s["logits"], s["experts"], s["dweights"], s["dlogits"], c["T"], c["E"], c["k"],
                                    score=c["score"], normalize=c["normalize"], scale=c["scale"])
    return s["dlogits"]


# ------------------------------------------------------------------ work and exact values

def work(case):
    c = case
    op = c["op"]
    size = {"f32": 4, "bf16": 2, "f16": 2}[c["type"]]

    def operand(rows, tile_rows):
        return rows * _code_bytes(c["K"]) + -(-rows // tile_rows) * _scale_pitch(c["K"]) * 4

    if op == "pack":
        read = min(c.get("source", c["rows"]), c["rows"]) * c["K"] * size + (4 * c["rows"] if c["form"] == "gather" else 0)
        return {"bytes": read + operand(c["rows"], c["tile_rows"]), "flops": 2 * c["rows"] * c["K"]}
    if op == "gemm":
        return {"bytes": operand(c["M"], 1) + operand(c["N"], BLOCK) + c["M"] * c["N"] * size,
                "flops": 2 * c["M"] * c["N"] * c["K"]}
    if op == "grouped":
        rows = c["T"] * c["k"]
        # experts that a routing of this many pairs reaches (all equally likely)
        active = c["E"] * (1 - (1 - 1 / c["E"]) ** rows)
        return {"bytes": int(operand(rows, 1) + active * operand(c["N"], BLOCK) + rows * c["N"] * size),
                "flops": 2 * rows * c["N"] * c["K"]}
    T, E, k = c["T"], c["E"], c["k"]
    if op == "route":
        return {"bytes": T * E * size + 16 * T * k + 8 * E + 4, "flops": 6 * T * E}
    # scores that are renormalised (and sigmoids) depend on the chosen logits alone
    dense = c["score"] == "softmax" and not c["normalize"]
    return {"bytes": T * E * size * (2 if dense else 1) + T * k * (8 + (0 if dense else size)),
            "flops": 4 * T * (E if dense else k) + 8 * T * k}


def _fp8_steps(fmt, device):
    """The values of the bytes 0 .. of the format's non-negative finite numbers, from their fields."""
    bits, bias, n = (3, 7, 127) if fmt == "e4m3" else (2, 15, 124)
    b = torch.arange(n, device=device)
    e, f = (b >> bits).double(), (b & (2 ** bits - 1)).double()
    return torch.where(e > 0, torch.exp2(e - bias) * (1 + f / 2 ** bits), 2.0 ** (1 - bias) * f / 2 ** bits)


def _exact_pack(x, fmt, tile_rows):
    """Bytes from the definition: the scale, its reciprocal and the products are each rounded to 32 bits, the codes
    are the nearest of the format's values (ties to the even byte)."""
    rows, K = x.shape
    steps = _fp8_steps(fmt, x.device)
    mids = (steps[1:] + steps[:-1]) / 2
    codes = torch.zeros((rows, _code_bytes(K)), dtype=torch.uint8, device=x.device)
    scales = torch.zeros((-(-rows // tile_rows), _scale_pitch(K)), dtype=torch.float64, device=x.device)
    for b in range(-(-K // BLOCK)):
        part = x[:, b * BLOCK:(b + 1) * BLOCK]
        amax = part.abs().max(-1).values
        if tile_rows > 1:
            amax = torch.cat([amax, amax.new_zeros(-rows % tile_rows)]).view(-1, tile_rows).max(-1).values
        s = torch.clamp((amax / LARGEST[fmt]).float(), min=2.0 ** -126).double()
        scales[:, b] = s
        r = (1.0 / s).float().double()
        y = (part * r.repeat_interleave(tile_rows)[:rows].unsqueeze(1)).float().double()
        mag = y.abs().clamp(max=LARGEST[fmt]).contiguous()
        lo, hi = torch.searchsorted(mids, mag), torch.searchsorted(mids, mag, right=True)
        q = torch.where(lo % 2 == 0, lo, hi) + 128 * torch.signbit(y)
        codes[:, b * BLOCK:b * BLOCK + part.shape[1]] = q.to(torch.uint8)
    return codes.view(FP8[fmt]), scales


def _exact_values(codes, scales, fmt, tile_rows, K):
    """The codes' values in 64 bits, from the fields of the formats (sign, exponent, fraction)."""
    steps = _fp8_steps(fmt, codes.device)
    q = codes.view(torch.uint8)[:, :K].int()
    v = steps[(q & 127).long()] * (1.0 - 2.0 * (q >> 7))
    row = torch.arange(codes.shape[0], device=codes.device) // tile_rows
    for b in range(-(-K // BLOCK)):
        v[:, b * BLOCK:(b + 1) * BLOCK] *= scales[row, b].double().unsqueeze(1)
    return v


def _exact_scores(x, score):
    """Scores of float64 logits, NaN as -inf."""
    if score == "sigmoid":
        with np.errstate(over="ignore"):
            return np.where(x >= 0, 1 / (1 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1 + np.exp(-np.abs(x))))
    m = x.max(-1, keepdims=True)
    s = np.exp(x - np.where(np.isfinite(m), m, 0.0))
    total = s.sum(-1, keepdims=True)
    return s / np.where(total > 0, total, 1.0)


def _exact_route(c, logits, bias):
    """Experts and weights token by token in 64 bits: groups by their scores, then experts by theirs."""
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    x = logits.double().cpu().numpy()
    x = np.where(np.isnan(x), -np.inf, x)
    s = _exact_scores(x, c["score"])
    pick = x if bias is None else s + bias.double().cpu().numpy()
    pick = np.where(x > -np.inf, pick, -np.inf)
    if G > 1:
        sums = s if bias is None and c["group_top"] > 1 else pick
        members = np.where(x > -np.inf, sums, -np.inf).reshape(T, G, E // G)
        best = -np.sort(-members, axis=-1)[..., : c["group_top"]]
        some = best[..., 0] > -np.inf
        group = np.where(some, np.where(best > -np.inf, best, 0.0).sum(-1), -np.inf)
        rank = np.lexsort((np.broadcast_to(np.arange(G), (T, G)), -group), axis=-1)
        out = np.ones((T, G), bool)
        np.put_along_axis(out, rank[:, : c["group_k"]], False, axis=-1)
        pick = np.where(np.repeat(out, E // G, axis=1), -np.inf, pick)
    order = np.lexsort((np.broadcast_to(np.arange(E), (T, E)), -pick), axis=-1)[:, :k]
    there = np.take_along_axis(pick, order, -1) > -np.inf
    chosen = np.where(there, np.take_along_axis(s, order, -1), 0.0)
    if c["normalize"]:
        total = chosen.sum(-1, keepdims=True)
        chosen = chosen / np.where(total > 0, total, 1.0)
    return np.where(there, order, -1).astype(np.int32), c["scale"] * chosen


def exact(case, seed):
    s = prepare(case, seed)
    c = case
    op = c["op"]
    if op == "pack":
        x = s["x"]
        out = []
        for i in range(0, c["rows"], 2048):
            if s["index"] is not None:
                at = s["index"][i:i + 2048].long()
                part = x[at.clamp(min=0)].double()
                part[at < 0] = 0
            else:
                part = x[i:i + 2048].double()
            out.append(_exact_pack(part, c["format"], c["tile_rows"]))
        return {"codes": torch.cat([o[0] for o in out]), "scales": torch.cat([o[1] for o in out])}
    if op in ("gemm", "grouped"):
        a = _exact_values(s["A"], s["SFA"], c["format"], 1, c["K"])
        if op == "gemm":
            ends, experts = [(0, c["M"])], [(s["B"], s["SFB"])]
        else:
            o = s["offsets"].tolist()
            ends, experts = list(zip(o[:-1], o[1:])), list(zip(s["B"], s["SFB"]))
        out = torch.zeros((a.shape[0], c["N"]), dtype=torch.float64, device="cuda")
        for e, (i, j) in enumerate(ends):
            if j > i:
                out[i:j] = torch.matmul(a[i:j], _exact_values(*experts[e], c["format"], BLOCK, c["K"]).t())
        return out
    T, E, k = c["T"], c["E"], c["k"]
    if op == "route":
        experts, weights = _exact_route(c, s["logits"], s["bias"])
        tokens, slots, offsets = np.full(T * k, -1, np.int32), np.full((T, k), -1, np.int32), np.zeros(E + 1, np.int32)
        t, j = np.nonzero(experts >= 0)
        by = np.lexsort((t, experts[t, j]))
        tokens[:by.size] = t[by]
        slots[t[by], j[by]] = np.arange(by.size)
        offsets[1:] = np.cumsum(np.bincount(experts[t, j], minlength=E))
        return {"experts": experts, "weights": weights, "offsets": offsets, "tokens": tokens, "slots": slots}
    # d w_j / d x_e by the quotient rule, summed against the weights' gradient
    x = s["logits"].double().cpu().numpy()
    x = np.where(np.isnan(x), -np.inf, x)
    experts, g = s["experts"].cpu().numpy(), s["dweights"].double().cpu().numpy()
    p = _exact_scores(x, c["score"])
    there = experts >= 0
    at = np.where(there, experts, 0)
    ds = np.zeros((T, E))  # gradient of the scores
    picked = np.where(there, np.take_along_axis(p, at, -1), 0.0)
    g = np.where(there, g, 0.0)
    if c["normalize"]:
        total = picked.sum(-1, keepdims=True)
        total = np.where(total > 0, total, 1.0)
        g = g / total - (g * picked).sum(-1, keepdims=True) / total ** 2
    for j in range(k):
        ds[np.arange(T), at[:, j]] += np.where(there[:, j], g[:, j], 0.0)
    out = p * (1 - p) * ds if c["score"] == "sigmoid" else p * (ds - (p * ds).sum(-1, keepdims=True))
    return c["scale"] * out
