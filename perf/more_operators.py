"""Measured cases of the dense block's 8-bit operators: norm, pack, matmul.

Rows and weights are held in E4M3 with an fp32 scale: rows' for each 128 columns of a row, weights' for each 128 x 128 block.

  norm    s = x + residual, rounded to the residual's type and kept; y = s / sqrt(mean(s^2) + eps) * gain; y in 8 bits
          with a scale for each 128 columns (scale = amax / 448, code = e4m3(y * fp32(448 / amax))), or in 16, or both.
          Without a gain nothing is normalised: the sum itself is quantised.
  pack    a weight matrix into 8 bits with a scale for each block of 128 x 128
  matmul  out[t][n] = add[t][n] + sum over blocks kb of 128 columns: row_scale[kb][t] * weight_scale[n / 128][kb] *
          (sum over the block of row_code * weight_code)

`own` chooses between elementary torch operations and the framework's kernels.
"""
import math

import torch

own = False

T_OF = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
E4M3 = torch.float8_e4m3fn
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's next token: what the expert block wrote joins the residual, on its way to the next layer's projection
        dict(name="norm-token", op="norm", rows=1, k=2048, x="f32", res="bf16", gain=True, y="", codes=True),
        # a serving batch's step; the norm's output is wanted in 16 bits too (a router reads it)
        dict(name="norm-batch", op="norm", rows=203, k=4096, x="f16", res="f16", gain=True, y="f16", codes=True),
        # prompts, in one call
        dict(name="norm-prompt", op="norm", rows=16384, k=2048, x="bf16", res="bf16", gain=True, y="", codes=True),
        # attention's output on its way to the output projection: quantised as it is
        dict(name="norm-none", op="norm", rows=6001, k=4096, x="bf16", res="", gain=False, y="", codes=True),
        # a layer's query, key and value projection at load time
        dict(name="pack-projection", op="pack", n=5120, k=2048, w="bf16"),
        # a vocabulary's head from a checkpoint in 32 bits
        dict(name="pack-head", op="pack", n=50021, k=4096, w="f32"),
        # one user's next token through the query, key and value projection: latency
        dict(name="matmul-token", op="matmul", rows=1, n=5120, k=2048, out="bf16", add=False),
        # a serving batch's step through the output projection, the residual added
        dict(name="matmul-batch", op="matmul", rows=61, n=2048, k=4096, out="bf16", add=True),
        # drafted tokens' logits: a long, odd weight matrix and few rows
        dict(name="matmul-head", op="matmul", rows=17, n=100003, k=2048, out="f32", add=False),
        # a short prompt, sizes that no tile divides
        dict(name="matmul-short", op="matmul", rows=333, n=6000, k=2000, out="f16", add=False),
        # prompts through the query, key and value projection
        dict(name="matmul-prompt", op="matmul", rows=4096, n=5120, k=2048, out="bf16", add=False),
        # a large projection over a chunk of long prompts, the residual added
        dict(name="matmul-large", op="matmul", rows=8191, n=8192, k=8192, out="bf16", add=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _features(rng, lo, hi):
    """Input features: multiples of 16, half of them of 128."""
    k = _log(rng, lo, hi)
    step = rng.choice([16, 128])
    return max(step, k // step * step)


def draw(rng):
    op = rng.choice(["norm", "norm", "pack", "matmul", "matmul", "matmul"])
    if op == "norm":
        k = _features(rng, 64, 16384)
        c = dict(op=op, rows=_log(rng, 1, max(2, min(20000, 67_000_000 // k))), k=k, x=rng.choice(["bf16", "bf16", "f16", "f32"]),
                 res="", gain=rng.random() < 0.75, y="", codes=True)
        kind = "f16" if c["x"] == "f16" else "bf16"
        if rng.random() < 0.7:
            c["res"] = rng.choice([kind, kind, "f32"])
        if rng.random() < 0.4:
            c.update(y=kind, codes=rng.random() < 0.7)
        return c
    if op == "pack":
        k = _features(rng, 128, 16384)
        return dict(op=op, n=_log(rng, 64, max(65, min(100000, 200_000_000 // k))), k=k, w=rng.choice(["bf16", "f16", "f32"]))
    k = _features(rng, 128, 12000)
    n = _log(rng, 100, min(110000, 200_000_000 // k))
    rows = _log(rng, 1, max(2, min(9000, 540_000_000_000 // (n * k), 120_000_000 // n)))
    return dict(op=op, rows=rows, n=n, k=k, out=rng.choice(["bf16", "bf16", "f16", "f32"]), add=rng.random() < 0.4)


def work(case):
    k, kb = case["k"], -(-case["k"] // 128)
    if case["op"] == "norm":
        t = case["rows"]
        per = SIZE[case["x"]] + 2 * SIZE.get(case["res"], 0) + SIZE.get(case["y"], 0) + (1 if case["codes"] else 0)
        return {"bytes": t * k * per + (4 * t * kb if case["codes"] else 0) + 4 * k * case["gain"], "flops": t * k * (4 + 4 * case["gain"])}
    n, nb = case["n"], -(-case["n"] // 128)
    if case["op"] == "pack":
        return {"bytes": n * k * (SIZE[case["w"]] + 1) + 4 * nb * kb, "flops": 2 * n * k}
    t, size = case["rows"], SIZE[case["out"]]
    return {"bytes": t * k + n * k + 4 * (t + nb) * kb + t * n * size * (2 if case["add"] else 1), "flops": 2 * t * n * k}


# ------------------------------------------------------------------ inputs
def _codes(g, rows, k):
    """Codes as a quantisation by blocks leaves them: normal values whose largest in a block is near 448."""
    return torch.randn((rows, k), generator=g, device=DEV, dtype=torch.float16).mul_(130.0).clamp_(-448, 448).to(E4M3)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    k, kb = case["k"], -(-case["k"] // 128)
    s = dict(case=dict(case))
    if case["op"] == "norm":
        t = case["rows"]
        # channels of different size, as a layer's outputs have them, a few of them large
        channel = torch.exp(0.7 * torch.randn(k, generator=g, device=DEV))
        s["x"] = (torch.randn((t, k), generator=g, device=DEV) * channel).to(T_OF[case["x"]])
        s["residual"] = None
        if case["res"]:
            s["residual"] = (3.0 * torch.randn((t, k), generator=g, device=DEV) * channel).to(T_OF[case["res"]])
        s["gain"] = torch.rand(k, generator=g, device=DEV) + 0.5 if case["gain"] else None
        s["eps"] = 1e-6
    elif case["op"] == "pack":
        s["w"] = (torch.randn((case["n"], k), generator=g, device=DEV) / math.sqrt(k)).to(T_OF[case["w"]])
    else:
        t, n = case["rows"], case["n"]
        s["codes"], s["w_codes"] = _codes(g, t, k), _codes(g, n, k)
        stride = (t + 3) // 4 * 4  # (a row of scales for each block of columns; whole 16 bytes)
        s["scales"] = torch.exp(0.3 * torch.randn((kb, stride), generator=g, device=DEV)) * (4.0 / 448)
        s["w_scales"] = torch.exp(0.2 * torch.randn((-(-n // 128), kb), generator=g, device=DEV)) * (4.0 / 448 / math.sqrt(k))
        s["add"] = torch.randn((t, n), generator=g, device=DEV).to(T_OF[case["out"]]) if case["add"] else None
    if own:
        _handles(s)
    return s


def _handles(s):
    """What a program that uses the framework keeps: the plan, the scratch, its buffers and their descriptions."""
    from quantized_moe_expert_gemv_gb300 import binding as si

    c = s["case"]
    k, kb = c["k"], -(-c["k"] // 128)
    s["si"] = si
    si.load_library()
    plan = s["plan"] = si.si_fp8_plan(si.make_fp8_desc(k, c.get("n", k)), 0)
    if c["op"] == "norm":
        t = c["rows"]
        stride = (t + 3) // 4 * 4
        s["s_out"] = torch.empty((t, k), dtype=T_OF[c["res"]], device=DEV) if c["res"] else None
        s["y_out"] = torch.empty((t, k), dtype=T_OF[c["y"]], device=DEV) if c["y"] else None
        s["codes_out"] = torch.empty((t, k), dtype=E4M3, device=DEV) if c["codes"] else None
        s["scales_out"] = torch.empty((kb, stride), device=DEV) if c["codes"] else None
        s["mats"] = [None if m is None else si.fp8_mat(m) for m in (s["x"], s["residual"], s["s_out"], s["y_out"])]
        s["rows"] = si.fp8_rows(s["codes_out"], s["scales_out"]) if c["codes"] else None
        return
    if c["op"] == "pack":
        s["codes_out"] = torch.empty((c["n"], k), dtype=E4M3, device=DEV)
        s["scales_out"] = torch.empty((-(-c["n"] // 128), kb), device=DEV)
        s["weight"], s["mat"] = si.fp8_weight(s["codes_out"], s["scales_out"]), si.fp8_mat(s["w"])
        return
    s["rows"], s["weight"] = si.fp8_rows(s["codes"], s["scales"]), si.fp8_weight(s["w_codes"], s["w_scales"])
    s["out"] = torch.empty((c["rows"], c["n"]), dtype=T_OF[c["out"]], device=DEV)
    s["mats"] = [si.fp8_mat(s["add"]) if c["add"] else None, si.fp8_mat(s["out"])]
    s["scratch"] = torch.empty(si.si_fp8_scratch_bytes(plan, c["rows"]), dtype=torch.uint8, device=DEV)
    si.si_fp8_scratch_init(plan, s["scratch"])


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_norm(s):
    x, residual, s_out, y = s["mats"]
    t = s["case"]["rows"]
    s["si"].si_fp8_norm(s["plan"], x, residual, s["gain"], s["eps"], s_out, y, s["rows"], t)
    scales = s["scales_out"]
    return dict(residual=s["s_out"], y=s["y_out"], codes=s["codes_out"], scales=None if scales is None else scales[:, :t])


def _own_pack(s):
    s["si"].si_fp8_pack(s["plan"], s["mat"], s["weight"])
    return dict(codes=s["codes_out"], scales=s["scales_out"])


def _own_matmul(s):
    add, out = s["mats"]
    s["si"].si_fp8_matmul(s["plan"], s["rows"], s["weight"], add, out, s["case"]["rows"], s["scratch"])
    return dict(out=s["out"])


_OWN = dict(norm=_own_norm, pack=_own_pack, matmul=_own_matmul)


# ---- the plain forms
def _quantise(y, dims):
    """Codes and scales of values whose blocks lie along `dims`."""
    amax = y.abs().amax(dims, keepdim=True)
    codes = (y * torch.where(amax >= 2.0 ** -100, 448.0 / amax, 0.0)).to(E4M3)
    return codes, amax / torch.full_like(amax, 448.0)


def _norm(s):
    c = s["case"]
    t, k, kb = c["rows"], c["k"], -(-c["k"] // 128)
    y, kept = s["x"].float(), None
    if c["res"]:
        kept = (y + s["residual"].float()).to(T_OF[c["res"]])
        y = kept.float()
    if c["gain"]:
        y = y * torch.rsqrt(y.square().mean(1, keepdim=True) + s["eps"]) * s["gain"]
    res = dict(residual=kept, y=y.to(T_OF[c["y"]]) if c["y"] else None, codes=None, scales=None)
    if c["codes"]:
        blocks = torch.nn.functional.pad(y, (0, kb * 128 - k)).view(t, kb, 128)
        codes, scales = _quantise(blocks, (2,))
        res["codes"] = codes.view(t, kb * 128)[:, :k].contiguous()
        res["scales"] = scales[:, :, 0].T.contiguous()
    return res


def _pack(s):
    n, k = s["w"].shape
    nb, kb = -(-n // 128), -(-k // 128)
    blocks = torch.nn.functional.pad(s["w"].float(), (0, kb * 128 - k, 0, nb * 128 - n)).view(nb, 128, kb, 128)
    codes, scales = _quantise(blocks, (1, 3))
    return dict(codes=codes.view(nb * 128, kb * 128)[:n, :k].contiguous(), scales=scales[:, 0, :, 0].contiguous())


def _matmul(s):
    c = s["case"]
    t, n, k = c["rows"], c["n"], c["k"]
    a = s["codes"].float() * s["scales"][:, :t].T.repeat_interleave(128, dim=1)[:, :k]
    w = s["w_codes"].float() * s["w_scales"].repeat_interleave(128, dim=0)[:n].repeat_interleave(128, dim=1)[:, :k]
    out = torch.matmul(a, w.T)
    if c["add"]:
        out = out + s["add"].float()
    return dict(out=out.to(T_OF[c["out"]]))


_PLAIN = dict(norm=_norm, pack=_pack, matmul=_matmul)


# ------------------------------------------------------------------ the definition in 64 bits
def exact(case, seed):
    """Codes as what they round: the value over its block's scale."""
    s = prepare(case, seed)
    k = case["k"]
    edges = list(range(0, k, 128)) + [k]
    spans = list(zip(edges, edges[1:]))
    if case["op"] == "norm":
        y = s["x"].double()
        kept = None
        if case["res"]:
            y = y + s["residual"].double()
            kept = y
            y = y.to(T_OF[case["res"]]).double()  # (the stream is kept in its own type, and what is kept is normalised)
        if case["gain"]:
            y = y / torch.sqrt((y * y).sum(1, keepdim=True) / k + s["eps"]) * s["gain"].double()
        res = dict(residual=kept, y=y if case["y"] else None, codes=None, scales=None)
        if case["codes"]:
            scales = torch.stack([y[:, a:b].abs().amax(1) / 448.0 for a, b in spans])
            res["scales"] = scales
            res["codes"] = torch.cat([y[:, a:b] / scales[i][:, None] for i, (a, b) in enumerate(spans)], dim=1)
        return res
    if case["op"] == "pack":
        n, w = case["n"], s["w"]
        codes, scales = [], []
        for at in range(0, n, 128):
            part = w[at:at + 128].double()
            top = torch.stack([part[:, a:b].abs().max() for a, b in spans]) / 448.0
            scales.append(top)
            codes.append(part / top.repeat_interleave(128)[:k])
        return dict(codes=torch.cat(codes), scales=torch.stack(scales))
    t, n = case["rows"], case["n"]
    out = torch.zeros((t, n), dtype=torch.float64, device=DEV)
    w_scales = s["w_scales"].double()
    for i, (a, b) in enumerate(spans):
        rows = s["codes"][:, a:b].double() * s["scales"][i, :t].double()[:, None]
        weight = s["w_codes"][:, a:b].double() * w_scales[:, i].repeat_interleave(128)[:n, None]
        out.addmm_(rows, weight.T)
    return dict(out=out if s["add"] is None else out + s["add"].double())
