"""The 8-bit cache's operators in 64 bits, on the host, from their definitions (torch on the CPU; no GPU code).

Tolerances (each test says which it takes):
  * out: the 16-bit rounding of the result, half a step of the type relative to the value; plus the
    weights' rounding to fp16 on the way into the second product (half a step, 2^-11 of the sum of p|v|),
    plus 2^-14 of that sum for the scores' and the exponential's 32-bit errors: a score is a sum of at
    most 256 products in 32 bits, off by less than 2^-17 of A = sum |q k| sm_scale, and the tests keep A
    below 8 on average of the weight, plus a floor for fp16's smallest values.
  * lse: 2^-17 A + 2^-21 (1 + |lse|).
  * weights: 2^-16 A + 2^-20 relative to the sum of the weights.
"""
from __future__ import annotations

import math
from dataclasses import dataclass, field

import torch

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
CODE = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
Q = {"int8": 127.0, "e4m3": 448.0}


@dataclass
class Shape:
    heads: int
    kv: int
    dim: int
    page: int
    code: str = "int8"
    dtype: str = "bf16"


@dataclass
class Cache:
    """Host copies of a cache and a call's description; .to_gpu() gives device tensors of the same names."""
    shape: Shape
    n_pages: int
    n_slots: int
    lens: list
    news: list
    table: torch.Tensor = None
    slots: torch.Tensor = None
    t: dict = field(default_factory=dict)


def quantise(x: torch.Tensor, code: str):
    """x [..., P, D] 16-bit values of a page and head -> (codes, scale [...]) by the definition, in 32 bits."""
    x = x.float()
    amax = x.abs().amax((-2, -1), keepdim=True)
    q = torch.tensor(Q[code], dtype=torch.float32)
    live = amax >= 2.0 ** -100
    bad = ~torch.isfinite(x).all(-1, keepdim=True).all(-2, keepdim=True)
    inv = torch.where(live & ~bad, q / amax, torch.zeros(()))
    y = torch.where(bad, torch.zeros(()), x * inv)
    codes = y.round().to(torch.int8) if code == "int8" else y.to(torch.float8_e4m3fn)
    scale = torch.where(bad, torch.tensor(math.nan), torch.where(live, amax / q, torch.zeros(())))
    return codes, scale[..., 0, 0]


def make_cache(shape: Shape, lens, news, seed, spare_pages=3, spare_slots=2, empty=False, cols=None) -> Cache:
    """Random codes, scales and rings for sequences of `lens` tokens (pages and slots in a random order)."""
    g = torch.Generator().manual_seed(seed)
    B, P = len(lens), shape.page
    total = [l + (n if empty else 0) for l, n in zip(lens, news)]
    need = [t // P for t in total]
    cols = cols or max(need + [1])
    n_pages = sum(need) + spare_pages
    order = torch.randperm(n_pages, generator=g)
    c = Cache(shape, n_pages, B + spare_slots, list(lens), list(news))
    c.table = torch.full((B, cols), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        c.table[b, :n] = order[at:at + n].to(torch.int32)
        at += n
    c.slots = torch.randperm(B + spare_slots, generator=g)[:B].to(torch.int32)
    full = (n_pages, shape.kv, P, shape.dim)
    for w in "kv":
        x = torch.randn(full, generator=g) * 36
        if shape.code == "int8":
            c.t[w + "_codes"] = x.round().clamp(-127, 127).to(torch.int8)
        else:
            c.t[w + "_codes"] = (x * 3).clamp(-448, 448).to(torch.float8_e4m3fn)
        c.t[w + "_scale"] = 4.0 / Q[shape.code] * torch.exp(0.3 * torch.randn(full[:2], generator=g))
        c.t[w + "_tail"] = torch.randn((B + spare_slots, shape.kv, 2 * P, shape.dim), generator=g).to(DT[shape.dtype])
    return c


def starts(news):
    s = [0]
    for n in news:
        s.append(s[-1] + n)
    return s


def history(c: Cache, w: str, b: int) -> torch.Tensor:
    """K or V of sequence b's tokens in 64 bits: [len, Hkv, D]."""
    P, L = c.shape.page, c.lens[b]
    pages = c.table[b, : L // P].long()
    x = c.t[w + "_codes"].float()[pages].double() * c.t[w + "_scale"][pages].double()[..., None, None]
    x = x.transpose(1, 2).reshape(-1, c.shape.kv, c.shape.dim)
    rows = torch.arange(L // P * P, L) % (2 * P)
    return torch.cat([x, c.t[w + "_tail"][int(c.slots[b])][:, rows].double().transpose(0, 1)])


def attend(c: Cache, q: torch.Tensor, sm: float):
    """out, lse, and what the tolerances go by: S = sum p|v| and A = sum p sum |q k| sm, for q [T, H, D]."""
    sh = c.shape
    G, T = sh.heads // sh.kv, q.shape[0]
    out = torch.zeros((T, sh.heads, sh.dim), dtype=torch.float64)
    lse = torch.full((T, sh.heads), -math.inf, dtype=torch.float64)
    S, A = torch.zeros_like(out), torch.zeros_like(lse)
    row = 0
    for b, n in enumerate(c.news):
        k, v = history(c, "k", b), history(c, "v", b)
        for i in range(n):
            see = c.lens[b] - n + i + 1
            if see > 0:
                qq = q[row].double().view(sh.kv, G, sh.dim)
                z = torch.einsum("hgd,thd->hgt", qq, k[:see]) * sm
                p = torch.softmax(z, 2)
                out[row] = torch.einsum("hgt,thd->hgd", p, v[:see]).reshape(sh.heads, sh.dim)
                S[row] = torch.einsum("hgt,thd->hgd", p, v[:see].abs()).reshape(sh.heads, sh.dim)
                lse[row] = torch.logsumexp(z, 2).reshape(-1)
                a = torch.einsum("hgd,thd->hgt", qq.abs(), k[:see].abs()) * sm
                A[row] = a.amax(2).reshape(-1)
            row += 1
    return out, lse, S, A


def weigh(c: Cache, q, lse, acc, decay, sm):
    """acc after the call, and the relative tolerance's A (the largest sum |q k| sm of the call)."""
    sh = c.shape
    G = sh.heads // sh.kv
    res = torch.zeros((len(c.lens), sh.kv, max(c.lens + [1])), dtype=torch.float64)
    row, A = 0, 0.0
    for b, n in enumerate(c.news):
        k = history(c, "k", b)
        old = max(0, c.lens[b] - n)
        if acc is not None:
            res[b, :, :old] += decay * acc[b, :, :old].double()
        for i in range(n):
            see = c.lens[b] - n + i + 1
            if see > 0:
                qq = q[row].double().view(sh.kv, G, sh.dim)
                z = torch.einsum("hgd,thd->hgt", qq, k[:see]) * sm
                A = max(A, float((torch.einsum("hgd,thd->hgt", qq.abs(), k[:see].abs()) * sm).max()))
                res[b, :, :see] += torch.exp(z - lse[row].double().view(sh.kv, G, 1)).sum(1)
            row += 1
    return res, A


def keep_pages(acc, length, page, budget, sink, recent):
    """The page numbers that one kv head keeps, for its sums acc [tokens] (64 bits, ties to the lower page)."""
    full = length // page
    score = acc[: full * page].double().reshape(full, page).sum(1).tolist()
    must = [j for j in range(full) if j < sink or j >= full - recent]
    if full <= budget:
        return list(range(full))
    rest = [j for j in range(full) if j not in set(must)]
    rest.sort(key=lambda j: (-(math.inf if math.isnan(score[j]) else score[j]), j))
    return sorted(must + rest[: budget - len(must)])
