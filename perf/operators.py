"""Measured cases of the 8-bit paged cache's operators: append, read, attend, weigh, evict.

A sequence's tokens lie in pages of P tokens, all kv heads' [P][D] codes (int8 or e4m3) of K and of V with one fp32 scale for each
page and head.  The last, unfinished page of a sequence is held in 16 bits in a ring of 2P rows (token t in row t mod 2P).

  append  new K and V rows of the unfinished page and of the one before go into the ring; a page whose last token arrives is quantised:
          scale = amax / Q, code = round(x * fp32(Q / amax)), Q = 127 (int8) or 448 (e4m3)
  read    pages back as 16-bit values, code * scale
  attend  causal attention of each sequence's last n tokens over its cache; the outputs and the rows' log-sum-exp
  weigh   each cached token's attention weight, summed over the rows of its kv head, added to decay * the earlier sum
  evict   each kv head keeps its pages of the largest summed weight (with the first and the latest ones), moved to new pages

`own` chooses between elementary torch operations and the framework's kernels.
"""
import math
import random

import torch

own = False

Q_OF = {"int8": 127.0, "e4m3": 448.0}
T_OF = {"bf16": torch.bfloat16, "f16": torch.float16}
C_OF = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one user's next token completes a page: the smallest call of the decode loop, all latency
        dict(name="append-token", op="append", dtype="bf16", code="int8", seqs=1, heads=32, kv=4, dim=128, page=64,
             old_lo=1023, old_hi=1023, new_lo=1, new_hi=1, key=1),
        # a batch of ragged prompts enters an empty cache
        dict(name="append-prompts", op="append", dtype="f16", code="e4m3", seqs=5, heads=32, kv=8, dim=128, page=32,
             old_lo=0, old_hi=0, new_lo=1500, new_hi=7001, key=2),
        # one user's next token over a short chat: latency
        dict(name="attend-token", op="attend", dtype="bf16", code="int8", seqs=1, heads=32, kv=4, dim=128, page=64,
             old_lo=1000, old_hi=1000, new_lo=1, new_hi=1, key=3),
        # a serving batch's decode step, ragged lengths
        dict(name="attend-batch", op="attend", dtype="bf16", code="int8", seqs=64, heads=32, kv=8, dim=128, page=64,
             old_lo=200, old_hi=16300, new_lo=1, new_hi=1, key=4),
        # few users with very long documents: one row group per head, the work lies along the keys
        dict(name="attend-long", op="attend", dtype="f16", code="e4m3", seqs=2, heads=64, kv=8, dim=64, page=16,
             old_lo=90000, old_hi=131071, new_lo=1, new_hi=1, key=5),
        # verification of drafted tokens: a few query tokens for each sequence, wide heads
        dict(name="attend-verify", op="attend", dtype="bf16", code="e4m3", seqs=24, heads=16, kv=8, dim=256, page=32,
             old_lo=300, old_hi=6000, new_lo=2, new_hi=6, key=6),
        # two whole prompts, causal
        dict(name="attend-prompts", op="attend", dtype="bf16", code="int8", seqs=2, heads=32, kv=4, dim=128, page=64,
             old_lo=0, old_hi=0, new_lo=2900, new_hi=4097, key=7),
        # one chunk of a long prompt over what is in the cache already
        dict(name="attend-chunk", op="attend", dtype="f16", code="e4m3", seqs=1, heads=32, kv=8, dim=128, page=32,
             old_lo=24000, old_hi=24000, new_lo=1024, new_hi=1024, key=8),
        # the weights of one decode step over a serving batch
        dict(name="weigh-step", op="weigh", dtype="bf16", code="int8", seqs=32, heads=32, kv=8, dim=128, page=64,
             old_lo=500, old_hi=9000, new_lo=1, new_hi=1, key=9),
        # the weights that a prompt's last tokens give its earlier ones
        dict(name="weigh-window", op="weigh", dtype="f16", code="e4m3", seqs=4, heads=32, kv=4, dim=128, page=16,
             old_lo=9000, old_hi=16000, new_lo=64, new_hi=64, key=10),
        # one user's cache goes back to its budget: latency
        dict(name="evict-one", op="evict", dtype="bf16", code="int8", seqs=1, heads=32, kv=4, dim=128, page=32,
             old_lo=1500, old_hi=1500, new_lo=1, new_hi=1, key=11, budget=24, sink=1, recent=4),
        # a batch of long caches to a quarter of their length
        dict(name="evict-batch", op="evict", dtype="f16", code="e4m3", seqs=8, heads=32, kv=8, dim=128, page=64,
             old_lo=20000, old_hi=32700, new_lo=1, new_hi=1, key=12, budget=128, sink=1, recent=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append-step", "append-prompt", "attend-step", "attend-step", "attend-step", "attend-verify",
                       "attend-prompt", "attend-prompt", "attend-chunk", "weigh-step", "weigh-window", "evict"])
    op = kind.split("-")[0]
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128, 128, 256] if kind in ("append-step", "attend-step", "attend-verify", "evict") else [64, 128])
    c = dict(op=op, dtype=rng.choice(["bf16", "f16"]), code=rng.choice(["int8", "e4m3"]), kv=kv,
             heads=kv * rng.choice([1, 2, 4, 5, 8]), dim=dim, page=rng.choice([16, 32, 64]), key=rng.randrange(1 << 20))
    if kind == "append-step":
        new = rng.choice([1, 1, 1, 2, 5])
        c.update(seqs=_log(rng, 1, 128), old_lo=rng.randrange(0, 200), old_hi=_log(rng, 200, 4000), new_lo=1, new_hi=new)
    elif kind == "append-prompt":
        hi = _log(rng, 100, 8000)
        c.update(seqs=rng.randrange(1, 6), old_lo=0, old_hi=0, new_lo=max(1, hi // 3), new_hi=hi)
    elif kind == "attend-step":
        hi = _log(rng, 30, 100000)
        most = max(1, min(128, (1 << 29) // (hi * kv * dim)))
        c.update(seqs=_log(rng, 1, most), old_lo=max(1, hi // rng.choice([1, 3, 20])), old_hi=hi, new_lo=1, new_hi=1)
    elif kind == "attend-verify":
        hi = _log(rng, 50, 12000)
        most = max(1, min(64, (1 << 28) // (hi * kv * dim)))
        c.update(seqs=_log(rng, 1, most), old_lo=max(1, hi // 4), old_hi=hi, new_lo=rng.randrange(1, 4), new_hi=rng.randrange(4, 12))
    elif kind == "attend-prompt":
        hi = _log(rng, 60, 3300)
        c.update(seqs=rng.randrange(1, 3), old_lo=0, old_hi=0, new_lo=max(1, hi // 2), new_hi=hi)
    elif kind == "attend-chunk":
        hi = _log(rng, 100, 24000)
        new = _log(rng, 40, max(60, min(800, 80_000_000_000 // (hi * c["heads"] * dim))))
        c.update(seqs=1, old_lo=hi, old_hi=hi, new_lo=new, new_hi=new)
    elif kind == "weigh-step":
        hi = _log(rng, 100, 16000)
        most = max(1, min(64, (1 << 28) // (hi * kv * dim)))
        c.update(seqs=_log(rng, 1, most), old_lo=max(1, hi // 4), old_hi=hi, new_lo=1, new_hi=rng.randrange(1, 5))
    elif kind == "weigh-window":
        hi = _log(rng, 500, 14000)
        c.update(seqs=rng.randrange(1, 5), old_lo=hi // 2, old_hi=hi, new_lo=32, new_hi=64)
    else:
        hi = _log(rng, 1000, 20000)
        pages = hi // c["page"]
        recent = rng.randrange(1, 1 + max(1, pages // 16))
        most = max(1, min(8, 90_000_000 // (hi * kv * dim)))
        c.update(seqs=rng.randrange(1, 1 + most), old_lo=hi // 2, old_hi=hi, new_lo=1, new_hi=1, sink=rng.randrange(0, 2), recent=recent,
                 budget=max(recent + 2, int(pages * rng.uniform(0.15, 0.7))))
    return c


def _lens(case):
    """Tokens of each sequence before the call, and its new ones: by the case alone.  The last sequence has the largest of both."""
    r = random.Random(case["key"])
    n, P = case["seqs"], case["page"]
    old = [r.randint(case["old_lo"], case["old_hi"]) for _ in range(n - 1)] + [case["old_hi"]]
    new = [r.randint(case["new_lo"], case["new_hi"]) for _ in range(n - 1)] + [case["new_hi"]]
    if case["op"] == "append" and case["old_hi"]:  # the last one's new tokens complete a page
        old[-1] += (P - 1 - old[-1]) % P
    return old, new


def work(case):
    old, new = _lens(case)
    Hk, H, D, P = case["kv"], case["heads"], case["dim"], case["page"]
    T, row = sum(new), Hk * D
    total = [a + b for a, b in zip(old, new)]
    seen = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, total))  # visible keys, summed over query tokens
    codes = sum(t // P * P * row + t % P * row * 2 for t in total)          # K, or V, as it lies in the cache
    op = case["op"]
    if op == "append":
        done = sum((t // P - a // P) * P for a, t in zip(old, total))
        ring = sum((a % P) * row for a, t in zip(old, total) if t // P > a // P)
        tail = sum(min(n, t % P + P) * row for n, t in zip(new, total))
        return {"bytes": 2 * (2 * T * row + 2 * ring + done * row + 2 * tail) + 2 * done * row * 3, "flops": 4 * done * row}
    if op == "attend":
        return {"bytes": 2 * codes + 2 * 2 * T * H * D + 4 * T * H, "flops": 4 * D * H * seen}
    if op == "weigh":
        return {"bytes": codes + 2 * T * H * D + 4 * T * H + 8 * Hk * sum(total), "flops": 2 * D * H * seen}
    kept = sum(min(case["budget"], t // P) for t in total) * P
    tail = sum(t % P for t in total)
    return {"bytes": 4 * Hk * (sum(total) + 2 * kept) + 4 * kept * row + 8 * tail * row + 2 * kept * row * 3,
            "flops": Hk * sum(total) + 2 * kept * row}


# ------------------------------------------------------------------ inputs
def _codes(g, code, shape):
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float16)
    if code == "int8":
        return x.mul_(36.0).round_().clamp_(-127, 127).to(torch.int8)
    return x.mul_(110.0).clamp_(-448, 448).to(torch.float8_e4m3fn)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    old, new = _lens(case)
    B, H, Hk, D, P = case["seqs"], case["heads"], case["kv"], case["dim"], case["page"]
    dt, Q = T_OF[case["dtype"]], Q_OF[case["code"]]
    total = [a + b for a, b in zip(old, new)]
    T = sum(new)
    cols = max(total) // P + 1
    budget = case.get("budget", 0)
    held = sum(t // P + 1 for t in total)
    n_pages = held + B * budget + 3
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, cols), -1, dtype=torch.int32)
    at = 0
    for b, t in enumerate(total):
        table[b, : t // P + 1] = torch.arange(at, at + t // P + 1, dtype=torch.int32)
        at += t // P + 1
    named = table >= 0
    table = torch.where(named.to(DEV), order[table.clamp(min=0).to(DEV).long()], -1).to(torch.int32).contiguous()

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEV)

    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    s = dict(case=dict(case), B=B, T=T, max_new=max(new), max_len=max(total), full=max(total) // P, table=table,
             q_start=ints(starts), old_lens=ints(old), lens=ints(total), sm=1.0 / math.sqrt(D))
    s["slots"] = torch.randperm(2 * B + 1, generator=g, device=DEV)[:B].to(torch.int32)
    if case["op"] == "append":
        s["k_codes"] = torch.zeros((n_pages, Hk, P, D), dtype=C_OF[case["code"]], device=DEV)
        s["v_codes"] = torch.zeros_like(s["k_codes"])
        s["k_scale"] = torch.zeros((n_pages, Hk), device=DEV)
        s["v_scale"] = torch.zeros((n_pages, Hk), device=DEV)
    else:
        s["k_codes"] = _codes(g, case["code"], (n_pages, Hk, P, D))
        s["v_codes"] = _codes(g, case["code"], (n_pages, Hk, P, D))
        amp = 4.0 / Q  # a page's largest value is about four times its spread
        s["k_scale"] = amp * torch.exp(0.2 * torch.randn((n_pages, Hk), generator=g, device=DEV))
        s["v_scale"] = amp * torch.exp(0.2 * torch.randn((n_pages, Hk), generator=g, device=DEV))
    s["k_tail"] = torch.randn((2 * B + 1, Hk, 2 * P, D), generator=g, device=DEV).to(dt)
    s["v_tail"] = torch.randn((2 * B + 1, Hk, 2 * P, D), generator=g, device=DEV).to(dt)
    # the projections' output: query, key and value heads side by side, so that each of the three is a strided view
    channel = torch.exp(0.5 * torch.randn((H + 2 * Hk, D), generator=g, device=DEV))
    channel[:H] = 1.2
    qkv = (torch.randn((T, H + 2 * Hk, D), generator=g, device=DEV) * channel).to(dt)
    s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hk], qkv[:, H + Hk:]
    if case["op"] == "append":
        done = [table[b, a // P:(a + n) // P] for b, (a, n) in enumerate(zip(old, new))]
        s["done"] = torch.cat(done).contiguous()
    if case["op"] == "weigh":
        s["lse"] = _attend(s)["lse"]
        s["decay"] = 0.875
        s["acc"] = torch.rand((B, Hk, cols * P), generator=g, device=DEV) * 0.01
        live = torch.arange(cols * P, device=DEV)[None, :] < s["lens"][:, None]
        s["acc"] *= live[:, None, :]
    if case["op"] == "evict":
        heavy = torch.randn((B, Hk, cols), generator=g, device=DEV).exp().repeat_interleave(P, dim=2)
        s["acc"] = torch.rand((B, Hk, cols * P), generator=g, device=DEV) * heavy
        s["new_table"] = order[held:held + B * budget].reshape(B, budget).contiguous()
        s["new_slots"] = ((s["slots"] + B + 1) % (2 * B + 1)).to(torch.int32) if B == 1 else _others(s["slots"], 2 * B + 1)
        kept = [min(t // P, budget) for t in total]
        s["done"] = torch.cat([s["new_table"][b, :n] for b, n in enumerate(kept)]).contiguous()
    if own:
        _handles(s)
    return s


def _others(slots, n):
    """As many tail slots that `slots` does not name."""
    free = torch.ones(n, dtype=torch.bool, device=slots.device)
    free[slots.long()] = False
    return torch.nonzero(free)[: slots.numel(), 0].to(torch.int32)


def _handles(s):
    """What a program that uses the framework keeps: the plan, the scratch, the descriptions of its buffers, and outputs."""
    from quantized_moe_expert_gemv_gb300 import binding as si

    c = s["case"]
    B, H, Hk, D, P = c["seqs"], c["heads"], c["kv"], c["dim"], c["page"]
    s["si"] = si
    si.load_library()
    plan = s["plan"] = si.si_kv_plan(si.make_kv_desc(H, Hk, D, P, code=c["code"], dtype=c["dtype"]), 0)
    s["cache"] = si.kv_cache(s["k_codes"], s["v_codes"], s["k_scale"], s["v_scale"], s["k_tail"], s["v_tail"])
    before = s["old_lens"] if c["op"] == "append" else s["lens"]
    s["batch"] = si.kv_batch(B, s["T"], s["max_new"], s["max_len"], s["q_start"], before, s["table"], s["slots"])
    size = si.si_kv_scratch_bytes(plan, B, s["T"], s["max_new"], s["max_len"])
    s["scratch"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    si.si_kv_scratch_init(plan, s["scratch"])
    dt = T_OF[c["dtype"]]
    if c["op"] in ("append", "evict"):
        n = s["done"].numel()
        s["k_read"] = torch.empty((n, Hk, P, D), dtype=dt, device=DEV)
        s["v_read"] = torch.empty((n, Hk, P, D), dtype=dt, device=DEV)
        s["lens_out"] = torch.empty(B, dtype=torch.int32, device=DEV)
    if c["op"] == "attend":
        s["out"] = torch.empty((s["T"], H, D), dtype=dt, device=DEV)
        s["lse_out"] = torch.empty((s["T"], H), device=DEV)
    if c["op"] in ("weigh", "evict"):
        s["acc_out"] = torch.zeros_like(s["acc"])
    if c["op"] == "evict":
        s["keep"] = torch.empty((B, Hk, c["budget"]), dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return _PLAIN[op](state)


def _own_append(s):
    si, plan, scratch = s["si"], s["plan"], s["scratch"]
    si.si_kv_append(plan, s["cache"], s["batch"], s["k"], s["v"], s["lens_out"], scratch)
    si.si_kv_read(plan, s["cache"], s["done"], s["done"].numel(), s["k_read"], s["v_read"], scratch)
    return dict(k=s["k_read"], v=s["v_read"], k_tail=s["k_tail"], v_tail=s["v_tail"], lens=s["lens_out"])


def _own_attend(s):
    s["si"].si_kv_attend(s["plan"], s["cache"], s["batch"], s["q"], s["out"], s["lse_out"], s["sm"], s["scratch"])
    return dict(out=s["out"], lse=s["lse_out"])


def _own_weigh(s):
    s["si"].si_kv_weigh(s["plan"], s["cache"], s["batch"], s["q"], s["lse"], s["acc"], s["acc_out"], s["decay"], s["sm"],
                        s["scratch"])
    return dict(acc=s["acc_out"])


def _own_evict(s):
    si, plan, scratch, c = s["si"], s["plan"], s["scratch"], s["case"]
    si.si_kv_evict(plan, s["cache"], s["batch"], s["acc"], s["acc_out"], c["budget"], c["sink"], c["recent"], s["new_table"],
                   s["new_slots"], s["keep"], s["lens_out"], scratch)
    si.si_kv_read(plan, s["cache"], s["done"], s["done"].numel(), s["k_read"], s["v_read"], scratch)
    return dict(k=s["k_read"], v=s["v_read"], k_tail=s["k_tail"], v_tail=s["v_tail"], keep=s["keep"], lens=s["lens_out"],
                acc=s["acc_out"])


_OWN = dict(append=_own_append, attend=_own_attend, weigh=_own_weigh, evict=_own_evict)


# ---- the plain forms
def _rows(s):
    """(sequence, index in it) of each row of q, k and v."""
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    b = torch.repeat_interleave(torch.arange(s["B"], device=DEV), n, output_size=s["T"])
    return b, torch.arange(s["T"], device=DEV) - s["q_start"].long()[b]


def _tokens(s, which):
    """K or V of every token in 32 bits: [B, Hkv, tokens padded to the longest, D]."""
    c = s["case"]
    P, n = c["page"], s["full"]
    pages = s["table"][:, :n].clamp(min=0).long()
    x = s[which + "_codes"].view(torch.int8)[pages].view(C_OF[c["code"]]).float() * s[which + "_scale"][pages][..., None, None]
    x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, 0, 0, 1)).transpose(1, 2).reshape(s["B"], c["kv"], (n + 1) * P, c["dim"])
    at = (s["lens"].long() // P * P)[:, None] + torch.arange(P, device=DEV)  # the tokens of the unfinished page
    b = torch.arange(s["B"], device=DEV)[:, None]
    x[b, :, at] = s[which + "_tail"][s["slots"].long()[:, None], :, at % (2 * P)].float()
    return x


def _scores(s):
    """Scores [B, Hkv, G * max_new, tokens] in 32 bits, -inf where a row does not see a token (and in rows that pad)."""
    c = s["case"]
    B, Hk, G, D, N = s["B"], c["kv"], c["heads"] // c["kv"], c["dim"], s["max_new"]
    b, i = _rows(s)
    q = torch.zeros((B, N, Hk, G, D), device=DEV)
    q[b, i] = s["q"].float().reshape(s["T"], Hk, G, D)
    q = q.permute(0, 2, 3, 1, 4).reshape(B, Hk, G * N, D)
    z = torch.matmul(q, _tokens(s, "k").transpose(2, 3)).mul_(s["sm"])
    n = (s["q_start"][1:] - s["q_start"][:-1]).long()
    row = torch.arange(N, device=DEV)
    last = (s["lens"].long() - n)[:, None] + row                       # the last token that a row sees
    see = (torch.arange(z.shape[3], device=DEV) <= last[..., None]) & (row < n[:, None])[..., None]
    return z.view(B, Hk, G, N, -1).masked_fill_(~see[:, None, None], -math.inf).view(z.shape), b, i


def _attend(s):
    c = s["case"]
    B, Hk, G, D, N = s["B"], c["kv"], c["heads"] // c["kv"], c["dim"], s["max_new"]
    z, b, i = _scores(s)
    m = z.amax(3, keepdim=True)
    p = z.sub_(m.clamp(min=-1e30)).exp_()
    total = p.sum(3, keepdim=True)
    out = torch.matmul(p, _tokens(s, "v")) / total.clamp(min=1e-30)
    lse = m + total.log()
    out = out.view(B, Hk, G, N, D).permute(0, 3, 1, 2, 4)[b, i].reshape(s["T"], c["heads"], D)
    lse = lse.view(B, Hk, G, N).permute(0, 3, 1, 2)[b, i].reshape(s["T"], c["heads"])
    return dict(out=out.to(T_OF[c["dtype"]]), lse=lse)


def _weigh(s):
    c = s["case"]
    B, Hk, G, N = s["B"], c["kv"], c["heads"] // c["kv"], s["max_new"]
    z, b, i = _scores(s)
    lse = torch.zeros((B, N, Hk, G), device=DEV)
    lse[b, i] = s["lse"].reshape(s["T"], Hk, G)
    w = z.sub_(lse.permute(0, 2, 3, 1).reshape(B, Hk, G * N, 1)).exp_().sum(2)
    t = torch.arange(s["acc"].shape[2], device=DEV)
    n = s["q_start"][1:] - s["q_start"][:-1]
    earlier = t < (s["lens"] - n)[:, None]
    return dict(acc=(s["acc"] * s["decay"] * earlier[:, None] + w) * (t < s["lens"][:, None])[:, None])


def _append(s):
    c = s["case"]
    P, Q, dt = c["page"], Q_OF[c["code"]], T_OF[c["dtype"]]
    b, i = _rows(s)
    slot, at = s["slots"].long(), s["old_lens"].long()
    pos = at[b] + i
    first = at // P                                                   # the page that the call begins in
    last = s["lens"].long() // P
    n = int(s["max_new"] + P - 1) // P + 1
    res = dict(lens=s["old_lens"] + (s["q_start"][1:] - s["q_start"][:-1]))
    whole = torch.arange(n, device=DEV) < (last - first)[:, None]     # the pages that the call completes
    for which in ("k", "v"):
        new, tail = s[which], s[which + "_tail"].clone()
        x = torch.zeros((s["B"], n * P, c["kv"], c["dim"]), dtype=dt, device=DEV)
        before = first[:, None] * P + torch.arange(P, device=DEV)
        x[:, :P] = tail[slot[:, None], :, before % (2 * P)]
        x[b, pos - first[b] * P] = new
        x = x.view(s["B"], n, P, c["kv"], c["dim"]).transpose(2, 3).float()
        amax = x.abs().amax((3, 4), keepdim=True)
        codes = x * torch.where(amax >= 2.0 ** -100, Q / amax, 0.0)
        codes = codes.round() if c["code"] == "int8" else codes.to(torch.float8_e4m3fn).float()
        res[which] = (codes * (amax / torch.full_like(amax, Q))).to(dt)[whole]
        keep = pos >= (last[b] - 1) * P                               # the unfinished page's tokens and the page's before
        tail[slot[b[keep]], :, pos[keep] % (2 * P)] = new[keep]
        res[which + "_tail"] = tail
    return res


def _evict(s):
    c = s["case"]
    B, Hk, P, n, dt = s["B"], c["kv"], c["page"], s["full"], T_OF[c["dtype"]]
    full = (s["lens"].long() // P)[:, None, None]
    j = torch.arange(n, device=DEV)
    score = s["acc"][:, :, : n * P].double().view(B, Hk, n, P).sum(3)
    score = score.masked_fill((j < c["sink"]) | (j >= full - c["recent"]), math.inf).masked_fill(j >= full, -math.inf)
    best = torch.sort(score, dim=2, descending=True, stable=True).indices
    count = full.clamp(max=c["budget"])
    best = torch.where(j < count, best, n)[:, :, : c["budget"]].sort(2).values
    best = torch.nn.functional.pad(best, (0, c["budget"] - best.shape[2]), value=n)
    kept = best < n
    src = s["table"][:, :n].long()[:, None].expand(B, Hk, n).gather(2, best.clamp(max=n - 1)).clamp(min=0)
    head = torch.arange(Hk, device=DEV)[None, :, None]
    lens = (count[:, 0, 0] * P + s["lens"].long() % P)
    acc = s["acc"][:, :, : n * P].view(B, Hk, n, P).gather(2, best.clamp(max=n - 1)[..., None].expand(-1, -1, -1, P))
    acc = torch.nn.functional.pad((acc * kept[..., None]).flatten(2), (0, max(0, s["acc"].shape[2] - c["budget"] * P)))[:, :, : s["acc"].shape[2]].clone()
    row = torch.arange(P, device=DEV)
    left = row < (s["lens"] % P)[:, None]                             # the unfinished page's tokens
    bs = torch.arange(B, device=DEV)[:, None].expand(B, P)[left]
    was, now = (full[:, 0] * P + row)[left], (count[:, 0] * P + row)[left]
    acc[bs, :, now] = s["acc"][bs, :, was]
    res = dict(keep=torch.where(kept, best, -1).to(torch.int32), lens=lens.to(torch.int32), acc=acc)
    live = kept[:, 0]
    for which in ("k", "v"):
        x = s[which + "_codes"].view(torch.int8)[src, head].view(C_OF[c["code"]]).float() * s[which + "_scale"][src, head][..., None, None]
        res[which] = x.to(dt).transpose(1, 2)[live]
        tail = s[which + "_tail"].clone()
        tail[s["new_slots"].long()[bs], :, now % (2 * P)] = s[which + "_tail"][s["slots"].long()[bs], :, was % (2 * P)]
        res[which + "_tail"] = tail
    return res


_PLAIN = dict(append=_append, attend=_attend, weigh=_weigh, evict=_evict)


# ------------------------------------------------------------------ the definition in 64 bits
def _history(s, which, b, h):
    """K or V of one sequence's tokens for one kv head, in 64 bits."""
    c = s["case"]
    P, length = c["page"], int(s["lens"][b])
    pages = s["table"][b, : length // P].long()
    codes = s[which + "_codes"].view(torch.int8)[pages, h].view(C_OF[c["code"]]).to(torch.float32).double()
    x = (codes * s[which + "_scale"][pages, h].double()[:, None, None]).reshape(-1, c["dim"])
    t = torch.arange(length // P * P, length, device=DEV) % (2 * P)
    return torch.cat([x, s[which + "_tail"][int(s["slots"][b]), h][t].double()])


def exact(case, seed):
    s = prepare(case, seed)
    old, new = _lens(case)
    Hk, G, D, P, dt = case["kv"], case["heads"] // case["kv"], case["dim"], case["page"], T_OF[case["dtype"]]
    op = case["op"]
    if op in ("attend", "weigh"):
        out = torch.zeros((s["T"], Hk, G, D), dtype=torch.float64, device=DEV)
        lse = torch.zeros((s["T"], Hk, G), dtype=torch.float64, device=DEV)
        acc = s["acc"].double() * 0 if op == "weigh" else None
        first = 0
        for b, (a, n) in enumerate(zip(old, new)):
            rows = slice(first, first + n)
            first += n
            hidden = torch.arange(a + n, device=DEV)[None, :] > (a + torch.arange(n, device=DEV))[:, None]
            for h in range(Hk):
                k = _history(s, "k", b, h)
                q = s["q"][rows, h * G:(h + 1) * G].double()
                z = torch.einsum("igd,td->git", q, k) * s["sm"]
                z[:, hidden] = -math.inf
                if op == "weigh":
                    w = (z - s["lse"][rows, h * G:(h + 1) * G].double().T[..., None]).exp().sum((0, 1))
                    w[:a] += s["decay"] * s["acc"][b, h, :a].double()
                    acc[b, h, : a + n] = w
                else:
                    lse[rows, h] = torch.logsumexp(z, 2).T
                    out[rows, h] = torch.einsum("git,td->igd", torch.softmax(z, 2), _history(s, "v", b, h))
        if op == "weigh":
            return dict(acc=acc)
        return dict(out=out.reshape(s["T"], Hk * G, D), lse=lse.reshape(s["T"], Hk * G))
    res = {}
    for which in ("k", "v"):
        pages = []
        if op == "append":
            first = 0
            for b, (a, n) in enumerate(zip(old, new)):
                tail = s[which + "_tail"][int(s["slots"][b])]
                at = torch.arange(a // P * P, a, device=DEV) % (2 * P)
                x = torch.cat([tail[:, at].transpose(0, 1), s[which][first:first + n]]).double()
                first += n
                for j in range((a + n) // P - a // P):
                    y = x[j * P:(j + 1) * P].transpose(0, 1)
                    top = y.abs().amax((1, 2), keepdim=True)
                    codes = y * (Q_OF[case["code"]] / top)
                    codes = codes.round() if case["code"] == "int8" else codes.float().to(torch.float8_e4m3fn).double()
                    pages.append(codes * top / Q_OF[case["code"]])
        else:
            keep = _kept(s)
            for b, n in enumerate(new):
                for j in range(len(keep[b][0])):
                    page = []
                    for h in range(Hk):
                        at = keep[b][h][j] * P
                        page.append(_history_page(s, which, b, h, at // P))
                    pages.append(torch.stack(page))
        res[which] = torch.stack(pages) if pages else None
        res[which + "_tail"] = None
    if op == "evict":
        res.update(keep=None, lens=None, acc=None)
    else:
        res.update(lens=None)
    return res


def _history_page(s, which, b, h, j):
    page = int(s["table_host"][b][j])
    return s[which + "_codes"][page, h].to(torch.float32).double() * s[which + "_scale"][page, h].double()


def _kept(s):
    """The pages that each sequence's kv heads keep: lists, by the definition."""
    if "kept" in s:
        return s["kept"]
    c = s["case"]
    P, acc = c["page"], s["acc"].double().cpu()
    s["table_host"] = s["table"].cpu().tolist()
    s["kept"] = []
    for b, length in enumerate(s["lens"].cpu().tolist()):
        full = length // P
        heads = []
        for h in range(c["kv"]):
            score = acc[b, h, : full * P].reshape(full, P).sum(1).tolist()
            must = [j for j in range(full) if j < c["sink"] or j >= full - c["recent"]]
            rest = sorted((j for j in range(full) if j not in set(must)), key=lambda j: (-score[j], j))
            heads.append(sorted(must + rest[: max(0, min(full, c["budget"]) - len(must))]))
        s["kept"].append(heads)
    return s["kept"]
