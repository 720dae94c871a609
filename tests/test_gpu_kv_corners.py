"""The 8-bit cache's operators where they can go wrong: empty rows, extreme values, loose bounds, broken neighbours."""
import math

import pytest
import torch

from quantized_moe_expert_gemv_gb300 import binding as si
import kv_reference as ref
from kv_reference import Shape
from test_gpu_kv import DEV, Dev, check_attend, make_q, run_evict

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ weigh
@pytest.mark.parametrize("code,dim,place", [("int8", 128, (63,)), ("e4m3", 64, (0,)), ("int8", 64, (31, 40)), ("e4m3", 128, (5, 6, 62))])
def test_weigh_a_window_among_sequences_without_rows(code, dim, place):
    """Sequences that only decay beside ones with a window of rows: a CTA takes several of the former in a row."""
    shape = Shape(16, 8, dim, 32, code, "bf16")
    lens = [100 + 7 * (b % 13) for b in range(64)]
    news = [64 if b in place else 0 for b in range(64)]
    c = ref.make_cache(shape, lens, news, seed=7)
    d = Dev(c)
    q, qd = make_q(c, 6)
    sm = dim ** -0.5
    _, lse, _, _ = ref.attend(c, q, sm)
    lse = lse.float()
    acc = torch.rand((64, 8, max(lens)), generator=torch.Generator().manual_seed(1))
    want, A = ref.weigh(c, q, lse, acc, 0.75, sm)
    for _ in range(20):
        out = torch.full_like(acc, 9.0).to(DEV)
        si.si_kv_weigh(d.plan, d.cache, d.batch, qd, lse.to(DEV), acc.to(DEV), out, 0.75, sm, d.scratch)
        assert d.status() == si.SI_OK
        got = out.cpu().double()
        for b, L in enumerate(lens):
            w = want[b, :, :L]
            assert ((got[b, :, :L] - w).abs() <= (2.0 ** -16 * A + 2.0 ** -19) * w + 1e-12).all(), b
            assert (got[b, :, L:] == 9.0).all()


# ------------------------------------------------------------------ loose bounds
def test_append_with_a_loose_bound():
    """max_new only bounds: the largest number completes the same pages as the exact one."""
    shape = Shape(4, 2, 64, 16, "int8", "bf16")
    g = torch.Generator().manual_seed(4)
    kv = torch.randn((140, 4, 64), generator=g).to(torch.bfloat16).to(DEV)
    res = []
    for most in (100, 2 ** 31 - 1):
        c = ref.make_cache(shape, [5, 60], [100, 40], seed=8, empty=True)
        d = Dev(c, max_len=110, max_new=most)
        out = torch.empty_like(d.lens)
        si.si_kv_append(d.plan, d.cache, d.batch, kv[:, :2], kv[:, 2:], out, d.scratch)
        assert out.tolist() == [105, 100] and d.status() == si.SI_OK
        res.append([d.k_codes, d.v_codes, d.k_scale, d.v_scale, d.k_tail.view(torch.int16), d.v_tail.view(torch.int16)])
    assert all(torch.equal(x, y) for x, y in zip(*res))


@pytest.mark.parametrize("lens,news", [([300, 90], [100, 40]), ([300, 90], [2, 1])], ids=["prompt", "step"])
def test_attend_and_weigh_with_a_loose_bound(lens, news):
    """The same outputs where max_new says no more than that a sequence may have all rows, or any number."""
    shape = Shape(8, 2, 64, 16, "int8", "bf16")
    c = ref.make_cache(shape, lens, news, seed=8)
    q, qd = make_q(c, 3)
    for most in (sum(news), 2 ** 31 - 1):
        d = Dev(c, max_new=most)
        out, lse = d.attend(qd, 0.125)
        check_attend(c, out, lse, q, 0.125)
        acc = torch.zeros((2, 2, 300), device=DEV)
        si.si_kv_weigh(d.plan, d.cache, d.batch, qd, lse, None, acc, 1.0, 0.125, d.scratch)
        want, A = ref.weigh(c, q, lse.cpu(), None, 1.0, 0.125)
        assert ((acc.cpu().double() - want).abs() <= (2.0 ** -16 * A + 2.0 ** -19) * want + 1e-12).all()
        assert d.status() == si.SI_OK


def test_attend_rows_without_a_token_past_32_bits():
    """2^20 rows of 64 heads of 256 of a sequence without tokens: 2^31 pieces of 16 bytes, all zeros."""
    n = 1 << 20
    c = ref.make_cache(Shape(64, 64, 256, 16, "int8", "bf16"), [0, 20], [n, 1], seed=1)
    d = Dev(c)
    q = torch.ones((1, 64, 256), dtype=torch.bfloat16, device=DEV).expand(n + 1, 64, 256)
    out, lse = d.attend(q, 0.06)
    assert d.status() == si.SI_OK
    for x, none in ((out, 0.0), (lse, -math.inf)):
        for part in x[:n].split(1 << 17):
            assert (part == none).all()
    assert torch.isfinite(out[n]).all() and (out[n] != 0).any() and torch.isfinite(lse[n]).all()


# ------------------------------------------------------------------ extreme scores
def low_cache(length, news, k):
    """Every key the same: `k` in the pages, twice that in the unfinished page's rows."""
    c = ref.make_cache(Shape(4, 2, 64, 16, "int8", "bf16"), [length], [news], seed=2)
    c.t["k_codes"].fill_(127)
    c.t["k_scale"].fill_(k / 127)
    c.t["k_tail"].fill_(2 * k)
    return c


@pytest.mark.parametrize("length,news", [(48, 1), (15, 1), (45, 10), (100, 100), (2000, 90), (5003, 1)])
def test_attend_scores_far_below_zero(length, news):
    """Scores of -8e34: a row takes what it sees as it would at any other height."""
    c = low_cache(length, news, 1e17)
    q = torch.full((news, 4, 64), -1e17).to(torch.bfloat16)
    d = Dev(c)
    out, lse = d.attend(q.to(DEV), 0.125)
    check_attend(c, out, lse, q, 0.125)
    assert d.status() == si.SI_OK


@pytest.mark.parametrize("length,news", [(48, 1), (100, 100), (5003, 1), (2000, 90)])
def test_attend_scores_past_the_range(length, news):
    """Scores of -8e38 and past all the range of 32 bits: NaN, as for +8e38, and not the zeros of a row that sees nothing."""
    c = low_cache(length, news, 1e19)
    d = Dev(c)
    for sign in (-1, 1):
        q = torch.full((news, 4, 64), sign * 1e19).to(torch.bfloat16)
        out, lse = d.attend(q.to(DEV), 0.125)
        assert torch.isnan(out).all() and not torch.isfinite(lse).any()


# ------------------------------------------------------------------ what a row does not see
@pytest.mark.parametrize("length,news,page", [(30, 12, 64), (300, 25, 64), (9, 3, 16), (200, 60, 32), (130, 130, 64), (1000, 150, 16)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attend_a_later_token_of_any_size(length, news, page, dim):
    """V of the last tokens 2^40 times as large as the others': the rows before them are within the usual bounds.  (Of the rows
    that see them, weights below 2^-36 of the largest V fall among fp16's smallest values: half a step for each token.)"""
    shape = Shape(8, 2, dim, page, "int8", "bf16")
    c = ref.make_cache(shape, [length, 20], [news, 1], seed=3)
    q, qd = make_q(c, 4)
    sm = dim ** -0.5
    out, lse, _, _ = ref.attend(c, q, sm)
    last = max(1, news // 3)
    for t in range(length - last, length):
        if t >= length // page * page:
            c.t["v_tail"][int(c.slots[0]), :, t % (2 * page)] *= 2.0 ** 40
        elif t % page == 0:  # (a page of later tokens alone)
            c.t["v_scale"][int(c.table[0, t // page])] *= 2.0 ** 40
    d = Dev(c)
    got, z = d.attend(qd, sm)
    first, half = max(0, news - last), torch.finfo(torch.bfloat16).eps / 2
    want, _, S, _ = ref.attend(c, q, sm)
    assert torch.equal(want[:first], out[:first])
    tol = half * want.abs() + (2.0 ** -11 + 2.0 ** -14) * S + 2.0 ** -25
    tol[first:news] += length * 2.0 ** -36 * ref.history(c, "v", 0).abs().amax()
    assert ((got.double().cpu() - want).abs() <= tol).all()
    assert ((z.double().cpu() - lse).abs() <= 2.0 ** -14).all()


@pytest.mark.parametrize("n", [20, 40])
def test_attend_a_page_without_a_v_scale_and_weights_that_vanish(n):
    """What attends to a token of such a page is NaN also where the token's weight is less than 32 bits hold."""
    c = ref.make_cache(Shape(4, 2, 64, 16, "int8", "bf16"), [40], [n], seed=2)
    c.t["k_codes"].fill_(127)
    c.t["k_codes"][int(c.table[0, 1])] = -127
    c.t["k_scale"].fill_(1.0 / 127)
    c.t["k_tail"].fill_(1.0)
    d = Dev(c)
    q = torch.ones((n, 4, 64), dtype=torch.bfloat16)
    good, z = d.attend(q.to(DEV), 4.0)
    check_attend(c, good, z, q, 4.0)
    d.v_scale[int(c.table[0, 1]), 1] = math.nan
    out, lse = d.attend(q.to(DEV), 4.0)
    sees = torch.arange(n, device=DEV) + 40 - n >= 16
    assert torch.equal(lse, z) and torch.equal(out[:, :2], good[:, :2]) and torch.equal(out[~sees], good[~sees])
    assert torch.isnan(out[sees, 2:]).all()


def test_attend_a_broken_start_leaves_the_other_sequences_whole():
    """A start outside the rows, in a call that is split along the keys: its two sequences are reported, the others right."""
    c = ref.make_cache(Shape(8, 2, 128, 64, "int8", "bf16"), [4000, 3900, 4000, 3800], [70, 70, 70, 70], seed=3)
    q, qd = make_q(c, 4)
    good, z = Dev(c).attend(qd, 0.09)
    check_attend(c, good, z, q, 0.09)
    for at, value, left in ((2, 99999, (0, 3)), (2, -5, (0, 3)), (1, 500, (2, 3)), (3, 0, (0, 1))):
        d = Dev(c)
        d.q_start[at] = value
        out, lse = d.attend(qd, 0.09)
        assert d.status() == si.SI_ERR_DEVICE
        for b in left:
            r = slice(70 * b, 70 * b + 70)
            assert torch.equal(out[r], good[r]) and torch.equal(lse[r], z[r]), (at, value, b)


# ------------------------------------------------------------------ evict
def test_evict_into_another_sequences_slot():
    """A new slot that holds another sequence's unfinished rows, or that two take, is reported and not written to."""
    shape = Shape(2, 2, 64, 16, "int8", "bf16")
    lens = [100, 107, 96, 55]  # the third has no unfinished rows
    c = ref.make_cache(shape, lens, [1] * 4, seed=7, spare_pages=20, spare_slots=4)
    s = c.slots.tolist()
    free = [x for x in range(c.n_slots) if x not in s]
    used = set(c.table[c.table >= 0].tolist())
    table = torch.tensor([p for p in range(c.n_pages) if p not in used][:16], dtype=torch.int32).view(4, 4)
    acc = torch.rand((4, 2, 107))
    for new, bad in (([s[1], s[0], s[2], s[3]], {0, 1}), ([s[1], s[1], s[2], s[3]], {0}), ([s[2], s[1], s[0], s[3]], set()),
                     ([free[0], s[0], s[2], free[1]], {1}), ([free[0], free[1], s[2], free[0]], {0, 3}),
                     ([s[0], s[1], s[1], s[3]], set())):
        d = Dev(c)
        acc_out, keep, lens_out = run_evict(d, acc.to(DEV), 4, 0, 1, table.to(DEV), torch.tensor(new, dtype=torch.int32, device=DEV))
        assert d.status() == (si.SI_ERR_DEVICE if bad else si.SI_OK), new
        assert lens_out.tolist() == [4 * 16 + 4, 4 * 16 + 11, 4 * 16, 3 * 16 + 7]
        want = {w: c.t[w].clone() for w in ("k_tail", "v_tail")}
        for b, L in enumerate(lens):
            n, r = min(4, L // 16), L % 16
            assert keep[b, 0, :n].tolist() == ref.keep_pages(acc[b, 0], L, 16, 4, 0, 1)
            if b not in bad:
                was, now = torch.arange(L - r, L) % 32, torch.arange(n * 16, n * 16 + r) % 32
                for w in want:
                    want[w][new[b], :, now] = c.t[w][s[b]][:, was]
        for w in want:
            assert torch.equal(getattr(d, w).cpu().view(torch.int16), want[w].view(torch.int16)), (new, w)


def kept_exactly(acc, length, page, budget):
    """keep_pages with sums that are rounded once (math.fsum)."""
    full = length // page
    score = [math.fsum(acc[j * page:(j + 1) * page].tolist()) for j in range(full)]
    return sorted(sorted(range(full), key=lambda j: (-score[j], j))[:budget])


def choose(acc, page, budget):
    """The pages that si_kv_evict keeps of one sequence, acc [heads, tokens]."""
    heads, length = acc.shape
    c = ref.make_cache(Shape(heads, heads, 64, page, "int8", "bf16"), [length], [1], seed=7, spare_pages=budget)
    used = set(c.table[c.table >= 0].tolist())
    table = torch.tensor([[p for p in range(c.n_pages) if p not in used][:budget]], dtype=torch.int32, device=DEV)
    d = Dev(c)
    _, keep, _ = run_evict(d, acc[None].to(DEV), budget, 0, 0, table, None)
    assert d.status() == si.SI_OK
    return keep[0].tolist()


@pytest.mark.parametrize("page", [16, 32, 64])
def test_evict_pages_of_the_same_values_tie(page):
    """A page's sum does not depend on the order of its tokens: ties stay with the lower pages, whatever the values' spread."""
    g = torch.Generator().manual_seed(3)
    acc = torch.empty((4, 300 * page))
    for h, spread in enumerate((2.0, 8.0, 24.0, 60.0)):
        x = torch.exp2(-spread * torch.rand(page, generator=g)) * torch.rand(page, generator=g)
        acc[h] = torch.cat([x[torch.randperm(page, generator=g)] for _ in range(300)])
    assert choose(acc, page, 120) == [list(range(120))] * 4


@pytest.mark.parametrize("page", [16, 32, 64])
def test_evict_pages_whose_sums_differ_in_the_last_bits(page):
    """Sums that differ near the last of 53 bits, their tokens in any order; negative, tiny and huge ones."""
    g = torch.Generator().manual_seed(5)
    rows = []
    for scale in (1.0, 2.0 ** -140, 2.0 ** 121, -1.0):
        pages = []
        step = torch.randperm(200, generator=g).tolist()
        for j in range(200):
            x = (torch.randint(1, 1 << 20, (page - 1,), generator=torch.Generator().manual_seed(9)).double() * 2.0 ** -20)
            small = 2.0 ** -24 + step[j] * 2.0 ** -47
            x = torch.cat([x, torch.tensor([small], dtype=torch.float64)]) * scale
            if abs(scale) < 2.0 ** -126:  # (the smallest values have fewer bits)
                x = x[torch.randperm(page, generator=g)] * torch.randint(1, 4, (1,), generator=g)
            pages.append(x[torch.randperm(page, generator=g)].float())
        rows.append(torch.cat(pages))
    acc = torch.stack(rows)
    got = choose(acc, page, 77)
    for h in range(4):
        assert got[h] == kept_exactly(acc[h], 200 * page, page, 77), h


def test_evict_sums_that_are_not_finite():
    """+inf above every sum, NaN above it, -inf below; sums past 32 bits' range are numbers."""
    acc = torch.rand((1, 8 * 16), generator=torch.Generator().manual_seed(1))
    acc[0, 16] = math.inf          # page 1
    acc[0, 40] = math.nan          # page 2
    acc[0, 50] = -math.inf         # page 3
    acc[0, 64:80] = 3.0e38         # page 4: 4.8e39
    acc[0, 80:96] = 2.9e38         # page 5
    acc[0, 96], acc[0, 97] = math.inf, -math.inf  # page 6: NaN
    for budget, want in ((1, [2]), (2, [2, 6]), (3, [1, 2, 6]), (4, [1, 2, 4, 6]), (5, [1, 2, 4, 5, 6]), (7, [0, 1, 2, 4, 5, 6, 7])):
        assert choose(acc, 16, budget) == [want]


@pytest.mark.parametrize("apart", [2, 20, 30, 40])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_weigh_a_window_of_rows_of_very_different_size(dtype, apart):
    """Each row keeps its bits beside one 2^apart as large.  (The large row has its values where the keys are zero, so that
    every score is of the order of one.)"""
    if dtype == "f16" and apart > 14:
        apart = 14
    shape = Shape(8, 2, 128, 32, "int8", dtype)
    c = ref.make_cache(shape, [400, 130], [32, 17], seed=4)
    for n in ("k_codes", "k_tail"):
        c.t[n][..., :32] = 0
    q, _ = make_q(c, 6)
    q[:, :, :32] = 0
    for row, head in ((3, 1), (20, 6), (40, 0)):
        q[row, head] = 0
        q[row, head, :32] = 2.0 ** apart
    d = Dev(c)
    sm = 128 ** -0.5
    _, lse, _, _ = ref.attend(c, q, sm)
    lse = lse.float()
    want, A = ref.weigh(c, q, lse, None, 1.0, sm)
    out = torch.zeros((2, 2, 400), device=DEV)
    si.si_kv_weigh(d.plan, d.cache, d.batch, q.to(DEV), lse.to(DEV), None, out, 1.0, sm, d.scratch)
    got = out.cpu().double()
    for b, L in enumerate(c.lens):
        w = want[b, :, :L]
        assert ((got[b, :, :L] - w).abs() <= (2.0 ** -16 * A + 2.0 ** -19) * w).all()
    assert d.status() == si.SI_OK


def test_weigh_a_window_with_rows_that_are_not_finite_or_zero():
    """A row with an infinity makes NaN of what it sees, in its kv head alone; rows of zeros weigh all tokens alike."""
    shape = Shape(8, 2, 64, 16, "e4m3", "bf16")
    c = ref.make_cache(shape, [200], [40], seed=4)
    q, _ = make_q(c, 6)
    q[5:9] = 0
    lse = ref.attend(c, q, 0.125)[1].float()
    want, A = ref.weigh(c, q, lse, None, 1.0, 0.125)
    d = Dev(c)
    out = torch.zeros((1, 2, 200), device=DEV)
    for bad in (None, math.inf, math.nan):
        if bad is not None:
            q[10, 1, 3] = bad
        si.si_kv_weigh(d.plan, d.cache, d.batch, q.to(DEV), lse.to(DEV), None, out, 1.0, 0.125, d.scratch)
        got = out.cpu().double()
        close = (got - want).abs() <= (2.0 ** -16 * A + 2.0 ** -19) * want
        assert close[0, 1].all()
        if bad is None:
            assert close[0, 0].all()
        else:
            assert torch.isnan(got[0, 0, :171]).all() and close[0, 0, 171:].all()


# ------------------------------------------------------------------ calls in a row
@pytest.mark.parametrize("code,dim", [("int8", 128), ("e4m3", 64)])
def test_steps_in_a_row_are_the_steps_one_by_one(code, dim):
    """Append, attend and weigh of 80 steps without a wait between them (each kernel starts while the one before it ends)
    give what they give with a wait after every call."""
    shape = Shape(8, 4, dim, 16, code, "bf16")
    B, steps = 40, 80
    lens = [20 + 11 * b for b in range(B)]
    g = torch.Generator().manual_seed(2)
    kv = torch.randn((steps, B, 8, dim), generator=g).bfloat16().to(DEV)
    q = torch.randn((steps, B, 8, dim), generator=g).bfloat16().to(DEV)

    def run(wait):
        c = ref.make_cache(shape, lens, [steps] * B, seed=5, empty=True)
        c.news = [1] * B
        most = max(lens) + steps
        d = Dev(c, max_len=most)
        outs, acc = [], torch.zeros((B, 4, most), device=DEV)
        before, after = d.lens, torch.empty_like(d.lens)
        for i in range(steps):
            b0 = si.kv_batch(B, B, 1, most, d.q_start, before, d.table, d.slots)
            b1 = si.kv_batch(B, B, 1, most, d.q_start, after, d.table, d.slots)
            out, lse = torch.empty_like(q[i]), torch.empty((B, 8), device=DEV)
            outs += [out, lse]
            si.si_kv_append(d.plan, d.cache, b0, kv[i, :, :4], kv[i, :, 4:], after, d.scratch)
            if wait:
                torch.cuda.synchronize()
            si.si_kv_attend(d.plan, d.cache, b1, q[i], out, lse, 0.1, d.scratch)
            if wait:
                torch.cuda.synchronize()
            si.si_kv_weigh(d.plan, d.cache, b1, q[i], lse, acc, acc, 0.9, 0.1, d.scratch)
            if wait:
                torch.cuda.synchronize()
            before, after = after, before
        assert d.status() == si.SI_OK
        return outs + [acc, before]
    want = run(True)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(run(False), want))


# ------------------------------------------------------------------ no rows at all
def test_calls_without_rows():
    """Nothing appended, nothing attended, sums that only decay: empty tensors are taken."""
    shape = Shape(4, 2, 64, 16, "int8", "bf16")
    c = ref.make_cache(shape, [40, 0, 33], [0, 0, 0], seed=3)
    d = Dev(c)
    none = torch.empty((0, 4, 64), dtype=torch.bfloat16, device=DEV)
    lse = torch.empty((0, 4), device=DEV)
    out = torch.full_like(d.lens, -7)
    si.si_kv_append(d.plan, d.cache, d.batch, none[:, :2], none[:, 2:], out, d.scratch)
    assert out.tolist() == c.lens
    si.si_kv_attend(d.plan, d.cache, d.batch, none, torch.empty_like(none), lse, 0.1, d.scratch)
    acc = torch.rand((3, 2, 40), device=DEV)
    got = torch.full_like(acc, 9.0)
    si.si_kv_weigh(d.plan, d.cache, d.batch, none, lse, acc, got, 0.5, 0.1, d.scratch)
    for b, L in enumerate(c.lens):
        assert torch.equal(got[b, :, :L], 0.5 * acc[b, :, :L]) and (got[b, :, L:] == 9.0).all()
    assert d.status() == si.SI_OK
    for t in (d.k_codes, d.v_codes):
        assert torch.equal(t.cpu().view(torch.uint8), c.t["k_codes" if t is d.k_codes else "v_codes"].view(torch.uint8))


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attend_and_weigh_a_chunk_among_steps(dim):
    """One call with a chunk of a prompt, steps of 30 sequences, one of two tokens and one without any."""
    shape = Shape(8, 2, dim, 32, "int8", "bf16")
    lens = [700] + [17 * b + 1 for b in range(30)] + [60, 45]
    c = ref.make_cache(shape, lens, [90] + [1] * 30 + [2, 0], seed=5)
    d = Dev(c)
    q, qd = make_q(c, 6)
    sm = dim ** -0.5
    out, lse = d.attend(qd, sm)
    check_attend(c, out, lse, q, sm)
    acc = torch.full((33, 2, 700), 9.0, device=DEV)
    si.si_kv_weigh(d.plan, d.cache, d.batch, qd, lse, None, acc, 1.0, sm, d.scratch)
    want, A = ref.weigh(c, q, lse.cpu(), None, 1.0, sm)
    for b, L in enumerate(lens):
        w = want[b, :, :L]
        assert ((acc[b, :, :L].cpu().double() - w).abs() <= (2.0 ** -16 * A + 2.0 ** -19) * w + 1e-12).all(), b
    assert d.status() == si.SI_OK
