"""The 8-bit cache's operators on the GPU against their definitions in 64 bits (kv_reference)."""
import math

import pytest
import torch

from quantized_moe_expert_gemv_gb300 import binding as si
import kv_reference as ref
from kv_reference import Shape

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Dev:
    """A reference cache's tensors on the device, with a plan and scratch for its sequences."""

    def __init__(self, c, max_len=None, max_new=None, lens=None):
        s = c.shape
        self.c = c
        self.plan = si.si_kv_plan(si.make_kv_desc(s.heads, s.kv, s.dim, s.page, s.code, s.dtype))
        for n, t in c.t.items():
            setattr(self, n, t.to(DEV))
        self.cache = si.kv_cache(self.k_codes, self.v_codes, self.k_scale, self.v_scale, self.k_tail, self.v_tail)
        self.q_start = torch.tensor(ref.starts(c.news), dtype=torch.int32, device=DEV)
        self.lens = torch.tensor(c.lens if lens is None else lens, dtype=torch.int32, device=DEV)
        self.table, self.slots = c.table.to(DEV), c.slots.to(DEV)
        self.T = sum(c.news)
        self.max_new = max(c.news) if max_new is None else max_new
        self.max_len = max(c.lens) if max_len is None else max_len
        self.batch = si.kv_batch(len(c.lens), self.T, self.max_new, self.max_len, self.q_start, self.lens, self.table,
                                 self.slots)
        n = si.si_kv_scratch_bytes(self.plan, len(c.lens), self.T, self.max_new, self.max_len)
        self.scratch = torch.empty(n, dtype=torch.uint8, device=DEV)
        si.si_kv_scratch_init(self.plan, self.scratch)

    def status(self):
        return si.si_kv_read_status(self.plan, self.scratch)

    def attend(self, q, sm, strided=False, lse=True, stream=None):
        s, T = self.c.shape, q.shape[0]
        if strided:  # heads apart and rows apart, in a larger buffer
            out = torch.full((s.heads, T, s.dim + 24), 7.0, dtype=q.dtype, device=DEV).transpose(0, 1)[:, :, :s.dim]
        else:
            out = torch.full((T, s.heads, s.dim), 7.0, dtype=q.dtype, device=DEV)
        z = torch.full((T, s.heads), 7.0, device=DEV) if lse else None
        si.si_kv_attend(self.plan, self.cache, self.batch, q, out, z, sm, self.scratch, stream)
        return out, z


def make_q(c, seed, strided=False):
    g = torch.Generator().manual_seed(seed)
    s, T = c.shape, sum(c.news)
    q = (torch.randn((T, s.heads, s.dim), generator=g) * 1.2).to(ref.DT[s.dtype])
    if strided:
        big = torch.zeros((T, s.heads + 3, s.dim + 8), dtype=q.dtype, device=DEV)
        big[:, 1:1 + s.heads, :s.dim] = q.to(DEV)
        return q, big[:, 1:1 + s.heads, :s.dim]
    return q, q.to(DEV)


def check_attend(c, got, lse, q, sm):
    out, z, S, A = ref.attend(c, q, sm)
    half = torch.finfo(ref.DT[c.shape.dtype]).eps / 2
    tol = half * out.abs() + (2.0 ** -11 + 2.0 ** -14) * S + 2.0 ** -25
    err = (got.double().cpu() - out).abs()
    assert torch.isfinite(got).all()
    assert (err <= tol).all(), f"out: {float((err / tol).max()):.2f} of the tolerance"
    if lse is not None:
        empty = torch.isinf(z)
        assert torch.equal(torch.isinf(lse.cpu()), empty)
        e = (lse.double().cpu() - z)[~empty].abs()
        t = (2.0 ** -17 * A + 2.0 ** -21 * (1 + z.abs()))[~empty]
        assert (e <= t).all(), f"lse: {float((e / t).max()):.2f} of the tolerance"


def shapes():
    return [Shape(8, 2, 128, 64, "int8", "bf16"), Shape(8, 8, 64, 16, "e4m3", "f16"), Shape(5, 1, 256, 32, "int8", "f16"),
            Shape(16, 1, 128, 16, "e4m3", "bf16"), Shape(6, 2, 64, 32, "int8", "bf16"), Shape(40, 2, 64, 64, "e4m3", "f16"),
            Shape(2, 1, 256, 64, "e4m3", "bf16"), Shape(32, 4, 128, 32, "int8", "f16")]


def ident(s):
    return f"{s.heads}x{s.kv}x{s.dim}-p{s.page}-{s.code}-{s.dtype}"


LENS = [
    ([1], [1]),                                       # one token in all
    ([0, 5, 0], [0, 1, 2]),                           # empty sequences, and rows without a token to see
    ([15, 16, 17, 63, 64, 65], [1, 1, 1, 1, 1, 1]),   # about a page
    ([3, 130, 1000], [3, 7, 2]),                      # few rows each
    ([2], [5]),                                       # more rows than tokens: the first see nothing
    ([700, 33], [40, 33]),                            # rows past one row group; a whole prompt
    ([257, 64, 511], [257, 64, 200]),                 # prompts
]


@pytest.mark.parametrize("lens,news", LENS, ids=[str(i) for i in range(len(LENS))])
@pytest.mark.parametrize("shape", shapes(), ids=ident)
def test_attend(shape, lens, news):
    c = ref.make_cache(shape, lens, news, seed=len(lens) + sum(lens))
    d = Dev(c)
    strided = sum(lens) % 2 == 1
    q, qd = make_q(c, 3, strided)
    sm = shape.dim ** -0.5
    out, lse = d.attend(qd, sm, strided)
    check_attend(c, out, lse, q, sm)
    assert d.status() == si.SI_OK
    again, z = d.attend(qd, sm, strided)
    assert torch.equal(out, again) and torch.equal(lse, z)


@pytest.mark.parametrize("shape,lens,news", [
    (Shape(8, 1, 128, 64, "int8", "bf16"), [20011, 3, 4097], [1, 1, 2]),
    (Shape(4, 4, 64, 16, "e4m3", "f16"), [9000], [1]),
    (Shape(4, 2, 256, 32, "e4m3", "bf16"), [5003, 200], [5, 1]),
    (Shape(8, 2, 128, 32, "e4m3", "f16"), [3000], [150]),
    (Shape(16, 2, 64, 64, "int8", "bf16"), [2500, 1500], [130, 513]),
], ids=["mqa", "mha", "wide", "chunk", "chunks"])
def test_attend_long(shape, lens, news):
    c = ref.make_cache(shape, lens, news, seed=9)
    d = Dev(c)
    q, qd = make_q(c, 4)
    sm = shape.dim ** -0.5
    out, lse = d.attend(qd, sm)
    check_attend(c, out, lse, q, sm)
    assert d.status() == si.SI_OK


def test_attend_many_sequences():
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 90, (300,), generator=g).tolist()
    c = ref.make_cache(Shape(4, 2, 64, 16, "int8", "bf16"), lens, [1] * 300, seed=6)
    d = Dev(c)
    q, qd = make_q(c, 4)
    out, lse = d.attend(qd, 0.125)
    check_attend(c, out, lse, q, 0.125)


@pytest.mark.parametrize("n", [1, 100], ids=["step", "prompt"])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_attend_scores_apart(code, n):
    """Scores far apart (one token takes all the weight), scores all equal, and pages of very different scale."""
    shape = Shape(4, 2, 128, 16, code, "bf16")
    for seed, sm in enumerate((0.0, 0.01, 0.1, 0.4, 0.1, 0.4, 0.2, 0.4)):
        g = torch.Generator().manual_seed(seed)
        c = ref.make_cache(shape, [300], [n], seed=2)
        c.t["v_scale"] *= torch.exp2(torch.randint(-12, 4, c.t["v_scale"].shape, generator=g).float())
        c.t["k_scale"] *= torch.exp2(torch.randint(-3, 2, c.t["k_scale"].shape, generator=g).float())
        d = Dev(c)
        q, qd = make_q(c, 4)
        out, lse = d.attend(qd, sm)
        o, z, S, A = ref.attend(c, q, sm)
        half = torch.finfo(torch.bfloat16).eps / 2
        tol = half * o.abs() + (2.0 ** -11 + 2.0 ** -15 * A[..., None]) * S + 2.0 ** -25
        far = float(((out.double().cpu() - o).abs() / tol).max())
        assert far <= 1, (seed, sm, far)
        assert ((lse.double().cpu() - z).abs() <= 2.0 ** -17 * A + 2.0 ** -21 * (1 + z.abs())).all()


@pytest.mark.parametrize("n", [1, 4, 100])
def test_attend_what_is_not_seen_does_not_matter(n):
    """NaN and infinities in the ring past the length, in other pages and slots, and in later tokens' places."""
    shape = Shape(8, 2, 128, 64, "int8", "bf16")
    c = ref.make_cache(shape, [200, 90], [n, min(n, 90)], seed=3)
    d = Dev(c)
    q, qd = make_q(c, 4)
    out, lse = d.attend(qd, 0.09)
    used = torch.unique(c.table[c.table >= 0]).long()
    others = torch.ones(c.n_pages, dtype=torch.bool)
    others[used] = False
    for w in "kv":
        getattr(d, w + "_scale")[others.to(DEV)] = math.nan
        tail = getattr(d, w + "_tail")
        live = torch.zeros(tail.shape[0], 2 * shape.page, dtype=torch.bool)
        for b, L in enumerate(c.lens):
            live[int(c.slots[b]), torch.arange(L // 64 * 64, L) % 128] = True
        tail.permute(0, 2, 1, 3)[~live.to(DEV)] = math.nan if w == "k" else math.inf
    again, z = d.attend(qd, 0.09)
    assert torch.equal(out, again) and torch.equal(lse, z)


@pytest.mark.parametrize("n", [8, 70])
def test_attend_a_later_token_that_is_nan(n):
    """A row sees no later token of the unfinished page, whatever it holds."""
    shape = Shape(8, 2, 128, 64, "e4m3", "f16")
    c = ref.make_cache(shape, [n + 2], [n], seed=3)
    if n >= 64:
        c = ref.make_cache(shape, [124], [n], seed=3)
    d = Dev(c)
    q, qd = make_q(c, 4)
    out, lse = d.attend(qd, 0.09)
    L = c.lens[0]
    for w, bad in (("k", math.nan), ("v", math.inf), ("v", math.nan), ("k", -math.inf)):
        e = Dev(c)
        getattr(e, w + "_tail")[int(c.slots[0]), :, (L - 1) % 128, 5] = bad
        again, z = e.attend(qd, 0.09)
        assert torch.equal(out[:-1], again[:-1]) and torch.equal(lse[:-1], z[:-1]), (w, bad)
        if w == "v" or math.isnan(bad):  # (a key of -inf may score +inf or -inf)
            assert not torch.isfinite(again[-1]).all()


def test_attend_a_page_without_a_scale_is_nan():
    shape = Shape(4, 2, 64, 16, "int8", "bf16")
    c = ref.make_cache(shape, [40, 40], [1, 1], seed=3)
    d = Dev(c)
    d.k_scale[int(c.table[0, 1]), 1] = math.nan
    q, qd = make_q(c, 4)
    out, lse = d.attend(qd, 0.1)
    assert torch.isnan(out[0, 2:]).all() and torch.isnan(lse[0, 2:]).all()
    assert torch.isfinite(out[0, :2]).all() and torch.isfinite(out[1]).all()


def test_indices_outside_the_cache_are_not_followed():
    """A page or slot outside the cache, a length or row range past the bounds: reported, and nothing else changes."""
    shape = Shape(4, 2, 64, 16, "int8", "bf16")
    c = ref.make_cache(shape, [40, 45, 50, 33], [1, 2, 1, 1], seed=3)
    q, qd = make_q(c, 4)
    good, _ = Dev(c).attend(qd, 0.1)
    rows = {0: slice(0, 1), 1: slice(1, 3), 2: slice(3, 4), 3: slice(4, 5)}

    def run(change, hit, nan):
        d = Dev(c)
        change(d)
        out, _ = d.attend(qd, 0.1)
        assert d.status() == si.SI_ERR_DEVICE and d.status() == si.SI_OK
        for b, r in rows.items():
            if b != hit:
                assert torch.equal(out[r], good[r])
            elif nan:
                assert torch.isnan(out[r]).all()
    run(lambda d: d.table[1].__setitem__(0, 10 ** 6), 1, True)
    run(lambda d: d.table[1].__setitem__(1, -5), 1, True)
    run(lambda d: d.slots.__setitem__(2, 99), 2, True)
    run(lambda d: d.slots.__setitem__(2, -1), 2, True)
    run(lambda d: d.lens.__setitem__(3, 51), 3, False)
    run(lambda d: d.lens.__setitem__(3, -4), 3, False)
    run(lambda d: d.q_start.__setitem__(4, 99), 3, False)


@pytest.mark.parametrize("dim", [64, 128])
def test_attend_reports_a_wait_that_runs_out(monkeypatch, dim):
    """The many-row kernel's waits are bounded: with a short budget and a wait that nothing ends, the call
    returns, the status says so, and the next call (of a plan without the test mode) is right."""
    shape = Shape(8, 2, dim, 64, "int8", "bf16")
    c = ref.make_cache(shape, [500], [200], seed=3)
    q, qd = make_q(c, 4)
    monkeypatch.setenv("SI_FAULT_WAIT_BUDGET", "20000")
    d = Dev(c)
    d.attend(qd, 0.1)
    assert d.status() == si.SI_ERR_TIMEOUT
    acc = torch.zeros((1, 2, 500), device=DEV)
    si.si_kv_weigh(d.plan, d.cache, d.batch, qd, torch.zeros((200, 8), device=DEV), None, acc, 1.0, 0.1, d.scratch)
    assert d.status() == si.SI_ERR_TIMEOUT
    start = torch.tensor([0, 20], dtype=torch.int32, device=DEV)
    few = si.kv_batch(1, 20, 20, 500, start, d.lens, d.table, d.slots)
    si.si_kv_weigh(d.plan, d.cache, few, qd, torch.zeros((200, 8), device=DEV), None, acc, 1.0, 0.1, d.scratch)
    assert d.status() == si.SI_ERR_TIMEOUT
    monkeypatch.delenv("SI_FAULT_WAIT_BUDGET")
    d = Dev(c)
    out, lse = d.attend(qd, 0.1)
    check_attend(c, out, lse, q, 0.1)
    assert d.status() == si.SI_OK


def test_refusals_launch_nothing_on_the_device():
    from test_kv_host import Call, refusals
    plan = si.si_kv_plan(si.make_kv_desc(8, 2, 128, 64))
    lib = si.load_library()
    for names, change, want in refusals():
        for name in names:
            call = Call(plan)
            change(call)
            assert call(lib, name) == want, (name, want)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ append, read
def run_append(d, k, v, lens_out=None):
    out = torch.full((len(d.c.lens),), -7, dtype=torch.int32, device=DEV) if lens_out is None else lens_out
    si.si_kv_append(d.plan, d.cache, d.batch, k, v, out, d.scratch)
    return out


APPEND = [([0], [1]), ([15], [1]), ([14, 0, 31], [2, 0, 1]), ([5, 60, 0], [70, 5, 200]), ([130, 64], [64, 63]),
          ([63, 1], [130, 191])]


@pytest.mark.parametrize("lens,news", APPEND, ids=[str(i) for i in range(len(APPEND))])
@pytest.mark.parametrize("shape", shapes(), ids=ident)
def test_append(shape, lens, news):
    P = shape.page
    c = ref.make_cache(shape, lens, news, seed=8, empty=True)
    total = [a + n for a, n in zip(lens, news)]
    d = Dev(c, max_len=max(total))
    g = torch.Generator().manual_seed(4)
    T = sum(news)
    kv = (torch.randn((T, 2 * shape.kv, shape.dim), generator=g) * torch.exp(torch.randn((2 * shape.kv, shape.dim), generator=g)))
    kv = kv.to(ref.DT[shape.dtype])
    kvd = kv.to(DEV)
    lens_out = run_append(d, kvd[:, :shape.kv], kvd[:, shape.kv:])
    assert lens_out.tolist() == total and d.status() == si.SI_OK
    for w, new in (("k", kv[:, :shape.kv]), ("v", kv[:, shape.kv:])):
        codes, scale, tail = (c.t[w + "_" + n].clone() for n in ("codes", "scale", "tail"))
        row = 0
        for b, (a, n) in enumerate(zip(lens, news)):
            slot = int(c.slots[b])
            old = c.t[w + "_tail"][slot][:, torch.arange(a // P * P, a) % (2 * P)].transpose(0, 1)
            x = torch.cat([old, new[row:row + n]])
            row += n
            first, last = a // P, (a + n) // P
            for j in range(first, last):
                page = int(c.table[b, j])
                codes[page], scale[page] = ref.quantise(x[(j - first) * P:(j - first + 1) * P].transpose(0, 1), shape.code)
            for t in range(max(a, (last - 1) * P), a + n):
                tail[slot, :, t % (2 * P)] = x[t - first * P]
        assert torch.equal(getattr(d, w + "_codes").cpu().view(torch.uint8), codes.view(torch.uint8)), w
        assert torch.equal(getattr(d, w + "_scale").cpu(), scale), w
        assert torch.equal(getattr(d, w + "_tail").cpu().view(torch.int16), tail.view(torch.int16)), w


def test_append_token_by_token_is_append_at_once():
    """The cache's contents do not depend on how the tokens came in, nor on a step that was taken back."""
    shape = Shape(4, 2, 64, 16, "int8", "bf16")
    g = torch.Generator().manual_seed(4)
    kv = torch.randn((53, 4, 64), generator=g).to(torch.bfloat16).to(DEV)

    def fill(steps):
        c = ref.make_cache(shape, [0], [53], seed=8, empty=True)
        d = Dev(c, max_len=53)
        for w in "kv":
            getattr(d, w + "_codes").zero_()
            getattr(d, w + "_scale").zero_()
            getattr(d, w + "_tail").zero_()
        lens, out = d.lens, torch.empty_like(d.lens)
        for at, n in steps:
            lens.fill_(at)
            start = torch.tensor([0, n], dtype=torch.int32, device=DEV)
            batch = si.kv_batch(1, n, n, 53, start, lens, d.table, d.slots)
            rows = kv[at:at + n]
            si.si_kv_append(d.plan, d.cache, batch, rows[:, :2], rows[:, 2:], out, d.scratch)
            assert int(out) == at + n
        live = torch.arange(48, 53, device=DEV) % 32
        return [d.k_codes, d.v_codes, d.k_scale, d.v_scale, d.k_tail[int(c.slots[0]), :, live]]

    once = fill([(0, 53)])
    single = fill([(t, 1) for t in range(53)])
    back = fill([(0, 13), (13, 7), (15, 9), (24, 10), (29, 16), (45, 8)])  # 20 -> 15, 34 -> 29: taken back in part
    for x, y, z in zip(once, single, back):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        assert torch.equal(x.view(torch.uint8), z.view(torch.uint8))


def test_append_zero_pages_and_pages_that_are_not_finite():
    shape = Shape(4, 4, 64, 16, "e4m3", "bf16")
    c = ref.make_cache(shape, [0], [16], seed=8, empty=True)
    d = Dev(c, max_len=16)
    k = torch.randn((16, 4, 64)).to(torch.bfloat16)
    k[:, 0] = 0
    k[:, 1] = 2.0 ** -110
    k[3, 2, 7] = math.inf
    k[9, 3, 1] = math.nan
    run_append(d, k.to(DEV), k.to(DEV))
    page = int(c.table[0, 0])
    assert d.k_scale[page, :2].tolist() == [0.0, 0.0] and torch.isnan(d.k_scale[page, 2:]).all()
    assert (d.k_codes[page].float() == 0).all()
    assert torch.equal(torch.isnan(d.v_scale[page]).cpu(), torch.tensor([False, False, True, True]))


def test_append_refuses_what_does_not_fit():
    """Past the host's bound, a bad slot, a bad page: reported; the other sequences are appended."""
    shape = Shape(4, 2, 64, 16, "int8", "bf16")
    g = torch.Generator().manual_seed(4)
    kv = torch.randn((6, 4, 64), generator=g).to(torch.bfloat16).to(DEV)

    def run(change):
        c = ref.make_cache(shape, [14, 14, 14], [2, 2, 2], seed=8, empty=True)
        d = Dev(c, max_len=16)
        before = {w: getattr(d, w).clone() for w in c.t}
        change(d)
        out = run_append(d, kv[:, :2], kv[:, 2:]).tolist()
        assert d.status() == si.SI_ERR_DEVICE
        for b in (0, 2):
            assert (d.k_codes[int(c.table[b, 0])] != before["k_codes"][int(c.table[b, 0])]).any()
        assert torch.equal(d.k_codes[int(c.table[1, 0])], before["k_codes"][int(c.table[1, 0])])
        return out, d, c, before
    out, d, c, before = run(lambda d: d.lens.__setitem__(1, 15))
    assert out == [16, 15, 16]
    assert torch.equal(d.k_tail[int(c.slots[1])].view(torch.int16), before["k_tail"][int(c.slots[1])].view(torch.int16))
    out, *_ = run(lambda d: d.slots.__setitem__(1, 77))
    assert out == [16, 14, 16]
    out, *_ = run(lambda d: d.table.__setitem__((1, 0), 1000))
    assert out == [16, 16, 16]


@pytest.mark.parametrize("shape", shapes(), ids=ident)
def test_read(shape):
    c = ref.make_cache(shape, [70], [1], seed=1, spare_pages=9)
    d = Dev(c)
    pages = torch.randperm(c.n_pages)[:5].to(torch.int32)
    dt = ref.DT[shape.dtype]
    k = torch.empty((5, shape.kv, shape.page, shape.dim), dtype=dt, device=DEV)
    v = torch.empty_like(k)
    si.si_kv_read(d.plan, d.cache, pages.to(DEV), 5, k, v, d.scratch)
    for w, got in (("k", k), ("v", v)):
        p = pages.long()
        want = (c.t[w + "_codes"].float()[p] * c.t[w + "_scale"][p][..., None, None]).to(dt)
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
    assert d.status() == si.SI_OK
    si.si_kv_read(d.plan, d.cache, torch.tensor([0, c.n_pages, -1, 1, 2], dtype=torch.int32, device=DEV), 5, k, v, d.scratch)
    assert d.status() == si.SI_ERR_DEVICE
    assert torch.isnan(k[1:3]).all() and torch.isnan(v[1:3]).all() and torch.isfinite(k[3:]).all()


# ------------------------------------------------------------------ weigh
WEIGH = [([1], [1]), ([0, 5, 0], [0, 1, 2]), ([15, 16, 17, 130], [1, 1, 1, 2]), ([3, 300], [3, 64]), ([2], [5]),
         ([900, 257], [5, 257]), ([3001], [1]), ([500, 2000, 64, 129], [60, 9, 17, 61])]


@pytest.mark.parametrize("lens,news", WEIGH, ids=[str(i) for i in range(len(WEIGH))])
@pytest.mark.parametrize("shape", shapes(), ids=ident)
def test_weigh(shape, lens, news):
    c = ref.make_cache(shape, lens, news, seed=5)
    d = Dev(c)
    q, qd = make_q(c, 6, strided=len(lens) % 2 == 1)
    sm = shape.dim ** -0.5
    _, lse, _, _ = ref.attend(c, q, sm)
    lse = lse.float()
    stride = max(lens) + 3
    acc = torch.rand((len(lens), shape.kv, stride))
    poison = acc.clone()  # what the call must not read: the call's own tokens and what lies past the length
    for b, (L, n) in enumerate(zip(lens, news)):
        poison[b, :, max(0, L - n):] = math.nan
    for first in (acc, None):
        want, A = ref.weigh(c, q, lse, first, 0.75, sm)
        out = torch.full((len(lens), shape.kv, stride), 9.0, device=DEV)
        si.si_kv_weigh(d.plan, d.cache, d.batch, qd, lse.to(DEV), None if first is None else poison.to(DEV), out, 0.75, sm,
                       d.scratch)
        got = out.cpu().double()
        for b, L in enumerate(lens):
            assert (got[b, :, L:] == 9.0).all()
            w = want[b, :, :L]
            tol = (2.0 ** -16 * A + 2.0 ** -19) * w + 1e-12
            assert ((got[b, :, :L] - w).abs() <= tol).all(), float(((got[b, :, :L] - w).abs() / tol).max())
        again = torch.full_like(out, 9.0)
        si.si_kv_weigh(d.plan, d.cache, d.batch, qd, lse.to(DEV), None if first is None else poison.to(DEV), again, 0.75,
                       sm, d.scratch)
        assert torch.equal(out, again)
    assert d.status() == si.SI_OK
    same = acc.to(DEV)  # in place
    si.si_kv_weigh(d.plan, d.cache, d.batch, qd, lse.to(DEV), same, same, 0.75, sm, d.scratch)
    want, _ = ref.weigh(c, q, lse, acc, 0.75, sm)
    for b, L in enumerate(lens):
        torch.testing.assert_close(same[b, :, :L].cpu().double(), want[b, :, :L], rtol=2.0 ** -16 * A + 2.0 ** -19, atol=1e-12)


def test_weigh_with_the_lse_of_attend_sums_to_the_rows():
    shape = Shape(8, 2, 128, 64, "int8", "bf16")
    c = ref.make_cache(shape, [1000, 333], [4, 4], seed=5)
    d = Dev(c)
    _, qd = make_q(c, 6)
    _, lse = d.attend(qd, 0.09)
    out = torch.zeros((2, 2, 1000), device=DEV)
    si.si_kv_weigh(d.plan, d.cache, d.batch, qd, lse, None, out, 1.0, 0.09, d.scratch)
    total = out.double().sum(2)  # four rows of four query heads, each of weight one
    assert ((total - 16).abs() <= 16 * 2.0 ** -14).all()


# ------------------------------------------------------------------ evict
EVICT = [([100], 4, 1, 1), ([500, 20, 0, 333], 6, 0, 0), ([1000, 64], 7, 2, 5), ([1000], 1, 0, 1), ([300, 290], 100, 0, 1),
         ([4000, 2111], 30, 1, 4)]


def run_evict(d, acc, budget, sink, recent, new_table, new_slots, stride=None):
    B, Hk = len(d.c.lens), d.c.shape.kv
    acc_out = torch.full_like(acc, 9.0)
    keep = torch.full((B, Hk, budget), -9, dtype=torch.int32, device=DEV)
    lens_out = torch.full((B,), -9, dtype=torch.int32, device=DEV)
    si.si_kv_evict(d.plan, d.cache, d.batch, acc, acc_out, budget, sink, recent, new_table, new_slots, keep, lens_out,
                   d.scratch)
    return acc_out, keep, lens_out


@pytest.mark.parametrize("scores", ["random", "ties", "zero", "nan"])
@pytest.mark.parametrize("lens,budget,sink,recent", EVICT, ids=[str(i) for i in range(len(EVICT))])
@pytest.mark.parametrize("shape", shapes()[:6], ids=ident)
def test_evict(shape, lens, budget, sink, recent, scores):
    P, B = shape.page, len(lens)
    c = ref.make_cache(shape, lens, [1] * B, seed=7, spare_pages=B * budget + 2, spare_slots=B + 1)
    d = Dev(c)
    g = torch.Generator().manual_seed(1)
    acc = torch.rand((B, shape.kv, max(lens) + 5), generator=g)
    if scores == "ties":
        acc = (acc * 2).round() * (torch.arange(acc.shape[2]) % P == 0)
    elif scores == "zero":
        acc = acc * 0
    elif scores == "nan":
        acc[torch.rand(acc.shape, generator=g) < 0.02] = math.nan
    used = set(c.table[c.table >= 0].tolist())
    free = [p for p in range(c.n_pages) if p not in used][:B * budget]
    new_table = torch.tensor(free, dtype=torch.int32).view(B, budget)
    new_slots = [s for s in range(c.n_slots) if s not in c.slots.tolist()][:B]
    for slots in (torch.tensor(new_slots, dtype=torch.int32, device=DEV), None):
        d = Dev(c)
        acc_out, keep, lens_out = run_evict(d, acc.to(DEV), budget, sink, recent, new_table.to(DEV), slots)
        assert d.status() == si.SI_OK
        want = {n: x.clone() for n, x in c.t.items()}
        for b, L in enumerate(lens):
            F, r = L // P, L % P
            n = min(F, budget)
            assert int(lens_out[b]) == n * P + r
            to = int(c.slots[b]) if slots is None else new_slots[b]
            for h in range(shape.kv):
                kept = ref.keep_pages(acc[b, h], L, P, budget, sink, recent)
                assert keep[b, h].tolist() == kept + [-1] * (budget - n)
                a = torch.cat([acc[b, h, j * P:(j + 1) * P] for j in kept] + [acc[b, h, F * P:L]])
                assert torch.equal(acc_out[b, h, :len(a)].cpu().nan_to_num(-1), a.nan_to_num(-1))
                assert (acc_out[b, h, len(a):] == 9.0).all()
                for w in "kv":
                    for i, j in enumerate(kept):
                        src, dst = int(c.table[b, j]), int(new_table[b, i])
                        want[w + "_codes"][dst, h] = c.t[w + "_codes"][src, h]
                        want[w + "_scale"][dst, h] = c.t[w + "_scale"][src, h]
                    was, now = torch.arange(F * P, L) % (2 * P), torch.arange(n * P, n * P + r) % (2 * P)
                    want[w + "_tail"][to, h, now] = c.t[w + "_tail"][int(c.slots[b]), h, was]
        for name, x in want.items():
            assert torch.equal(getattr(d, name).cpu().view(torch.uint8), x.view(torch.uint8)), name


def test_evict_many_pages():
    shape = Shape(2, 2, 64, 16, "int8", "f16")
    c = ref.make_cache(shape, [16 * 5000 + 3], [1], seed=7, spare_pages=800)
    d = Dev(c)
    acc = torch.rand((1, 2, 16 * 5000 + 3)) ** 8
    used = set(c.table[c.table >= 0].tolist())
    free = [p for p in range(c.n_pages) if p not in used][:777]
    _, keep, lens = run_evict(d, acc.to(DEV), 777, 3, 20, torch.tensor([free], dtype=torch.int32, device=DEV), None)
    for h in range(2):
        assert keep[0, h].tolist() == ref.keep_pages(acc[0, h], c.lens[0], 16, 777, 3, 20)
    assert int(lens) == 777 * 16 + 3


def test_evict_indices_outside_the_cache():
    shape = Shape(2, 2, 64, 16, "int8", "bf16")
    c = ref.make_cache(shape, [100, 100], [1, 1], seed=7, spare_pages=9, spare_slots=4)
    acc = torch.rand((2, 2, 100))
    used = set(c.table[c.table >= 0].tolist())
    free = torch.tensor([p for p in range(c.n_pages) if p not in used][:8], dtype=torch.int32).view(2, 4)
    for change in ("page", "new", "slot"):
        d = Dev(c)
        table, slots = free.clone(), None
        if change == "page":
            d.table[0] = c.n_pages + 5
        if change == "new":
            table[0] = -3
        if change == "slot":
            slots = torch.tensor([99, int(c.slots[1])], dtype=torch.int32, device=DEV)
        run_evict(d, acc.to(DEV), 4, 0, 1, table.to(DEV), slots)
        assert d.status() == si.SI_ERR_DEVICE
        kept = ref.keep_pages(acc[1, 0], 100, 16, 4, 0, 1)
        for i, j in enumerate(kept):
            assert torch.equal(d.k_codes[int(free[1, i]), 0].cpu(), c.t["k_codes"][int(c.table[1, j]), 0])
        if change == "page":
            assert torch.isnan(d.k_scale[free[0].long().to(DEV)]).all()


# ------------------------------------------------------------------ together
def test_offsets_past_32_bits():
    """Pages whose bytes lie past 2^32 in the code arrays."""
    shape = Shape(2, 2, 256, 64, "int8", "bf16")
    per = 2 * 64 * 256
    n = (1 << 32) // per + 40
    c = ref.make_cache(shape, [200], [3], seed=1)
    d = Dev(c)
    q, qd = make_q(c, 4)
    want, z = d.attend(qd, 0.06)
    shift = n - c.n_pages
    big = {}
    for w in "kv":
        big[w] = torch.zeros((n, 2, 64, 256), dtype=torch.int8, device=DEV)
        big[w + "s"] = torch.zeros((n, 2), device=DEV)
        big[w][shift:] = getattr(d, w + "_codes")
        big[w + "s"][shift:] = getattr(d, w + "_scale")
    d.table += shift
    d.cache = si.kv_cache(big["k"], big["v"], big["ks"], big["vs"], d.k_tail, d.v_tail)
    got, z2 = d.attend(qd, 0.06)
    assert torch.equal(want, got) and torch.equal(z, z2)
    k = torch.empty((1, 2, 64, 256), dtype=torch.bfloat16, device=DEV)
    v = torch.empty_like(k)
    si.si_kv_read(d.plan, d.cache, d.table[0, 1:2].contiguous(), 1, k, v, d.scratch)
    assert torch.equal(k[0].float(), (d.k_codes[int(c.table[0, 1])].float() * d.k_scale[int(c.table[0, 1])][:, None, None]).bfloat16().float())
    _, lse, _, _ = ref.attend(c, q, 0.06)
    acc = torch.zeros((1, 2, 200), device=DEV)
    si.si_kv_weigh(d.plan, d.cache, d.batch, qd, lse.float().to(DEV), None, acc, 1.0, 0.06, d.scratch)
    w, A = ref.weigh(c, q, lse.float(), None, 1.0, 0.06)
    assert ((acc.cpu().double() - w).abs() <= (2.0 ** -16 * A + 2.0 ** -19) * w + 1e-12).all()
    assert d.status() == si.SI_OK


@pytest.mark.parametrize("n", [1, 200])
def test_another_stream_and_a_graph(n):
    """The calls run on the stream they are given, and a captured step replays on new contents."""
    shape = Shape(8, 2, 128, 64, "int8", "bf16")
    c = ref.make_cache(shape, [1000, 270], [n, n], seed=5)
    d = Dev(c)
    _, qd = make_q(c, 6)
    k = torch.randn((2 * n, 2, 128), device=DEV).bfloat16()
    old = torch.tensor([1000 - n, 270 - n], dtype=torch.int32, device=DEV)
    before = si.kv_batch(2, 2 * n, n, 1000, d.q_start, old, d.table, d.slots)
    lens = torch.zeros_like(old)
    after = si.kv_batch(2, 2 * n, n, 1000, d.q_start, lens, d.table, d.slots)
    out, lse = torch.empty_like(qd), torch.empty((2 * n, 8), device=DEV)
    acc = torch.zeros((2, 2, 1000), device=DEV)
    rings = [(d.k_tail, d.k_tail.clone()), (d.v_tail, d.v_tail.clone())]

    def back():  # a call of more than a page may write over the rows that it began with: put them back
        for ring, was in rings:
            ring.copy_(was)

    def step(stream=None):
        si.si_kv_append(d.plan, d.cache, before, k, k, lens, d.scratch, stream)
        si.si_kv_attend(d.plan, d.cache, after, qd, out, lse, 0.09, d.scratch, stream)
        si.si_kv_weigh(d.plan, d.cache, after, qd, lse, None, acc, 1.0, 0.09, d.scratch, stream)

    step()
    want = [x.clone() for x in (out, lse, acc, lens)]
    back()
    for x in (out, lse, acc, lens):
        x.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((out, lse, acc, lens), want))
    back()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    k2 = torch.randn_like(k)
    k.copy_(k2)
    graph.replay()
    torch.cuda.synchronize()
    got = [x.clone() for x in (out, lse, acc, lens)]
    back()
    step()
    assert all(torch.equal(x, y) for x, y in zip((out, lse, acc, lens), got))
    assert not torch.equal(got[0], want[0])
    assert d.status() == si.SI_OK


@pytest.mark.parametrize("lens,news", [([2600, 900], [2600, 900]), ([6000], [150]), ([4000, 31, 2500], [4, 1, 3])],
                         ids=["prompts", "chunk", "steps"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_every_repetition_gives_the_same_bits(code, dim, lens, news):
    """Warps and CTAs meet in another order each time; the sums keep theirs."""
    shape = Shape(8, 2, dim, 32, code, "bf16")
    c = ref.make_cache(shape, lens, news, seed=dim)
    d = Dev(c)
    _, qd = make_q(c, 4)
    want = None
    for _ in range(40):
        out, lse = d.attend(qd, dim ** -0.5)
        acc = torch.zeros((len(lens), 2, max(lens)), device=DEV)
        si.si_kv_weigh(d.plan, d.cache, d.batch, qd, lse, None, acc, 1.0, dim ** -0.5, d.scratch)
        if want is None:
            want = (out, lse, acc)
        assert all(torch.equal(x, y) for x, y in zip((out, lse, acc), want))
    assert d.status() == si.SI_OK
