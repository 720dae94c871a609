"""The dense block's products where one call's shared memory passes to the next at once, waits that run out in each of the
kernels, and memory that no call takes."""
import pytest
import torch

import fp8_reference as ref
from test_gpu_fp8 import DEV, Product, empty_rows, randn
from quantized_moe_expert_gemv_gb300 import binding as si

pytestmark = pytest.mark.gpu


def check_back_to_back(sizes, reps):
    """Calls of all sizes in turn with nothing between them, each into outputs of its own: the bits of its first call, which
    are those of the definition."""
    ps = [Product(t, n, k, seed=t + n) for t, n, k in sizes]
    firsts = []
    for p in ps:
        firsts.append(p(torch.empty((p.t, p.n), device=DEV)))
        ref.check_out(firsts[-1], *p.want(), p.k)
    outs = [[torch.empty((p.t, p.n), device=DEV) for _ in range(8)] for p in ps]
    off = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(reps // 8):
        for mine in outs:
            for out in mine:
                out.fill_(7)
        for i in range(8):
            for p, mine in zip(ps, outs):
                p(mine[i])
        off += sum((out != first).sum() for mine, first in zip(outs, firsts) for out in mine)
    assert off.item() == 0
    assert all(p.status() == si.SI_OK for p in ps)


# A CTA pair of which the odd CTA has no rows (up to 128) ends as early as it can: its last signals come from products that
# the even one issued, and the next call's barriers take the place of the ones that they are meant for.
@pytest.mark.parametrize("sizes", [[(100, 5120, 16)], [(128, 5120, 1024)], [(65, 12800, 128)], [(128, 5120, 144), (120, 12800, 640)],
                                   [(100, 5120, 256), (300, 640, 256)]], ids=str)
def test_pairs_hand_over_their_memory(sizes):
    check_back_to_back(sizes, 1600)


# A call of few rows and blocks ends right after its products; kernels of all kinds take each other's place.
@pytest.mark.parametrize("sizes", [[(1, 5120, 16)], [(3, 5120, 640), (40, 5120, 128)], [(64, 2048, 512), (17, 2048, 144)],
                                   [(128, 5120, 640), (3, 5120, 640), (120, 12800, 128), (64, 2048, 512)]], ids=str)
def test_few_rows_hand_over_their_memory(sizes):
    check_back_to_back(sizes, 1600)


# 304 and 5000 columns: outputs by boxes, alone, with `add` by boxes, and with one of another type; 300: rows that end anywhere
@pytest.mark.parametrize("out,add", [("f32", None), ("bf16", None), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f32")])
@pytest.mark.parametrize("t,n", [(1, 304), (40, 304), (300, 304), (300, 5000), (300, 300)])
def test_each_wait_that_runs_out_is_reported(monkeypatch, t, n, out, add):
    monkeypatch.setenv("SI_FAULT_WAIT_BUDGET", "2000000")
    p = Product(t, n, 512, seed=1)
    monkeypatch.delenv("SI_FAULT_WAIT_BUDGET")
    q = Product(t, n, 512, seed=1)
    a = None if add is None else randn(p.g, t, n, dtype=ref.TYPES[add])
    got = torch.empty((t, n), dtype=ref.TYPES[out], device=DEV)
    for _ in range(2):
        p(got, a)
        assert p.status() == si.SI_ERR_TIMEOUT and p.status() == si.SI_OK
        q(got, a)  # (the next call, right after it, is as good as ever)
        ref.check_out(got, *q.want(a), 512)
        assert q.status() == si.SI_OK


def test_calls_take_no_memory():
    """Neither the device's, once the kernels have been loaded, nor torch's."""
    plans = []
    for t, n, k in ((1, 640, 512), (40, 640, 512), (300, 640, 512), (300, 5000, 512), (300, 301, 512)):
        p = Product(t, n, k, seed=2)
        codes, scales = empty_rows(t, k)
        weight = si.fp8_weight(torch.empty_like(p.w_codes), torch.empty_like(p.w_scales))
        w, x = randn(p.g, n, k), randn(p.g, t, k, dtype=torch.bfloat16)
        plans.append((p, w, weight, x, torch.empty_like(x), torch.ones(k, device=DEV), si.fp8_rows(codes, scales),
                      torch.empty((t, n), dtype=torch.bfloat16, device=DEV)))

    def calls():
        for p, w, weight, x, y, gain, rows, out in plans:
            si.si_fp8_pack(p.plan, w, weight)
            si.si_fp8_norm(p.plan, x, x, gain, 1e-6, y, None, rows, p.t)
            for add in (None, out):
                si.si_fp8_matmul(p.plan, rows, weight, add, out, p.t, p.scratch)

    def held():
        torch.cuda.synchronize()
        return torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()
    calls()
    before = held()
    for _ in range(20):
        calls()
    assert held() == before
