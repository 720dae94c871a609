"""The dense block's products where one call's shared memory passes to the next at once."""
import pytest
import torch

import fp8_reference as ref
from test_gpu_fp8 import DEV, Product
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
