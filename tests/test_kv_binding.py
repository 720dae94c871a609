"""What the binding refuses before a call: tensors whose shapes the C side, which sees addresses alone, cannot check."""
import pytest
import torch

from quantized_moe_expert_gemv_gb300 import binding as si


def cache(**kw):
    t = dict(k_codes=torch.zeros(9, 2, 16, 64, dtype=torch.int8), v_codes=torch.zeros(9, 2, 16, 64, dtype=torch.int8),
             k_scale=torch.zeros(9, 2), v_scale=torch.zeros(9, 2), k_tail=torch.zeros(3, 2, 32, 64, dtype=torch.bfloat16),
             v_tail=torch.zeros(3, 2, 32, 64, dtype=torch.bfloat16))
    return si.kv_cache(**{**t, **kw})


def ints(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def batch(**kw):
    t = dict(n_seqs=3, total_new=5, max_new=2, max_len=64, q_start=ints(4), lens=ints(3), page_table=ints(3, 4), slots=ints(3))
    return si.kv_batch(**{**t, **kw})


def test_cache():
    assert cache().n_pages == 9 and cache().n_slots == 3
    assert cache(k_codes=torch.zeros(9, 2, 16, 64, dtype=torch.float8_e4m3fn)).n_pages == 9
    for kw in (dict(v_codes=torch.zeros(8, 2, 16, 64, dtype=torch.int8)), dict(k_scale=torch.zeros(9, 4)), dict(v_scale=torch.zeros(8, 2)),
               dict(k_scale=torch.zeros(9, 2, dtype=torch.float64)), dict(k_tail=torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)),
               dict(v_tail=torch.zeros(2, 2, 32, 64, dtype=torch.bfloat16)), dict(k_tail=torch.zeros(3, 2, 32, 64)),
               dict(k_codes=torch.zeros(9, 2, 16, 64)), dict(k_codes=torch.zeros(9, 2, 64, 16, dtype=torch.int8).transpose(2, 3)),
               dict(k_codes=torch.zeros(9, 2, 16 * 64, dtype=torch.int8), v_codes=torch.zeros(9, 2, 16 * 64, dtype=torch.int8))):
        with pytest.raises(ValueError):
            cache(**kw)


def test_batch():
    assert batch().table_stride == 4 and batch(slots=None, page_table=ints(5, 9)[:, :4]).table_stride == 9
    for kw in (dict(q_start=ints(3)), dict(lens=ints(2)), dict(slots=ints(2)), dict(page_table=ints(2, 4)), dict(page_table=ints(12)),
               dict(lens=torch.zeros(3, dtype=torch.int64)), dict(page_table=ints(3, 4).float()), dict(lens=ints(3, 2)[:, 0]),
               dict(page_table=ints(4, 3).T), dict(q_start=ints(4).to(torch.int64))):
        with pytest.raises(ValueError):
            batch(**kw)


def test_sums():
    plan = si.KvPlan(0, si.make_kv_desc(4, 2, 64, 16))
    q, lse = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 4)
    good, scratch = torch.zeros(3, 2, 64), torch.zeros(64)
    for acc_in, acc_out in ((torch.zeros(3, 2, 65), good), (good, torch.zeros(3, 2, 63)), (None, torch.zeros(2, 2, 64)),
                            (torch.zeros(3, 2, 128)[:, :, ::2], good), (good, torch.zeros(2, 3, 64).transpose(0, 1)), (None, torch.zeros(6, 64))):
        with pytest.raises(ValueError):
            si.si_kv_weigh(plan, cache(), batch(), q, lse, acc_in, acc_out, 1.0, 0.1, scratch)
        with pytest.raises(ValueError):
            si.si_kv_evict(plan, cache(), batch(), torch.zeros(3, 2, 66) if acc_in is None else acc_in, acc_out, 4, 0, 0, ints(3, 4), None,
                           ints(3, 2, 4), ints(3), scratch)
    for table, keep in ((ints(3, 5), ints(3, 2, 4)), (ints(3, 4), ints(3, 2, 5)), (ints(3, 8)[:, ::2], ints(3, 2, 4)), (ints(3, 4), ints(2, 3, 4).transpose(0, 1))):
        with pytest.raises(ValueError):
            si.si_kv_evict(plan, cache(), batch(), good, good.clone(), 4, 0, 0, table, None, keep, ints(3), scratch)
