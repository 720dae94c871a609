"""The example layer's bookkeeping: sums of tokens that never had one, and the status across calls of any size."""
import pytest
import torch

import kv_reference as ref
from test_gpu_decoder_layer import snapshot

pytestmark = pytest.mark.gpu


def tiny(**kw):
    from quantized_moe_expert_gemv_gb300 import synth
    from quantized_moe_expert_gemv_gb300.decoder_layer import DecoderLayer
    args = dict(heads=4, kv=2, dim=64, page=16, code="int8", n_seqs=3, max_len=256, budget=5, sink=1, recent=2, window=8)
    return DecoderLayer(synth.TINY, **{**args, **kw})


def rows(n, seed):
    return torch.randn((n, 256), generator=torch.Generator(device="cuda:0").manual_seed(seed), device="cuda:0").bfloat16()


def test_a_second_prompt_starts_without_sums():
    """Prompts longer than the window, after evictions have left old sums past the lengths: the sums afterwards are the
    decayed ones of the cached tokens and the window's weights alone."""
    layer = tiny()
    layer.prompts(rows(140, 1), [100, 33, 7])
    layer.prompts(rows(180, 2), [40, 60, 80])
    assert max(layer.host_lens) <= 6 * 16 and layer.acc.any()
    evict, layer.evict = layer.evict, lambda: False
    for counts, seed in (([70, 20, 30], 3), ([3, 40, 9], 4)):
        before, lens = layer.acc.cpu().clone(), list(layer.host_lens)
        layer.prompts(rows(sum(counts), seed), counts)
        for b, L in enumerate(lens):
            before[b, :, L:] = 0
        last = [min(n, layer.window) for n in counts]
        c = snapshot(layer, last, "int8")
        at, pick = 0, []
        for n, m in zip(counts, last):
            pick += range(at + n - m, at + n)
            at += n
        q, _, lse = (t.cpu() for t in layer.last)
        want, A = ref.weigh(c, q[pick], lse[pick], before, layer.decay, layer.sm)
        for b, L in enumerate(layer.host_lens):
            got, w = layer.acc[b, :, :L].cpu().double(), want[b, :, :L]
            assert ((got - w).abs() <= (2.0 ** -16 * A + 2.0 ** -19) * w + 1e-12).all(), b
    layer.evict = evict
    assert layer.evict() and layer.status() == 0


def test_an_error_before_a_larger_call_is_still_reported():
    from quantized_moe_expert_gemv_gb300 import binding as si
    layer = tiny()
    layer.attention(rows(60, 1), [20, 20, 20])
    layer.table[1, 0] = 10 ** 6
    layer.attention(rows(3, 2), [1, 1, 1])
    layer.table[1, 0] = layer.pages[1][0]
    layer.attention(rows(400, 3), [150, 130, 120])
    assert layer.status() == si.SI_ERR_DEVICE and layer.status() == si.SI_OK
