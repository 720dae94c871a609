"""The example layer (quantized_moe_expert_gemv_gb300/decoder_layer.py) runs the cache's operators and the expert
block together: its attention is that of its own cache, its lengths and kept pages follow the rules."""
import pytest
import torch

import kv_reference as ref
from kv_reference import Shape

pytestmark = pytest.mark.gpu


def snapshot(layer, counts, code):
    """The layer's cache as a reference cache."""
    shape = Shape(layer.heads, layer.kv, layer.dim, layer.page, code, "bf16")
    c = ref.Cache(shape, layer.tensors[0].shape[0], layer.n, list(layer.host_lens), list(counts))
    c.table, c.slots = layer.table.cpu(), torch.arange(layer.n, dtype=torch.int32)
    c.t = dict(zip(("k_codes", "v_codes", "k_scale", "v_scale", "k_tail", "v_tail"), (t.cpu() for t in layer.tensors)))
    return c


def check_attention(layer, c):
    q, out, lse = (t.cpu() for t in layer.last)
    want, z, S, A = ref.attend(c, q, layer.sm)
    half = torch.finfo(torch.bfloat16).eps / 2
    assert ((out.double() - want).abs() <= half * want.abs() + (2.0 ** -11 + 2.0 ** -14) * S + 2.0 ** -25).all()
    assert ((lse.double() - z).abs() <= 2.0 ** -17 * A + 2.0 ** -21 * (1 + z.abs())).all()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_layer(code):
    from quantized_moe_expert_gemv_gb300 import binding as si, synth
    from quantized_moe_expert_gemv_gb300.decoder_layer import DecoderLayer
    layer = DecoderLayer(synth.TINY, heads=4, kv=2, dim=64, page=16, code=code, n_seqs=3, max_len=256, budget=5, sink=1,
                         recent=2, window=8)
    counts = [100, 33, 7]
    g = torch.Generator(device="cuda:0").manual_seed(3)
    x = torch.randn((sum(counts), 256), generator=g, device="cuda:0").bfloat16()
    evict, layer.evict = layer.evict, lambda: False
    y = layer.prompts(x, counts)
    assert y.shape == x.shape and torch.isfinite(y).all()
    check_attention(layer, snapshot(layer, counts, code))
    sums = layer.acc.double().sum(2)  # a weight of one from each of the window's rows and of the group's two heads
    want = torch.tensor([[2.0 * min(n, 8)] for n in counts], dtype=torch.float64, device="cuda:0")
    assert ((sums - want).abs() <= want * 2.0 ** -14).all()
    layer.evict = evict
    assert layer.evict() and layer.host_lens == [5 * 16 + 4, 33, 7] == layer.lens.tolist()
    kept = layer.kept.cpu()
    assert (kept[0, :, 0] == 0).all() and (kept[0, :, 3:] == torch.tensor([4, 5])).all() and (kept[1, :, 2:] == -1).all()
    x = y[torch.tensor([99, 132, 139], device="cuda:0")]
    for i in range(60):
        before = None if i % 12 else True
        layer.evict = (lambda: False) if before else evict
        y = layer.step(x)
        assert torch.isfinite(y).all()
        if before:
            check_attention(layer, snapshot(layer, [1, 1, 1], code))
            evict()
        assert layer.lens.tolist() == layer.host_lens and max(layer.host_lens) < 6 * 16
    assert layer.positions == [160, 93, 67]
    assert len(set(sum(layer.pages, []))) == sum(map(len, layer.pages)) and not set(layer.free) & set(sum(layer.pages, []))
    assert layer.status() == si.SI_OK
