"""Prefill calls whose shared memory passes to the next one at once."""
import pytest
import torch

from quantized_moe_expert_gemv_gb300 import binding, build, device, synth

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 33, 300])
def test_calls_back_to_back_repeat_bit_for_bit(tokens):
    """Sums have a fixed order, so each call has the bits of the first.  One token leaves one chunk a pass, of which the
    second issuing thread has none."""
    build.build()
    binding.load_library()
    layer = device.to_device(synth.make_layer(synth.TINY, seed=3))
    plan = binding.si_moe_plan(device.desc_for(synth.TINY, max_tokens=tokens))
    scratch = device.alloc_scratch(plan, binding.SI_MODE_PREFILL, tokens)
    x = device.tokens_to_device(synth.make_tokens(synth.TINY, seed=5, n_tokens=tokens))
    outs = [torch.full((tokens, synth.TINY.hidden), 7.0, device="cuda") for _ in range(21)]
    for first in (True, False, False, False):
        for out in outs[:1] if first else outs[1:]:
            binding.si_moe_forward_prefill(plan, layer.struct(), x, tokens, out, None, scratch)
        assert torch.isfinite(outs[0]).all()
        if not first:
            assert all(torch.equal(out, outs[0]) for out in outs[1:])
            for out in outs[1:]:
                out.fill_(7)
    assert binding.si_moe_read_status(plan, scratch) == binding.SI_OK
