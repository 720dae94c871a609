"""What the dense block's calls and its binding refuse, beside the arguments that no call takes."""
import pytest
import torch

from quantized_moe_expert_gemv_gb300 import binding
from test_fp8_host import BAD, OK, Call, checks  # noqa: F401 (a fixture)


def test_the_status_is_read_on_the_plans_device_alone(checks):  # noqa: F811
    """Another device's stream does not wait for the plan's kernels: the word would be read while they run."""
    c = Call(checks)
    assert checks.si_fp8_read_status(c.h, 0x1000, None) == OK
    before = checks.stub_launches()
    checks.stub_device(1)
    try:
        assert checks.si_fp8_read_status(c.h, 0x1000, None) == BAD and checks.stub_launches() == before
    finally:
        checks.stub_device(0)


def test_the_binding_reads_the_status_in_the_plans_stream(monkeypatch):
    plan = binding.Fp8Plan(0, binding.make_fp8_desc(512, 300), 1)
    with pytest.raises(ValueError, match="device 1"):  # (a scratch in host memory)
        binding.si_fp8_read_status(plan, torch.zeros(512, dtype=torch.uint8))

    class Lib:
        def si_fp8_read_status(self, *args):
            return args
    monkeypatch.setattr(binding, "load_library", Lib)
    monkeypatch.setattr(binding, "_fp8_raw_stream", lambda device: 1000 + device)
    monkeypatch.setattr(binding, "_fp8_scratch", lambda plan, scratch: 77)
    assert binding.si_fp8_read_status(plan, None) == (0, 77, 1001)
    assert binding.si_fp8_read_status(plan, None, 5) == (0, 77, 5)
