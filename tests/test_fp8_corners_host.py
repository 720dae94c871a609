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


@pytest.mark.parametrize("dtype", [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.int8, torch.bool], ids=str)
def test_codes_of_another_8_bit_type_are_refused(dtype):
    """Their bits would be read as E4M3."""
    codes = torch.zeros(6, 300, dtype=torch.uint8).view(dtype)
    for make, scales in ((binding.fp8_rows, torch.zeros(3, 8)), (binding.fp8_weight, torch.zeros(1, 3))):
        with pytest.raises(ValueError, match="8 bits"):
            make(codes, scales)


@pytest.mark.parametrize("dtype", [torch.float8_e4m3fn, torch.uint8], ids=str)
def test_codes_in_e4m3_or_its_bytes_are_taken(dtype, monkeypatch):
    monkeypatch.setattr(binding, "_on_device", lambda *tensors: 0)  # (tensors in host memory here)
    codes = torch.zeros(6, 300, dtype=torch.uint8).view(dtype)
    assert binding.fp8_rows(codes, torch.zeros(3, 8)).rows == 6 and binding.fp8_weight(codes, torch.zeros(1, 3)).rows == 6
