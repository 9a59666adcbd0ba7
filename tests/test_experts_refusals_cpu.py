"""More refusals of the routed-expert operators, on the CPU: no call here
reaches a kernel launch."""
import os

import pytest

import adapter_lora_serving_amd as L
from adapter_lora_serving_amd import build

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
A16 = 0x10000   # a device address that is never dereferenced here


@pytest.fixture(scope="module")
def lib():
    if not (os.path.exists(L.lib_path()) and os.path.exists(build.BINDING_PATH)):
        build.build()
    return L.lib()


@pytest.mark.parametrize("T,k", [(1 << 59, 32), ((1 << 59) + 1, 32), (1 << 62, 4), ((1 << 63) - 1, 2),
                                 (1 << 31, 1), (1 << 30, 2)])
def test_choices_past_64_bits_are_refused(lib, T, k):
    """T * k is a multiple of 2^64 in the first rows, so its low bits look small."""
    assert lib.lora_route_experts(1, A16, T, 64, k, 0, None, 1, 1, 0, 1, 1.0, A16, A16,
                                  None) == INVALID
    assert lib.lora_expert_rows(A16, T, k, 8, None, A16, A16, A16, None, None, 0, None) == INVALID
    assert lib.lora_expert_rows_workspace_bytes(T, k, 8) == 0
    assert lib.lora_combine_experts(1, A16, 8, 64, A16, A16, T, k, None, A16, None) == INVALID


@pytest.mark.parametrize("n", [(1 << 31) - 1, (1 << 31) - 255, (1 << 31) - 1023])
@pytest.mark.parametrize("E", [8, 1023, 1024])
def test_rows_whose_blocks_pass_32_bits_are_refused(lib, n, E):
    """Rounded up to whole blocks of 1024 choices, n is 2^31."""
    need = lib.lora_expert_rows_workspace_bytes(n, 1, E)
    assert need == 0
    assert lib.lora_expert_rows(A16, n, 1, E, None, A16, A16, A16, None, A16, 1 << 40,
                                None) == INVALID
    need = lib.lora_expert_rows_workspace_bytes((1 << 31) - 1024, 1, E)
    assert need == (0 if E == 1024 else ((1 << 21) - 1) * (E + 1) * 4)


@pytest.mark.parametrize("off", [1, 2, 3])
def test_route_bias_between_floats_is_refused(lib, off):
    assert lib.lora_route_experts(1, A16, 4, 64, 2, 0, A16 + off, 1, 1, 0, 1, 1.0, A16, A16,
                                  None) == ALIGN


def test_compiled_binding_refuses_cpu_tensors(lib):
    """Its own message: without the binding the same type says that it is not built."""
    import torch
    x = torch.zeros(2, 64)
    i = torch.zeros(2, 2, dtype=torch.int32)
    q = L.MXFP4(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 4, dtype=torch.uint8))
    for f in (lambda: L.route_experts(x, 2), lambda: L.expert_rows(i, 4),
              lambda: L.combine_experts(x, i, torch.zeros(2, 2)), lambda: L.quantize_mxfp4(x),
              lambda: L.gather_quantize_mxfp4(x, i[0]), lambda: L.silu_mul_quantize_mxfp4(x),
              lambda: L.dequantize_mxfp4(q), lambda: L.mxfp4_linear(q, q),
              lambda: L.mxfp4_expert_linear(q, q, i[0])):
        with pytest.raises(L.LoraError, match="must be on the GPU"):
            f()
    for f in (lambda: L.route_experts([[0.0]], 1), lambda: L.dequantize_mxfp4([q[0], q[1]])):
        with pytest.raises(L.LoraError, match="must be"):
            f()
