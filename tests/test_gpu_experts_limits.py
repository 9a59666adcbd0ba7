"""The routed-expert operators at the ends of their limits, on the GPU.

Inputs repeat or are constant, so that what is expected needs no second pass
over gigabytes on the host."""
import pytest

import adapter_lora_serving_amd as L
from gpu_util import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T", [(1 << 23) + 1, (1 << 24) - 1, 1 << 24, (1 << 25) + 3])
def test_combine_of_many_tokens(T):
    """From 2^24 tokens on, a workgroup a token is 2^32 threads and more."""
    t = torch()
    rows = t.stack([t.full((8,), float(v), device=DEV) for v in range(1, 5)]).bfloat16()
    pos = (t.arange(T, device=DEV) % 5 - 1).int().unsqueeze(1)   # -1: adds nothing
    y = t.full((T, 8), -1.0, device=DEV).bfloat16()
    L.combine_experts(rows, pos, t.full((T, 1), 2.0, device=DEV), y=y)
    want = 2 * (pos + 1).bfloat16().expand(T, 8)
    assert t.equal(y, want)
