"""Arguments of another kind that are looked at after the tensors."""
import pytest

import adapter_lora_serving_amd as L
from gpu_util import torch
from test_gpu_dense import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [32, None, 1.5, ("32",), (32.0,)])
def test_out_slices(bad):
    t = torch()
    x, w = t.zeros(4, 64, device=DEV).bfloat16(), t.zeros(32, 64, device=DEV).bfloat16()
    d = L.Delta(t.zeros(4, 8, device=DEV), t.zeros(2, 32, 8, device=DEV).bfloat16(),
                L.build_addressing(t.zeros(4, dtype=t.int32, device=DEV), 2),
                t.zeros(2, dtype=t.int32, device=DEV), t.zeros(2, device=DEV), bad)
    for f in (L.epilogue_linear, L.gated_linear):
        with pytest.raises(L.LoraError, match="out_slices must be"):
            f(x, w, delta=d)
