"""Arguments of another kind are refused as any other invalid one is: by LoraError."""
import os

import pytest

import adapter_lora_serving_amd as L
from adapter_lora_serving_amd import build


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(build.DENSE_BINDING_PATH):
        build.build()


@pytest.mark.parametrize("bad", ["1e-6", None, [1e-6], 1 << 2000])
def test_norm_numbers(bad):
    import torch
    x = torch.zeros(2, 64).bfloat16()
    for f in (L.add_rms_norm, L.add_rms_norm_quantize_mxfp8):
        with pytest.raises(L.LoraError, match="eps must be a number"):
            f(x, x[0], eps=bad)
        with pytest.raises(L.LoraError, match="weight_offset must be a number"):
            f(x, x[0], weight_offset=bad)


def test_an_error_of_the_argument_s_own_is_raised():
    import torch

    class Mine(Exception):
        pass

    class Odd:
        def __float__(self):
            raise Mine

    with pytest.raises(Mine):
        L.add_rms_norm(torch.zeros(2, 64), torch.zeros(64), eps=Odd())
