"""Scale byte 0, 2^-127, in the products, the quantisation and back."""
import numpy as np
import pytest

import adapter_lora_serving_amd as L
from gpu_util import f64, torch
from oracle import dense_oracle as D
from test_gpu_dense import DEV

pytestmark = pytest.mark.gpu


# a kernel for few rows and one of tiles, for either result type
@pytest.mark.parametrize("T", [3, 20, 50, 100, 300])
@pytest.mark.parametrize("code", [0x7E, 0x40, 0x3C, 0xC1])
def test_byte_0_is_2_to_the_minus_127(T, code):
    """Every code of x under byte 0 against ones of a W that is large: values of 2^-126 and
    more come out as they are, whichever way the result is formed."""
    t = torch()
    K, N = 160, 96
    v = D.E4M3[code & 127] * (-1.0 if code > 127 else 1.0) * 2.0**-127
    # 1.5 2^-127 is below bf16's normal values, which a float32 y may take for 0
    exact = (t.bfloat16, t.float32) if abs(v) >= 2.0**-126 else (t.bfloat16,)
    x = L.MXFP8(t.full((T, K), code, dtype=t.uint8, device=DEV), t.zeros(T, 16, dtype=t.uint8, device=DEV))
    w = L.MXFP8(t.full((2 * N, K), 0x38, dtype=t.uint8, device=DEV),
                t.full((2 * N, 16), 240, dtype=t.uint8, device=DEV))
    ref = K * v * 2.0**113
    for dt in exact:
        for a, b, rows in ((x, w, 2 * N), (L.MXFP8(w.codes[:T].contiguous(), w.scales[:T].contiguous()),
                                           L.MXFP8(x.codes[:T].contiguous(), x.scales[:T].contiguous()), T)):
            if a.codes.shape[0] < T:
                continue
            y = f64(L.epilogue_linear(a, b, dtype=dt))
            assert y.shape == (T, rows) and (y == ref).all(), (dt, y[0, 0], ref)
    if abs(v) >= 2.0**-126:
        for held in (False, True):
            f = L.gated_linear_quantize_mxfp8 if held else L.gated_linear
            bias = t.ones(2 * N, device=DEV)
            bias[:N] = 0
            out = f(x, w, bias=bias, activation=None)
            rows = f64(out[0] if held else out)
            want = np.float64(t.tensor(ref * (ref + 1), dtype=t.float64).bfloat16().double().item())
            assert (rows == want).all(), (held, rows[0, 0], want)


def test_byte_0_from_and_to_float32():
    t = torch()
    x = t.zeros(2, 64, device=DEV)
    x[0, :6] = t.tensor([2.0**-126, -(2.0**-127), 3 * 2.0**-128, 2.0**-133, 2.0**-149, 0.0])
    x[1, 32:36] = t.tensor([448 * 2.0**-127, 2.0**-127, -17 * 2.0**-127, 19 * 2.0**-127])
    q = L.quantize_mxfp8(x)
    codes, scales = D.quantize(f64(x))
    assert np.array_equal(q.codes.view(t.uint8).cpu().numpy(), codes) and np.array_equal(q.scales.cpu().numpy(), scales)
    assert not q.scales.any()
    assert np.array_equal(f64(L.dequantize_mxfp8(q, t.float32)), D.dequantize(codes, scales))
