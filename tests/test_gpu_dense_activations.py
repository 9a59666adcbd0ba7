"""The products' activations in float32 against their formulas in fp64: a product of
zeros leaves act(bias), so every z is met as it is. The bounds are those of the
kernels' own comments; values below 2^-120 may be 0."""
import math

import numpy as np
import pytest

import adapter_lora_serving_amd as L
from gpu_util import f64, torch
from test_gpu_dense import DEV, gpu

pytestmark = pytest.mark.gpu


def ref(z, act):
    """The activation by its formula, without cancellation on the negative side."""
    z = z.astype(np.float64)
    if act == "gelu":
        return z / 2 * np.array([math.erfc(-v / math.sqrt(2)) for v in z])
    u = z if act == "silu" else 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z**3)
    with np.errstate(over="ignore"):
        return z / (1 + np.exp(-u))


def bound(z, act):
    z = np.abs(z.astype(np.float64))
    if act == "gelu":
        return 2.0**-19
    if act == "silu":
        return (z + 4) * 2.0**-23
    return (4 * 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z**3) + 4) * 2.0**-23


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T", [1, 70])
def test_relative_error(T, act):
    t = torch()
    rng = np.random.default_rng(T)
    z = np.concatenate([rng.uniform(-13, 13, 40000), rng.uniform(-1, 1, 20000), np.linspace(-6, 6, 20000),
                        np.exp2(rng.uniform(-60, 4, 4000)) * rng.choice([-1, 1], 4000)]).astype(np.float32)
    x, w = t.zeros(T, 8, device=DEV).bfloat16(), t.zeros(len(z), 8, device=DEV).bfloat16()
    y = f64(L.epilogue_linear(x, w, bias=gpu(z), activation=act, dtype=t.float32))
    assert (y == y[:1]).all()
    want = ref(z, act)
    err = np.abs(y[0] - want)
    over = err / (bound(z, act) * np.abs(want) + np.where(np.abs(want) < 2.0**-120, 2.0**-120, 0.0))
    worst = over.argmax()
    print(act, "worst relative error", (err / np.abs(want))[np.abs(want) > 2.0**-120].max())
    assert over[worst] <= 1, (float(z[worst]), float(err[worst]), float(want[worst]))


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("T", [1, 70])
def test_ends(T, act):
    """Far out a gate is open or shut; infinity, zero and a NaN."""
    t = torch()
    z = t.tensor([20.0, 1e10, 3e38, float("inf"), -100.0, -1e10, -3e38, 0.0, -0.0, float("nan")], device=DEV)
    x, w = t.zeros(T, 8, device=DEV).bfloat16(), t.zeros(10, 8, device=DEV).bfloat16()
    y = L.epilogue_linear(x, w, bias=z, activation=act, dtype=t.float32)
    assert (y[:, :4] == z[:4]).all() and (y[:, 4:9].abs() < 2.0**-120).all() and t.isnan(y[:, 9]).all()
