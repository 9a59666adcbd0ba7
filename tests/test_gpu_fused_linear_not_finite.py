"""An adapter whose B is not finite, in the base projection with the delta in its
epilogue (fused_column_linear): the rows of other slots and of none keep the bits
that they have without it."""
import numpy as np
import pytest

import adapter_lora_serving_amd as L
from gpu_util import f64, torch
from test_gpu_dense import bf16, gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [40, 300, 1100])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_rows_of_other_slots_keep_their_bits(T, bad):
    t = torch()
    rng = np.random.default_rng(T)
    slots, R, K, slices = 5, 40, 128, (256, 512)
    out = sum(slices)
    slot = rng.integers(-1, slots, T)
    slot[T // 2] = 3
    ranks = np.array([16, 0, 40, 33, 7], np.int32)
    x, w = bf16(rng, T, K)[1], bf16(rng, out, K, std=0.1)[1]
    a, b = bf16(rng, slots, 2 * R, K, std=0.1)[1], bf16(rng, slots, out, R, std=0.3)[1]
    addr = L.build_addressing(gpu(slot.astype(np.int32)), slots)
    scal = gpu(np.array([1.0, 2.0, 0.5, 0.75, 1.5], np.float32))

    def run(bb):
        return L.fused_column_linear(x, w, a, bb, addr, gpu(ranks), scal, slices)

    clean = run(b)
    assert t.isfinite(clean).all()
    for column in (0, 255, 700):
        pb = b.clone()
        pb[3, column, 32] = bad
        y = run(pb)
        hit = t.zeros(T, out, dtype=t.bool, device=y.device)
        hit[gpu(slot == 3), column] = True
        assert t.equal(y[~hit], clean[~hit])
        assert not t.isfinite(y[hit]).any()
        if np.isinf(bad):   # infinity times a finite h, of the product's sign
            h = L.shrink(x, a, addr, gpu(ranks), 2)
            sign = np.sign(f64(h)[slot == 3, (0 if column < 256 else R) + 32]) * np.sign(bad)
            assert np.array_equal(f64(y)[slot == 3, column], sign * np.inf)
