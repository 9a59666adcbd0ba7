"""MXFP4 products: the bits of a row do not depend on the tile that forms it,
and scales hold over their whole range.

The sizes are those at which 256 compute units take each shape of tile."""
import numpy as np
import pytest

import adapter_lora_serving_amd as L
from gpu_util import torch
from test_gpu_experts import DEV, held

pytestmark = pytest.mark.gpu
HELD = {}


def part(q, lo, hi):
    return L.MXFP4(q.codes[lo:hi].contiguous(), q.scales[lo:hi].contiguous())


def operands(rows, N, K):
    """Operands and the y of all of them, made once for a K."""
    if K not in HELD:
        HELD.clear()
        x, w = held(rows, K, K), held(N, K, K + 1)
        HELD[K] = x, w, L.mxfp4_linear(x, w, dtype=torch().float32)
    return HELD[K]


# (first row, rows, columns) of a product cut out of 5120 x 33024 x 1056, which
# 256 x 256 tiles form
DEEP = {
    "256x256": (37, 1024, 12288), "256x256 and halves": (0, 5120, 3840),
    "128x128": (9, 512, 12288), "64x64, four stages": (100, 65, 500),
    "64x64, one row": (77, 1, 6000), "32x128": (3, 8, 20000), "64x128, three stages": (50, 40, 17000),
    "64x128, scale registers": (300, 600, 5300), "64x64, scale registers": (11, 40, 33024),
}
# the same out of 1024 x 12288 x 480, by 128 x 128 tiles
SHALLOW = {"64x128, shallow": (100, 65, 500), "64x128, one row": (5, 1, 12288),
           "128x128, shallow": (24, 1000, 12160)}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name", list(DEEP) + list(SHALLOW))
def test_same_bits_in_every_tiling(name, dtype):
    t = torch()
    deep = name in DEEP
    x, w, whole = operands(5120, 33024, 1056) if deep else operands(1024, 12288, 480)
    at, rows, cols = (DEEP if deep else SHALLOW)[name]
    dt = t.float32 if dtype == "f32" else t.bfloat16
    y = L.mxfp4_linear(part(x, at, at + rows), part(w, 0, cols), dtype=dt)
    assert t.equal(y, whole[at:at + rows, :cols].to(dt))


# rows of each expert, columns; what the averages make of them
GROUPED = {
    "256x256": ([1500, 0, 1400, 1], 8192), "256x256 and halves": ([1293, 1, 1299, 1290], 4700),
    "128x128": ([130, 60, 129, 100], 8192), "64x64, four stages": ([3, 0, 70, 1], 600),
    "32x128": ([8, 1, 5, 9], 8192), "64x128, three stages": ([20, 1, 2, 30], 8192),
    "64x128, scale registers": ([65, 130, 64, 200], 3500),
    "64x64, scale registers": ([30, 65, 2, 64], 8256),
}


@pytest.mark.parametrize("K", [1056, 480])
@pytest.mark.parametrize("name", list(GROUPED))
def test_grouped_rows_have_the_dense_bits(name, K):
    t = torch()
    counts, N = GROUPED[name]
    off = np.concatenate([[0], np.cumsum(counts)])
    x = held(int(off[-1]), K, N)
    w = held(4 * N, K, N + 1)
    y = L.mxfp4_expert_linear(x, L.MXFP4(w.codes.view(4, N, -1), w.scales.view(4, N, -1)),
                              t.from_numpy(off).to(DEV), dtype=t.float32)
    for e in range(4):
        lo, hi = int(off[e]), int(off[e + 1])
        one = L.mxfp4_linear(part(x, lo, hi), part(w, e * N, (e + 1) * N), dtype=t.float32)
        assert t.equal(y[lo:hi], one), e


@pytest.mark.parametrize("code", [1, 2, 7])
@pytest.mark.parametrize("K", [32, 544])
def test_every_pair_of_scales(code, K):
    """One product a value, 2^-127 to 2^127 against the same: it is exact or
    fp32's rounding of the exact product, denormal and infinite ones too."""
    t = torch()
    c = t.zeros(255, K // 2, dtype=t.uint8, device=DEV)
    c[:, 0] = code
    s = t.zeros(255, -(-(K // 32) // 4) * 4, dtype=t.uint8, device=DEV)
    s[:, 0] = t.arange(255, device=DEV)
    y = L.mxfp4_linear(L.MXFP4(c, s), L.MXFP4(c, s), dtype=t.float32)
    e = np.arange(255) - 127.0
    v = {1: 0.5, 2: 1.0, 7: 6.0}[code]
    with np.errstate(over="ignore"):
        want = (v * v * np.exp2(e[:, None] + e[None, :])).astype(np.float32)
    assert np.array_equal(y.cpu().numpy(), want)


@pytest.mark.parametrize("rows,N,K", [(5, 70, 96), (65, 129, 1024), (300, 5300, 736), (1024, 12288, 544)])
@pytest.mark.parametrize("shift", [-109, -60, 60, 106])
def test_operands_at_opposite_ends(rows, N, K, shift):
    """Scales of x multiplied by 2^shift and those of w divided by it: the same
    products, hence the same bits."""
    t = torch()
    x, w = held(rows, K, 1), held(N, K, 2)   # bytes 118 to 131
    want = L.mxfp4_linear(x, w, dtype=t.float32)
    x.scales.copy_((x.scales.int() + shift).byte())
    w.scales.copy_((w.scales.int() - shift).byte())
    assert int(x.scales.int().min()) >= 0 and int(w.scales.int().max()) <= 254
    assert t.equal(L.mxfp4_linear(x, w, dtype=t.float32), want)
