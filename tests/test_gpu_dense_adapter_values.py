"""What an adapter's own rows get from the dense layer's products: h in all the bits
that the result shows, and h and B at the ends of their types as the formula has
them."""
import numpy as np
import pytest

import adapter_lora_serving_amd as L
from gpu_util import f64, torch
from oracle import dense_oracle as D
from test_gpu_dense import DEV, EPS, bf16, codes_of, gpu, near

pytestmark = pytest.mark.gpu


def delta_of(h, b, scal, slices, slot=None):
    """A Delta of every rank over T tokens, all of slot 0 unless told, and the
    formula's value in fp64."""
    T, slots, R = h.shape[0], b.shape[0], b.shape[2]
    slot = np.zeros(T, np.int32) if slot is None else slot
    ranks = np.full(slots, R, np.int32)
    d = L.Delta(gpu(h), gpu(b).bfloat16(), L.build_addressing(gpu(slot.astype(np.int32)), slots), gpu(ranks),
                gpu(scal), slices)
    with np.errstate(invalid="ignore", over="ignore"):
        return d, D.delta(h, f64(d.b), slot, ranks, scal, slices)


# rows by the kernel for few rows and by tiles
@pytest.mark.parametrize("T", [4, 70, 300])
@pytest.mark.parametrize("which", ["b", "h"])
def test_infinite_values_are_the_formula_s(T, which):
    """An infinite B times a finite h, and an infinite h times a finite B, are infinite, of
    the product's sign."""
    t = torch()
    rng = np.random.default_rng(T)
    N, R = 20016, 16
    h = rng.standard_normal((T, R)).astype(np.float32)
    h[: T // 2] = np.round(h[: T // 2] * 4) / 4 + 0.125   # of few bits: what is left of them is zero
    b = rng.standard_normal((2, N, R)).astype(np.float32)
    if which == "b":
        b[0, ::3, 5], b[0, 1::3, 7] = np.inf, -np.inf
    else:
        h[1, 3], h[2, 9] = np.inf, -np.inf
    d, (ref, _) = delta_of(h, b, np.array([0.75, 1.0], np.float32), (N,))
    x, w = bf16(rng, T, 8)[1], bf16(rng, N, 8)[1]
    for dt in (t.bfloat16, t.float32):
        y = f64(L.epilogue_linear(x, w, delta=d, dtype=dt))
        assert np.isinf(ref).any()
        assert np.array_equal(y[np.isinf(ref)], ref[np.isinf(ref)])
        assert np.isfinite(y[np.isfinite(ref)]).all()
    rows = f64(L.gated_linear(x, w, activation="relu", delta=d._replace(out_slices=(N // 2, N // 2),
                                                                         h=gpu(np.concatenate([h, h], 1)))))
    z = f64(x) @ f64(w).T + ref
    g, u = np.maximum(z[:, : N // 2], 0), z[:, N // 2:]
    sure = np.abs(z[:, : N // 2]) > 1e-4   # a gate next to 0 may be 0 in fp32, and 0 times infinity is not a number
    with np.errstate(invalid="ignore"):
        ref = g * u
    assert np.array_equal(rows[sure & np.isinf(ref)], ref[sure & np.isinf(ref)])
    assert np.array_equal(np.isnan(rows)[sure], np.isnan(ref)[sure])


@pytest.mark.parametrize("T", [4, 70, 300])
def test_h_at_the_end_of_float32(T):
    """A finite h that bf16 rounds to infinity, as it is and by its scaling."""
    t = torch()
    rng = np.random.default_rng(T)
    N, R = 20016, 8
    most = float(np.finfo(np.float32).max)
    # bf16 rounds what is past 255.5 / 256 of 2^128 up; its own largest value is below that
    ends = np.array([most, 2.0**128 * (255.75 / 256), 2.0**128 * (255.5 / 256), 2.0**128 * (255.25 / 256),
                     2.0**128 * (255.0 / 256)])
    h = np.zeros((T, R), np.float32)
    h[:, 2] = rng.choice(ends, T) * rng.choice([-1.0, 1.0], T)
    h[1::2, 2] /= 2   # twice that with its scaling
    b = np.zeros((2, N, R), np.float32)
    b[:, :, 2] = 2.0**-120 * rng.standard_normal((2, N))
    slot = np.arange(T) % 2
    d, (ref, mag) = delta_of(h, b, np.array([1.0, 2.0], np.float32), (N,), slot)
    assert np.isfinite(ref).all() and np.abs(ref).max() < 4096
    x, w = t.zeros(T, 8, device=DEV).bfloat16(), t.ones(N, 8, device=DEV).bfloat16()
    # three parts of h or all of it: one rounding of each product and of each sum
    near(f64(L.epilogue_linear(x, w, delta=d, dtype=t.float32)), ref, 8 * EPS * mag, "y")
    two = d._replace(out_slices=(N // 2, N // 2), h=gpu(np.concatenate([h, h], 1)))
    rows = f64(L.gated_linear(x, w, activation=None, delta=two))
    g, u = ref[:, : N // 2], ref[:, N // 2:]
    # two parts of h leave 2^-17 of it, three nothing
    near(rows, g * u, 2.1 * (2.0**-17 + 8 * EPS) * np.abs(g * u), "rows", t.bfloat16)


@pytest.mark.parametrize("T", [4, 70, 300, 2000])
def test_codes_show_all_bits_of_h(T):
    """Rows that go on to their codes take h in 24 bits, also of bf16 operands: what is left
    of 1 + 2^-10 + 2^-20 by a base product of -1 and a bias of -2^-10 is 2^-20."""
    t = torch()
    N, K, R = 4064, 32, 8
    h = np.full((T, 2 * R), 1.0 + 2.0**-10 + 2.0**-20, np.float32)
    b = np.zeros((1, 2 * N, R), np.float32)
    b[0, :N, 3] = 1.0
    d, _ = delta_of(h, b, np.ones(1, np.float32), (N, N))
    x, w = t.zeros(T, K, device=DEV), t.zeros(2 * N, K, device=DEV)
    x[:, 0], w[:N, 0], w[N:, 0] = 1.0, -1.0, 1.0
    bias = t.zeros(2 * N, device=DEV)
    bias[:N] = -2.0**-10
    x, w = x.bfloat16(), w.bfloat16()
    for xo, wo in ((x, w), (L.quantize_mxfp8(x), L.quantize_mxfp8(w))):
        rows, q = L.gated_linear_quantize_mxfp8(xo, wo, bias=bias, activation=None, delta=d)
        assert (rows == 2.0**-20).all()
        assert (L.dequantize_mxfp8(q) == 2.0**-20).all()
