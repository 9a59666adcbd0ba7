"""Adapter values that are not finite, or nearly not, in the dense layer's
products: by the definition delta[t] depends on t's slot alone, and on column n
only through B's row n and the h of n's slice. So an infinity or a NaN in one
slot's B, scaling or h leaves every other row, and every column of another slice,
the bits that it has without it."""
import numpy as np
import pytest

import adapter_lora_serving_amd as L
from gpu_util import torch
from test_gpu_dense import DEV, bf16, codes_of, gpu, operand

pytestmark = pytest.mark.gpu
R = 24
POISON = {"b_inf": np.inf, "b_nan": np.nan, "scaling_inf": np.inf, "scaling_nan": np.nan,
          "h_inf": -np.inf, "h_nan": np.nan}


class Adapters:
    """A delta over T tokens in slots of ranks 1 to R, in which token T // 2 has an adapter."""

    def __init__(self, rng, T, slices, slots):
        t = torch()
        self.slices, self.slots = slices, slots
        self.slot = rng.integers(-1, slots, T)
        self.row = T // 2
        self.bad = self.slot[self.row] = max(self.slot[self.row], 0)
        self.ranks = rng.integers(1, R + 1, slots)
        self.scal = gpu((0.5 + rng.random(slots)).astype(np.float32))
        self.h = gpu(rng.standard_normal((T, len(slices) * R)).astype(np.float32))
        self.b = bf16(rng, slots, sum(slices), R, std=0.3)[1]
        self.addr = L.build_addressing(gpu(self.slot.astype(np.int32)), slots)
        self.rank = int(self.ranks[self.bad]) - 1   # the last one that counts
        self.rows = t.from_numpy(self.slot == self.bad).to(DEV)

    def delta(self, poison=None, part=0, column=None):
        """The Delta; a poison goes to the bad slot's B at `column`, to its scaling, or to
        token `row`'s h of slice `part`."""
        h, b, scal = self.h, self.b, self.scal
        if poison and poison[0] == "b":
            b = b.clone()
            b[self.bad, column, self.rank] = POISON[poison]
        elif poison and poison[0] == "s":
            scal = scal.clone()
            scal[self.bad] = POISON[poison]
        elif poison:
            h = h.clone()
            h[self.row, part * R + self.rank] = POISON[poison]
        return L.Delta(h, b, self.addr, gpu(self.ranks.astype(np.int32)), scal, self.slices)

    def reached(self, poison, part, column):
        """Which values of x W^T + delta the poison belongs to, [T, out]."""
        t = torch()
        hit = t.zeros(len(self.slot), sum(self.slices), dtype=t.bool, device=DEV)
        if poison[0] == "b":
            hit[:, column] = self.rows
        elif poison[0] == "s":
            hit |= self.rows[:, None]
        else:
            lo = sum(self.slices[:part])
            hit[self.row, lo:lo + self.slices[part]] = True
        return hit


# T, N: rows of one and of several slots in a tile of every size, the kernel for few
# rows; N leaves a slice's end inside a tile
SHAPES = [(5, 328), (16, 72), (40, 328), (60, 5000), (130, 328), (300, 328), (509, 6136), (1021, 6136),
          (2045, 6136)]


@pytest.mark.parametrize("poison", sorted(POISON))
@pytest.mark.parametrize("form,out", [("bf16", "bf16"), ("bf16", "f32"), ("mx", "bf16"), ("mx", "f32")])
@pytest.mark.parametrize("T,N", SHAPES)
def test_linear_keeps_them_where_they_belong(T, N, form, out, poison):
    t = torch()
    rng = np.random.default_rng(T + N)
    dt = t.bfloat16 if out == "bf16" else t.float32
    x, w = operand(rng, T, 128, form)[1], operand(rng, N, 128, form, std=0.1)[1]
    slices = (N - 48, 8, 40)
    a = Adapters(rng, T, slices, 6)
    clean = L.epilogue_linear(x, w, delta=a.delta(), dtype=dt)
    assert t.isfinite(clean).all()
    for part, column in ((0, 3), (1, N - 47), (2, N - 1)):
        y = L.epilogue_linear(x, w, delta=a.delta(poison, part, column), dtype=dt)
        hit = a.reached(poison, part, column)
        assert t.equal(y[~hit], clean[~hit]), (part, int((y[~hit] != clean[~hit]).sum()))
        assert not t.isfinite(y[hit]).any()


GATED_SHAPES = [(5, 96), (16, 64), (40, 544), (130, 96), (187, 4064), (509, 4064), (763, 4064), (1531, 4064)]


@pytest.mark.parametrize("poison", sorted(POISON))
@pytest.mark.parametrize("form,held", [("bf16", False), ("bf16", True), ("mx", False), ("mx", True)])
@pytest.mark.parametrize("T,N", GATED_SHAPES)
def test_gated_keeps_them_where_they_belong(T, N, form, held, poison):
    t = torch()
    rng = np.random.default_rng(T + N)
    x, w = operand(rng, T, 128, form)[1], operand(rng, 2 * N, 128, form, std=0.1)[1]
    a = Adapters(rng, T, (N - 24, 24, N), 6)   # the gates' last 24 columns are a slice of their own

    def run(d):
        if held:
            rows, q = L.gated_linear_quantize_mxfp8(x, w, activation=None, delta=d)
            assert np.array_equal(codes_of(q)[0], codes_of(L.quantize_mxfp8(rows))[0])
            return rows
        return L.gated_linear(x, w, activation=None, delta=d)

    clean = run(a.delta())
    for part, column in ((0, 5), (1, N - 1), (2, N), (2, 2 * N - 3)):
        y = run(a.delta(poison, part, column))
        hit = a.reached(poison, part, column)
        hit = hit[:, :N] | hit[:, N:]
        assert t.equal(y[~hit], clean[~hit]), (part, int((y[~hit] != clean[~hit]).sum()))
        assert not t.isfinite(y[hit]).any()


def test_malformed_addressing_with_them():
    """Positions, bounds and ranks out of range beside values that are not finite: some y, and
    no access outside."""
    t = torch()
    rng = np.random.default_rng(3)
    T, N, slots = 130, 128, 4
    x, w = bf16(rng, T, 64)[1], bf16(rng, N, 64)[1]
    b = bf16(rng, slots, N, R)[1]
    b[1:] = float("nan")
    h = t.full((T, R), float("inf"), device=DEV)
    big = 2**31 - 1
    for order, indptr, ranks in ((np.full(T, big), [0, 20, 40, 60, T], [24, 99, -3, big]),
                                 (np.full(T, -5), [0, 20, 40, 60, T], [24] * 4),
                                 (np.arange(T), [50, 20, big, -7, T], [24] * 4),
                                 (np.arange(T), [-big, 3, 200, T, big], [24] * 4)):
        i32 = lambda v: gpu(np.asarray(v).astype(np.int32))   # noqa: E731
        d = L.Delta(h, b, L.Addressing(i32(order), i32(indptr)), i32(ranks), t.ones(slots, device=DEV), (N,))
        L.epilogue_linear(x, w, delta=d, activation="relu")
        L.gated_linear(x, w, delta=d)
    t.cuda.synchronize()


@pytest.mark.parametrize("T", [20, 150])
def test_replayed_as_a_graph(T):
    """A captured call whose adapters become bad, and good again, between its replays."""
    t = torch()
    rng = np.random.default_rng(T)
    x, w = bf16(rng, T, 64)[1], bf16(rng, 192, 64)[1]
    a = Adapters(rng, T, (96, 96), 5)
    good, bad = a.delta().b.clone(), a.delta("b_inf", 1, 100).b
    d = a.delta()._replace(b=good.clone())

    def step():
        return L.epilogue_linear(x, w, delta=d), L.gated_linear_quantize_mxfp8(x, w, delta=d)[0]

    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        step()
        g = t.cuda.CUDAGraph()
        with t.cuda.graph(g, stream=side):
            out = step()
    t.cuda.synchronize()
    for b in (good, bad, good, bad, good):
        d.b.copy_(b)
        eager = step()
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        for e, o in zip(eager, out):
            assert t.equal(e.view(t.int16), o.view(t.int16))
