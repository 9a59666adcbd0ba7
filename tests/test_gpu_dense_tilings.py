"""Every kernel of the dense layer's products against fp64, in all that they form at
once: base product, delta over many slots, bias, activation, residual, codes.

Bounds as in test_gpu_dense.py, with those of exact products and all of h wherever the
result is float32 or has codes. Codes say more: rows formed by the scaled instruction
(2^-16 of their size off, root mean square) come to another bf16 value than the exact
ones about once in 65, those of exact products and fp32 sums less than once in 1000
(an error of 4 roundings, 2^-22, against a bf16 step of 2^-9 or more: 2^-12)."""
import threading

import numpy as np
import pytest

import adapter_lora_serving_amd as L
from dense_shapes import GATED, PLAIN
from gpu_util import torch
from test_gpu_dense import DEV, EPS

pytestmark = pytest.mark.gpu
R = 24


def values(q):
    """fp64 values of an operand, on the GPU."""
    t = torch()
    if t.is_tensor(q):
        return q.double()
    s = t.exp2(q.scales[:, : q.codes.shape[1] // 32].double() - 127)
    return q.codes.double() * s.repeat_interleave(32, 1)


class Case:
    def __init__(self, T, out, K, form, slices, seed):
        t = torch()
        g = t.Generator(device=DEV)
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)
        x = t.randn(T, K, device=DEV, generator=g).bfloat16()
        w = (t.randn(out, K, device=DEV, generator=g) * K**-0.5).bfloat16()
        self.x, self.w = (x, w) if form == "bf16" else (L.quantize_mxfp8(x), L.quantize_mxfp8(w))
        xv, wv = values(self.x), values(self.w)
        self.z, mag = xv @ wv.T, xv.abs() @ wv.abs().T
        slots = 70
        slot = t.from_numpy(rng.integers(-1, slots, T)).to(DEV)
        ranks = t.from_numpy(rng.integers(0, R + 1, slots).astype(np.int32)).to(DEV)
        scal = (0.5 + t.rand(slots, device=DEV, generator=g))
        h = t.randn(T, len(slices) * R, device=DEV, generator=g)
        b = (0.3 * t.randn(slots, out, R, device=DEV, generator=g)).bfloat16()
        dmag = t.zeros_like(mag)
        for s in range(slots):
            r, rows = int(ranks[s]), (slot == s).nonzero()[:, 0]
            first = 0
            for i, n in enumerate(slices):
                hs = h[rows, i * R:i * R + r].double() * scal[s].double()
                bs = b[s, first:first + n, :r].double()
                self.z[rows, first:first + n] += hs @ bs.T
                dmag[rows, first:first + n] = hs.abs() @ bs.abs().T
                h[rows, i * R + r:(i + 1) * R] = float("nan")
                first += n
            b[s, :, r:] = float("nan")
        h[slot < 0] = float("nan")
        self.delta = L.Delta(h, b, L.build_addressing(slot.int(), slots), ranks, scal, slices)
        self.bias = t.randn(out, device=DEV, generator=g)
        self.z += self.bias.double()
        self.residual = t.randn(T, out, device=DEV, generator=g)
        self.exact = (K + R + 8) * EPS * (mag + dmag) + 2.0**-23 * dmag + 2 * EPS * (
            self.z.abs() + self.bias.double().abs())
        self.scaled = self.exact + 2.0**-12 * mag + 2.0**-17 * dmag


def silu(z):
    return z / (1 + (-z).exp())


def silu_bound(z, dz, ref):
    """Of the activation's own error and of dz, where its slope is at most 1.1."""
    return 1.1 * dz + (z.abs() + 4) * 2 * EPS * ref.abs() + 2.0**-120


def near(got, ref, bound):
    """The result lies between the roundings of the bound's ends."""
    t = torch()
    if got.dtype == t.bfloat16:
        # to bf16 by way of float32: widened by its half step, so that no end is rounded inwards
        wide = bound + EPS * ref.abs()
        ok = ((ref - wide).float().bfloat16() <= got) & (got <= (ref + wide).float().bfloat16())
    else:
        ok = (got.double() - ref).abs() <= bound + EPS * ref.abs()
    assert ok.all(), (int((~ok).sum()), (~ok).nonzero()[0].tolist())


PLAIN_CASES = [(form, out, kernel) for (form, out), shapes in PLAIN.items() for kernel in shapes]


@pytest.mark.parametrize("form,out,kernel", PLAIN_CASES, ids=lambda v: v if isinstance(v, str) else "x".join(map(str, v)))
def test_plain(form, out, kernel):
    t = torch()
    T, N, K = PLAIN[form, out][kernel]
    c = Case(T, N, K, form, (N - 16, 8, 8), T + N)
    dt = t.bfloat16 if out == "bf16" else t.float32
    ref = silu(c.z)
    bound = silu_bound(c.z, c.exact if out == "f32" or form == "bf16" else c.scaled, ref)
    res = c.residual.to(dt)
    ref = ref + res.double()
    bound = bound + 2 * EPS * (ref.abs() + res.double().abs())
    y = L.epilogue_linear(c.x, c.w, bias=c.bias, activation="silu", residual=res, delta=c.delta, dtype=dt)
    near(y, ref, bound)


GATED_CASES = [(form, held, kernel) for form, shapes in GATED.items() for held in (False, True) for kernel in shapes]


@pytest.mark.parametrize("form,held,kernel", GATED_CASES, ids=lambda v: v if isinstance(v, str) else
                         ("codes" if v else "rows") if isinstance(v, bool) else "x".join(map(str, v)))
def test_gated(form, held, kernel):
    t = torch()
    T, N, K = GATED[form][kernel]
    c = Case(T, 2 * N, K, form, (N, N), T + N)
    g, u = c.z[:, :N], c.z[:, N:]
    dz = c.exact if held or form == "bf16" else c.scaled
    a = silu(g)
    da, du = silu_bound(g, dz[:, :N], a), dz[:, N:]
    ref = a * u
    bound = da * (u.abs() + du) + a.abs() * du + 2 * EPS * ref.abs()
    if not held:
        near(L.gated_linear(c.x, c.w, bias=c.bias, delta=c.delta), ref, bound)
        return
    rows, q = L.gated_linear_quantize_mxfp8(c.x, c.w, bias=c.bias, delta=c.delta)
    near(rows, ref, bound)
    again = L.quantize_mxfp8(rows)
    assert t.equal(again.codes.view(t.uint8), q.codes.view(t.uint8)) and t.equal(again.scales, q.scales)
    if rows.numel() > 100000:
        other = (rows != ref.float().bfloat16()).double().mean()
        assert other < 1e-3, float(other)


@pytest.mark.parametrize("T,form", [(5, "mx"), (140, "mx"), (140, "bf16")])
def test_codes_of_two_threads(T, form):
    """Rows, codes and scales of calls from two threads, each on a stream of its own."""
    t = torch()
    c = Case(T, 2 * 576, 544, form, (576, 576), T)
    want = L.gated_linear_quantize_mxfp8(c.x, c.w, bias=c.bias, delta=c.delta)
    norm = L.add_rms_norm_quantize_mxfp8(want[0], want[0][0].contiguous())
    t.cuda.synchronize()
    wrong = []

    def work():
        s = t.cuda.Stream()
        with t.cuda.stream(s):
            for _ in range(20):
                rows, q = L.gated_linear_quantize_mxfp8(c.x, c.w, bias=c.bias, delta=c.delta)
                n, _, nq = L.add_rms_norm_quantize_mxfp8(rows, rows[0].contiguous())
                s.synchronize()
                for got, ref in ((rows, want[0]), (q.codes, want[1].codes), (q.scales, want[1].scales),
                                 (n, norm[0]), (nq.codes, norm[2].codes), (nq.scales, norm[2].scales)):
                    if not t.equal(got.view(t.uint8), ref.view(t.uint8)):
                        wrong.append(1)

    threads = [threading.Thread(target=work) for _ in range(2)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong


@pytest.mark.parametrize("form", ["bf16", "mx"])
@pytest.mark.parametrize("T", [5, 30, 130])
@pytest.mark.parametrize("N,slices", [(100, (96, 104)), (36, (72,)), (44, (8, 72, 8)), (96, (40, 112, 40))])
def test_slices_across_gates_and_ups(N, slices, T, form):
    """A slice may hold the last gates and the first ups; N may end within 8 columns."""
    c = Case(T, 2 * N, 160, form, slices, T + N)
    g, u = c.z[:, :N], c.z[:, N:]
    dz = c.exact if form == "bf16" else c.scaled
    a = silu(g)
    da, du = silu_bound(g, dz[:, :N], a), dz[:, N:]
    bound = da * (u.abs() + du) + a.abs() * du + 2 * EPS * (a * u).abs()
    near(L.gated_linear(c.x, c.w, bias=c.bias, delta=c.delta), a * u, bound)
