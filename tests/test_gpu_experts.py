"""The routed-expert operators on the GPU against the fp64 definitions.

Tolerances. eps = 2^-24 is the relative half step of fp32; the bounds are on
the fp32 value. A bf16 result is that value rounded once: rounding keeps order,
so the result lies between the roundings of the bound's two ends.
  weights   a score is an exponential (2 ulp), a sum rounded once and a
            quotient; a weight divides it by a sum of k of them: relative
            error at most (k + 8) 2 eps.
  products  the products are exact, K of them are added in fp32 in some order:
            |error| <= K eps sum |x w|.
  combine   k + 1 terms, each product rounded once: (k + 2) 2 eps sum |w r|.
  silu      the exponential, a sum, a quotient and a product: 8 eps relative.
Whatever is whole (ids, rows, codes, scales) is equal."""
import importlib.util
import math
import os
import random

import numpy as np
import pytest

import adapter_lora_serving_amd as L
from gpu_util import f64, torch
from oracle import experts_oracle as X

pytestmark = pytest.mark.gpu
EPS = 2.0**-24
DEV = "cuda:0"


def gen(seed):
    t = torch()
    g = t.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def bf16(a):
    return torch().from_numpy(np.asarray(a, np.float32)).to(DEV).bfloat16()


def rounded(a, dtype):
    """fp64 values rounded to dtype (by way of fp32), in fp64."""
    return torch().from_numpy(np.asarray(a)).float().to(dtype).double().numpy()


def near(got, ref, bound, what="", dtype=None):
    """|value - ref| <= bound for the fp32 value that was rounded to dtype."""
    if dtype == torch().bfloat16:
        bad = ~((rounded(ref - bound, dtype) <= got) & (got <= rounded(ref + bound, dtype)))
    else:
        bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), f"{what}: {int(bad.sum())} values off, worst {np.max(np.abs(got - ref))}"


# ---- routing --------------------------------------------------------------

def grid_logits(rng, T, E):
    """Logits and biases on coarse grids: equal choices are equal in any
    precision, others far apart (checked by the caller)."""
    return rng.integers(-32, 33, (T, E)) / 8.0, rng.integers(-3, 4, E) / 16.0


ROUTES = [
    # T, E, k, dtype, scores, bias, groups, top_groups, group_score
    (1, 64, 2, "bf16", "softmax", False, 1, 1, "max"),
    (1, 1, 1, "f32", "sigmoid", True, 1, 1, "max"),
    (37, 8, 8, "bf16", "softmax", True, 1, 1, "max"),
    (130, 7, 3, "f32", "sigmoid", True, 1, 1, "max"),
    (65, 256, 8, "f32", "sigmoid", True, 8, 4, "sum2"),
    (33, 256, 8, "bf16", "softmax", False, 16, 3, "max"),
    (20, 60, 4, "f32", "softmax", True, 5, 2, "sum2"),
    (20, 90, 6, "f32", "sigmoid", False, 6, 3, "max"),
    (9, 16, 4, "bf16", "sigmoid", True, 16, 5, "sum2"),
    (17, 300, 32, "f32", "softmax", True, 4, 3, "sum2"),
    (5, 512, 10, "bf16", "sigmoid", True, 8, 2, "sum2"),
    (6, 1024, 20, "f32", "softmax", False, 16, 7, "max"),
    (3, 1001, 32, "bf16", "sigmoid", False, 1, 1, "max"),
]


@pytest.mark.parametrize("case", ROUTES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("holes", [False, True])
def test_route(case, holes):
    t = torch()
    T, E, k, dtype, scores, bias, G, tg, gsc = case
    rng = np.random.default_rng(T * 1000 + E)
    x, b = grid_logits(rng, T, E)
    if holes:   # closed experts, whole rows of them among these
        x[rng.random((T, E)) < 0.5] = -np.inf
        x[rng.random((T, E)) < 0.1] = np.nan
        x[T // 2] = -np.inf
    logits = t.from_numpy(x.astype(np.float32)).to(DEV)
    logits = logits.bfloat16() if dtype == "bf16" else logits
    r = L.route_experts(logits, k, scores=scores,
                        bias=t.from_numpy(b.astype(np.float32)).to(DEV) if bias else None,
                        groups=G, top_groups=tg, group_score=gsc, scaling=2.5)
    ids, w, choice = X.route(x, k, scores, b if bias else None, G, tg, gsc, scaling=2.5)
    for row in choice:   # no two choices that fp32 could confuse
        v = np.unique(row[np.isfinite(row)])
        gap = np.diff(v)
        gap = gap[gap > 1e-14]   # equal but for the last bit of fp64
        assert not gap.size or gap.min() > 2e-7
    got = r.ids.cpu().numpy()
    assert np.array_equal(got, ids)
    near(f64(r.weights), w, (k + 8) * 2 * EPS * np.abs(w), "weights")
    assert (f64(r.weights)[ids < 0] == 0).all()


def test_route_infinite_and_extreme_logits():
    t = torch()
    inf, nan, big = math.inf, math.nan, 3e38
    x = t.tensor([[0, inf, 1, inf], [-inf, nan, -inf, nan], [big, -big, 0, big],
                  [-big, -big, -inf, -big]], device=DEV)
    for scores in ("softmax", "sigmoid"):
        r = L.route_experts(x, 3, scores=scores)
        ids, w, _ = X.route(f64(x), 3, scores)
        assert np.array_equal(r.ids.cpu().numpy(), ids)
        near(f64(r.weights), w, 1e-5 * np.abs(w), scores)
    # a bias closes an expert by -inf or NaN, whatever its logit
    r = L.route_experts(x[:1], 4, scores="sigmoid",
                        bias=t.tensor([-inf, 0.0, nan, 0.0], device=DEV))
    assert r.ids.tolist() == [[1, 3, -1, -1]]


def test_route_ties_and_plain_weights():
    t = torch()
    r = L.route_experts(t.zeros(3, 100, device=DEV), 5, renormalize=False)
    assert r.ids.tolist() == [[0, 1, 2, 3, 4]] * 3
    near(f64(r.weights), np.full((3, 5), 0.01), 0.01 * 8 * EPS)
    r = L.route_experts(t.zeros(2, 96, device=DEV), 4, groups=8, top_groups=2)
    assert r.ids.tolist() == [[0, 1, 2, 3]] * 2
    # sigmoid scores that are all 0: weights 0, not NaN
    r = L.route_experts(t.full((1, 8), -2e38, device=DEV), 2, scores="sigmoid")
    assert r.ids.tolist() == [[0, 1]] and r.weights.tolist() == [[0.0, 0.0]]
    assert L.route_experts(t.zeros(0, 8, device=DEV), 2).ids.shape == (0, 2)


def test_route_into_given_buffers():
    t = torch()
    x = t.randn(6, 32, device=DEV, generator=gen(0))
    out = L.Routing(t.empty(6, 4, dtype=t.int32, device=DEV), t.empty(6, 4, device=DEV))
    r = L.route_experts(x, 4, out=out)
    assert r.ids.data_ptr() == out.ids.data_ptr()
    assert t.equal(out.ids, L.route_experts(x, 4).ids)
    with pytest.raises(L.LoraError):
        L.route_experts(x, 3, out=out)
    with pytest.raises(L.LoraError):
        L.route_experts(x.t(), 2)          # not contiguous
    with pytest.raises(L.LoraError):
        L.route_experts(x, 2, scores="tanh")
    with pytest.raises(L.LoraError):
        L.route_experts(x, 2, bias=t.zeros(31, device=DEV))
    with pytest.raises(L.LoraError):
        L.route_experts(x.half(), 2)
    with pytest.raises(L.LoraError):
        L.route_experts(x, 33)


# ---- expert-sorted rows ---------------------------------------------------

@pytest.mark.parametrize("T,k,E", [(0, 2, 8), (1, 1, 1), (1, 8, 256), (3, 2, 63), (5, 3, 64),
                                   (256, 2, 8), (512, 2, 63), (513, 2, 40), (300, 8, 1024),
                                   (8191, 8, 256), (8192, 8, 512), (9001, 8, 256),
                                   (20000, 4, 1024)])
@pytest.mark.parametrize("dead", [0.0, 0.3, 1.0])
def test_rows(T, k, E, dead):
    t = torch()
    rng = np.random.default_rng(T + E)
    ids = np.minimum(rng.integers(0, E, (T, k)), rng.integers(0, E, (T, k))).astype(np.int32)
    gone = rng.random((T, k)) < dead
    ids[gone] = rng.choice([-1, -7, E, 1 << 30], gone.sum())
    slot = rng.integers(-1, 50, T).astype(np.int32)
    d_ids, d_slot = (t.from_numpy(v).to(DEV) for v in (ids, slot))
    ref = X.expert_rows(ids, E, slot)
    r = L.expert_rows(d_ids, E, d_slot)
    for got, want, name in zip(r, ref, r._fields):
        assert np.array_equal(got.cpu().numpy(), want), name
    r = L.expert_rows(d_ids, E)
    assert r.row_slot is None
    for got, want in zip(r[:3], ref[:3]):
        assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("shift", [1, 2, 3])
def test_rows_from_any_address(shift):
    t = torch()
    rng = np.random.default_rng(shift)
    ids = rng.integers(-1, 100, (700, 3)).astype(np.int32)
    buf = t.empty(shift + ids.size, dtype=t.int32, device=DEV)
    view = buf[shift:].view(700, 3)
    view.copy_(t.from_numpy(ids))
    r = L.expert_rows(view, 100)
    for got, want in zip(r[:3], X.expert_rows(ids, 100)[:3]):
        assert np.array_equal(got.cpu().numpy(), want)


def test_rows_feed_the_expert_addressing():
    t = torch()
    ids = t.randint(0, 8, (100, 2), device=DEV, generator=gen(3), dtype=t.int32)
    slot = t.randint(-1, 5, (100,), device=DEV, generator=gen(4), dtype=t.int32)
    r = L.expert_rows(ids, 8, slot)
    from adapter_lora_serving_amd import build_addressing_experts
    addr = build_addressing_experts(r.row_slot, r.offsets, 8, 5)
    assert int(addr.slot_indptr[-1]) == int((slot >= 0).sum()) * 2


def test_rows_refusals():
    t = torch()
    ids = t.zeros(4, 2, dtype=t.int32, device=DEV)
    for f in (lambda: L.expert_rows(ids, 0), lambda: L.expert_rows(ids, 1025),
              lambda: L.expert_rows(ids.view(-1), 4),
              lambda: L.expert_rows(ids, 4, t.zeros(5, dtype=t.int32, device=DEV)),
              lambda: L.expert_rows(t.zeros(4, 33, dtype=t.int32, device=DEV), 4),
              lambda: L.expert_rows(ids.t(), 4)):
        with pytest.raises(L.LoraError):
            f()


# ---- quantisation ---------------------------------------------------------

def check_quantized(q, x):
    codes, scales = X.quantize(x)
    assert np.array_equal(q.scales.cpu().numpy(), scales)
    assert np.array_equal(q.codes.cpu().numpy(), codes)


def test_quantize_every_bf16():
    t = torch()
    bits = np.arange(65536, dtype=np.uint16)
    order = np.random.default_rng(0).permutation(65536)   # blocks that mix sizes
    for b in (bits, bits[order]):
        x = t.from_numpy(b.view(np.int16)).view(t.bfloat16).to(DEV).view(-1, 128)
        check_quantized(L.quantize_mxfp4(x), f64(x))


@pytest.mark.parametrize("rows,K", [(0, 64), (1, 32), (3, 96), (7, 4096), (129, 160), (1000, 544)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize(rows, K, dtype):
    t = torch()
    rng = np.random.default_rng(rows + K)
    x = rng.standard_normal((rows, K)) * np.exp2(rng.integers(-20, 20, (rows, K // 32)).repeat(32, 1))
    if rows:
        x[0] = 0.0
        x[-1, :32] = np.exp2(-126.0) * rng.standard_normal(32)   # denormal results
        x[rows // 2, 5] = np.nan
        x[rows // 2, K - 1] = -np.inf
    d = t.from_numpy(x.astype(np.float32)).to(DEV)
    d = d.bfloat16() if dtype == "bf16" else d
    q = L.quantize_mxfp4(d)
    check_quantized(q, f64(d))
    for out in (t.bfloat16, t.float32):
        v = L.dequantize_mxfp4(q, out)
        want = t.from_numpy(X.dequantize(*X.quantize(f64(d)))).to(out)
        assert np.array_equal(f64(v), want.double().numpy(), equal_nan=True)


def test_quantize_halves_round_to_even():
    t = torch()
    # every midpoint of the grid, at every scale that bf16 has
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = np.zeros((240, 32))
    x[:, 0] = 4.0
    x[:, 1:8] = mids
    x[:, 8:15] = -mids
    x[:, 15:22] = mids * (1 + 2.0**-7)
    x[:, 22:29] = mids * (1 - 2.0**-7)
    x *= np.exp2(np.arange(-120, 120))[:, None]
    for d in (bf16(x), t.from_numpy(x.astype(np.float32)).to(DEV)):
        check_quantized(L.quantize_mxfp4(d), f64(d))


def test_dequantize_every_code_at_every_scale():
    t = torch()
    codes = t.arange(256, dtype=t.uint8, device=DEV).repeat(256, 1)      # both halves of a byte
    scales = t.arange(256, dtype=t.uint8, device=DEV).unsqueeze(1).repeat(1, 16)
    want = t.from_numpy(X.dequantize(codes.cpu().numpy(), scales.cpu().numpy()))
    for out in (t.bfloat16, t.float32):
        v = L.dequantize_mxfp4(L.MXFP4(codes, scales), out)
        assert np.array_equal(f64(v), want.to(out).double().numpy(), equal_nan=True)


def test_quantize_stacked_weights():
    t = torch()
    w = t.randn(3, 40, 96, device=DEV, generator=gen(1))
    q = L.quantize_mxfp4(w)
    assert q.codes.shape == (3, 40, 48) and q.scales.shape == (3, 40, 4)
    one = L.quantize_mxfp4(w[1].contiguous())
    assert t.equal(q.codes[1], one.codes) and t.equal(q.scales[1], one.scales)
    assert L.dequantize_mxfp4(q).shape == (3, 40, 96)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gather_quantize(dtype):
    t = torch()
    x = t.randn(50, 224, device=DEV, generator=gen(2))
    x = x.bfloat16() if dtype == "bf16" else x
    idx = np.random.default_rng(0).integers(-5, 60, 333).astype(np.int32)   # clamped
    rows, q = L.gather_quantize_mxfp4(x, t.from_numpy(idx).to(DEV))
    want = x[t.from_numpy(np.clip(idx, 0, 49)).long().to(DEV)]
    assert t.equal(rows, want)
    check_quantized(q, f64(want))


@pytest.mark.parametrize("rows,K", [(1, 32), (9, 96), (70, 14336), (257, 736)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_silu_mul_quantize(rows, K, dtype):
    t = torch()
    gu = 3 * t.randn(rows, 2 * K, device=DEV, generator=gen(rows))
    gu = gu.bfloat16() if dtype == "bf16" else gu
    act, q = L.silu_mul_quantize_mxfp4(gu)
    g, u = np.split(f64(gu), 2, 1)
    want = g / (1 + np.exp(-g)) * u
    near(f64(act), want, 8 * EPS * np.abs(want) + 1e-38, "act", act.dtype)
    check_quantized(q, f64(act))   # the codes are those of the rounded rows


def test_quantize_refusals():
    t = torch()
    x = t.zeros(4, 64, device=DEV)
    for f in (lambda: L.quantize_mxfp4(x[:, :48].contiguous()), lambda: L.quantize_mxfp4(x.t()),
              lambda: L.quantize_mxfp4(x.half()), lambda: L.silu_mul_quantize_mxfp4(x[:, :32].contiguous()),
              lambda: L.silu_mul_quantize_mxfp4(t.zeros(4, 65, device=DEV)),
              lambda: L.gather_quantize_mxfp4(x[:0], t.zeros(3, dtype=t.int32, device=DEV)),
              lambda: L.dequantize_mxfp4(L.MXFP4(x, x)),
              lambda: L.dequantize_mxfp4(L.quantize_mxfp4(x), t.float16),
              lambda: L.dequantize_mxfp4(L.MXFP4(L.quantize_mxfp4(x).codes,
                                                 L.quantize_mxfp4(x).scales[:3]))):
        with pytest.raises(L.LoraError):
            f()


# ---- products -------------------------------------------------------------

def held(rows, K, seed):
    """Random MXFP4 rows with the full range of codes and a few scales."""
    t = torch()
    g = gen(seed)
    codes = t.randint(0, 256, (rows, K // 2), dtype=t.uint8, device=DEV, generator=g)
    scales = t.randint(118, 132, (rows, -(-(K // 32) // 4) * 4), dtype=t.uint8, device=DEV,
                       generator=g)
    return L.MXFP4(codes, scales)


def values(q):
    """fp64 values on the GPU, apart from the kernels."""
    t = torch()
    grid = t.tensor(np.concatenate([X.GRID, -X.GRID]), device=DEV)
    v = t.stack([grid[(q.codes & 15).long()], grid[(q.codes >> 4).long()]], -1).flatten(-2)
    s = t.exp2(q.scales.double() - 127).masked_fill(q.scales == 255, math.nan)
    return v * s.repeat_interleave(32, -1)[..., :v.shape[-1]]


def check_product(y, xv, wv, K, what=""):
    t = torch()
    ref = xv @ wv.t()
    bound = K * EPS * (xv.abs() @ wv.abs().t())
    lo, hi = ref - bound, ref + bound
    if y.dtype == t.bfloat16:
        lo, hi = (v.float().bfloat16().double() for v in (lo, hi))
    bad = ~((lo <= y.double()) & (y.double() <= hi))
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {y.numel()} values off"


SHAPES = [
    # rows, N, K: single rows and odd sizes, and sizes that take each tile
    (1, 1, 32), (1, 100, 544), (2, 33, 96), (33, 70, 480), (65, 129, 1024), (64, 64, 512),
    (700, 6000, 256), (1000, 5300, 736), (30, 19878, 544), (1024, 4096, 544), (40, 40001, 544),
    (1024, 12288, 576), (1111, 12290, 2336), (257, 515, 4128), (5, 300, 14336),
]


@pytest.mark.parametrize("rows,N,K", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear(rows, N, K, dtype):
    t = torch()
    x, w = held(rows, K, rows), held(N, K, N + 1)
    y = L.mxfp4_linear(x, w, dtype=t.bfloat16 if dtype == "bf16" else t.float32)
    assert y.shape == (rows, N)
    check_product(y, values(x), values(w), K)


@pytest.mark.parametrize("rows,N,K", [(3, 72, 96), (64, 256, 544), (1111, 12292, 672)])
def test_linear_writes_its_own_rows_alone(rows, N, K):
    t = torch()
    x, w = held(rows, K, 1), held(N, K, 2)
    buf = t.full((rows + 2, N), 7.0, device=DEV)
    y = buf[1:-1]
    if y.data_ptr() % 16:
        pytest.skip("the view is not 16-byte aligned")
    L.mxfp4_linear(x, w, y=y)
    check_product(y, values(x), values(w), K)
    assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())


@pytest.mark.parametrize("rows,N,K", [(70, 90, 96), (70, 90, 544), (1024, 12288, 736)])
def test_linear_scales(rows, N, K):
    """A NaN scale stays in its row and column, and scale padding is no scale."""
    t = torch()
    x, w = held(rows, K, 3), held(N, K, 4)
    clean = L.mxfp4_linear(x, w)
    if (K // 32) % 4:
        for q in (x, w):
            q.scales[:, K // 32:] = 255
        assert t.equal(L.mxfp4_linear(x, w), clean)
    x.scales[rows // 2, 1] = 255
    w.scales[N // 3, 0] = 255
    y = L.mxfp4_linear(x, w)
    bad = t.zeros(rows, N, dtype=t.bool, device=DEV)
    bad[rows // 2] = True
    bad[:, N // 3] = True
    assert bool(t.isnan(y[bad]).all()) and t.equal(y[~bad], clean[~bad])


def test_linear_same_bits_every_time_and_in_every_tiling():
    t = torch()
    x, w = held(1024, 1056, 5), held(12288, 1056, 6)
    y = L.mxfp4_linear(x, w)
    assert t.equal(y, L.mxfp4_linear(x, w))
    for lo, hi, cols in ((0, 1, 12288), (100, 165, 500), (300, 900, 5300)):
        part = L.mxfp4_linear(L.MXFP4(x.codes[lo:hi].contiguous(), x.scales[lo:hi].contiguous()),
                              L.MXFP4(w.codes[:cols].contiguous(), w.scales[:cols].contiguous()))
        assert t.equal(part, y[lo:hi, :cols])


@pytest.mark.parametrize("rows,N", [(5120, 3840), (4910, 3740), (5000, 3700)])
def test_linear_half_tiles(rows, N):
    """Some 300 tiles of 256 x 256, the last ones as halves: the second half of
    the last columns is whole, 28 columns and nothing."""
    x, w = held(rows, 544, rows), held(N, 544, N)
    check_product(L.mxfp4_linear(x, w, dtype=torch().float32), values(x), values(w), 544)


@pytest.mark.parametrize("rows,N,K", [(40, 17000, 1312), (70, 12200, 2080), (9, 20000, 1184),
                                      (130, 10900, 800)])
def test_linear_scale_groups(rows, N, K):
    """64 x 128 tiles, whose scales come for four stages of 256 at a time: six,
    nine, five and four stages, the last one short."""
    x, w = held(rows, K, rows), held(N, K, N)
    check_product(L.mxfp4_linear(x, w, dtype=torch().float32), values(x), values(w), K)


@pytest.mark.parametrize("rows,N,K", [(32, 17000, 1312), (1, 20011, 544), (17, 16500, 2080)])
@pytest.mark.parametrize("E", [1, 3])
def test_linear_32_rows(rows, N, K, E):
    t = torch()
    x = held(rows, K, rows)
    if E == 1:
        w = held(N, K, N)
        check_product(L.mxfp4_linear(x, w), values(x), values(w), K)
        return
    N //= 3
    W = L.MXFP4(*(v.view(E, N, -1) for v in held(E * N, K, E)))
    off = [0, rows // 2, rows // 2, rows]
    y = L.mxfp4_expert_linear(x, W, t.tensor(off, dtype=t.int32, device=DEV))
    xv = values(x)
    for e in range(E):
        check_product(y[off[e]:off[e + 1]], xv[off[e]:off[e + 1]],
                      values(L.MXFP4(W.codes[e], W.scales[e])), K, f"expert {e}")


@pytest.mark.parametrize("K", [544, 1184, 1312, 2336])
def test_expert_linear_scale_groups_across_tiles(K):
    """65 rows of each expert: more tiles than workgroups, so the ring of scale
    groups runs on from one tile into the next."""
    t = torch()
    rows, E, N = 520, 8, 2400
    x = held(rows, K, 3)
    W = L.MXFP4(*(v.view(E, N, -1) for v in held(E * N, K, E)))
    off = [65 * e for e in range(E + 1)]
    y = L.mxfp4_expert_linear(x, W, t.tensor(off, dtype=t.int32, device=DEV), dtype=t.float32)
    xv = values(x)
    for e in range(E):
        check_product(y[off[e]:off[e + 1]], xv[off[e]:off[e + 1]],
                      values(L.MXFP4(W.codes[e], W.scales[e])), K, f"expert {e}")


def test_expert_linear_half_tiles():
    t = torch()
    rows, E, N, K = 3900, 4, 4700, 544   # 19 tiles of columns and 17 or so of rows
    x = held(rows, K, 3)
    W = L.MXFP4(*(v.view(E, N, -1) for v in held(E * N, K, E)))
    off = [7, 1300, 1301, 2600, 3890]
    y = L.mxfp4_expert_linear(x, W, t.tensor(off, dtype=t.int32, device=DEV))
    xv = values(x)
    assert bool((y[:7] == 0).all()) and bool((y[3890:] == 0).all())
    for e in range(E):
        check_product(y[off[e]:off[e + 1]], xv[off[e]:off[e + 1]],
                      values(L.MXFP4(W.codes[e], W.scales[e])), K, f"expert {e}")


@pytest.mark.parametrize("bounds", [
    [0, 0, 5, 5, 40, 40], [0, 70, 70, 70, 70, 70], [3, 10, 10, 30, 31, 60], [0, 0, 0, 0, 0, 0],
    [0, 1, 2, 3, 4, 70], [70, 70, 70, 70, 70, 70]])
@pytest.mark.parametrize("N,K", [(40, 96), (301, 544)])
def test_expert_linear_bounds(bounds, N, K):
    t = torch()
    x = held(70, K, 7)
    w = [held(N, K, 8 + e) for e in range(5)]
    W = L.MXFP4(*(t.stack(p) for p in zip(*w)))
    y = t.full((70, N), math.nan, device=DEV)
    L.mxfp4_expert_linear(x, W, t.tensor(bounds, dtype=t.int32, device=DEV), y=y)
    xv = values(x)
    dead = t.ones(70, dtype=t.bool, device=DEV)
    for e in range(5):
        lo, hi = bounds[e], bounds[e + 1]
        dead[lo:hi] = False
        check_product(y[lo:hi], xv[lo:hi], values(w[e]), K, f"expert {e}")
    assert bool((y[dead] == 0).all())


@pytest.mark.parametrize("rows,E,N,K,dtype", [
    (512, 8, 3000, 544, "bf16"), (300, 300, 70, 64, "f32"), (20, 1000, 33, 544, "bf16"),
    (4000, 3, 6100, 576, "bf16"), (1500, 5, 700, 2336, "f32"), (1, 4, 129, 4096, "bf16"),
    (3000, 40, 1100, 160, "bf16")])
def test_expert_linear(rows, E, N, K, dtype):
    t = torch()
    x = held(rows, K, rows)
    W = L.MXFP4(*(v.view(E, N, -1) for v in held(E * N, K, E)))
    ids = np.sort(np.random.default_rng(E).zipf(1.3, rows) % E)
    off = np.concatenate([[0], np.cumsum(np.bincount(ids, minlength=E))]).astype(np.int32)
    y = L.mxfp4_expert_linear(x, W, t.from_numpy(off).to(DEV),
                              dtype=t.bfloat16 if dtype == "bf16" else t.float32)
    xv = values(x)
    for e in range(E):
        if off[e + 1] > off[e]:
            check_product(y[off[e]:off[e + 1]], xv[off[e]:off[e + 1]],
                          values(L.MXFP4(W.codes[e], W.scales[e])), K, f"expert {e}")


@pytest.mark.parametrize("bad", [[5, 3, 9, 2, 70, 1], [-4, 10, 1 << 30, 20, 30, -9],
                                 [1 << 30] * 6, [-1] * 6])
def test_expert_linear_malformed_bounds_stay_inside(bad):
    t = torch()
    x = held(70, 96, 1)
    W = L.MXFP4(*(v.view(5, 64, -1) for v in held(320, 96, 2)))
    buf = t.full((72, 64), 7.0, device=DEV)
    L.mxfp4_expert_linear(x, W, t.tensor(bad, dtype=t.int32, device=DEV), y=buf[1:-1])
    t.cuda.synchronize()
    assert bool((buf[0] == 7).all()) and bool((buf[-1] == 7).all())


def test_expert_linear_past_32_bit_offsets():
    t = torch()
    E, N, K = 5, 131072, 8192   # 2.7 GB of codes
    W = L.MXFP4(t.zeros(E, N, K // 2, dtype=t.uint8, device=DEV),
                t.full((E, N, K // 32), 127, dtype=t.uint8, device=DEV))
    last = held(N, K, 9)
    W.codes[-1] = last.codes
    x = held(6, K, 10)
    off = t.tensor([0, 2, 2, 2, 2, 6], dtype=t.int32, device=DEV)
    y = L.mxfp4_expert_linear(x, W, off, dtype=t.float32)
    assert bool((y[:2] == 0).all())
    check_product(y[2:], values(x)[2:], values(L.MXFP4(last.codes, W.scales[-1])), K)


def test_product_refusals():
    t = torch()
    x, w = held(4, 64, 1), held(8, 64, 2)
    W = L.MXFP4(w.codes.view(2, 4, -1), w.scales.view(2, 4, -1))
    off = t.zeros(3, dtype=t.int32, device=DEV)
    for f in (lambda: L.mxfp4_linear(x, held(8, 96, 3)), lambda: L.mxfp4_linear(x, W),
              lambda: L.mxfp4_linear(x, w, dtype=t.float16),
              lambda: L.mxfp4_linear(x, w, y=t.empty(4, 9, device=DEV)),
              lambda: L.mxfp4_linear(L.MXFP4(x.codes, x.scales[:, :2].contiguous()), w),
              lambda: L.mxfp4_linear(L.MXFP4(x.codes.int(), x.scales), w),
              lambda: L.mxfp4_expert_linear(x, w, off),
              lambda: L.mxfp4_expert_linear(x, W, off[:2]),
              lambda: L.mxfp4_expert_linear(x, W, off.cpu())):
        with pytest.raises(L.LoraError):
            f()
    assert L.mxfp4_linear(held(0, 64, 1), w).shape == (0, 8)


# ---- the weighted sum -----------------------------------------------------

@pytest.mark.parametrize("T,k,H,n", [(0, 2, 64, 4), (1, 1, 8, 1), (7, 3, 104, 30), (256, 2, 4096, 512),
                                     (33, 32, 520, 100), (1000, 8, 200, 8000), (5, 2, 64, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("add", [False, True])
def test_combine(T, k, H, n, dtype, add):
    t = torch()
    dt = t.bfloat16 if dtype == "bf16" else t.float32
    rng = np.random.default_rng(T + H)
    rows = t.randn(n, H, device=DEV, generator=gen(H)).to(dt)
    pos = rng.integers(-3, n + 3, (T, k)).astype(np.int32)
    w = rng.standard_normal((T, k)).astype(np.float32)
    w[(pos < 0) | (pos >= n)] = np.nan   # never read
    res = t.randn(T, H, device=DEV, generator=gen(H + 1)).to(dt) if add else None
    d_pos, d_w = t.from_numpy(pos).to(DEV), t.from_numpy(w).to(DEV)
    y = L.combine_experts(rows, d_pos, d_w, residual=res)
    ref = X.combine(f64(rows), pos, w, None if res is None else f64(res))
    size = X.combine(np.abs(f64(rows)), pos, np.abs(w), None if res is None else np.abs(f64(res)))
    near(f64(y), ref, (k + 2) * 2 * EPS * size, "y", dt)
    if add:   # in place
        same = L.combine_experts(rows, d_pos, d_w, residual=res, y=res)
        assert same.data_ptr() == res.data_ptr() and t.equal(res, y)


def test_combine_leaves_unused_rows_unread():
    t = torch()
    rows = t.full((10, 64), math.nan, device=DEV)
    rows[3], rows[8] = 1.0, 2.0
    y = L.combine_experts(rows, t.tensor([[3, -1, 8]], dtype=t.int32, device=DEV),
                          t.tensor([[0.5, math.inf, 0.25]], device=DEV))
    assert bool((y == 1.0).all())


def test_combine_past_32_bit_offsets():
    t = torch()
    rows = t.zeros(300000, 4096, dtype=t.bfloat16, device=DEV)   # 2.4 GB
    rows[-1] = 3.0
    y = L.combine_experts(rows, t.tensor([[299999, 0]], dtype=t.int32, device=DEV),
                          t.tensor([[2.0, 1.0]], device=DEV))
    assert bool((y == 6.0).all())


def test_combine_refusals():
    t = torch()
    rows = t.zeros(4, 64, device=DEV)
    pos = t.zeros(2, 2, dtype=t.int32, device=DEV)
    w = t.zeros(2, 2, device=DEV)
    for f in (lambda: L.combine_experts(rows, pos, w.double()),
              lambda: L.combine_experts(rows, pos, w[:1]),
              lambda: L.combine_experts(rows, pos.view(-1), w),
              lambda: L.combine_experts(rows, pos, w, residual=t.zeros(2, 60, device=DEV)),
              lambda: L.combine_experts(rows, pos, w, y=t.zeros(2, 64, device=DEV).bfloat16()),
              lambda: L.combine_experts(t.zeros(4, 62, device=DEV), pos, w),
              lambda: L.combine_experts(rows.half(), pos, w)):
        with pytest.raises(L.LoraError):
            f()


# ---- together -------------------------------------------------------------

def example():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("routed_experts",
                                                  os.path.join(root, "examples", "routed_experts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def layer_inputs(T, hidden, slots, seed):
    t = torch()
    g = gen(seed)
    return (t.randn(T, hidden, device=DEV, generator=g).bfloat16(),
            t.randn(T, hidden, device=DEV, generator=g).bfloat16(),
            t.randint(-1, slots, (T,), device=DEV, generator=g, dtype=t.int32))


@pytest.mark.parametrize("T,experts,top_k", [(1, 8, 2), (50, 8, 2), (300, 16, 4)])
def test_layer_stage_by_stage(T, experts, top_k):
    """Every stage of the layer against its definition on the stage's inputs."""
    t = torch()
    hidden, inter, slots = 256, 512, 4
    layer = example().RoutedExperts(hidden, inter, experts, slots, top_k)
    x, residual, slot = layer_inputs(T, hidden, slots, T)
    s = layer.step(x, residual, slot)
    ids, w, _ = X.route(f64(s["logits"]), top_k)
    got = s["routing"].ids.cpu().numpy()
    assert np.array_equal(got, ids)
    near(f64(s["routing"].weights), w, (top_k + 8) * 2 * EPS * np.abs(w))
    row_token, positions, offsets, row_slot = X.expert_rows(ids, experts, slot.cpu().numpy())
    for a, b in zip(s["sorted"], (row_token, positions, offsets, row_slot)):
        assert np.array_equal(a.cpu().numpy(), b)
    assert t.equal(s["rows"], x[t.from_numpy(row_token).long().to(DEV)])
    check_quantized(s["x"], f64(s["rows"]))
    for base, q, wt, K in (("base_gate_up", s["x"], layer.gate_up, hidden),
                           ("base_down", s["h"], layer.down, inter)):
        xv = values(q)
        for e in range(experts):
            lo, hi = int(offsets[e]), int(offsets[e + 1])
            if hi > lo:
                check_product(s[base][lo:hi], xv[lo:hi],
                              values(L.MXFP4(wt.codes[e], wt.scales[e])), K, base)

    def lora(xr, y0, a, b, entries, ranks, scalings, widths):
        y = f64(y0).copy()
        R = b.shape[2]
        a, b, xr = f64(a), f64(b), f64(xr)
        for r, e in enumerate(entries):
            if e < 0:
                continue
            n, at = int(ranks[e]), 0
            for i, width in enumerate(widths):
                h = a[e, i * R:i * R + n] @ xr[r]
                y[r, at:at + width] += float(scalings[e]) * (b[e, at:at + width, :n] @ h)
                at += width
        return y

    expert = np.searchsorted(offsets[1:], np.arange(T * top_k), side="right")
    entry = np.where(row_slot >= 0, expert * slots + row_slot, -1)
    pr, ps = layer.pool_ranks.cpu().numpy(), layer.pool_scalings.cpu().numpy()
    ref = lora(s["rows"], s["base_gate_up"], *layer.gate_up_lora, entry, pr, ps, (inter, inter))
    near(f64(s["gate_up"]), ref, 1e-2 + 1e-2 * np.abs(ref), "gate_up delta")
    ref = lora(s["act"], s["base_down"], *layer.down_lora, entry, pr, ps, (hidden,))
    near(f64(s["down"]), ref, 1e-2 + 1e-2 * np.abs(ref), "down delta")
    ref = lora(x, s["base_logits"], *layer.router_lora, slot.cpu().numpy(),
               layer.ranks.cpu().numpy(), layer.scalings.cpu().numpy(), (experts,))
    near(f64(s["logits"]), ref, 1e-2 + 1e-2 * np.abs(ref), "router delta")
    check_quantized(s["h"], f64(s["act"]))
    ref = X.combine(f64(s["down"]), positions, f64(s["routing"].weights), f64(residual))
    size = X.combine(np.abs(f64(s["down"])), positions, f64(s["routing"].weights),
                     np.abs(f64(residual)))
    near(f64(s["y"]), ref, (top_k + 2) * 2 * EPS * size, "y", t.bfloat16)


def test_layer_as_a_graph_and_on_another_stream():
    t = torch()
    layer = example().RoutedExperts(256, 512, 8, 4, 2)
    x, residual, slot = layer_inputs(64, 256, 4, 5)
    eager = layer.step(x, residual, slot)["y"].clone()
    stream = t.cuda.Stream()
    stream.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(stream):
        other = layer.step(x, residual, slot)["y"]
        t.cuda.synchronize()
        assert t.equal(other, eager)
        graph = t.cuda.CUDAGraph()
        with t.cuda.graph(graph, stream=stream):
            y = layer.step(x, residual, slot)["y"]
    for seed in (6, 7, 8):   # new inputs in the graph's buffers, eager work between
        nx, nr, ns = layer_inputs(64, 256, 4, seed)
        x.copy_(nx), residual.copy_(nr), slot.copy_(ns)
        want = layer.step(nx, nr, ns)["y"].clone()
        t.cuda.synchronize()
        graph.replay()
        t.cuda.synchronize()
        assert t.equal(y, want), seed


def test_random_shapes_agree_with_the_plain_forms():
    """Drawn sizes of every operator against its elementary form in fp32."""
    t = torch()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location("operators", os.path.join(root, "perf", "operators.py"))
    P = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(P)
    rng = random.Random(11)
    for i in range(40):
        c = P.draw(rng)
        print("case", c, flush=True)
        s = P.prepare(c, i)
        P.own = False
        want = P.run(s)
        P.own = True
        got = P.run(s)
        for key, v in want.items():
            if not v.dtype.is_floating_point:
                assert t.equal(got[key], v), (c, key)
                continue
            # fp32 sums in another order, and one rounding step where bf16
            # rounds them: 2-norms within 2^-9 (bf16) or 1e-5 of each other
            off = float((got[key].double() - v.double()).norm())
            assert off <= (2.0**-9 if v.dtype == t.bfloat16 else 1e-5) * float(v.double().norm()), (c, key)
