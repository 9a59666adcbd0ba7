"""The routed-expert operators at the ends of their limits, on the GPU.

Inputs repeat or are constant, so that what is expected needs no second pass
over gigabytes on the host."""
import numpy as np
import pytest

import adapter_lora_serving_amd as L
from gpu_util import f64, torch
from oracle import experts_oracle as X
from test_gpu_experts import check_product, check_quantized, held, values

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("T", [(1 << 23) + 1, (1 << 24) - 1, 1 << 24, (1 << 25) + 3])
def test_combine_of_many_tokens(T):
    """From 2^24 tokens on, a workgroup a token is 2^32 threads and more."""
    t = torch()
    rows = t.stack([t.full((8,), float(v), device=DEV) for v in range(1, 5)]).bfloat16()
    pos = (t.arange(T, device=DEV) % 5 - 1).int().unsqueeze(1)   # -1: adds nothing
    y = t.full((T, 8), -1.0, device=DEV).bfloat16()
    L.combine_experts(rows, pos, t.full((T, 1), 2.0, device=DEV), y=y)
    want = 2 * (pos + 1).bfloat16().expand(T, 8)
    assert t.equal(y, want)


@pytest.mark.parametrize("T,E,live", [((1 << 28) + 5, 2, 1), ((1 << 28) - 1, 2, 1),
                                      ((1 << 26) + 3, 257, 256)])
def test_route_of_many_tokens(T, E, live):
    """16 lanes a token (64 past 256 experts): from 2^28 (2^26) tokens on that
    is 2^32 threads and more."""
    t = torch()
    x = t.zeros(T, E, dtype=t.bfloat16, device=DEV)
    x[:, live] = 1.0
    x[1::2, 0] = 2.0
    out = L.Routing(t.full((T, 1), -5, dtype=t.int32, device=DEV), t.zeros(T, 1, device=DEV))
    L.route_experts(x, 1, out=out)
    del x
    assert bool((out.ids[0::2] == live).all()) and bool((out.ids[1::2] == 0).all())
    assert bool((out.weights == 1).all())


@pytest.mark.parametrize("rows,K", [(1 << 27, 32), (1 << 20, 4096)])
def test_quantize_of_2_to_the_32_values(rows, K):
    """The largest quantisation: with 32 columns its rows and their padding are
    2^31 pieces of 8."""
    t = torch()
    part = t.randn(1 << 10, K, device=DEV).bfloat16()
    x = part.repeat(rows >> 10, 1)
    x[-1] = 7.0
    want, last = L.quantize_mxfp4(part), L.quantize_mxfp4(x[-1:].contiguous())
    q = L.quantize_mxfp4(x)
    assert t.equal(q.codes[-1:], last.codes) and t.equal(q.scales[-1:], last.scales)
    q.codes[-1], q.scales[-1] = want.codes[-1], want.scales[-1]
    for got, one in zip(q, want):
        assert bool((got.view(-1, *one.shape) == one).all())
    back = L.dequantize_mxfp4(q)
    assert bool((back.view(-1, *part.shape) == L.dequantize_mxfp4(want)).all())


@pytest.mark.parametrize("grouped", [False, True])
def test_product_of_2_to_the_31_rows(grouped):
    """One row less than 2^31, whose number and a tile's pass 31 bits."""
    t = torch()
    rows, N, K = (1 << 31) - 1, 2, 32
    part = L.quantize_mxfp4(t.randn(1 << 15, K, device=DEV))
    x = L.MXFP4(t.empty(rows, K // 2, dtype=t.uint8, device=DEV),
                t.empty(rows, 4, dtype=t.uint8, device=DEV))
    for to, one in zip(x, part):
        whole = to[:rows >> 15 << 15].view(-1, *one.shape)
        whole.copy_(one.expand_as(whole))
        to[rows >> 15 << 15:].copy_(one[:rows & 0x7fff])
    w = L.quantize_mxfp4(t.randn(2, N, K, device=DEV))
    one = [L.mxfp4_linear(part, L.MXFP4(w.codes[e], w.scales[e])) for e in range(2)]
    if grouped:   # a row of expert 0, the others of expert 1 but for the last
        y = L.mxfp4_expert_linear(x, w, t.tensor([0, 1, rows - 1], device=DEV))
        assert t.equal(y[0], one[0][0]) and bool((y[-1] == 0).all())
        y[0], y[-1] = one[1][0], one[1][(rows - 1) & 0x7fff]
    else:
        y = L.mxfp4_linear(x, L.MXFP4(w.codes[1], w.scales[1]))
    assert bool((y[:rows >> 15 << 15].view(-1, 1 << 15, N) == one[1]).all())
    assert t.equal(y[rows >> 15 << 15:], one[1][:rows & 0x7fff])


@pytest.mark.parametrize("T,k,E", [(16384, 8, 1024), (16385, 8, 1024), (1 << 17, 32, 1024), (74899, 7, 1023),
                                   (209715, 20, 1024), ((1 << 17) + 1, 32, 1024), (1 << 22, 1, 1024)])
def test_rows_of_many_choices_and_experts(T, k, E):
    """Around the largest sort of one launch, 2^22 choices of 1024 experts."""
    t = torch()
    rng = np.random.default_rng(T)
    ids = rng.integers(-3, E + 3, (T, k)).astype(np.int32)
    slot = rng.integers(-1, 50, T).astype(np.int32)
    r = L.expert_rows(t.from_numpy(ids).to(DEV), E, t.from_numpy(slot).to(DEV))
    key = ids.reshape(-1)
    key = np.where((key < 0) | (key >= E), E, key)
    order = np.argsort(key, kind="stable")
    live = key[order] < E
    positions = np.empty(T * k, np.int32)
    positions[order] = np.arange(T * k)
    counts = np.bincount(key, minlength=E + 1)[:E]
    want = (order // k, np.where(key < E, positions, -1).reshape(T, k),
            np.concatenate([[0], np.cumsum(counts)]), np.where(live, slot[order // k], -1))
    for got, ref, name in zip(r, want, r._fields):
        assert np.array_equal(got.cpu().numpy(), ref), name


@pytest.mark.parametrize("rows,N,K", [(3, 40, 1 << 20), (300, 130, (1 << 20) - 32), (40, 1 << 20, 96),
                                      (1, (1 << 20) - 1, 544), (700, 1 << 20, 544)])
def test_product_of_the_widest_operands(rows, N, K):
    t = torch()
    x, w = held(rows, K, 1), held(N, K, 2)
    y = L.mxfp4_linear(x, w, dtype=t.float32)
    check_product(y, values(x), values(w), K)


@pytest.mark.parametrize("rows", [40, 5000])
def test_product_of_the_most_experts(rows):
    t = torch()
    E, N, K = 1024, 72, 544
    x, w = held(rows, K, 1), held(E * N, K, 2)
    W = L.MXFP4(w.codes.view(E, N, -1), w.scales.view(E, N, -1))
    off = np.sort(np.random.default_rng(rows).integers(0, rows + 1, E + 1)).astype(np.int32)
    y = L.mxfp4_expert_linear(x, W, t.from_numpy(off).to(DEV), dtype=t.float32)
    xv, wv = values(x), values(w).view(E, N, K)
    dead = t.ones(rows, dtype=t.bool, device=DEV)
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        dead[lo:hi] = False
        if hi > lo:
            check_product(y[lo:hi], xv[lo:hi], wv[e], K, f"expert {e}")
    assert bool((y[dead] == 0).all())


@pytest.mark.parametrize("K", [1 << 20, (1 << 20) - 32])
def test_quantize_the_widest_rows(K):
    t = torch()
    x = t.randn(3, 2 * K, device=DEV).bfloat16()
    act, q = L.silu_mul_quantize_mxfp4(x)
    check_quantized(q, f64(act))
    rows, g = L.gather_quantize_mxfp4(act, t.tensor([2, 0, 2, 1], device=DEV))
    assert t.equal(rows, act[[2, 0, 2, 1]]) and t.equal(g.codes, q.codes[[2, 0, 2, 1]])
    assert t.equal(L.dequantize_mxfp4(q), t.from_numpy(X.dequantize(*X.quantize(f64(act)))).to(DEV).bfloat16())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_combine_the_widest_rows(dtype):
    t = torch()
    rows = t.randint(-8, 9, (5, 1 << 20), device=DEV).to(t.bfloat16 if dtype == "bf16" else t.float32)
    pos = t.tensor([[4, 0], [5, 3], [-1, 9]], device=DEV)
    y = L.combine_experts(rows, pos, t.tensor([[2.0, 1.0], [1.0, -4.0], [1.0, 1.0]], device=DEV))
    assert t.equal(y[0], 2 * rows[4] + rows[0]) and t.equal(y[1], -4 * rows[3])   # exact
    assert bool((y[2] == 0).all())
