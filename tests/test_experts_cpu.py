"""CPU checks of the routed-expert operators: the oracle against hand-worked
cases, and the C ABI's refusals (no call here reaches a kernel launch)."""
import os

import numpy as np
import pytest

import adapter_lora_serving_amd as L
from oracle import experts_oracle as X

OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
A16, MIS = 0x10000, 0x10008   # device addresses that are never dereferenced here


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.lib_path()):
        from adapter_lora_serving_amd import build
        build.build()
    return L.lib()


# ---- the oracle -----------------------------------------------------------

def test_route_by_hand():
    # softmax of (log 1, log 2, log 4, log 1) is (1, 2, 4, 1) / 8
    x = np.log(np.array([[1.0, 2.0, 4.0, 1.0]]))
    ids, w, _ = X.route(x, 2)
    assert ids.tolist() == [[2, 1]] and np.allclose(w, [[4 / 6, 2 / 6]])
    ids, w, _ = X.route(x, 2, bias=[0.5, 0.0, 0.0, 0.0], renormalize=False, scaling=2.0)
    assert ids.tolist() == [[0, 2]] and np.allclose(w, [[0.25, 1.0]])   # weights without the bias
    ids, _, _ = X.route(x, 4)
    assert ids.tolist() == [[2, 1, 0, 3]]                               # the tie to the lowest
    # groups {0, 1} and {2, 3}: best 2/8 against 4/8, sums 3/8 against 5/8
    assert X.route(x, 1, groups=2, top_groups=1)[0].tolist() == [[2]]
    y = np.log(np.array([[3.0, 3.0, 4.0, 1.0]]))
    assert X.route(y, 2, groups=2, top_groups=1, group_score="max")[0].tolist() == [[2, 3]]
    assert X.route(y, 2, groups=2, top_groups=1, group_score="sum2")[0].tolist() == [[0, 1]]


def test_route_closed_experts():
    inf, nan = np.inf, np.nan
    ids, w, _ = X.route(np.array([[-inf, 0.0, nan, -inf], [-inf, nan, -inf, nan],
                                  [1.0, inf, 0.0, inf]]), 2, scores="softmax")
    assert ids.tolist() == [[1, -1], [-1, -1], [1, 3]]
    assert np.allclose(w, [[1, 0], [0, 0], [0.5, 0.5]])


def test_rows_by_hand():
    rt, pos, off, slot = X.expert_rows(np.array([[2, 0], [0, -1], [2, 5]]), 3, [7, 8, 9])
    assert rt.tolist() == [0, 1, 0, 2, 1, 2]
    assert pos.tolist() == [[2, 0], [1, -1], [3, -1]]
    assert off.tolist() == [0, 2, 2, 4] and slot.tolist() == [7, 8, 7, 9, -1, -1]


def test_quantize_by_hand():
    x = np.zeros((1, 32))
    # largest 6: scale 1. Ties: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    x[0, :10] = [6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.26, -3.0]
    codes, scales = X.quantize(x)
    assert scales.tolist() == [[127, 0, 0, 0]]
    assert X.dequantize(codes, scales)[0, :10].tolist() == [6, 0, 1, 1, 2, 2, 4, 4, -0.5, -3]
    # 7.9 has the exponent of 6's scale and saturates; 8 takes the next scale
    for top, byte, back in ((7.9, 127, 6.0), (8.0, 128, 8.0), (2.0**-130, 0, 0.0), (0.0, 0, 0.0)):
        x = np.zeros((1, 32))
        x[0, 3] = top
        codes, scales = X.quantize(x)
        assert scales[0, 0] == byte and X.dequantize(codes, scales)[0, 3] == back, top
    for v in (np.nan, np.inf):
        x[0, 0] = v
        codes, scales = X.quantize(x)
        assert scales[0, 0] == 255 and not codes.any() and np.isnan(X.dequantize(codes, scales)).all()


def test_quantize_is_nearest():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 96)) * np.exp(rng.standard_normal((50, 1)) * 4)
    codes, scales = X.quantize(x)
    v = X.dequantize(codes, scales).reshape(50, 3, 32)
    s = np.exp2(scales[:, :3].astype(float) - 127)
    grid = np.concatenate([-X.GRID, X.GRID])
    d = np.abs(x.reshape(50, 3, 32, 1) - grid * s[:, :, None, None]).min(3)
    assert np.allclose(np.abs(v - x.reshape(50, 3, 32)), d, rtol=1e-12, atol=0)
    top = np.abs(x.reshape(50, 3, 32)).max(2) / s
    assert (top >= 4).all() and (top < 8).all()


# ---- refusals -------------------------------------------------------------

def test_route_refusals(lib):
    def call(dtype=1, x=A16, T=4, E=64, k=2, scores=0, bias=None, G=1, tg=1, gsc=0, ids=A16, w=A16):
        return lib.lora_route_experts(dtype, x, T, E, k, scores, bias, G, tg, gsc, 1, 1.0, ids, w,
                                      None)
    assert call(dtype=2) == UNSUPPORTED
    assert call(T=-1) == INVALID
    for kw in (dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(G=0), dict(G=17)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(scores=2), dict(gsc=2), dict(G=3), dict(G=4, tg=0), dict(G=4, tg=5),
               dict(k=20, G=4, tg=1), dict(E=4, k=5), dict(x=None), dict(ids=None), dict(w=None)):
        assert call(**kw) == INVALID, kw
    assert call(T=1 << 30, k=2) == INVALID          # 2^31 choices
    assert call(x=MIS) == ALIGN
    assert call(T=0, x=None, ids=None, w=None) == OK


def test_rows_refusals(lib):
    def call(ids=A16, T=4, k=2, E=8, ts=A16, rt=A16, pos=A16, off=A16, rs=A16, ws=None, wsb=0):
        return lib.lora_expert_rows(ids, T, k, E, ts, rt, pos, off, rs, ws, wsb, None)
    assert call(T=-1) == INVALID
    for kw in (dict(k=0), dict(k=33), dict(E=0), dict(E=1025)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(ids=None), dict(rt=None), dict(pos=None), dict(off=None), dict(rs=None),
               dict(ts=None)):
        assert call(**kw) == INVALID, kw
    need = lib.lora_expert_rows_workspace_bytes(10000, 8, 256)
    assert need > 0 and lib.lora_expert_rows_workspace_bytes(8192, 8, 256) == 0
    assert lib.lora_expert_rows_workspace_bytes(-1, 8, 256) == 0
    assert call(T=10000, k=8, E=256) == WORKSPACE
    assert call(T=10000, k=8, E=256, ws=A16, wsb=need - 1) == WORKSPACE
    assert call(T=10000, k=8, E=256, ws=MIS, wsb=need) == ALIGN


def test_combine_refusals(lib):
    def call(dtype=1, rows=A16, n=8, H=64, pos=A16, w=A16, T=4, k=2, res=None, y=A16):
        return lib.lora_combine_experts(dtype, rows, n, H, pos, w, T, k, res, y, None)
    assert call(dtype=5) == UNSUPPORTED
    assert call(k=33) == UNSUPPORTED
    for kw in (dict(T=-1), dict(n=-1), dict(H=0), dict(rows=None), dict(pos=None), dict(w=None),
               dict(y=None)):
        assert call(**kw) == INVALID, kw
    assert call(H=1 << 21) == UNSUPPORTED
    for kw in (dict(H=60), dict(dtype=0, H=62), dict(rows=MIS), dict(res=MIS), dict(y=MIS)):
        assert call(**kw) == ALIGN, kw
    assert call(T=0, rows=None, n=0, pos=None, w=None, y=None) == OK


def test_quantize_refusals(lib):
    def call(dtype=1, form=0, x=A16, xr=4, ri=None, rows=4, K=64, ro=None, c=A16, s=A16):
        return lib.lora_quantize_mxfp4(dtype, form, x, xr, ri, rows, K, ro, c, s, None)
    assert call(dtype=3) == UNSUPPORTED
    assert call(K=(1 << 20) + 32) == UNSUPPORTED
    assert call(rows=1 << 13, xr=1 << 13, K=1 << 20) == UNSUPPORTED       # 2^33 values
    for kw in (dict(form=3), dict(rows=-1), dict(K=0), dict(xr=-1), dict(x=None), dict(c=None),
               dict(s=None), dict(xr=3), dict(form=1, ro=A16), dict(form=1, ri=A16),
               dict(form=1, ri=A16, ro=A16, xr=0), dict(form=2)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(K=48), dict(x=MIS), dict(c=MIS), dict(s=A16 + 2), dict(form=2, ro=MIS)):
        assert call(**kw) == ALIGN, kw
    assert call(rows=0, x=None, c=None, s=None) == OK
    assert lib.lora_mxfp4_scale_row_bytes(4096) == 128
    assert lib.lora_mxfp4_scale_row_bytes(96) == 4
    assert lib.lora_mxfp4_scale_row_bytes(100) == 0
    d = lib.lora_dequantize_mxfp4
    assert d(7, A16, A16, 4, 64, A16, None) == UNSUPPORTED
    assert d(1, A16, A16, 4, 65, A16, None) == ALIGN
    assert d(1, None, A16, 4, 64, A16, None) == INVALID
    assert d(1, A16, A16, 4, 64, MIS, None) == ALIGN
    assert d(1, None, None, 0, 64, None, None) == OK


def test_linear_refusals(lib):
    def call(dtype=1, x=A16, xs=A16, rows=4, w=A16, ws=A16, N=64, K=64, y=A16):
        return lib.lora_mxfp4_linear(dtype, x, xs, rows, w, ws, N, K, y, None)

    def grouped(off=A16, E=4, rows=4):
        return lib.lora_mxfp4_expert_linear(1, A16, A16, rows, A16, A16, 64, 64, off, E, A16, None)
    assert call(dtype=2) == UNSUPPORTED
    for kw in (dict(N=1 << 21), dict(K=1 << 21)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(rows=-1), dict(N=0), dict(K=0), dict(x=None), dict(xs=None), dict(w=None),
               dict(ws=None), dict(y=None)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(K=16), dict(x=MIS), dict(w=MIS), dict(y=MIS), dict(xs=A16 + 1), dict(ws=A16 + 1)):
        assert call(**kw) == ALIGN, kw
    assert call(rows=0, x=None, xs=None, w=None, ws=None, y=None) == OK
    assert grouped(off=None) == INVALID
    assert grouped(E=0) == UNSUPPORTED and grouped(E=1025) == UNSUPPORTED
    assert grouped(rows=0, off=None) == OK


def test_binding_refuses_cpu_tensors(lib):
    import torch
    x = torch.zeros(2, 64)
    for f in (lambda: L.route_experts(x, 2), lambda: L.quantize_mxfp4(x),
              lambda: L.silu_mul_quantize_mxfp4(x),
              lambda: L.expert_rows(torch.zeros(2, 2, dtype=torch.int32), 4)):
        with pytest.raises(L.LoraError):
            f()
