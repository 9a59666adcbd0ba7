"""The rule that picks a product's kernel: the sizes of dense_shapes.py reach the kernels
that they name, and there are no others."""
import ctypes
import os

import pytest

import adapter_lora_serving_amd as L
from adapter_lora_serving_amd import build
from dense_shapes import GATED, PLAIN


@pytest.fixture(scope="module")
def choice():
    if not os.path.exists(L.lib_path()):
        build.build()
    f = L.lib().lora_test_linear_choice
    f.restype, f.argtypes = None, [ctypes.c_int] * 8 + [ctypes.c_void_p]

    def call(mx, gated, f32, residual, T, N, K):
        out = (ctypes.c_int32 * 3)()
        f(mx, gated, f32, residual, T, N, K, 256, out)
        return tuple(out)

    return call


def test_shapes_reach_the_kernels_they_name(choice):
    for (form, out), shapes in PLAIN.items():
        for kernel, size in shapes.items():
            assert choice(form == "mx", 0, out == "f32", 1, *size) == kernel, (form, out, kernel)
    for form, shapes in GATED.items():
        for kernel, size in shapes.items():
            assert choice(form == "mx", 1, 0, 0, *size) == kernel, (form, kernel)


def test_tiles_are_ragged_and_in_several_rounds():
    for (form, _), shapes in list(PLAIN.items()) + [((form, None), s) for form, s in GATED.items()]:
        for (rows, cols, each), (T, N, K) in shapes.items():
            if not each:
                continue
            if shapes in GATED.values():
                cols //= 2
            tiles = -(-T // rows) * -(-N // cols)
            assert tiles > 256 * each and T % rows and N % cols
            stages = -(-K * (1 if form == "mx" else 2) // 128)
            assert stages % 2 and K * (1 if form == "mx" else 2) % 128


def test_no_other_kernels(choice):
    sizes = [1, 8, 9, 16, 17, 32, 33, 64, 65, 100, 128, 200, 256, 300, 500, 512, 700, 1024, 1500, 2048, 4096, 8192]
    for (form, out), shapes in PLAIN.items():
        mx = form == "mx"
        met = {choice(mx, 0, out == "f32", r, T, N, K) for T in sizes for K in (64, 512, 4096, 14336)
               for N in (1, 64, 500, 1024, 4096, 6144, 14336, 28672, 131072) for r in (0, 1)}
        assert met == set(shapes), (form, out)
    for form, shapes in GATED.items():
        met = {choice(form == "mx", 1, 0, 0, T, N, K) for T in sizes for K in (64, 512, 4096, 14336)
               for N in (1, 64, 500, 1024, 4096, 6144, 14336, 28672, 131072)}
        assert met == set(shapes), form
