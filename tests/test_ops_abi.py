"""Refusals of the grouped matmul, the FP8 matmul, its quantisers and the layer
norm: every bad argument is answered before CUDA is touched (no GPU here)."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p(1 << 20)          # 256-byte aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)  # not 16-byte aligned
WS16 = ctypes.c_void_p((1 << 20) + 16)  # not 256-byte aligned
N = None


@pytest.fixture(scope="module")
def L():
    import os

    from sparse_moe_layer_limited_b200 import _lib, build
    if not os.path.exists(build.LIB_PATH):
        build.build()
    return _lib


def test_grouped_matmul(L):
    f = L.lib()
    for fn in (f.moe_grouped_matmul, f.moe_grouped_matmul_dx):
        ok = [P, 4, P, 2, P, 16, 24, L.DTYPE_BF16, P, P, N]

        def call(i, v):
            a = list(ok)
            a[i] = v
            return fn(*a)
        for i, v in ((1, -1), (3, 0), (3, -2), (5, 0), (6, -8)):
            assert call(i, v) == L.ERR_ARG, (i, v)
        for i in (0, 2, 4, 8, 9):
            assert call(i, N) == L.ERR_ARG and call(i, ODD) == L.ERR_ARG, i
        assert call(9, WS16) == L.ERR_ARG
        assert call(2, N) == L.ERR_ARG                     # two experts need offsets
        assert call(3, 385) == L.ERR_UNSUPPORTED
        assert call(5, 12) == L.ERR_UNSUPPORTED and call(6, 20) == L.ERR_UNSUPPORTED
        assert call(7, L.DTYPE_E4M3) == L.ERR_UNSUPPORTED and call(7, 9) == L.ERR_UNSUPPORTED
        assert call(1, 1 << 40) == L.ERR_UNSUPPORTED
        # no rows: nothing to do, and the row pointers may be NULL
        assert fn(N, 0, P, 2, P, 16, 24, L.DTYPE_BF16, N, P, N) == L.OK
        assert fn(N, 0, N, 1, P, 16, 24, L.DTYPE_FP32, N, P, N) == L.OK


def test_grouped_matmul_dw(L):
    f = L.lib().moe_grouped_matmul_dw
    ok = [P, P, 4, P, 2, 16, 24, L.DTYPE_BF16, P, P, N]

    def call(i, v):
        a = list(ok)
        a[i] = v
        return f(*a)
    for i, v in ((2, -1), (4, 0), (5, 0), (6, 0)):
        assert call(i, v) == L.ERR_ARG, (i, v)
    for i in (0, 1, 3, 8, 9):
        assert call(i, N) == L.ERR_ARG and call(i, ODD) == L.ERR_ARG, i
    assert call(4, 385) == L.ERR_UNSUPPORTED
    assert call(5, 12) == L.ERR_UNSUPPORTED and call(6, 20) == L.ERR_UNSUPPORTED
    assert call(7, 9) == L.ERR_UNSUPPORTED
    assert f(P, P, 4, P, 384, 1 << 24, 1 << 20, L.DTYPE_BF16, P, P, N) == L.ERR_UNSUPPORTED


def test_fp8_matmul(L):
    f = L.lib()
    for fn in (f.moe_matmul_fp8, f.moe_matmul_fp8_dx):
        ok = [P, 0, P, 4, 4, P, 2, P, P, 32, 48, P, P, N]

        def call(i, v):
            a = list(ok)
            a[i] = v
            return fn(*a)
        for i, v in ((3, 3), (4, -1), (6, 0), (9, 0), (10, 0)):
            assert call(i, v) == L.ERR_ARG, (i, v)
        for i in (0, 2, 5, 7, 8, 11, 12):
            assert call(i, N) == L.ERR_ARG and call(i, ODD) == L.ERR_ARG, i
        assert call(1, 2) == L.ERR_UNSUPPORTED and call(1, -1) == L.ERR_UNSUPPORTED
        assert call(6, 385) == L.ERR_UNSUPPORTED and call(10, 40) == L.ERR_UNSUPPORTED
        assert fn(N, 0, N, 0, 0, P, 2, P, P, 32, 48, N, P, N) == L.OK
    assert f.moe_matmul_fp8_dx(P, 0, P, 4, 4, P, 2, P, P, 33, 48, P, P, N) == L.ERR_UNSUPPORTED


def test_quantisers(L):
    f = L.lib()
    r = f.moe_quantize_rows_fp8
    assert r(P, -1, 128, 0, P, P, 4, N) == L.ERR_ARG
    assert r(P, 4, 0, 0, P, P, 4, N) == L.ERR_ARG
    assert r(P, 4, 128, 0, P, P, 3, N) == L.ERR_ARG
    assert r(P, 4, 120, 0, P, P, 4, N) == L.ERR_UNSUPPORTED
    assert r(P, 4, 128, 2, P, P, 4, N) == L.ERR_UNSUPPORTED
    for a in ((N, P, P), (P, N, P), (P, P, N), (ODD, P, P), (P, ODD, P), (P, P, ODD)):
        assert r(a[0], 4, 128, 0, a[1], a[2], 4, N) == L.ERR_ARG
    assert r(N, 0, 128, 0, N, N, 0, N) == L.OK
    b = f.moe_quantize_blocks_fp8
    assert b(P, 0, 128, 128, P, P, N) == L.ERR_ARG
    assert b(P, 1, 0, 128, P, P, N) == L.ERR_ARG
    assert b(P, 1, 128, 100, P, P, N) == L.ERR_UNSUPPORTED
    assert b(N, 1, 128, 128, P, P, N) == L.ERR_ARG
    assert b(P, 1, 128, 128, ODD, P, N) == L.ERR_ARG


def test_layer_norm(L):
    f = L.lib()
    ok = [P, P, P, 1e-5, 4, 64, L.DTYPE_BF16, P, P, P, N]

    def call(i, v):
        a = list(ok)
        a[i] = v
        return f.moe_layer_norm(*a)
    for i in (0, 1, 7, 8, 9):
        assert call(i, N) == L.ERR_ARG and call(i, ODD) == L.ERR_ARG, i
    assert call(2, ODD) == L.ERR_ARG
    for eps in (-1e-5, float("nan"), float("inf")):
        assert call(3, eps) == L.ERR_ARG
    assert call(4, -1) == L.ERR_ARG and call(5, 0) == L.ERR_ARG
    assert call(5, 16385) == L.ERR_UNSUPPORTED and call(4, 1 << 31) == L.ERR_UNSUPPORTED
    assert call(6, L.DTYPE_E4M3) == L.ERR_UNSUPPORTED
    assert f.moe_layer_norm(N, P, N, 1e-5, 0, 64, 0, N, N, N, N) == L.OK
    ok = [P, P, P, P, P, 4, 64, L.DTYPE_BF16, P, P, P, P, N]

    def back(i, v):
        a = list(ok)
        a[i] = v
        return f.moe_layer_norm_backward(*a)
    for i in (0, 1, 2, 3, 4, 8, 9, 11):
        assert back(i, N) == L.ERR_ARG and back(i, ODD) == L.ERR_ARG, i
    assert back(10, ODD) == L.ERR_ARG and back(11, WS16) == L.ERR_ARG
    assert back(5, -1) == L.ERR_ARG and back(6, 0) == L.ERR_ARG
    assert back(6, 16385) == L.ERR_UNSUPPORTED and back(7, 2) == L.ERR_UNSUPPORTED
    assert f.moe_layer_norm_workspace_size(4, 64) > 0
    assert f.moe_layer_norm_workspace_size(-1, 64) == 0
    assert f.moe_layer_norm_workspace_size(4, 16385) == 0


def test_the_binding_refuses_wrong_tensors(L):
    """Types, shapes and places are checked before the library is called."""
    from sparse_moe_layer_limited_b200 import (moe_grouped_matmul, moe_grouped_matmul_dw,
                                               moe_layer_norm, moe_matmul_fp8,
                                               moe_quantize_rows_fp8)
    bf = torch.bfloat16
    x, w, y = torch.zeros(4, 24, dtype=bf), torch.zeros(2, 16, 24, dtype=bf), torch.zeros(4, 16, dtype=bf)
    off, ws = torch.zeros(3, dtype=torch.int32), torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        moe_grouped_matmul(x, off, w, y, ws)
    with pytest.raises(ValueError, match="dimensions"):
        moe_grouped_matmul(x, off, w[0], y, ws)
    with pytest.raises(TypeError):
        moe_grouped_matmul(x.half(), off, w, y, ws)
    with pytest.raises(ValueError):
        moe_grouped_matmul_dw(x[0], x, off, w, ws)
    with pytest.raises(TypeError):
        moe_quantize_rows_fp8(x, x, torch.zeros(1, 4))
    with pytest.raises(TypeError):
        moe_matmul_fp8(x, torch.zeros(1, 4), off, w, torch.zeros(2, 1, 1), y, ws)
    with pytest.raises(TypeError):
        moe_layer_norm(x.half(), torch.ones(24), None, 1e-5, x, torch.ones(4), torch.ones(4))


WIDE = (1 << 31) - 16  # a C int whose rounding up to whole tiles is none


def test_widths_next_to_31_bits(L):
    f = L.lib()
    U = L.ERR_UNSUPPORTED
    for n, k in ((WIDE, 16), (16, WIDE)):
        for dt in (L.DTYPE_BF16, L.DTYPE_FP32):
            assert f.moe_grouped_matmul(P, 4, N, 1, P, n, k, dt, P, P, N) == U
            assert f.moe_grouped_matmul_dx(P, 4, N, 1, P, n, k, dt, P, P, N) == U
            assert f.moe_grouped_matmul_dw(P, P, 4, N, 1, n, k, dt, P, P, N) == U
        assert f.moe_matmul_fp8(P, 0, P, 4, 4, N, 1, P, P, n, k, P, P, N) == U
        assert f.moe_matmul_fp8_dx(P, 0, P, 4, 4, N, 1, P, P, n, k, P, P, N) == U
        assert f.moe_quantize_blocks_fp8(P, 1, n, k, P, P, N) == U
    assert f.moe_quantize_rows_fp8(P, 4, WIDE, 0, P, P, 4, N) == U


def test_dimensions_past_31_bits(L):
    """A view of that many columns, refused before its memory is looked at."""
    w = torch.empty(1).expand(1, 8, (1 << 32) + 8)
    x = torch.empty(1).expand(1, (1 << 32) + 8)
    with pytest.raises(ValueError, match="31 bits"):
        L.moe_grouped_matmul(x, None, w, x, x)
    with pytest.raises(ValueError, match="31 bits"):
        L.moe_quantize_rows_fp8(x, x, x)
