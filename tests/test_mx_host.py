"""Microscaled 4-bit formats and the standalone dropout, without a GPU: pins of
the oracle (oracle.mx), workspace and scale-array sizes, and every refusal of
the entry points."""

import ctypes as C
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import mx
from qlora_linear_layers_b200 import _lib
from qlora_linear_layers_b200.build import build


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


# ---------------------------------------------------------------------------
# The oracle
# ---------------------------------------------------------------------------

def test_element_and_scale_tables():
    """E2M1 over 6 is the FP4 table (fp32); E4M3 is torch's float8 type."""
    assert np.array_equal((mx.E2M1 / 6).astype(np.float32), oracle.fp4_table()[:8])
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(mx.E4M3, codes.view(torch.float8_e4m3fn).double().numpy())


def test_nearest_even_against_torch_float8():
    """The search reproduces torch's rounding to E4M3, midpoints included."""
    rng = np.random.default_rng(5)
    mid = (mx.E4M3[:-1] + mx.E4M3[1:]) / 2
    v = np.concatenate([rng.random(5000) * 448, 2.0 ** rng.uniform(-12, 8.8, 5000), mid, mx.E4M3])
    v = v.astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(mx.nearest_even(v.astype(np.float64), mx.E4M3), want)
    # E2M1 by hand: midpoints 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5 go to the even code
    got = mx.nearest_even(np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.001, 9.0]), mx.E2M1)
    assert list(got) == [0, 2, 2, 4, 4, 6, 6, 7, 7]


@pytest.mark.parametrize("fmt", [mx.MXFP4, mx.NVFP4])
def test_quantise_error_and_invariants(fmt):
    """Half a step of E2M1 under the chosen scale; powers of two scale the
    result; requantising returns the same values."""
    rng = np.random.default_rng(fmt)
    x = rng.standard_normal((9, 128)) * np.exp2(rng.integers(-20, 20, (9, 1)))
    codes, scale, s = mx.quantize(x, fmt)
    v = mx.dequantize(codes, scale, s, fmt)
    full = mx.scale_values(scale, fmt) * (1 if s is None else s[:, None])
    m = np.abs(x).reshape(9, -1, mx.BLOCK[fmt]) / full[:, :, None]
    step = np.where(m < 2, 0.5, np.where(m < 4, 1.0, 2.0))
    err = np.abs(v - x).reshape(m.shape) / full[:, :, None]
    assert np.all(err <= np.maximum(step / 2, m - 6) + 1e-12)
    assert np.all(m < 8)
    assert np.array_equal(mx.dequantize(*mx.quantize(x * 2.0 ** 7, fmt), fmt), v * 2.0 ** 7)
    assert np.array_equal(mx.fake_quantize(v, fmt), v) or fmt == mx.NVFP4
    if fmt == mx.NVFP4:
        a = np.max(np.abs(x), axis=1)
        assert np.all(a <= 2688 * s) and np.all(a > 2688 * s / 2)


def test_tile_layout_by_hand():
    s = np.arange(130 * 6).reshape(130, 6) % 251
    t = mx.tile_scales(s.astype(np.uint8))
    assert t.size == 2 * 2 * 512
    assert t[0] == s[0, 0] and t[3] == s[0, 3] and t[4] == s[32, 0] and t[16] == s[1, 0]
    assert t[512] == s[0, 4] and t[512 + 2] == 0 and t[1024 + 16] == s[129, 0]
    assert t[31 * 16 + 12 + 1] == s[127, 1]


def test_layer_gradients_by_autograd_and_differences():
    """dA, dB of the layer's formula equal autograd's and central differences
    (the layer is linear in A and in B)."""
    rng = np.random.default_rng(8)
    M, N, K, r, alpha = 5, 8, 64, 8, 16.0
    X, W, A, B, dY = (rng.standard_normal(s) for s in ((M, K), (N, K), (r, K), (N, r), (M, N)))
    dX, dA, dB = oracle.linear_bwd(X, dY, W, A, B, alpha, r)
    tA, tB = (torch.from_numpy(v).requires_grad_() for v in (A, B))
    xq = torch.from_numpy(mx.fake_quantize(X, mx.NVFP4))
    Y = xq @ torch.from_numpy(W).T + alpha / r * (torch.from_numpy(X) @ tA.T) @ tB.T
    Y.backward(torch.from_numpy(dY))
    assert np.allclose(tA.grad, dA) and np.allclose(tB.grad, dB)

    def loss(A, B):
        return float(np.sum(dY * mx.linear_fwd(X, W, A, B, alpha, r, mx.NVFP4)[0]))

    D = rng.standard_normal(A.shape)
    assert math.isclose((loss(A + D, B) - loss(A - D, B)) / 2, np.sum(D * dA), rel_tol=1e-9)
    D = rng.standard_normal(B.shape)
    assert math.isclose((loss(A, B + D) - loss(A, B - D)) / 2, np.sum(D * dB), rel_tol=1e-9)


# ---------------------------------------------------------------------------
# Sizes
# ---------------------------------------------------------------------------

def test_scale_bytes(lib):
    f = lib.qlora_mx_scale_bytes
    assert f(mx.NVFP4, 1, 32) == 512 and f(mx.NVFP4, 128, 64) == 512 and f(mx.NVFP4, 129, 96) == 2048
    assert f(mx.MXFP4, 128, 128) == 512 and f(mx.MXFP4, 1, 160) == 1024
    assert f(2, 1, 32) == 0 and f(0, 0, 32) == 0 and f(0, 1, 40) == 0
    assert f(mx.NVFP4, 28672, 8192) == 28672 * 8192 // 16


def test_workspace_sizes(lib):
    ws = lib.qlora_workspace_bytes
    for M, N, K in ((1, 1024, 1024), (16, 18944, 3584), (8192, 4096, 4096)):
        base = ws(_lib.QLORA_OP_MX_FWD, M, N, K, 0)
        assert base >= M * K // 2 + lib.qlora_mx_scale_bytes(1, M, K) + 4 * M
        assert ws(_lib.QLORA_OP_MX_FWD, M, N, K, 16) > base
        assert ws(_lib.QLORA_OP_MX_BWD, M, N, K, 0) >= 2 * N * K
        assert ws(_lib.QLORA_OP_MX_BWD, M, N, K, 16) > ws(_lib.QLORA_OP_MX_BWD, M, N, K, 0)
        for plain, drop in ((_lib.QLORA_OP_MX_FWD, _lib.QLORA_OP_MX_FWD_DROPOUT),
                            (_lib.QLORA_OP_MX_BWD, _lib.QLORA_OP_MX_BWD_DROPOUT)):
            assert ws(drop, M, N, K, 16) >= ws(plain, M, N, K, 16) + 2 * M * K       # X'
        assert ws(_lib.QLORA_OP_MX_FWD, M, N, K, 12) == 0 == ws(_lib.QLORA_OP_MX_BWD, M, N, K, -1)


# ---------------------------------------------------------------------------
# Refusals (the addresses are never dereferenced: validation fails first)
# ---------------------------------------------------------------------------

FAKE = 1 << 20
INVALID, SHAPE, ALIGN, WORKSPACE = (_lib.QLORA_ERR_INVALID_ARG, _lib.QLORA_ERR_SHAPE,
                                    _lib.QLORA_ERR_ALIGN, _lib.QLORA_ERR_WORKSPACE)


def _t(**kw):
    d = dict(packed=FAKE, rows=64, cols=128, format=1, reserved=0, scales=FAKE, row_scale=FAKE)
    d.update(kw)
    return _lib.MXTensor(**d)


def test_quantise_refusals(lib):
    def f(X=FAKE, dt=1, rows=4, cols=64, ld=64, fmt=1, p=FAKE, s=FAKE, r=FAKE):
        return lib.qlora_mx_quantize(X, dt, rows, cols, ld, fmt, p, s, r, None)
    assert f(X=None) == f(p=None) == f(s=None) == f(r=None) == INVALID
    assert f(dt=2) == f(fmt=2) == f(fmt=-1) == INVALID
    assert f(rows=0) == f(cols=0) == f(cols=48, ld=48) == f(ld=32) == f(ld=68) == SHAPE
    assert f(dt=0, ld=66) == f(rows=-5) == f(ld=1 << 50) == SHAPE
    assert f(X=FAKE + 2) == f(p=FAKE + 8) == f(s=FAKE + 4) == f(r=FAKE + 4) == ALIGN


def test_dequantise_and_product_refusals(lib):
    def deq(**kw):
        return lib.qlora_mx_dequantize(C.byref(_t(**kw)), FAKE, None)
    assert lib.qlora_mx_dequantize(None, FAKE, None) == INVALID
    assert lib.qlora_mx_dequantize(C.byref(_t()), None, None) == INVALID
    assert lib.qlora_mx_dequantize(C.byref(_t()), FAKE + 2, None) == ALIGN
    assert deq(packed=None) == deq(scales=None) == deq(row_scale=None) == deq(format=3) == INVALID
    assert deq(rows=0) == deq(cols=16) == deq(cols=80) == deq(rows=1 << 31) == SHAPE
    assert deq(packed=FAKE + 8) == deq(scales=FAKE + 1) == deq(row_scale=FAKE + 4) == ALIGN

    def mm(x, w, Y=FAKE):
        return lib.qlora_mx_matmul(C.byref(x), C.byref(w), Y, None)
    assert mm(_t(), _t(format=0)) == INVALID
    assert mm(_t(), _t(), None) == INVALID
    assert mm(_t(), _t(cols=256)) == SHAPE
    assert mm(_t(rows=0), _t()) == SHAPE
    assert mm(_t(), _t(), FAKE + 4) == ALIGN
    assert lib.qlora_mx_matmul(None, C.byref(_t()), FAKE, None) == INVALID


def _drop(p=0.1):
    return C.byref(_lib.Dropout(p=p, reserved=0, seed=1))


def test_layer_refusals(lib):
    def fwd(w=None, X=FAKE, M=4, A=FAKE, B=FAKE, r=8, alpha=16.0, d=None, Y=FAKE, T=None, ws=FAKE, n=1 << 30):
        return lib.qlora_mx_linear_fwd(C.byref(w or _t()), X, M, A, B, r, alpha, d, Y, T, ws, n, None)
    assert fwd(X=None) == fwd(Y=None) == fwd(A=None) == fwd(B=None) == fwd(r=0) == INVALID
    assert fwd(r=12) == fwd(r=256) == fwd(r=-8) == fwd(alpha=float("nan")) == fwd(alpha=float("inf")) == INVALID
    assert fwd(d=_drop(1.0)) == fwd(d=_drop(-0.1)) == fwd(d=_drop(float("nan"))) == INVALID
    assert fwd(A=None, B=None, r=0, d=_drop()) == fwd(A=None, B=None, r=0, T=FAKE) == INVALID
    assert fwd(M=0) == fwd(w=_t(rows=60)) == fwd(w=_t(cols=96)) == SHAPE
    assert fwd(X=FAKE + 8) == fwd(A=FAKE + 8) == fwd(Y=FAKE + 8) == fwd(T=FAKE + 8) == fwd(ws=FAKE + 8) == ALIGN
    assert fwd(ws=None) == fwd(n=100) == WORKSPACE

    def bwd(X=FAKE, dY=FAKE, M=4, A=FAKE, B=FAKE, r=8, d=None, T=None, dX=FAKE, dA=FAKE, dB=FAKE, n=1 << 30):
        return lib.qlora_mx_linear_bwd(C.byref(_t()), X, dY, M, A, B, r, 16.0, d, T, dX, dA, dB, FAKE, n, None)
    assert bwd(dY=None) == bwd(dX=None) == bwd(dA=None) == bwd(dB=None) == bwd(r=0) == INVALID
    assert bwd(A=None, B=None, r=0) == bwd(A=None, B=None, r=0, dA=None, dB=None, T=FAKE) == INVALID
    assert bwd(dY=FAKE + 8) == bwd(dX=FAKE + 8) == bwd(T=FAKE + 8) == bwd(dB=FAKE + 8) == ALIGN
    assert bwd(M=0) == SHAPE and bwd(n=100) == WORKSPACE


def test_dropout_refusals(lib):
    def f(X=FAKE, ldx=8, R=None, ldr=0, dt=1, rows=2, cols=8, d=None, first=0, Y=FAKE, ldy=8):
        return lib.qlora_dropout_fwd(X, ldx, R, ldr, dt, rows, cols, d or _drop(), first, Y, ldy, None)
    assert lib.qlora_dropout_fwd(FAKE, 8, None, 0, 1, 2, 8, None, 0, FAKE, 8, None) == INVALID
    assert f(X=None) == f(Y=None) == f(dt=2) == f(d=_drop(1.0)) == f(d=_drop(-1.0)) == INVALID
    assert f(rows=0) == f(cols=0) == f(ldx=7) == f(ldy=7) == f(R=FAKE, ldr=7) == f(first=-1) == SHAPE
    assert f(rows=1 << 40, cols=1 << 40, ldx=1 << 40, ldy=1 << 40) == SHAPE
    assert f(X=FAKE + 2) == f(Y=FAKE + 2) == f(R=FAKE + 2, ldr=8) == ALIGN
    assert lib.qlora_dropout_bwd(None, 8, 1, 2, 8, _drop(), 0, FAKE, 8, None) == INVALID
    assert lib.qlora_dropout_bwd(FAKE, 8, 1, 2, 8, _drop(), 0, FAKE, 4, None) == SHAPE


def test_python_refuses_host_tensors():
    import qlora_linear_layers_b200 as q
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.mx_quantize(x)
    with pytest.raises(ValueError):
        q.dropout_fwd(x, 0.1, 1)
    with pytest.raises(ValueError):
        q.dropout_bwd(x, 0.1, 1)
