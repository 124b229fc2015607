"""GPU parity of the microscaled product and layer where row scales are far
from 1, against fp64 on the tensors' own values: the product of a token's scale and
a weight row's may leave fp32's range although the result does not.
"""

import numpy as np
import pytest
import torch

from oracle import mx

pytestmark = pytest.mark.gpu

H = 2.0 ** -8            # half a bf16 step
U = 2.0 ** -23           # a truncated fp32 step
TINY = 2.0 ** -134 * 1.01        # half of bf16's fixed step below 2^-126, and fp32's below that
BF16_MAX = 255 * 2.0 ** 120


@pytest.fixture(scope="module")
def q():
    from qlora_linear_layers_b200.build import build
    build()
    import qlora_linear_layers_b200 as q
    return q


def stored(q, rows, cols, exps, seed, low):
    """Random codes (row 0: zeros) under E4M3 scales that are small (low) or large,
    row scales 2^exps in turn; and the fp64 values."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    codes[0] = 0
    scale = rng.integers(1, 9, (rows, cols // 16)) if low else rng.integers(90, 127, (rows, cols // 16))
    s = np.exp2(np.resize(exps, rows)).astype(np.float32)
    t = q.MXTensor(torch.from_numpy(mx.pack(codes)).cuda(), torch.from_numpy(mx.tile_scales(scale.astype(np.uint8))).cuda(),
                   torch.from_numpy(s).cuda(), rows, cols, mx.NVFP4)
    return t, torch.from_numpy(mx.dequantize(codes, scale, s, mx.NVFP4)).cuda()


def check(got, ref, bound):
    """Within the bound, and infinite past bf16's range (between, either is right)."""
    got = got.double()
    fits, past = ref.abs() + bound < BF16_MAX, ref.abs() - bound > 2.0 ** 128
    assert bool(got[past].isinf().all()) and bool((got[past].sign() == ref[past].sign()).all())
    assert bool(got[fits].isfinite().all())
    assert float(((got - ref).abs() - bound - TINY)[fits].max()) <= 0


# every kernel of the product: up to 16 and 32 tokens, 128 wide whole and split, paired in one round and more
SIZES = [(5, 136, 192), (16, 256, 4096), (24, 136, 4096), (40, 136, 192), (100, 128, 8192), (33, 264, 4096), (2000, 4096, 512)]


@pytest.mark.parametrize("low", [False, True])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_product_far_row_scales(q, M, N, K, low):
    x, vx = stored(q, M, K, [-100, -70, 100, 0, 60, -3, 70], M, low)
    w, vw = stored(q, N, K, [100, -100, -80, -1, 64], N, low)
    ref, mag = vx @ vw.T, vx.abs() @ vw.abs().T
    check(q.mx_matmul(x, w), ref, H * ref.abs() + (1 + H) * (K + 3) * U * mag)
    assert q.qlora_check_status() == 0


@pytest.mark.parametrize("M,N,K", SIZES)
def test_layer_far_row_scales(q, M, N, K):
    """Rows of W near 2^-90 and of X near 2^-50 (and far smaller): the adapter's
    term is all that is left of them, whichever way it is added."""
    r, s = 16, 2.0
    g = torch.Generator("cuda").manual_seed(M)
    rn = lambda *k: torch.randn(*k, generator=g, device="cuda")
    rows = lambda n, e: torch.exp2(torch.tensor(e, device="cuda").repeat(n // len(e) + 1)[:n, None].float())
    X = (rn(M, K) * rows(M, [-50, 0, -95, 30])).bfloat16()
    w = q.mx_quantize(rn(N, K) * rows(N, [-90, 0, -95, -6, -60]))
    A, B = (rn(r, K) * 0.1).bfloat16(), rn(N, r).bfloat16()
    Y, T = q.mx_linear_fwd(w, X, A, B, s * r)
    assert q.qlora_check_status() == 0
    vx, vw = q.mx_dequantize(q.mx_quantize(X)).double(), q.mx_dequantize(w).double()
    x, a, b = X.double(), A.double(), B.double()
    t, t_mag = x @ a.T, x.abs() @ a.abs().T
    ref, mag = vx @ vw.T + s * t @ b.T, vx.abs() @ vw.abs().T
    assert float(((T.double() - t).abs() - H * t.abs() - (1 + H) * K * U * t_mag - TINY).max()) <= 0
    ad = s * (H * t.abs() + (1 + H) * K * U * t_mag) @ b.abs().T       # T's sum, and s T in bf16
    check(Y, ref, H * ref.abs() + (1 + H) * (ad + (K + r + 3) * U * (mag + (1 + H) * s * t_mag @ b.abs().T)))


@pytest.mark.parametrize("fmt", [mx.MXFP4, mx.NVFP4])
@pytest.mark.parametrize("p", [0.0, 0.25])
@pytest.mark.parametrize("M,N,K", [(1, 136, 256), (20, 136, 4096), (40, 136, 192), (200, 520, 320), (33, 264, 4096), (600, 264, 128)])
def test_zero_rows_of_the_weight(q, fmt, p, M, N, K):
    """Rows of zeros in W, forward and backward: the adapter's term is all of their
    outputs, and they add nothing but it to dX."""
    r, s, seed, bf = 16, 2.0, 11, torch.bfloat16
    g = torch.Generator("cuda").manual_seed(M + K)
    rn = lambda *k: torch.randn(*k, generator=g, device="cuda")
    W = rn(N, K)
    W[8:80] = 0
    X, A, B, dY = rn(M, K).to(bf), (rn(r, K) * 0.1).to(bf), rn(N, r).to(bf), rn(M, N).to(bf)
    X[M // 2] = 0
    w = q.mx_quantize(W, fmt)
    Y, T = q.mx_linear_fwd(w, X, A, B, s * r, p=p, seed=seed)
    dX, dA, dB = q.mx_linear_bwd(w, X, dY, A, B, s * r, p=p, seed=seed, T=T)
    assert q.qlora_check_status() == 0
    vx, vw = q.mx_dequantize(q.mx_quantize(X, fmt)).double(), q.mx_dequantize(w).double()
    assert bool((vw[8:80] == 0).all())
    xd = q.dropout_fwd(X, p, seed).double()
    keep = (q.dropout_fwd(torch.ones_like(X), p, seed) != 0).double() / (1 - p)
    a, b, d = A.double(), B.double(), dY.double()
    t, t_mag = xd @ a.T, xd.abs() @ a.abs().T
    ref, mag = vx @ vw.T + s * t @ b.T, vx.abs() @ vw.abs().T
    ad = s * (H * t.abs() + (1 + H) * K * U * t_mag) @ b.abs().T
    check(Y, ref, H * ref.abs() + (1 + H) * (ad + (K + r + 3) * U * (mag + (1 + H) * s * t_mag @ b.abs().T)))
    assert bool((Y[M // 2] == 0).all())
    u, u_mag = d @ b, d.abs() @ b.abs()
    ue = s * (H * u.abs() + (1 + H) * N * U * u_mag)            # s U: its sum, and its rounding
    ref, mag = d @ vw + keep * s * (u @ a), d.abs() @ vw.abs()
    ad = keep * (ue @ a.abs() + (N + r + 4) * U * (1 + H) * s * (u_mag @ a.abs()))
    twice = H * (d @ vw).abs() if p else 0                      # with dropout dX is rounded twice
    check(dX, ref, H * ref.abs() + (1 + 2 * H) * (ad + twice + (N + 1) * U * mag))
    ref = s * u.T @ xd
    check(dA, ref, H * ref.abs() + (1 + H) * (ue.T @ xd.abs() + M * U * (1 + H) * s * u_mag.T @ xd.abs()))
    ref = s * d.T @ T.double()
    check(dB, ref, H * ref.abs() + (1 + H) * (M + 1) * U * s * d.abs().T @ T.double().abs())
