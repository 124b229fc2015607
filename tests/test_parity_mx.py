"""GPU parity of the microscaled 4-bit operators and the QLoRA layer on them
against the fp64 oracle (oracle.mx).

Quantisation, its scales and dequantised values are compared bit for bit.  The
product of two stored tensors is bounded element by element: with S = sum |x w|
over the contraction, fp32 sums of K exact products in any order, truncating,
err by at most K 2^-23 S, and the result is rounded to bf16 once (2^-8).  The
adapter's rank-r factor is rounded to bf16 (2^-8 of sum |s T B|), and in the
backward s U likewise; with dropout dX is rounded to bf16 twice.
"""

import numpy as np
import pytest
import torch

import oracle
from oracle import dropout as OD
from oracle import mx
from qlora_linear_layers_b200 import synth

pytestmark = pytest.mark.gpu

FMTS = [mx.MXFP4, mx.NVFP4]
H = 2.0 ** -8            # half a bf16 step
U = 2.0 ** -23           # a truncated fp32 step


@pytest.fixture(scope="module")
def q():
    from qlora_linear_layers_b200.build import build
    build()
    import qlora_linear_layers_b200 as q
    return q


def f64(t):
    return t.detach().double().cpu().numpy()


def within(got, ref, bound):
    got = f64(got)
    assert got.shape == ref.shape
    # the bf16 grid below 2^-126 has a fixed step: 2^-134 covers half of it
    worst = np.max(np.abs(got - ref) - bound - 2.0 ** -134)
    assert worst <= 0, f"exceeds its bound by {worst:.3e}"


def check_quantised(q, X, fmt):
    t = q.mx_quantize(X, fmt)
    assert q.qlora_check_status() == 0
    codes, scale, s = mx.quantize(f64(X), fmt)
    want = mx.dequantize(codes, scale, s, fmt)
    assert np.array_equal(t.block_scales().cpu().numpy(), scale)
    assert np.array_equal(t.scales.cpu().numpy(), mx.tile_scales(scale))
    if fmt == mx.NVFP4:
        assert np.array_equal(f64(t.row_scale), s)
    got = mx.unpack(t.packed.cpu().numpy(), *X.shape)
    differ = got != codes                       # a zero may be stored as -0
    assert np.all((got[differ] & 7) == 0) and np.all((codes[differ] & 7) == 0)
    assert np.array_equal(f64(q.mx_dequantize(t)), mx.bf16(want))
    return t


# ---------------------------------------------------------------------------
# Quantisation
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols,pad", [
    (1, 32, 0), (3, 64, 0), (37, 96, 8), (129, 160, 64), (5, 1024, 0), (4, 8192, 0), (3, 8224, 32),
    (2, 18944, 0), (1, 33024, 0), (2, 66016, 0)])
def test_quantise_exact(q, fmt, dtype, rows, cols, pad):
    g = torch.Generator().manual_seed(rows * 1000 + cols)
    X = torch.randn(rows, cols + pad, generator=g) * torch.exp2(torch.randint(-12, 12, (rows, 1), generator=g))
    X = X.to(dtype).cuda()[:, :cols]
    check_quantised(q, X, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quantise_edges(q, fmt, dtype):
    """Midpoints and their neighbours under every significand of the scale,
    zero rows and blocks, -0, the type's largest and smallest values, scales
    that round to zero, rows whose scale is clamped."""
    rows = []
    base = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, -5])
    for m in range(8, 16):                                     # block maxima 6 * m / 8 * 2^k
        for k in (-3, 0, 5):
            b = base * m / 8 * 2.0 ** k
            t = torch.tensor(b, dtype=dtype)
            up = torch.nextafter(t, torch.full_like(t, 1e30))
            down = torch.nextafter(t, torch.full_like(t, -1e30))
            up[14], down[14] = t[14], t[14]                    # the maximum stays
            rows.append(torch.cat([t, up, down, -t]))
    tiny = 2.0 ** -126
    z = torch.zeros(64, dtype=dtype)
    rows += [z, -z]
    for v in (3e38, 1e-30, 1e-36, tiny, 2.0 ** -120, 2.0 ** -100 * 2688, 2688.0, 2690.0):
        a = z.clone()
        a[3], a[17], a[40] = v, -v / 3, v / 4096
        rows.append(a)
    a = z.clone()
    a[0], a[16:32], a[33] = 2688.0, 2.0 ** -12, -(2.0 ** -9)     # blocks whose E4M3 scale underflows
    rows.append(a)
    check_quantised(q, torch.stack(rows).cuda(), fmt)


@pytest.mark.parametrize("k", [0, -40, 90])
def test_midpoints_under_every_block_scale(q, k):
    """The seven midpoints and the floats on both sides of each, under all 126 E4M3 scales."""
    S = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()[:, None]
    t = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]) * S            # exact: 4 and 3 bits
    X = torch.zeros(126, 64)
    X[:, 0] = 2688.0                                                         # the row scale is 2^k
    X[:, 16] = X[:, 32] = X[:, 48] = (6 * S)[:, 0]
    X[:, 17:24] = t
    X[:, 33:40] = torch.nextafter(t, torch.full_like(t, 1e30))
    X[:, 49:56] = -torch.nextafter(t, torch.zeros_like(t))
    codes, scale, s = mx.quantize(X.double().numpy() * 2.0 ** k, mx.NVFP4)
    assert np.all(s == 2.0 ** k) and np.all(scale[:, 1:4] == np.arange(1, 127)[:, None])
    check_quantised(q, (X * 2.0 ** k).cuda(), mx.NVFP4)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(300, 32), (1, 96), (129, 224), (257, 480), (130, 544), (40, 20480), (33, 26624)])
def test_quantise_row_lengths(q, fmt, dtype, rows, cols):
    """Rows that share a CTA, a warp or part of one, and rows longer than a CTA's registers."""
    X = torch.randn(rows, cols, generator=torch.Generator().manual_seed(cols))
    check_quantised(q, (X * torch.logspace(-12, 12, rows)[:, None]).to(dtype).cuda(), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_non_finite_blocks(q, fmt, dtype, bad):
    """A NaN or infinity makes its block NaN, leaves the others as they are
    without it, and is reported."""
    X = torch.randn(4, 128, generator=torch.Generator().manual_seed(1)).to(dtype)
    Y = X.clone()
    b = mx.BLOCK[fmt]
    Y[2, 70 // b * b: 70 // b * b + b] = 0
    X[2, 70] = bad
    t = q.mx_quantize(X.cuda(), fmt)
    assert q.qlora_check_status() == q._lib.QLORA_ERR_NONFINITE
    assert q.qlora_check_status() == 0
    v, ref = f64(q.mx_dequantize(t)), mx.bf16(mx.fake_quantize(f64(Y), fmt))
    nan = np.zeros((4, 128), bool)
    nan[2, 70 // b * b: 70 // b * b + b] = True
    assert np.all(np.isnan(v[nan])) and np.array_equal(v[~nan], ref[~nan])
    w = q.mx_quantize(torch.ones(8, 128, device="cuda"), fmt)
    P = f64(q.mx_matmul(t, w))
    assert np.all(np.isnan(P[2])) and np.all(np.isfinite(P[[0, 1, 3]]))
    assert np.all(np.isnan(f64(q.mx_matmul(w, t))[:, 2]))


def stored(q, rows, cols, fmt, seed, any_scale=False):
    """A stored tensor with random codes and scales, and its fp64 values."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 16, (rows, cols)).astype(np.uint8)
    n = cols // mx.BLOCK[fmt]
    scale = rng.integers(30, 90, (rows, n)) if fmt == mx.NVFP4 else rng.integers(117, 131, (rows, n))
    s = None
    if fmt == mx.NVFP4:
        s = (rng.random(rows) + 0.5 if any_scale else 2.0 ** rng.integers(-8, 3, rows)).astype(np.float32)
    t = q.MXTensor(torch.from_numpy(mx.pack(codes)).cuda(), torch.from_numpy(mx.tile_scales(scale.astype(np.uint8))).cuda(),
                   None if s is None else torch.from_numpy(s).cuda(), rows, cols, fmt)
    return t, mx.dequantize(codes, scale, s, fmt)


def test_dequantise_any_row_scale(q):
    """An arbitrary fp32 row scale: RNbf16(RN32(q S s))."""
    t, v = stored(q, 70, 96, mx.NVFP4, 4, any_scale=True)
    assert np.array_equal(f64(q.mx_dequantize(t)), mx.bf16(v))


# ---------------------------------------------------------------------------
# Product
# ---------------------------------------------------------------------------

def product_bound(x, w):
    # one more fp32 rounding for each row scale
    S = np.abs(x) @ np.abs(w).T
    return H * np.abs(x @ w.T) + (x.shape[1] + 2) * U * S


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [
    (1, 1, 32), (1, 8, 64), (2, 130, 96), (16, 256, 1024), (17, 77, 352), (31, 129, 256), (32, 128, 4096),
    (33, 300, 288), (64, 64, 128), (65, 1000, 544), (128, 256, 2080), (129, 512, 512), (255, 136, 800),
    (300, 1001, 1056), (513, 384, 1984), (1100, 640, 320), (1, 4096, 18944), (40, 200, 8000)])
def test_product(q, fmt, M, N, K):
    x, vx = stored(q, M, K, fmt, M + N)
    w, vw = stored(q, N, K, fmt, M + K, any_scale=True)
    Y = q.mx_matmul(x, w)
    assert q.qlora_check_status() == 0
    within(Y, vx @ vw.T, product_bound(vx, vw))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,r", [(4096, 4096, 512, 8), (4000, 4090, 544, 0), (2040, 2568, 576, 64), (2220, 2560, 256, 0),
                                     (8100, 600, 2048, 128)])
def test_product_in_rounds_of_tiles(q, fmt, M, N, K, r):
    """More tiles than pairs of SMs, the last round in halves or not, on the GPU in fp64."""
    g = torch.Generator("cuda").manual_seed(M)
    x = q.mx_quantize(torch.randn(M, K, generator=g, device="cuda"), fmt)
    w = q.mx_quantize(torch.randn(N, K, generator=g, device="cuda"), fmt)
    vx, vw = q.mx_dequantize(x).double(), q.mx_dequantize(w).double()
    ref, mag = vx @ vw.T, vx.abs() @ vw.abs().T
    err = (q.mx_matmul(x, w).double() - ref).abs()
    assert float((err - H * ref.abs() - (1 + H) * (K + 2) * U * mag).max()) <= 0
    if r:
        X = q.mx_dequantize(x)                     # X quantised again is X
        A, B = (torch.randn(*k, generator=g, device="cuda").bfloat16() for k in ((r, K), (N, r)))
        Y, T = q.mx_linear_fwd(w, X, A, B, float(r))
        t = vx @ A.double().T
        b, ref = B.double().abs(), ref + t @ B.double().T
        t_mag = vx.abs() @ A.double().abs().T      # T: its sum, and its rounding
        ad = (H * t.abs() + (1 + H) * K * U * t_mag) @ b.T
        bound = H * ref.abs() + (1 + H) * (ad + (K + r + 2) * U * (mag + (1 + H) * t_mag @ b.T))
        assert float(((Y.double() - ref).abs() - bound).max()) <= 0
    assert q.qlora_check_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_product_reads_out_the_weight(q, fmt):
    """One-hot rows of x return columns of the stored weight, rounded once (an
    NVFP4 block of a single 1 stores 6 * E4M3(2^11 / 6) * 2^-11 = 1.03125)."""
    K, N = 288, 200
    x = torch.zeros(K, K)
    x[range(K), range(K)] = 1.0
    w, vw = stored(q, N, K, fmt, 9)
    Y = q.mx_matmul(q.mx_quantize(x.cuda(), fmt), w)
    one = 1.03125 if fmt == mx.NVFP4 else 1.0
    assert np.array_equal(f64(Y), mx.bf16(one * vw.T))


@pytest.mark.parametrize("fmt", FMTS)
def test_product_rows_stand_alone(q, fmt):
    """A row's result depends on that row alone: shuffled rows, and NaN scales
    in others, leave it bit for bit."""
    M, N, K = 300, 264, 1120
    X = synth.activations(M, K, 3).cuda()
    w = q.mx_quantize(synth.weight(N, K, 4).cuda(), fmt)
    Y = q.mx_matmul(q.mx_quantize(X, fmt), w)
    perm = torch.randperm(M, generator=torch.Generator().manual_seed(0)).cuda()
    assert torch.equal(q.mx_matmul(q.mx_quantize(X[perm].contiguous(), fmt), w), Y[perm])
    X[5] = float("nan")
    P = q.mx_matmul(q.mx_quantize(X, fmt), w)
    assert q.qlora_check_status() == q._lib.QLORA_ERR_NONFINITE
    keep = torch.arange(M, device="cuda") != 5
    assert torch.equal(P[keep], Y[keep]) and bool(P[5].isnan().all())


def test_rows_past_the_last_are_left(q):
    x, vx = stored(q, 19, 256, mx.NVFP4, 1)
    w, vw = stored(q, 72, 256, mx.NVFP4, 2)
    buf = torch.full((40, 72), 7.0, dtype=torch.bfloat16, device="cuda")
    q.qlora_mx_matmul(x, w, buf[:19])
    assert torch.equal(buf[:19], q.mx_matmul(x, w)) and bool((buf[19:] == 7).all())


# ---------------------------------------------------------------------------
# The layer
# ---------------------------------------------------------------------------

def layer(q, fmt, M, N, K, r, seed):
    W = synth.weight(N, K, seed + 1)
    X = synth.activations(M, K, seed + 2)
    A = synth.activations(r, K, seed + 3, sigma=0.02) if r else None
    B = synth.activations(N, r, seed + 4, sigma=0.02) if r else None
    w = q.mx_quantize(W.cuda(), fmt)
    return X, A, B, w, mx.fake_quantize(f64(W), fmt)


LAYERS = [
    (1, 1024, 1024, 16, 16.0, 0.0), (4, 264, 576, 8, 16.0, 0.1), (16, 512, 1024, 64, 32.0, 0.0),
    (17, 136, 320, 128, 8.0, 0.0), (100, 200, 192, 32, 16.0, 0.05), (257, 384, 640, 16, 32.0, 0.0),
    (300, 1000, 2048, 64, 16.0, 0.3), (300, 104, 64, 0, 0.0, 0.0), (9, 264, 704, 0, 0.0, 0.0),
    (700, 136, 256, 128, 64.0, 0.0)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K,r,alpha,p", LAYERS)
def test_layer_forward_backward(q, fmt, M, N, K, r, alpha, p):
    seed = 100 * M + r
    X, A, B, w, vw = layer(q, fmt, M, N, K, r, seed)
    dY = synth.activations(M, N, seed + 5)
    g = [None if t is None else t.cuda() for t in (X, A, B, dY)]
    Y, T = q.mx_linear_fwd(w, g[0], g[1], g[2], alpha, p=p, seed=seed)
    dX, dA, dB = q.mx_linear_bwd(w, g[0], g[3], g[1], g[2], alpha, p=p, seed=seed, T=T)
    assert q.qlora_check_status() == 0
    x, d = f64(X), f64(dY)
    a, b = (np.zeros((8, K)), np.zeros((N, 8))) if not r else (f64(A), f64(B))
    s = alpha / r if r else 0.0
    mask = OD.keep_mask(M, K, p, seed) if p else np.ones((M, K), bool)
    xd = OD.dropped_input(X.float().numpy(), mask, p).astype(np.float64) if p else x
    c = float(OD.keep_scale(p)) if p else 1.0
    xq = mx.fake_quantize(x, fmt)
    t = xd @ a.T
    ad = np.abs(xd) @ np.abs(a).T
    y = xq @ vw.T + s * (t @ b.T)
    within(Y, y, H * np.abs(y) + product_bound(xq, vw) + 1.01 * H * s * (np.abs(t) @ np.abs(b).T)
           + (K + 130) * U * s * (ad @ np.abs(b).T))
    if r:
        within(T, t, H * np.abs(t) + K * U * ad)
        t = f64(T)                               # the backward reads the saved T
    u, ua = d @ b, np.abs(d) @ np.abs(b)
    dx = d @ vw + np.where(mask, c, 0) * (s * (u @ a))
    terms = np.abs(d) @ np.abs(vw)
    once = H * np.abs(dx) + (2 * H if p else 0) * np.abs(d @ vw) + N * U * terms
    within(dX, dx, once + c * s * (1.01 * H * (np.abs(u) @ np.abs(a)) + (N + 130) * U * (ua @ np.abs(a))))
    if r:
        da = s * (u.T @ xd)
        within(dA, da, H * np.abs(da) + 1.01 * H * s * (np.abs(u).T @ np.abs(xd)) + (N + M) * U * s * (ua.T @ np.abs(xd)))
        db = s * (d.T @ t)
        within(dB, db, H * np.abs(db) + (M + 1) * U * s * (np.abs(d).T @ np.abs(t)))
        # T not passed: recomputed by the call, the same bits
        again = q.mx_linear_bwd(w, g[0], g[3], g[1], g[2], alpha, p=p, seed=seed)
        assert all(torch.equal(i, j) for i, j in zip((dX, dA, dB), again))


@pytest.mark.parametrize("fmt", FMTS)
def test_adapter_gradients_by_differences(q, fmt):
    """The layer is linear in A and in B: central differences of sum(dY * Y)
    equal the gradients up to the bf16 roundings of Y, T and the gradient."""
    M, N, K, r, alpha = 64, 136, 256, 16, 16.0
    X, A, B, w, vw = layer(q, fmt, M, N, K, r, 77)
    B = synth.activations(N, r, 5, sigma=1.0)
    dY = synth.activations(M, N, 6)
    X, A, B, dY = X.cuda(), A.cuda(), B.cuda(), dY.cuda()
    _, dA, dB = q.mx_linear_bwd(w, X, dY, A, B, alpha)
    s = alpha / r

    def both(A, B):
        Y, _ = q.mx_linear_fwd(w, X, A, B, alpha)
        y, d = f64(Y), f64(dY)
        # what the roundings of Y and of s T can move the sum by
        t = np.abs(f64(X) @ f64(A).T) * s
        slack = H * np.sum(np.abs(d) * np.abs(y)) + 1.01 * H * np.sum(np.abs(d) * (t @ np.abs(f64(B)).T))
        return np.sum(d * y), slack

    for name, grad in (("A", dA), ("B", dB)):
        D = torch.ones_like(grad) * torch.sign(grad)           # +-1: the sum moves by sum |grad|
        hi = both(A + D, B) if name == "A" else both(A, B + D)
        lo = both(A - D, B) if name == "A" else both(A, B - D)
        plus = (A + D, A - D) if name == "A" else (B + D, B - D)
        step = f64(plus[0]) - f64(plus[1])                     # the step actually taken, in bf16
        want = np.sum(step * f64(grad))
        slack = hi[1] + lo[1] + 2 * H * np.sum(np.abs(step) * np.abs(f64(grad)))
        assert slack < 0.25 * abs(want)
        assert abs(hi[0] - lo[0] - want) <= slack


def test_streams_and_workspace_contents(q):
    """On a stream that is not the current one, and with a workspace full of
    NaN bytes, the results are the same bits."""
    for fmt in FMTS:
        X, A, B, w, _ = layer(q, fmt, 150, 264, 448, 16, 5)
        X, A, B = X.cuda(), A.cuda(), B.cuda()
        dY = synth.activations(150, 264, 8).cuda()
        Y, T = q.mx_linear_fwd(w, X, A, B, 16.0, p=0.1, seed=3)
        G = q.mx_linear_bwd(w, X, dY, A, B, 16.0, p=0.1, seed=3, T=T)
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        Y2, T2 = q.mx_linear_fwd(w, X, A, B, 16.0, p=0.1, seed=3, stream=st)
        G2 = q.mx_linear_bwd(w, X, dY, A, B, 16.0, p=0.1, seed=3, T=T2, stream=st)
        st.synchronize()
        assert torch.equal(Y, Y2) and torch.equal(T, T2) and all(torch.equal(a, b) for a, b in zip(G, G2))
        n = q.workspace_bytes(q._lib.QLORA_OP_MX_FWD_DROPOUT, 150, 264, 448, 16)
        ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        Y3, T3 = torch.empty_like(Y), torch.empty_like(T)
        q.qlora_mx_linear_fwd(w, X, A, B, 16.0, Y3, T3, 0.1, 3, ws=ws)
        assert torch.equal(Y, Y3) and torch.equal(T, T3)


@pytest.mark.parametrize("M", [3, 200])
def test_graph_capture_and_replay(q, M):
    """Two captured graphs that share one workspace, replayed in turn on new
    inputs, give the eager results."""
    X, A, B, w, _ = layer(q, mx.NVFP4, M, 264, 448, 16, 5)
    X, A, B = X.cuda(), A.cuda(), B.cuda()
    n = q.workspace_bytes(q._lib.QLORA_OP_MX_FWD, M, 264, 448, 16)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    xs = [X.clone(), X.clone()]
    ys = [torch.empty(M, 264, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    q.qlora_mx_linear_fwd(w, xs[0], A, B, 16.0, ys[0], ws=ws)
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            q.qlora_mx_linear_fwd(w, xs[i], A, B, 16.0, ys[i], ws=ws)
        graphs.append(g)
    for rep in range(3):
        for i in (1, 0):
            xs[i].copy_(X * (rep + 1) + i)
            graphs[i].replay()
        for i in (0, 1):
            assert torch.equal(ys[i], q.mx_linear_fwd(w, xs[i], A, B, 16.0)[0])
    assert q.qlora_check_status() == 0


@pytest.mark.parametrize("fmt", FMTS)
def test_a_block_as_it_is_used(q, fmt):
    """Quantise a weight, run a training step (layer, dropout with residual,
    both backwards) and one-token serving of the same layer."""
    M, D, r, alpha, p, seed = 130, 320, 16, 32.0, 0.2, 99
    X, A, B, w, vw = layer(q, fmt, M, D, D, r, 50)
    Xc, Ac, Bc = X.cuda(), A.cuda(), B.cuda()
    Y, T = q.mx_linear_fwd(w, Xc, Ac, Bc, alpha, p=p, seed=seed)
    Z = q.dropout_fwd(Y, p, seed + 1, residual=Xc)
    dZ = synth.activations(M, D, 60).cuda()
    dY = q.dropout_bwd(dZ, p, seed + 1)
    dX, dA, dB = q.mx_linear_bwd(w, Xc, dY, Ac, Bc, alpha, p=p, seed=seed, T=T)
    dX = dX + dZ
    assert q.qlora_check_status() == 0
    x, a, b = f64(X), f64(A), f64(B)
    m0, m1 = OD.keep_mask(M, D, p, seed), OD.keep_mask(M, D, p, seed + 1)
    xd = OD.dropped_input(X.float().numpy(), m0, p)
    c = float(OD.keep_scale(p))
    y, t = mx.linear_fwd(x, vw, a, b, alpha, r, fmt, Xd=xd)
    z = np.where(m1, c * f64(Y), 0) + x
    within(Z, z, H * np.abs(z) + 3 * U * (np.abs(f64(Y)) * c + np.abs(x)))
    dy = np.where(m1, c * f64(dZ), 0)
    within(dY, dy, 1.01 * H * np.abs(dy))
    gx, ga, gb = OD.linear_bwd_dropout(x, f64(dY), vw, a, b, alpha, r, m0, p)
    for got, ref in ((Y, y), (dX, gx + f64(dZ)), (dA, ga), (dB, gb)):
        # four bf16 roundings at most lie between these and the formula
        assert np.max(np.abs(f64(got) - ref)) <= 4 * H * np.max(np.abs(ref))
    one, _ = q.mx_linear_fwd(w, Xc[7:8].contiguous(), Ac, Bc, alpha)
    y1, _ = mx.linear_fwd(x[7:8], vw, a, b, alpha, r, fmt)
    assert np.max(np.abs(f64(one) - y1)) <= 2 * H * np.max(np.abs(y1))


def test_python_checks(q):
    x = q.mx_quantize(torch.randn(4, 64, device="cuda"))
    w = q.mx_quantize(torch.randn(8, 64, device="cuda"))
    with pytest.raises(q.QLoraError):
        q.mx_quantize(torch.randn(4, 80, device="cuda"))
    with pytest.raises(q.QLoraError):
        q.mx_matmul(x, q.mx_quantize(torch.randn(8, 64, device="cuda"), mx.MXFP4))
    with pytest.raises(ValueError):
        q.mx_quantize(torch.randn(64, 4, device="cuda").t())
    with pytest.raises(ValueError):
        q.mx_quantize(torch.randn(4, 64, device="cuda").half())
    with pytest.raises(ValueError):
        q.qlora_mx_matmul(x, w, torch.empty(4, 9, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError):
        q.mx_matmul(q.MXTensor(x.packed, x.scales, None, 4, 64, 1), w)
    X = torch.randn(4, 64, device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        q.mx_linear_fwd(w, X.float())
    with pytest.raises(ValueError):
        q.mx_linear_fwd(w, X, torch.zeros(8, 64, device="cuda", dtype=torch.bfloat16),
                        torch.zeros(9, 8, device="cuda", dtype=torch.bfloat16), 1.0)
    with pytest.raises(q.QLoraError):
        q.mx_linear_fwd(w, X, p=0.5)                          # dropout needs an adapter
    assert q.qlora_check_status() == 0


# ---------------------------------------------------------------------------
# Calls that the documentation allows at its edges
# ---------------------------------------------------------------------------

def layer_bounds(x, vx, vw, a, b, s, K):
    """(Y in fp64, its bound) as in test_layer_forward_backward, no dropout."""
    t = x @ a.T
    y = vx @ vw.T + s * (t @ b.T)
    ad = np.abs(x) @ np.abs(a).T
    return y, (H * np.abs(y) + product_bound(vx, vw) + 1.01 * H * s * (np.abs(t) @ np.abs(b).T)
               + (K + 130) * U * s * (ad @ np.abs(b).T))


@pytest.mark.parametrize("M,N,K,r", [(5, 136, 192, 16), (40, 136, 192, 64), (200, 520, 320, 32), (1500, 40, 64, 8)])
def test_layer_any_row_scale(q, M, N, K, r):
    """A weight whose row scales are no powers of two (a tensor scale repeated,
    say): the adapter's factor B / s may be rounded once more, deq(W) too."""
    rng = np.random.default_rng(M)
    w, vw = stored(q, N, K, mx.NVFP4, M, any_scale=True)
    X, A = synth.activations(M, K, 1), synth.activations(r, K, 2, sigma=0.1)
    B, dY = synth.activations(N, r, 3), synth.activations(M, N, 4)
    Y, T = q.mx_linear_fwd(w, X.cuda(), A.cuda(), B.cuda(), 16.0)
    dX, dA, dB = q.mx_linear_bwd(w, X.cuda(), dY.cuda(), A.cuda(), B.cuda(), 16.0, T=T)
    assert q.qlora_check_status() == 0
    x, a, b, d, s = f64(X), f64(A), f64(B), f64(dY), 16.0 / r
    y, bound = layer_bounds(x, mx.fake_quantize(x, mx.NVFP4), vw, a, b, s, K)
    within(Y, y, bound + 1.02 * H * s * (np.abs(x @ a.T) @ np.abs(b).T))
    wb = mx.bf16(vw)                                    # what the backward multiplies by
    u, ua = d @ b, np.abs(d) @ np.abs(b)
    dx = d @ wb + s * (u @ a)
    within(dX, dx, H * np.abs(dx) + N * U * (np.abs(d) @ np.abs(wb)) + s * (1.01 * H * (np.abs(u) @ np.abs(a))
           + (N + 130) * U * (ua @ np.abs(a))))


@pytest.mark.parametrize("fmt", FMTS)
def test_wide_tokens(q, fmt):
    """A contraction past what one pass of the token kernel holds in registers."""
    M, N, K, r = 3, 72, 24640, 8
    X, A, B, w, vw = layer(q, fmt, M, N, K, r, 9)
    Y, T = q.mx_linear_fwd(w, X.cuda(), A.cuda(), B.cuda(), 16.0)
    x = f64(X)
    y, bound = layer_bounds(x, mx.fake_quantize(x, fmt), vw, f64(A), f64(B), 2.0, K)
    within(Y, y, bound)
    t = x @ f64(A).T
    within(T, t, H * np.abs(t) + K * U * (np.abs(x) @ np.abs(f64(A)).T))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M", [1, 30, 60, 300])
def test_zero_and_nan_tokens_stay_in_their_rows(q, fmt, M):
    """A zero token gives zeros, a NaN token NaNs, and neither touches the rest."""
    N, K, r = 264, 576, 16
    X, A, B, w, _ = layer(q, fmt, M + 2, N, K, r, 21)
    X, A, B = X.cuda(), A.cuda(), B.cuda()
    Y, T = q.mx_linear_fwd(w, X, A, B, 16.0)
    Z = X.clone()
    Z[M // 2], Z[M] = 0, float("nan")
    P, S = q.mx_linear_fwd(w, Z, A, B, 16.0)
    assert q.qlora_check_status() == q._lib.QLORA_ERR_NONFINITE
    keep = torch.ones(M + 2, dtype=torch.bool, device="cuda")
    keep[M // 2] = keep[M] = False
    assert torch.equal(P[keep], Y[keep]) and torch.equal(S[keep], T[keep])
    assert bool((P[M // 2] == 0).all()) and bool((S[M // 2] == 0).all())
    assert bool(P[M].isnan().all()) and bool(S[M].isnan().all())


@pytest.mark.parametrize("fmt", FMTS)
def test_zero_weight_rows(q, fmt):
    """Rows of zeros in W leave the adapter's term alone, forward and backward."""
    M, N, K, r = 20, 136, 256, 16
    W = synth.weight(N, K, 1)
    W[8:80] = 0
    X, A, B = synth.activations(M, K, 2), synth.activations(r, K, 3, sigma=0.02), synth.activations(N, r, 4)
    w = q.mx_quantize(W.cuda(), fmt)
    for m in (M, 1):
        Y, T = q.mx_linear_fwd(w, X[:m].cuda(), A.cuda(), B.cuda(), 16.0)
        y = f64(X[:m]) @ f64(A).T @ f64(B).T
        bound = 4 * H * (np.abs(f64(X[:m]) @ f64(A).T) @ np.abs(f64(B)).T)
        got = f64(Y)[:, 8:80]
        assert np.all(np.abs(got - y[:, 8:80]) <= bound[:, 8:80])


def test_the_same_bits_every_time(q):
    """Split contractions add in a fixed order: ten runs, one result."""
    for M, N, K, r in ((1, 264, 4096, 16), (24, 520, 2048, 8), (100, 136, 8192, 64), (300, 1024, 512, 16)):
        X, A, B, w, _ = layer(q, mx.NVFP4, M, N, K, r, 5)
        X, A, B, dY = X.cuda(), A.cuda(), B.cuda(), synth.activations(M, N, 6).cuda()
        first = None
        for _ in range(10):
            Y, T = q.mx_linear_fwd(w, X, A, B, 16.0, p=0.0)
            out = (Y, T) + q.mx_linear_bwd(w, X, dY, A, B, 16.0, T=T)
            if first is None:
                first = out
            assert all(torch.equal(a, b) for a, b in zip(first, out))


def test_two_streams_at_once(q):
    """Calls that overlap on two streams, each with its own buffers."""
    parts = []
    for i, (M, fmt) in enumerate(((20, mx.NVFP4), (20, mx.MXFP4), (700, mx.NVFP4), (150, mx.MXFP4))):
        X, A, B, w, _ = layer(q, fmt, M, 520, 1024, 16, 30 + i)
        X, A, B, dY = X.cuda(), A.cuda(), B.cuda(), synth.activations(M, 520, i).cuda()
        Y, T = q.mx_linear_fwd(w, X, A, B, 16.0, p=0.1, seed=i)
        want = (Y, T) + q.mx_linear_bwd(w, X, dY, A, B, 16.0, p=0.1, seed=i, T=T)
        parts.append((X, A, B, dY, w, want))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in parts]
    got = []
    for rep in range(3):
        for i, (X, A, B, dY, w, want) in enumerate(parts):
            Y, T = q.mx_linear_fwd(w, X, A, B, 16.0, p=0.1, seed=i, stream=streams[i])
            got.append((i, (Y, T) + q.mx_linear_bwd(w, X, dY, A, B, 16.0, p=0.1, seed=i, T=T, stream=streams[i])))
    torch.cuda.synchronize()
    for i, out in got:
        assert all(torch.equal(a, b) for a, b in zip(parts[i][5], out))
    assert q.qlora_check_status() == 0


@pytest.mark.parametrize("M", [20, 200])
def test_backward_in_a_graph(q, M):
    """The backward captured and replayed on new gradients."""
    X, A, B, w, _ = layer(q, mx.MXFP4, M, 264, 448, 16, 5)
    X, A, B = X.cuda(), A.cuda(), B.cuda()
    dY = synth.activations(M, 264, 1).cuda()
    out = [torch.empty_like(t) for t in (X, A, B)]
    n = q.workspace_bytes(q._lib.QLORA_OP_MX_BWD_DROPOUT, M, 264, 448, 16)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    q.qlora_mx_linear_bwd(w, X, dY, A, B, 16.0, *out, p=0.2, seed=4, ws=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qlora_mx_linear_bwd(w, X, dY, A, B, 16.0, *out, p=0.2, seed=4, ws=ws)
    for i in range(3):
        dY.copy_(synth.activations(M, 264, 10 + i))
        g.replay()
        want = q.mx_linear_bwd(w, X, dY, A, B, 16.0, p=0.2, seed=4)
        assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("M,N,K", [(16, 4096, 4096), (70, 1024, 4096), (130, 2048, 1024), (600, 1024, 2048),
                                   (2100, 512, 1024), (33, 264, 8192), (1111, 320, 2432), (777, 2048, 3520),
                                   (250, 4096, 4032)])
def test_larger_layers_by_their_norm(q, fmt, M, N, K):
    """Sizes that reach every kernel of the layer, against fp64 products on the
    GPU of the tensors' own dequantised values: the bf16 roundings are
    independent, so the error's norm is below half a step of the result's."""
    r, s = 16, 1.0
    X, A, B, w, _ = layer(q, fmt, M, N, K, r, M + K)
    X, A, B, dY = X.cuda(), A.cuda(), B.cuda(), synth.activations(M, N, 9).cuda()
    Y, T = q.mx_linear_fwd(w, X, A, B, 16.0)
    dX, dA, dB = q.mx_linear_bwd(w, X, dY, A, B, 16.0, T=T)
    vw, vx = q.mx_dequantize(w).double(), q.mx_dequantize(q.mx_quantize(X, fmt)).double()
    x, a, b, d = X.double(), A.double(), B.double(), dY.double()
    u = d @ b
    for got, ref in ((Y, vx @ vw.T + s * (x @ a.T) @ b.T), (T, x @ a.T), (dX, d @ vw + s * u @ a),
                     (dA, s * u.T @ x), (dB, s * d.T @ T.double())):
        assert float((got.double() - ref).norm()) <= H * float(ref.norm())
    assert q.qlora_check_status() == 0


@pytest.mark.slow
@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_past_32_bits(q, fmt):
    """More than 2^32 elements quantised and dequantised, more than 2^31 outputs
    of a product: the last rows equal the same rows on their own."""
    rows, K = 66000, 65536
    g = torch.Generator(device="cuda").manual_seed(1)
    X = torch.empty(rows, K, dtype=torch.bfloat16, device="cuda")
    X.zero_()
    X[-256:] = torch.randn(256, K, generator=g, device="cuda")
    t = q.mx_quantize(X, fmt)
    tail = q.mx_quantize(X[-256:].contiguous(), fmt)
    assert torch.equal(t.packed.view(rows, -1)[-256:], tail.packed.view(256, -1))
    assert torch.equal(q.mx_dequantize(t)[-256:], q.mx_dequantize(tail))
    del X
    one = q.mx_quantize(torch.randn(3, K, generator=g, device="cuda"), fmt)
    assert torch.equal(q.mx_matmul(t, one)[-256:], q.mx_matmul(tail, one))
    del t
    w = q.mx_quantize(torch.randn(60000, 64, generator=g, device="cuda"), fmt)
    x = torch.randn(40000, 64, generator=g, device="cuda")
    Y = q.mx_matmul(q.mx_quantize(x, fmt), w)
    assert torch.equal(Y[-200:], q.mx_matmul(q.mx_quantize(x[-200:].contiguous(), fmt), w))


@pytest.mark.parametrize("fmt", FMTS)
def test_more_tiles_of_tokens_than_65535(q, fmt):
    """The last rows of 65536 tiles of tokens and a piece, against fp64 products of them alone."""
    M, N, K, r, s, p, seed, n = 65536 * 128 + 5, 8, 64, 8, 2.0, 0.25, 7, 300
    bf, g = torch.bfloat16, torch.Generator("cuda").manual_seed(1)
    X, dY = (torch.randn(M, k, generator=g, device="cuda", dtype=bf) for k in (K, N))
    A, B = (torch.randn(*k, generator=g, device="cuda", dtype=bf) * 0.1 for k in ((r, K), (N, r)))
    w = q.mx_quantize(torch.randn(N, K, generator=g, device="cuda", dtype=bf), fmt)
    Y, T = q.mx_linear_fwd(w, X, A, B, s * r, p=p, seed=seed)
    dX, dA, dB = q.mx_linear_bwd(w, X, dY, A, B, s * r, p=p, seed=seed, T=T)
    Y0 = q.mx_matmul(q.mx_quantize(X, fmt), w)
    x, d = X[-n:], dY[-n:].double()
    xd = q.dropout_fwd(x, p, seed, first=(M - n) * K).double()
    keep = q.dropout_fwd(torch.ones_like(x), p, seed, first=(M - n) * K) != 0
    vw, vx, a, b = q.mx_dequantize(w).double(), q.mx_dequantize(q.mx_quantize(x, fmt)).double(), A.double(), B.double()
    t, u = xd @ a.T, d @ b
    for got, ref, halves in ((Y0, vx @ vw.T, 1), (Y, vx @ vw.T + s * t @ b.T, 1), (T, t, 1),
                             (dX, d @ vw + keep * (s / (1 - p)) * (u @ a), 2)):   # dX is rounded twice
        assert float((got[-n:].double() - ref).norm()) <= halves * H * float(ref.norm())
    assert torch.isfinite(dA.double()).all() and torch.isfinite(dB.double()).all()
    assert q.qlora_check_status() == 0
