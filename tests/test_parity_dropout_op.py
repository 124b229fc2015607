"""GPU parity of the standalone dropout (forward, with a residual, backward)
against the oracle's mask and scaling: bit for bit without a residual, and one
fp32 and one output rounding with it."""

import numpy as np
import pytest
import torch

from oracle import dropout as OD
from qlora_linear_layers_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    from qlora_linear_layers_b200.build import build
    build()
    import qlora_linear_layers_b200 as q
    return q


def make(M, K, dtype, seed):
    return torch.randn(M, K, generator=torch.Generator().manual_seed(seed)).to(dtype)


def expected(X, mask, p, residual=None):
    """RN(RN32(D c X) + R) with the roundings made by NumPy and torch."""
    v = np.where(mask, X.float().numpy() * OD.keep_scale(p), np.float32(0)).astype(np.float32)
    if residual is not None:
        v = v + residual.float().numpy()
    return torch.from_numpy(v).to(X.dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K,p,seed", [
    (1, 1, 0.5, 3), (1, 7, 0.5, 3), (3, 8, 0.1, 2 ** 64 - 1), (5, 9, 0.9, 1), (33, 55, 0.25, 7), (16, 64, 0.05, 11),
    (130, 257, 0.3, 5), (7, 1024, 0.1, 6), (2, 4100, 0.5, 8)])
def test_forward_and_backward(q, dtype, M, K, p, seed):
    X, R = make(M, K, dtype, 1), make(M, K, dtype, 2)
    mask = OD.keep_mask(M, K, p, seed)
    assert torch.equal(q.dropout_fwd(X.cuda(), p, seed).cpu(), expected(X, mask, p))
    assert torch.equal(q.dropout_bwd(R.cuda(), p, seed).cpu(), expected(R, mask, p))
    assert torch.equal(q.dropout_fwd(X.cuda(), p, seed, residual=R.cuda()).cpu(), expected(X, mask, p, R))
    assert q.qlora_check_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_apart_and_in_place(q, dtype):
    """Slices of wider buffers, aligned and not in their width; the output
    written over an input."""
    p, seed = 0.3, 12
    for M, K, wide in ((20, 48, 64), (20, 45, 64), (20, 48, 61 if dtype == torch.bfloat16 else 53)):
        X, R = make(M, wide, dtype, 1), make(M, wide + 8, dtype, 2)
        want = expected(X[:, :K], OD.keep_mask(M, K, p, seed), p, R[:, :K])
        x, r = X.cuda(), R.cuda()
        assert torch.equal(q.dropout_fwd(x[:, :K], p, seed, residual=r[:, :K]).cpu(), want)
        q.qlora_dropout_fwd(x[:, :K], p, seed, x[:, :K], r[:, :K])
        assert torch.equal(x[:, :K].cpu(), want)
        assert torch.equal(x[:, K:].cpu(), X[:, K:])            # what lies beside is left


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [40, 37])
def test_parts_get_the_whole_mask(q, dtype, K):
    X = make(24, K, dtype, 1).cuda()
    whole = q.dropout_fwd(X, 0.4, 5)
    for cut in (1, 8, 13):
        # a part starts on a 16-byte boundary of its own: copies
        top, rest = X[:cut].clone(), X[cut:].clone()
        parts = [q.dropout_fwd(top, 0.4, 5), q.dropout_fwd(rest, 0.4, 5, first=cut * K)]
        assert torch.equal(torch.cat(parts), whole)


def test_far_element_numbers(q):
    """Numbers past 32 bits reach the generator whole."""
    first = (1 << 40) + 3
    X = torch.ones(1, 21)
    thr = OD.keep_threshold(0.5)
    want = []
    for e in range(first, first + 21):
        w = OD.philox4x64_10((e // 8, 0, 0, 0), (9, 0))
        want.append(((w[e % 8 // 2] >> (16 if e % 2 else 40)) & 0xFFFFFF) >= thr)
    got = q.dropout_fwd(X.cuda(), 0.5, 9, first=first).cpu()
    assert torch.equal(got[0] != 0, torch.tensor(want))


def test_dropped_values_are_zero_whatever_they_hold(q):
    X = torch.full((4, 64), float("nan"))
    mask = torch.from_numpy(OD.keep_mask(4, 64, 0.5, 2))
    Y = q.dropout_fwd(X.cuda(), 0.5, 2).cpu()
    assert torch.equal(Y.isnan(), mask) and bool((Y[~mask] == 0).all())


def test_no_dropout_is_the_identity(q):
    X, R = make(5, 33, torch.bfloat16, 1).cuda(), make(5, 33, torch.bfloat16, 2).cuda()
    assert torch.equal(q.dropout_fwd(X, 0.0, 1), X)
    assert torch.equal(q.dropout_fwd(X, 0.0, 1, residual=R), X + R)


def test_it_is_the_layers_adapter_input(q):
    """T of the layer with dropout is T of the plain layer on dropout(X)."""
    M, N, K, r = 40, 64, 256, 16
    w = q.quantize(synth.weight(N, K, 1).cuda())
    X, A = synth.activations(M, K, 2).cuda(), synth.activations(r, K, 3, sigma=0.02).cuda()
    B = synth.activations(N, r, 4).cuda()
    _, T = q.linear_fwd_dropout(w, X, A, B, 16.0, 0.2, 77)
    _, T2 = q.linear_fwd_dropout(w, q.dropout_fwd(X, 0.2, 77), A, B, 16.0, 0.0, 0)
    assert torch.equal(T, T2)


@pytest.mark.slow
def test_offsets_past_32_bits(q):
    """More than 2^32 elements: the last rows equal the same rows with their number."""
    M, K = 66000, 65544
    X = torch.ones(M, K, dtype=torch.bfloat16, device="cuda")
    Y = q.dropout_fwd(X, 0.5, 3)
    assert torch.equal(Y[-9:], q.dropout_fwd(X[-9:].contiguous(), 0.5, 3, first=(M - 9) * K))
    assert not torch.equal(Y[-9:], Y[:9])


def test_captured_and_replayed(q):
    X = make(40, 96, torch.bfloat16, 1).cuda()
    Y = torch.empty_like(X)
    q.qlora_dropout_fwd(X, 0.3, 8, Y)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q.qlora_dropout_fwd(X, 0.3, 8, Y)
    X.mul_(3)
    g.replay()
    assert torch.equal(Y, q.dropout_fwd(X, 0.3, 8))


def test_python_checks(q):
    X = make(4, 8, torch.bfloat16, 1).cuda()
    for bad in (X.t(), X.half(), X[0]):
        with pytest.raises(ValueError):
            q.dropout_fwd(bad, 0.1, 1)
    with pytest.raises(ValueError):
        q.dropout_fwd(X, 0.1, 1, residual=X.float())
    with pytest.raises(ValueError):
        q.dropout_fwd(X, 0.1, 1, residual=X[:2])
    for p in (1.0, -0.1, float("nan")):
        with pytest.raises(q.QLoraError):
            q.dropout_fwd(X, p, 1)
    with pytest.raises(q.QLoraError):
        q.dropout_bwd(X, 0.1, 1, first=-1)
    assert q.qlora_check_status() == 0
