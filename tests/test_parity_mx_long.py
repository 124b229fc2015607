"""GPU parity of the microscaled layer's adapter products over long contractions.

The tensor core truncates the sum that it adds to, so terms of one sign are
where a long chain of additions shows.  All inputs are positive and U = dY B and
s U are exact in bf16, so that what is left of an error is the sum's and the
result's own rounding to bf16.  The roundings of n results are independent and
uniform (the results' significands are spread by the columns of X and rows of A):
their relative errors are at most H, of mean 0 and standard deviation H / sqrt(3),
so that the mean's is H / sqrt(3 n); five of these, and 2^-12 for the sum.
"""

import pytest
import torch

pytestmark = pytest.mark.gpu

H = 2.0 ** -8            # half a bf16 step


@pytest.fixture(scope="module")
def q():
    from qlora_linear_layers_b200.build import build
    build()
    import qlora_linear_layers_b200 as q
    return q


def check(got, ref):
    rel = (got.double() - ref) / ref
    assert float(rel.abs().max()) <= H + 2.0 ** -12
    assert abs(float(rel.mean())) <= 5 * H / (3 * ref.numel()) ** 0.5 + 2.0 ** -12


def spread(n, lo=1.0):
    """Distinct factors in [lo, 2 lo)."""
    return lo * torch.exp2(torch.arange(n, device="cuda") / n)


@pytest.mark.parametrize("M,N,r", [(65536 * 128 + 5, 64, 8), (8 * 512 * 64 + 1, 72, 128), (8 * 1024 * 64 + 70, 16, 16),
                                   (2 * 512 * 64 * 8, 64, 64)])
def test_gradients_over_many_tokens(q, M, N, r):
    """dA and dB: a contraction over the tokens, one run of each rank to many."""
    K, s, bf = 128, 2.0, torch.bfloat16
    g = torch.Generator("cuda").manual_seed(M)
    X = (torch.rand(M, K, generator=g, device="cuda").add_(0.5).mul_(spread(K))).to(bf)
    A = (torch.rand(r, K, generator=g, device="cuda") * spread(r, 2.0 ** -8)[:, None]).to(bf)
    B = torch.zeros(N, r, dtype=bf, device="cuda")
    B[torch.arange(r, device="cuda") % N, torch.arange(r, device="cuda")] = 1.0        # U: columns of dY
    dY = torch.randint(1, 128, (M, N), generator=g, device="cuda").to(bf)
    w = q.mx_quantize(torch.ones(N, K, dtype=bf, device="cuda"))
    T = torch.empty(M, r, dtype=bf, device="cuda")
    q.qlora_mx_linear_fwd(w, X, A, B, s * r, torch.empty(M, N, dtype=bf, device="cuda"), T)
    dX, dA, dB = q.mx_linear_bwd(w, X, dY, A, B, s * r, T=T)
    assert q.qlora_check_status() == 0
    rA, rB = (torch.zeros(*n, dtype=torch.float64, device="cuda") for n in ((r, K), (N, r)))
    for c in range(0, M, 1 << 17):
        d, x, t = (v[c:c + (1 << 17)].double() for v in (dY, X, T))
        rA += s * (d @ B.double()).T @ x
        rB += s * d.T @ t
    check(dA, rA)
    check(dB, rB)


@pytest.mark.parametrize("L", [8 * 512 * 64 + 64, 1 << 22])
def test_down_projections_of_wide_matrices(q, L):
    """T = X A^T over L columns, and U = dY B over L rows of W."""
    M, r, bf = 5, 16, torch.bfloat16
    g = torch.Generator("cuda").manual_seed(L)
    rnd = lambda *n: torch.rand(*n, generator=g, device="cuda").add_(0.5)
    X, A = (rnd(M, L) * spread(M)[:, None]).to(bf), (rnd(r, L) * spread(r)[:, None]).to(bf)
    w = q.mx_quantize(torch.ones(8, L, dtype=bf, device="cuda"))
    # more than 64 tokens: T by itself, not beside their quantisation
    Xm = X.repeat(14, 1)
    T = q.mx_linear_fwd(w, Xm, A, torch.zeros(8, r, dtype=bf, device="cuda"), 1.0)[1]
    check(T[:M], X.double() @ A.double().T)
    assert torch.equal(T, T[:M].repeat(14, 1))
    # dX = dY deq(W) + s U A with W = 0 and A = e_j e_j^T: U, rounded to bf16 once
    w = q.mx_quantize(torch.zeros(L, 64, dtype=bf, device="cuda"))
    E = torch.eye(r, 64, dtype=bf, device="cuda")
    dY, B = X, A.t().contiguous()
    dX = q.mx_linear_bwd(w, torch.zeros(M, 64, dtype=bf, device="cuda"), dY, E, B, float(r))[0]
    check(dX[:, :r], X.double() @ A.double().T)
    assert bool((dX[:, r:] == 0).all())
    assert q.qlora_check_status() == 0
