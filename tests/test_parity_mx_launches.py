"""GPU tests of the microscaled layer's chained launches, whose kernels start while
the one before still runs."""

import pytest
import torch

from qlora_linear_layers_b200 import synth

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def q():
    from qlora_linear_layers_b200.build import build
    build()
    import qlora_linear_layers_b200 as q
    return q


def layer(q, M, N, K, r, fmt):
    X, dY = synth.activations(M, K, 1).cuda(), synth.activations(M, N, 2).cuda()
    A, B = synth.activations(r, K, 3, sigma=0.02).cuda(), synth.activations(N, r, 4, sigma=0.02).cuda()
    return q.mx_quantize(synth.weight(N, K, 5).cuda(), fmt), X, dY, A, B


@pytest.mark.parametrize("p", [0.0, 0.1])
@pytest.mark.parametrize("M,N,K,r", [(16, 8192, 1024, 16), (200, 4096, 512, 128), (1000, 4096, 2048, 64), (2000, 2048, 2048, 16)])
def test_waits_count_the_work_alone(q, M, N, K, r, p):
    """At the shortest limit of a bounded wait, two streams busy at once: no wait of a
    kernel that started early counts the time of the one before it."""
    w, X, dY, A, B = layer(q, M, N, K, r, 1)
    run = lambda s=None: q.mx_linear_bwd(w, X, dY, A, B, 16.0, p=p, seed=3, stream=s)
    want = run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    lib = q._lib.load()
    assert lib.qlora_set_wait_limit(1_000_000) == 0
    try:
        got = [run(s) for _ in range(5) for s in streams]
        torch.cuda.synchronize()
    finally:
        assert lib.qlora_set_wait_limit(0) == 0
    assert q.qlora_check_status() == 0
    assert all(torch.equal(a, b) for out in got for a, b in zip(want, out))
