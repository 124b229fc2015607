"""The workspace that a caller of the microscaled layer passes: refused where the
kernels could not write to it, counted in bytes whatever its type."""

import pytest
import torch

import qlora_linear_layers_b200 as q


def test_checks():
    host = torch.empty(64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="ws"):
        q._scratch(host, 0)                                       # a host tensor for a call on a GPU
    with pytest.raises(ValueError, match="ws"):
        q._scratch(host[::2], -1)                                 # gaps that the kernels would write to
    assert q._scratch(host, -1) == (host.data_ptr(), 64)
    assert q._scratch(torch.empty(16, dtype=torch.float32), -1)[1] == 64


@pytest.mark.gpu
def test_layer_refuses_and_takes():
    M, N, K, r = 20, 64, 128, 8
    bf = torch.bfloat16
    g = torch.Generator("cuda").manual_seed(1)
    X, A, B, dY = (torch.randn(*n, generator=g, device="cuda", dtype=bf) for n in ((M, K), (r, K), (N, r), (M, N)))
    w = q.mx_quantize(torch.randn(N, K, generator=g, device="cuda"))
    want, dwant = q.mx_linear_fwd(w, X, A, B, 16.0), q.mx_linear_bwd(w, X, dY, A, B, 16.0)
    out, grads = [torch.empty_like(t) for t in want], [torch.empty_like(t) for t in dwant]
    n = max(q.workspace_bytes(op, M, N, K, r) for op in (q._lib.QLORA_OP_MX_FWD, q._lib.QLORA_OP_MX_BWD))
    fwd = lambda ws: q.qlora_mx_linear_fwd(w, X, A, B, 16.0, *out, ws=ws)
    bwd = lambda ws: q.qlora_mx_linear_bwd(w, X, dY, A, B, 16.0, *grads, ws=ws)
    for call in (fwd, bwd):
        for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(n, dtype=torch.uint8, pin_memory=True),
                   torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
            with pytest.raises(ValueError):
                call(ws)
        with pytest.raises(q.QLoraError):
            call(torch.empty(64, dtype=torch.uint8, device="cuda"))
        call(torch.empty((n + 3) // 4, dtype=torch.float32, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(out + grads, want + dwant))
    assert q.qlora_check_status() == 0
