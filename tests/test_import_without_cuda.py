"""The package imports, and its host-only queries answer, where torch was built
without CUDA: such a build has none of torch's CUDA bindings."""

import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import torch
for name in [n for n in dir(torch._C) if n.startswith("_cuda_")]:
    delattr(torch._C, name)
import qlora_linear_layers_b200 as q
import qlora_linear_layers_b200.dp
assert q.workspace_bytes(q._lib.QLORA_OP_MX_FWD, 16, 1024, 1024, 16) > 0
assert q.mx_scale_bytes(1, 128, 64) == 512 and len(q.code_table()) == 16
x = torch.zeros(4, 64, dtype=torch.bfloat16)
for call in (lambda: q.mx_quantize(x), lambda: q.dropout_fwd(x, 0.1, 1)):
    try:
        call()
    except ValueError:
        continue
    raise SystemExit("a host tensor was taken")
"""


def test_import_and_host_queries():
    from qlora_linear_layers_b200.build import build
    build()
    p = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr
