"""The microscaled 4-bit operators and the standalone dropout: cases, plain forms and exact values.

Operators
---------
quantise   microscaled 4-bit floating point and back: MXFP4 (blocks of 32, power-of-two
           scales) and NVFP4 (blocks of 16, E4M3 scales, one fp32 scale per row)
product    Y = deq(x) deq(w)^T of two quantised operands
layer      the QLoRA layer on a microscaled base: Y = deq(Q(X)) deq(W)^T + s (X' A^T) B^T
grad       its gradients: dX = dY deq(W) + D c s U A, dA = s U^T X', dB = s dY^T T, U = dY B
dropout    Y = D * c * X (+ residual) or dX = D * c * dY, the keep mask D from Philox4x64-10

Storage: two codes a byte, element 2j in the low nibble; scales in tiles of 128 rows x 4 scale
columns, 512 bytes each, byte (r % 32) * 16 + (r // 32) * 4 + c, tiles of a row block consecutive.
"""

import math

import numpy as np
import torch

own = False

MXFP4, NVFP4 = 0, 1
BLOCK = {MXFP4: 32, NVFP4: 16}
BF16, F32 = torch.bfloat16, torch.float32

# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # a 70B-class MLP weight taken to 4 bits once, before training or serving
        dict(name="quantise-70b-nv", op="quantise", fmt=NVFP4, M=28672, K=8192, dtype="bf16", pad=0),
        # fp32 activations of a ragged batch, a slice of a wider buffer
        dict(name="quantise-ragged-mx", op="quantise", fmt=MXFP4, M=777, K=18944, dtype="fp32", pad=64),
        # the smallest call: latency
        dict(name="product-tiny-nv", op="product", fmt=NVFP4, M=16, N=1024, K=1024),
        # one token through a 70B-class projection, served: a read of the weight
        dict(name="product-1-70b-mx", op="product", fmt=MXFP4, M=1, N=28672, K=8192),
        # a prompt of 4096 tokens through an attention projection
        dict(name="product-4096-nv", op="product", fmt=NVFP4, M=4096, N=4096, K=4096),
        # a decode batch through the 7B-class gate projection with its adapter
        dict(name="layer-16-7b-nv", op="layer", fmt=NVFP4, M=16, N=18944, K=3584, r=64, alpha=16.0, p=0.0),
        # a training step's forward through the same projection
        dict(name="layer-8192-7b-mx", op="layer", fmt=MXFP4, M=8192, N=18944, K=3584, r=64, alpha=16.0, p=0.0),
        # a ragged batch through the down projection, adapter dropout on
        dict(name="layer-777-down-nv", op="layer", fmt=NVFP4, M=777, N=3584, K=18944, r=16, alpha=32.0, p=0.05),
        # a training step's backward on an attention projection
        dict(name="grad-8192-nv", op="grad", fmt=NVFP4, M=8192, N=4096, K=4096, r=64, alpha=128.0, p=0.0),
        # the same of a ragged batch with adapter dropout, a small rank
        dict(name="grad-1111-7b-mx", op="grad", fmt=MXFP4, M=1111, N=18944, K=3584, r=8, alpha=16.0, p=0.1),
        # dropout of a block's output before the residual sum
        dict(name="dropout-residual", op="dropout", M=8192, K=3584, dtype="bf16", p=0.1, residual=True, back=False),
        # its gradient on an odd-sized fp32 tensor
        dict(name="dropout-grad-odd", op="dropout", M=4097, K=4095, dtype="fp32", p=0.05, residual=False, back=True),
    ]


def _log(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["quantise", "product", "layer", "grad", "dropout"])
    fmt = rng.choice([MXFP4, NVFP4])
    if op == "quantise":
        return dict(op=op, fmt=fmt, M=_log(rng, 1, 8192), K=_log(rng, 64, 19000, 32),
                    dtype=rng.choice(["bf16", "fp32"]), pad=rng.choice([0, 0, 32, 4096]))
    if op == "dropout":
        back = rng.random() < 0.5
        return dict(op=op, M=_log(rng, 1, 8192), K=_log(rng, 64, 4096), dtype=rng.choice(["bf16", "fp32"]),
                    p=rng.choice([0.05, 0.1, 0.25, 0.5]), residual=not back and rng.random() < 0.5, back=back)
    N, K = _log(rng, 1024, 19000, 8), _log(rng, 1024, 19000, 64)
    most = 8192 * 18944 * 3584 // (N * K + 4 * N)      # no dearer than the largest listed case
    if op == "product":
        return dict(op=op, fmt=fmt, M=min(most, _log(rng, 1, 8192)), N=N + rng.choice([0, 0, 1, 3]), K=K - rng.choice([0, 32]))
    return dict(op=op, fmt=fmt, M=min(most, _log(rng, 1 if op == "layer" else 16, 8192)), N=N, K=K, r=rng.choice([8, 16, 32, 64, 128]),
             alpha=rng.choice([16.0, 32.0]), p=rng.choice([0.0, 0.0, 0.05]))


def _dt(case):
    return BF16 if case["dtype"] == "bf16" else F32


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _scale_columns(fmt, K):
    return (K // BLOCK[fmt] + 3) // 4 * 4


def _tile(codes):
    """Row-major scale bytes [rows, columns] -> the tiled byte array."""
    rows, cols = codes.shape
    R, C = (rows + 127) // 128 * 128, (cols + 3) // 4 * 4
    full = torch.zeros(R, C, dtype=torch.uint8, device=codes.device)
    full[:rows, :cols] = codes
    return full.view(R // 128, 4, 32, C // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile(scales, rows, cols):
    R, C = (rows + 127) // 128 * 128, (cols + 3) // 4 * 4
    full = scales.view(R // 128, C // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(R, C)
    return full[:rows, :cols]


def _pow2(field):
    """2^(field - 127) from an exponent field (0 stands for 2^-127)."""
    normal = (field.to(torch.int32) << 23).view(F32)
    return torch.where(field == 0, torch.full_like(normal, 2.0 ** -127), normal)


def _quantise(X, fmt):
    """codes [rows, K] (uint8), scale bytes [rows, K / block], row scale [rows] (or None)."""
    x = X.float()
    rows, K = x.shape
    b = BLOCK[fmt]
    if fmt == NVFP4:
        bits = x.abs().amax(1).view(torch.int32)
        f = (bits >> 23) - 11 + ((bits & 0x7FFFFF) > 0x280000).to(torch.int32)
        f = torch.where(bits == 0, torch.full_like(f, 127), f.clamp(min=27))      # at least 2^-100
        s = _pow2(f)
        x = x * _pow2(254 - f)[:, None]
        amax = x.abs().view(rows, K // b, b).amax(2)
        code = (amax / torch.full_like(amax, 6.0)).to(torch.float8_e4m3fn)   # a true division
        S = code.float()
        code = code.view(torch.uint8)
    else:
        s = None
        field = (x.abs().view(rows, K // b, b).amax(2).view(torch.int32) >> 23) - 2
        code = field.clamp(min=0).to(torch.uint8)
        S = _pow2(code)
    y = x.view(rows, K // b, b)
    m, S3 = y.abs(), S[:, :, None]
    # the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times S, ties to the even code: products t * S are exact
    q = (m > 0.25 * S3).to(torch.uint8)
    q += m >= 0.75 * S3
    q += m > 1.25 * S3
    q += m >= 1.75 * S3
    q += m > 2.5 * S3
    q += m >= 3.5 * S3
    q += m > 5.0 * S3
    q = torch.where(S3 == 0, torch.zeros_like(q), q) | (torch.signbit(y).to(torch.uint8) << 3)
    return q.view(rows, K), code, s


def _values(codes, code, s, fmt):
    """fp32 values of codes under their scales."""
    rows, K = codes.shape
    table = torch.tensor(_E2M1, dtype=F32, device=codes.device)
    S = code.view(torch.float8_e4m3fn).float() if fmt == NVFP4 else _pow2(code)
    v = table[codes.int()].view(rows, -1, BLOCK[fmt]) * S[:, :, None]
    v = v.view(rows, K)
    return v * s[:, None] if s is not None else v


def _pack(codes):
    return codes[:, 0::2] | (codes[:, 1::2] << 4)


def _unpacked_values(t, fmt, rows, K):
    p = t["packed"].view(rows, K // 2)
    codes = torch.stack((p & 15, p >> 4), 2).view(rows, K)
    return _values(codes, _untile(t["scales"], rows, K // BLOCK[fmt]).contiguous(), t["row_scale"], fmt)


_M32 = 0xFFFFFFFF


def _mulhilo(c, m):
    """High and low words of the unsigned 64 x 64-bit product, on int64."""
    a0, a1, m0, m1 = c & _M32, (c >> 32) & _M32, m & _M32, m >> 32
    p00, p10, p01, p11 = a0 * m0, a1 * m0, a0 * m1, a1 * m1
    mid = ((p00 >> 32) & _M32) + (p10 & _M32) + (p01 & _M32)
    hi = p11 + ((p10 >> 32) & _M32) + ((p01 >> 32) & _M32) + ((mid >> 32) & _M32)
    return hi, (p00 & _M32) | (mid << 32)


def _signed(v):
    v &= (1 << 64) - 1
    return v - (1 << 64) if v >> 63 else v


def _keep(n, p, seed, device):
    """Keep mask of elements 0..n-1."""
    c0 = torch.arange((n + 7) // 8, dtype=torch.int64, device=device)
    c1, c2, c3 = torch.zeros_like(c0), torch.zeros_like(c0), torch.zeros_like(c0)
    for r in range(10):
        k0, k1 = _signed(seed + r * 0x9E3779B97F4A7C15), _signed(r * 0xBB67AE8584CAA73B)
        h0, l0 = _mulhilo(c0, 0xD2E7470EE14C6C93)
        h1, l1 = _mulhilo(c2, 0xCA5A826395121157)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
    u = torch.stack([(w >> sh) & 0xFFFFFF for w in (c0, c1, c2, c3) for sh in (40, 16)], 1)
    thr = int(math.floor(float(np.float32(p)) * (1 << 24) + 0.5))
    return u.view(-1)[:n] >= thr


def _factor(p):
    return float(np.float32(1) / (np.float32(1) - np.float32(p)))


def _dropped(X, p, seed):
    """The adapter's input X' (fp32 values of bf16) and the mask times its factor."""
    if p == 0:
        return X.float(), None
    keep = _keep(X.numel(), p, seed, X.device).view(X.shape)
    c = _factor(p)
    return torch.where(keep, (X.float() * c).to(BF16).float(), 0.0), keep.float() * c


def _plain(st):
    c = st["case"]
    op = c["op"]
    if op == "quantise":
        q, code, s = _quantise(st["X"], c["fmt"])
        out = {"values": _values(q, code, s, c["fmt"]).to(BF16)}
        return out if s is None else {**out, "row_scale": s}
    if op == "product":
        x = _unpacked_values(st["x"], c["fmt"], c["M"], c["K"])
        w = _unpacked_values(st["w"], c["fmt"], c["N"], c["K"])
        return (x @ w.t()).to(BF16)
    if op == "dropout":
        x = st["X"]
        y = torch.where(_keep(x.numel(), c["p"], st["seed"], x.device).view(x.shape), x.float() * _factor(c["p"]), 0.0)
        return (y + st["R"].float() if c["residual"] else y).to(x.dtype)
    s = c["alpha"] / c["r"]
    w = _unpacked_values(st["w"], c["fmt"], c["N"], c["K"])
    A, B = st["A"].float(), st["B"].float()
    Xd, mask = _dropped(st["X"], c["p"], st["seed"])
    if op == "layer":
        x = _values(*_quantise(st["X"], c["fmt"]), c["fmt"])
        T = Xd @ A.t()
        return {"Y": (x @ w.t() + s * (T @ B.t())).to(BF16), "T": T.to(BF16)}
    dY = st["dY"].float()
    U = dY @ B
    ad = s * (U @ A)
    dX = dY @ w + (ad if mask is None else mask * ad)
    return {"dX": dX.to(BF16), "dA": (s * (U.t() @ Xd)).to(BF16), "dB": (s * (dY.t() @ st["T"].float())).to(BF16)}


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------


def _own(st):
    import qlora_linear_layers_b200 as q

    c = st["case"]
    op = c["op"]
    if op == "dropout":
        if c["back"]:
            return q.dropout_bwd(st["X"], c["p"], st["seed"])
        return q.dropout_fwd(st["X"], c["p"], st["seed"], residual=st["R"])
    if op == "quantise":
        t = q.mx_quantize(st["X"], c["fmt"])
        out = {"values": q.mx_dequantize(t)}
        return out if t.row_scale is None else {**out, "row_scale": t.row_scale}
    w = q.MXTensor(rows=c["N"], cols=c["K"], format=c["fmt"], **st["w"])
    if op == "product":
        return q.mx_matmul(q.MXTensor(rows=c["M"], cols=c["K"], format=c["fmt"], **st["x"]), w)
    if op == "layer":
        Y, T = q.mx_linear_fwd(w, st["X"], st["A"], st["B"], c["alpha"], p=c["p"], seed=st["seed"])
        return {"Y": Y, "T": T}
    dX, dA, dB = q.mx_linear_bwd(w, st["X"], st["dY"], st["A"], st["B"], c["alpha"], p=c["p"], seed=st["seed"], T=st["T"])
    return {"dX": dX, "dA": dA, "dB": dB}


# ---------------------------------------------------------------------------
# What the tools call
# ---------------------------------------------------------------------------


def _activations(g, M, K, dtype=BF16):
    """Gaussian rows with a few channels eight times as large, and rows of unequal size."""
    x = torch.randn(M, K, generator=g, device="cuda")
    x *= 1 + 7 * (torch.rand(K, generator=g, device="cuda") < 0.005)
    x *= torch.exp2(torch.rand(M, 1, generator=g, device="cuda") * 4 - 2)
    return x.to(dtype)


def _packed(X, fmt):
    q, code, s = _quantise(X, fmt)
    return {"packed": _pack(q).view(-1), "scales": _tile(code), "row_scale": s}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    st = {"case": c, "seed": seed * 0x9E3779B97F4A7C15 % (1 << 64)}
    op, K = c["op"], c["K"]
    if op == "quantise":
        wide = torch.randn(c["M"], K + c["pad"], generator=g, device="cuda") if c["dtype"] == "fp32" else \
            _activations(g, c["M"], K + c["pad"])
        st["X"] = wide[:, :K]
        return st
    if op == "dropout":
        st["X"] = torch.randn(c["M"], K, generator=g, device="cuda").to(_dt(c))
        st["R"] = torch.randn(c["M"], K, generator=g, device="cuda").to(_dt(c)) if c["residual"] else None
        return st
    st["w"] = _packed((torch.randn(c["N"], K, generator=g, device="cuda") * 0.02).to(BF16), c["fmt"])
    X = _activations(g, c["M"], K)
    if op == "product":
        st["x"] = _packed(X, c["fmt"])
        return st
    st["X"] = X
    st["A"] = (torch.randn(c["r"], K, generator=g, device="cuda") * 0.02).to(BF16)
    st["B"] = (torch.randn(c["N"], c["r"], generator=g, device="cuda") * 0.02).to(BF16)
    if op == "grad":
        st["dY"] = torch.randn(c["M"], c["N"], generator=g, device="cuda").to(BF16)
        st["T"] = (_dropped(X, c["p"], st["seed"])[0] @ st["A"].float().t()).to(BF16)
    return st


def run(state):
    if own:
        return _own(state)
    return _plain(state)


def _stored(fmt, rows, K):
    return rows * K / 2 + rows * K / BLOCK[fmt] + (4 * rows if fmt == NVFP4 else 0)


def work(case):
    c = case
    op, M, K = c["op"], c["M"], c["K"]
    if op == "dropout":
        e = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": M * K * e * (3 if c["residual"] else 2), "flops": 2 * M * K}
    if op == "quantise":
        e = 2 if c["dtype"] == "bf16" else 4
        # the input, the 4-bit tensor written and read back, the values
        return {"bytes": M * K * (e + 2) + 2 * _stored(c["fmt"], M, K), "flops": 4 * M * K}
    N = c["N"]
    w = _stored(c["fmt"], N, K)
    if op == "product":
        return {"bytes": w + _stored(c["fmt"], M, K) + 2 * M * N, "flops": 2 * M * N * K}
    r = c["r"]
    ad = 2 * r * (N + K)
    if op == "layer":
        return {"bytes": w + ad + 2 * M * (K + N + r), "flops": 2 * M * N * K + 2 * M * r * (N + K)}
    return {"bytes": w + 2 * ad + 2 * M * (2 * K + N + r), "flops": 2 * M * N * K + 4 * M * r * (N + K)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_grid(v, emin, bits, top):
    """Nearest value with `bits` fraction bits and exponents >= emin, ties to even, at most top."""
    e = (torch.frexp(v)[1] - 1).clamp(min=emin)
    step = torch.ldexp(torch.ones_like(v), e - bits)
    return torch.minimum(torch.round(v / step) * step, torch.full_like(v, top))


def _exact_quantised(X, fmt):
    """(values, row scale) in 64 bits."""
    x = X.double()
    rows, K = x.shape
    if fmt == NVFP4:
        top = x.abs().amax(1) / 2688
        one = torch.ones_like(top)
        mant, e = torch.frexp(top)                     # top = mant 2^e, mant in [0.5, 1)
        s = torch.ldexp(one, torch.where(mant == 0.5, e - 1, e).clamp(min=-100))
        s = torch.where(top == 0, one, s)
        y = (x / s[:, None]).view(rows, -1, 16)
        S = _exact_grid(y.abs().amax(2) / 6, -6, 3, 448.0)[:, :, None]
    else:
        s = None
        y = x.view(rows, -1, 32)
        a = y.abs().amax(2)
        e = torch.where(a == 0, torch.full_like(a, -127).int(), torch.frexp(a)[1] - 3).clamp(min=-127)
        S = torch.ldexp(torch.ones_like(a), e)[:, :, None]
    safe = torch.where(S == 0, torch.ones_like(S), S)
    v = torch.copysign(_exact_grid(y.abs() / safe, 0, 1, 6.0) * S, y).view(rows, K)
    return (v if s is None else v * s[:, None]), s


def _exact_stored(t, fmt, rows, K):
    """64-bit values of a stored tensor, from its bytes."""
    p = t["packed"].view(rows, K // 2).long()
    code = torch.empty(rows, K, dtype=torch.int64, device=p.device)
    code[:, 0::2], code[:, 1::2] = p % 16, p // 16
    e, m = code // 2 % 4, code % 2
    mag = torch.where(e == 0, m * 0.5, (1 + 0.5 * m) * torch.exp2(e.double() - 1))
    mag = torch.where(code >= 8, -mag, mag)
    r = torch.arange(rows, device=p.device)[:, None]
    j = torch.arange(K // BLOCK[fmt], device=p.device)[None]
    tiles = (K // BLOCK[fmt] + 3) // 4
    b = t["scales"][(r // 128 * tiles + j // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + j % 4].long()
    if fmt == NVFP4:
        S = torch.where(b // 8 == 0, b * 2.0 ** -9, (1 + b % 8 / 8.0) * torch.exp2((b // 8).double() - 7))
        S = S * t["row_scale"].double()[:, None]
    else:
        S = torch.exp2(b.double() - 127)
    return (mag.view(rows, -1, BLOCK[fmt]) * S[:, :, None]).view(rows, K)


def _exact_keep(n, p, seed, device):
    """The keep mask from the generator's published definition, on the host."""
    u64, blocks = np.uint64, (n + 7) // 8
    low = u64(_M32)

    def product(a, m):
        m0, m1 = u64(m & _M32), u64(m >> 32)
        a0, a1 = a & low, a >> u64(32)
        t = a0 * m0
        k = t >> u64(32)
        t2 = a1 * m0 + k
        t3 = a0 * m1 + (t2 & low)
        return a1 * m1 + (t2 >> u64(32)) + (t3 >> u64(32)), a * u64(m)

    with np.errstate(over="ignore"):
        c = [np.arange(blocks, dtype=u64)] + [np.zeros(blocks, u64) for _ in range(3)]
        k0, k1 = u64(seed), u64(0)
        for i in range(10):
            if i:
                k0, k1 = u64((int(k0) + 0x9E3779B97F4A7C15) % (1 << 64)), u64((int(k1) + 0xBB67AE8584CAA73B) % (1 << 64))
            h0, l0 = product(c[0], 0xD2E7470EE14C6C93)
            h1, l1 = product(c[2], 0xCA5A826395121157)
            c = [h1 ^ c[1] ^ k0, l1, h0 ^ c[3] ^ k1, l0]
    u = np.empty((blocks, 8), np.uint32)
    for i in range(8):
        u[:, i] = (c[i // 2] >> u64(16 if i % 2 else 40)) & u64(0xFFFFFF)
    thr = int(math.floor(float(np.float32(p)) * (1 << 24) + 0.5))
    return torch.from_numpy(u.reshape(-1)[:n] >= thr).to(device)


def exact(case, seed):
    st, c = prepare(case, seed), dict(case)
    op, M, K, fmt = c["op"], c["M"], c["K"], c.get("fmt")
    if c.get("p") and M * K > 60_000_000:
        return None
    if op == "quantise":
        v, s = _exact_quantised(st["X"], fmt)
        return {"values": v} if s is None else {"values": v, "row_scale": s}
    if op == "product":
        return _exact_stored(st["x"], fmt, M, K) @ _exact_stored(st["w"], fmt, c["N"], K).t()
    keep = _exact_keep(M * K, c["p"], st["seed"], "cuda").view(M, K) if c["p"] else None
    factor = _factor(c["p"])
    if op == "dropout":
        y = torch.where(keep, st["X"].double() * factor, 0.0)
        return y + st["R"].double() if c["residual"] else y
    s = c["alpha"] / c["r"]
    w, A, B, Xd = _exact_stored(st["w"], fmt, c["N"], K), st["A"].double(), st["B"].double(), st["X"].double()
    if keep is not None:                                # X' is a bf16 tensor by definition
        Xd = torch.where(keep, (Xd * factor).float().to(BF16).double(), 0.0)
    if op == "layer":
        T = Xd @ A.t()
        return {"Y": _exact_quantised(st["X"], fmt)[0] @ w.t() + s * (T @ B.t()), "T": T}
    dY = st["dY"].double()
    U = dY @ B
    ad = s * (U @ A)
    if keep is not None:
        ad = torch.where(keep, ad * factor, 0.0)
    return {"dX": dY @ w + ad, "dA": s * (U.t() @ Xd), "dB": s * (dY.t() @ st["T"].double())}
