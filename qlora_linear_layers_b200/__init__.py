"""B200-native QLoRA NF4 linear layers.

Thin Python binding over libqlora_nf4.so (C ABI in include/qlora_nf4.h).
PyTorch supplies device memory and streams only; every step of the path runs
in the library's sm_100a kernels.  The functions named like the C entry
points (nf4_quantize, nf4_double_quantize, nf4_dequantize, qlora_linear_fwd,
qlora_linear_bwd, qlora_check_status) marshal tensors to pointers; `quantize`,
`dequantize`, `linear_fwd`, `linear_bwd` are conveniences that allocate the
outputs and the workspace with torch and call them.  The microscaled 4-bit
formats (`mx_quantize`, `mx_dequantize`, `mx_matmul`, `mx_linear_fwd`,
`mx_linear_bwd`) and the standalone dropout (`dropout_fwd`, `dropout_bwd`) have
the same two layers.
"""

from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import QLoraError  # noqa: F401

BLOCKSIZE = 64
DQ_BLOCKSIZE = 256


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


@dataclass
class NF4Tensor:
    """A quantised weight: the buffers of `nf4_weight` plus its shape."""
    packed: torch.Tensor            # uint8 [rows*cols/2]
    rows: int
    cols: int
    absmax: torch.Tensor            # fp32 [rows*cols/64]
    qabsmax: torch.Tensor | None    # int8 [rows*cols/64]
    dq_scale: torch.Tensor | None   # fp32 [ceil(n_absmax/256)]
    dq_mean: torch.Tensor | None    # fp32 [1]
    double_quant: int = 1           # 0 none, 1 int8 codes, 2 E4M3 codes (True = 1)
    quant_type: int = _lib.QLORA_QUANT_NF4

    def c_struct(self) -> _lib.NF4Weight:
        return _lib.NF4Weight(
            packed=_ptr(self.packed), rows=self.rows, cols=self.cols, blocksize=BLOCKSIZE,
            double_quant=int(self.double_quant),
            absmax=_ptr(self.absmax), qabsmax=_ptr(self.qabsmax), dq_scale=_ptr(self.dq_scale),
            dq_mean=_ptr(self.dq_mean), dq_blocksize=DQ_BLOCKSIZE, quant_type=self.quant_type)

    def stored_bytes(self) -> int:
        """Bytes the quantised weight occupies (codes + constants in use)."""
        if self.double_quant:
            return (self.packed.numel() + self.qabsmax.numel() + 4 * self.dq_scale.numel()
                    + 4 * self.dq_mean.numel())
        return self.packed.numel() + 4 * self.absmax.numel()


@dataclass
class MXTensor:
    """A microscaled 4-bit matrix: the buffers of `qlora_mx_tensor` plus its shape."""
    packed: torch.Tensor            # uint8 [rows*cols/2], element 2j in the low nibble
    scales: torch.Tensor            # uint8, tiles of 128 rows x 4 scale columns
    row_scale: torch.Tensor | None  # fp32 [rows] (NVFP4)
    rows: int
    cols: int
    format: int = _lib.QLORA_NVFP4

    def c_struct(self) -> _lib.MXTensor:
        rows, cols, nv = self.rows, self.cols, self.format == _lib.QLORA_NVFP4
        p, sc, rs = self.packed, self.scales, self.row_scale
        dev = p.get_device()
        # a width that the library refuses has no tiles
        tiles = 0 if cols % 32 else (rows + 127) // 128 * -(-cols // (64 if nv else 128))
        if not (p.is_contiguous() and sc.is_contiguous() and dev >= 0 and sc.get_device() == dev
                and p.dtype is torch.uint8 and sc.dtype is torch.uint8
                and p.numel() == rows * cols // 2
                and sc.numel() >= tiles * 512):
            raise ValueError("packed and scales must be contiguous uint8 CUDA tensors of a "
                             f"{rows} x {cols} matrix")
        if nv and (rs is None or rs.numel() != rows or rs.dtype is not torch.float32
                   or not rs.is_contiguous() or rs.get_device() != dev):
            raise ValueError(f"row_scale must be a contiguous fp32 CUDA tensor of {rows} values")
        return _lib.MXTensor(p.data_ptr(), rows, cols, self.format, 0, sc.data_ptr(),
                             rs.data_ptr() if nv else None)

    def block_scales(self) -> torch.Tensor:
        """The scale bytes as a row-major [rows, cols / block] tensor (a copy)."""
        n = self.cols // (16 if self.format == _lib.QLORA_NVFP4 else 32)
        rb, tiles = (self.rows + 127) // 128, (n + 3) // 4
        t = self.scales[:rb * tiles * 512].view(rb, tiles, 32, 4, 4).permute(0, 3, 2, 1, 4)
        return t.reshape(rb * 128, tiles * 4)[:self.rows, :n].contiguous()

    def stored_bytes(self) -> int:
        """Bytes the quantised matrix occupies."""
        rs = 4 * self.rows if self.format == _lib.QLORA_NVFP4 else 0
        return self.packed.numel() + self.scales.numel() + rs


# ---------------------------------------------------------------------------
# Entry points with the C names
# ---------------------------------------------------------------------------

def nf4_quantize(W: torch.Tensor, packed: torch.Tensor, absmax: torch.Tensor, stream=None):
    _need_cuda(W, packed, absmax)
    dt = {torch.float32: _lib.QLORA_F32, torch.bfloat16: _lib.QLORA_BF16}.get(W.dtype)
    if dt is None:
        raise ValueError("W must be fp32 or bf16")
    _lib.check(_lib.load().nf4_quantize(_ptr(W), dt, W.shape[0], W.shape[1], BLOCKSIZE,
                                        _ptr(packed), _ptr(absmax), _stream(stream)),
               "nf4_quantize")


def qlora_quantize_4bit(W: torch.Tensor, packed: torch.Tensor, absmax: torch.Tensor,
                        quant_type: int = _lib.QLORA_QUANT_NF4, dq_hist: torch.Tensor | None = None,
                        stream=None):
    """Quantise W (fp32/bf16 [rows, cols]); with dq_hist (int64 [256]) also
    write the exponent histogram of the block absmax values."""
    _need_cuda(W, packed, absmax, dq_hist)
    dt = {torch.float32: _lib.QLORA_F32, torch.bfloat16: _lib.QLORA_BF16}.get(W.dtype)
    if dt is None:
        raise ValueError("W must be fp32 or bf16")
    if dq_hist is not None and (dq_hist.dtype != torch.int64 or dq_hist.numel() != 256):
        raise ValueError("dq_hist must be int64 [256]")
    _lib.check(_lib.load().qlora_quantize_4bit(_ptr(W), dt, W.shape[0], W.shape[1], BLOCKSIZE,
                                               int(quant_type), _ptr(packed), _ptr(absmax),
                                               _ptr(dq_hist), _stream(stream)),
               "qlora_quantize_4bit")


def nf4_double_quantize_hist(absmax: torch.Tensor, dq_hist: torch.Tensor, n_total: int,
                             qabsmax: torch.Tensor, dq_scale: torch.Tensor, dq_mean: torch.Tensor,
                             stream=None, dq_type: int = _lib.QLORA_DQ_INT8):
    """Second double-quantisation pass from a complete histogram over n_total
    absmax values (summed over shards when the weight is sharded); dq_type
    picks int8 or E4M3 codes."""
    _need_cuda(absmax, dq_hist, qabsmax, dq_scale, dq_mean)
    _lib.check(_lib.load().qlora_double_quantize_hist(_ptr(absmax), absmax.numel(), _ptr(dq_hist),
                                                      int(n_total), DQ_BLOCKSIZE, int(dq_type),
                                                      _ptr(qabsmax), _ptr(dq_scale), _ptr(dq_mean),
                                                      _stream(stream)),
               "qlora_double_quantize_hist")


def workspace_bytes(op: int, M: int, N: int, K: int, r: int) -> int:
    return int(_lib.load().qlora_workspace_bytes(op, M, N, K, r))


def _workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)


def nf4_double_quantize(absmax: torch.Tensor, qabsmax: torch.Tensor, dq_scale: torch.Tensor,
                        dq_mean: torch.Tensor, ws: torch.Tensor | None = None, stream=None):
    _need_cuda(absmax, qabsmax, dq_scale, dq_mean)
    need = workspace_bytes(_lib.QLORA_OP_DOUBLE_QUANT, 0, absmax.numel(), 0, 0)
    if ws is None:
        ws = _workspace(need, absmax.device)
    _lib.check(_lib.load().nf4_double_quantize(_ptr(absmax), absmax.numel(), DQ_BLOCKSIZE,
                                               _ptr(qabsmax), _ptr(dq_scale), _ptr(dq_mean),
                                               _ptr(ws), ws.numel(), _stream(stream)),
               "nf4_double_quantize")


def nf4_dequantize(w: NF4Tensor, out: torch.Tensor, stream=None):
    _need_cuda(out)
    cw = w.c_struct()
    _lib.check(_lib.load().nf4_dequantize(C.byref(cw), _ptr(out), _stream(stream)),
               "nf4_dequantize")


def qlora_merge(w: NF4Tensor, A, B, alpha: float, out, stream=None):
    """out[N, K] bf16 = RNbf16(deq(W) + (alpha / r) B A)."""
    _need_cuda(A, B, out)
    cw = w.c_struct()
    _lib.check(_lib.load().qlora_merge(C.byref(cw), _ptr(A), _ptr(B), A.shape[0], float(alpha),
                                       _ptr(out), _stream(stream)),
               "qlora_merge")


def qlora_linear_fwd(w: NF4Tensor, X, A, B, alpha: float, Y, T_save=None, ws=None, stream=None):
    _need_cuda(X, A, B, Y, T_save)
    M, r = X.shape[0], A.shape[0]
    need = workspace_bytes(_lib.QLORA_OP_FWD, M, w.rows, w.cols, r)
    if ws is None:
        ws = _workspace(need, X.device)
    cw = w.c_struct()
    _lib.check(_lib.load().qlora_linear_fwd(C.byref(cw), _ptr(X), M, _ptr(A), _ptr(B), r,
                                            float(alpha), _ptr(Y), _ptr(T_save), _ptr(ws),
                                            ws.numel(), _stream(stream)),
               "qlora_linear_fwd")


def qlora_linear_bwd(w: NF4Tensor, X, dY, A, B, alpha: float, dX, dA, dB, T=None, ws=None,
                     stream=None):
    _need_cuda(X, dY, A, B, dX, dA, dB, T)
    M, r = X.shape[0], A.shape[0]
    need = workspace_bytes(_lib.QLORA_OP_BWD, M, w.rows, w.cols, r)
    if ws is None:
        ws = _workspace(need, X.device)
    cw = w.c_struct()
    _lib.check(_lib.load().qlora_linear_bwd(C.byref(cw), _ptr(X), _ptr(dY), M, _ptr(A), _ptr(B),
                                            r, float(alpha), _ptr(T), _ptr(dX), _ptr(dA),
                                            _ptr(dB), _ptr(ws), ws.numel(), _stream(stream)),
               "qlora_linear_bwd")


def qlora_linear_fwd_dropout(w: NF4Tensor, X, A, B, alpha: float, p: float, seed: int, Y,
                             T_save=None, ws=None, stream=None):
    """The forward with LoRA dropout (rate p, Philox seed) on the adapter input."""
    _need_cuda(X, A, B, Y, T_save)
    M, r = X.shape[0], A.shape[0]
    if ws is None:
        ws = _workspace(workspace_bytes(_lib.QLORA_OP_FWD_DROPOUT, M, w.rows, w.cols, r), X.device)
    cw = w.c_struct()
    dr = _lib.Dropout(p=float(p), reserved=0, seed=int(seed))
    _lib.check(_lib.load().qlora_linear_fwd_dropout(C.byref(cw), _ptr(X), M, _ptr(A), _ptr(B), r,
                                                    float(alpha), C.byref(dr), _ptr(Y), _ptr(T_save),
                                                    _ptr(ws), ws.numel(), _stream(stream)),
               "qlora_linear_fwd_dropout")


def qlora_linear_bwd_dropout(w: NF4Tensor, X, dY, A, B, alpha: float, p: float, seed: int, dX, dA,
                             dB, T=None, ws=None, stream=None):
    """The backward with LoRA dropout; the mask is regenerated from (p, seed)."""
    _need_cuda(X, dY, A, B, dX, dA, dB, T)
    M, r = X.shape[0], A.shape[0]
    if ws is None:
        ws = _workspace(workspace_bytes(_lib.QLORA_OP_BWD_DROPOUT, M, w.rows, w.cols, r), X.device)
    cw = w.c_struct()
    dr = _lib.Dropout(p=float(p), reserved=0, seed=int(seed))
    _lib.check(_lib.load().qlora_linear_bwd_dropout(C.byref(cw), _ptr(X), _ptr(dY), M, _ptr(A),
                                                    _ptr(B), r, float(alpha), C.byref(dr), _ptr(T),
                                                    _ptr(dX), _ptr(dA), _ptr(dB), _ptr(ws),
                                                    ws.numel(), _stream(stream)),
               "qlora_linear_bwd_dropout")


# None where torch was built without CUDA: no tensor gets as far as a call of these there
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)    # without the initialisation that a CUDA tensor implies


class _On:
    """Device and stream of a call: entered, it gives the raw stream.  With a
    stream that is not the current one, buffers allocated inside belong to it,
    so that the allocator orders their reuse after the call's work."""

    def __init__(self, dev: int, stream):
        self.dev, self.stream, self.ctx = dev, stream, None

    def __enter__(self) -> int:
        if self.stream is not None:
            if self.stream.device.index != self.dev:
                raise ValueError("the stream is on another device than the tensors")
            self.ctx = torch.cuda.stream(self.stream)
        elif self.dev != _current_device():
            self.ctx = torch.cuda.device(self.dev)
        if self.ctx is not None:
            self.ctx.__enter__()
        return _raw_stream(self.dev)

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def _dense(dev: int, dtype, shape: tuple, t, what: str) -> int | None:
    """Address of a contiguous tensor of this device, type and shape, or of None."""
    if t is None:
        return None
    if (t.get_device() != dev or dev < 0 or t.dtype is not dtype or t.shape != shape
            or not t.is_contiguous()):
        raise ValueError(f"{what}: expected a contiguous {dtype} tensor {shape} on CUDA device {dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _scratch(ws, dev: int) -> tuple:
    """(address, bytes) of a workspace tensor of any type on this device."""
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"ws: expected a contiguous tensor on CUDA device {dev}, got one on {ws.device}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _rows_of(t, what: str) -> int:
    """Row stride in elements of a 2-D CUDA tensor whose rows are contiguous."""
    if t.get_device() < 0 or t.dim() != 2:
        raise ValueError(f"{what}: expected a 2-D CUDA tensor")
    n, k = t.shape
    if (k > 1 and t.stride(1) != 1) or (n > 1 and t.stride(0) < k):
        raise ValueError(f"{what}: expected contiguous rows")
    return t.stride(0) if n > 1 else k


def _float_type(t) -> int:
    if t.dtype is torch.bfloat16:
        return _lib.QLORA_BF16
    if t.dtype is torch.float32:
        return _lib.QLORA_F32
    raise ValueError("expected fp32 or bf16")


def mx_scale_bytes(format: int, rows: int, cols: int) -> int:
    return int(_lib.load().qlora_mx_scale_bytes(int(format), rows, cols))


def _mx_quantize(X, out, format, stream):
    ld, dev, (rows, cols) = _rows_of(X, "X"), X.get_device(), X.shape
    lib = _lib.load()
    with _On(dev, stream) as s:
        if out is None:
            nv = format == _lib.QLORA_NVFP4
            out = MXTensor(X.new_empty(rows * cols // 2, dtype=torch.uint8),
                           X.new_empty(lib.qlora_mx_scale_bytes(format, rows, cols), dtype=torch.uint8),
                           X.new_empty(rows, dtype=torch.float32) if nv else None, rows, cols, format)
            p, sc, rs = out.packed.data_ptr(), out.scales.data_ptr(), _ptr(out.row_scale)
        else:
            if (out.rows, out.cols) != (rows, cols) or out.packed.get_device() != dev:
                raise ValueError("out does not fit X")
            cw = out.c_struct()
            p, sc, rs = cw.packed, cw.scales, cw.row_scale
        _lib.check(lib.qlora_mx_quantize(X.data_ptr(), _float_type(X), rows, cols, ld, out.format, p, sc,
                                         rs, s),
                   "qlora_mx_quantize")
    return out


def qlora_mx_quantize(X: torch.Tensor, out: MXTensor, stream=None):
    """Quantise X (fp32/bf16, rows contiguous, any row stride) into `out`."""
    if out is None:
        raise ValueError("out is missing")
    _mx_quantize(X, out, out.format, stream)


def _mx_dequantize(t: MXTensor, out, stream):
    cw, dev = t.c_struct(), t.packed.get_device()
    with _On(dev, stream) as s:
        if out is None:
            out = t.packed.new_empty((t.rows, t.cols), dtype=torch.bfloat16)
        else:
            _dense(dev, torch.bfloat16, (t.rows, t.cols), out, "out")
        _lib.check(_lib.load().qlora_mx_dequantize(C.byref(cw), out.data_ptr(), s), "qlora_mx_dequantize")
    return out


def qlora_mx_dequantize(t: MXTensor, out: torch.Tensor, stream=None):
    if out is None:
        raise ValueError("out is missing")
    _mx_dequantize(t, out, stream)


def _mx_matmul(x: MXTensor, w: MXTensor, Y, stream):
    cx, cw, dev = x.c_struct(), w.c_struct(), x.packed.get_device()
    if w.packed.get_device() != dev:
        raise ValueError("x and w are on different devices")
    with _On(dev, stream) as s:
        if Y is None:
            Y = x.packed.new_empty((x.rows, w.rows), dtype=torch.bfloat16)
            y = Y.data_ptr()
        else:
            y = _dense(dev, torch.bfloat16, (x.rows, w.rows), Y, "Y")
        _lib.check(_lib.load().qlora_mx_matmul(C.byref(cx), C.byref(cw), y, s), "qlora_mx_matmul")
    return Y


def qlora_mx_matmul(x: MXTensor, w: MXTensor, Y: torch.Tensor, stream=None):
    """Y[M, N] bf16 = deq(x) deq(w)^T, both of one format."""
    _mx_matmul(x, w, Y, stream)


def _mx_layer(w: MXTensor, X, A, B, p, seed):
    """Checked arguments that the layer's forward and backward share."""
    cw, dev, bf = w.c_struct(), w.packed.get_device(), torch.bfloat16
    M, r = X.shape[0], 0 if A is None else A.shape[0]
    x = _dense(dev, bf, (M, w.cols), X, "X")
    a = _dense(dev, bf, (r, w.cols), A, "A")
    b = _dense(dev, bf, (w.rows, r), B, "B")
    dr = None if p == 0 else C.byref(_lib.Dropout(float(p), 0, int(seed)))
    return C.byref(cw), dev, M, r, x, a, b, dr


def _mx_fwd(w, X, A, B, alpha, Y, T, save_T, p, seed, ws, stream):
    cw, dev, M, r, x, a, b, dr = _mx_layer(w, X, A, B, p, seed)
    with _On(dev, stream) as s:
        if Y is None:
            Y = X.new_empty((M, w.rows))
            if save_T and r:
                T = X.new_empty((M, r))
        else:
            _dense(dev, torch.bfloat16, (M, w.rows), Y, "Y")
            _dense(dev, torch.bfloat16, (M, r), T, "T_save")
        if ws is None:
            op = _lib.QLORA_OP_MX_FWD if dr is None else _lib.QLORA_OP_MX_FWD_DROPOUT
            ws = _mx_workspace(op, M, w, r, X)
        _lib.check(_lib.load().qlora_mx_linear_fwd(cw, x, M, a, b, r, alpha, dr, Y.data_ptr(), _ptr(T),
                                                   *_scratch(ws, dev), s),
                   "qlora_mx_linear_fwd")
    return Y, T


def _mx_workspace(op, M, w, r, X):
    return X.new_empty(max(16, _lib.load().qlora_workspace_bytes(op, M, w.rows, w.cols, r)),
                       dtype=torch.uint8)


def qlora_mx_linear_fwd(w: MXTensor, X, A, B, alpha: float, Y, T_save=None, p: float = 0.0,
                        seed: int = 0, ws=None, stream=None):
    """The QLoRA layer on a microscaled base (A = B = None: no adapter)."""
    if Y is None:
        raise ValueError("Y is missing")
    _mx_fwd(w, X, A, B, alpha, Y, T_save, False, p, seed, ws, stream)


def _mx_bwd(w, X, dY, A, B, alpha, dX, dA, dB, T, p, seed, ws, stream):
    cw, dev, M, r, x, a, b, dr = _mx_layer(w, X, A, B, p, seed)
    bf = torch.bfloat16
    dy = _dense(dev, bf, (M, w.rows), dY, "dY")
    t = _dense(dev, bf, (M, r), T, "T")
    with _On(dev, stream) as s:
        if dX is None:
            dX = torch.empty_like(X)
            if r:
                dA, dB = torch.empty_like(A), torch.empty_like(B)
        else:
            _dense(dev, bf, (M, w.cols), dX, "dX")
            _dense(dev, bf, (r, w.cols), dA, "dA")
            _dense(dev, bf, (w.rows, r), dB, "dB")
        if ws is None:
            op = _lib.QLORA_OP_MX_BWD if dr is None else _lib.QLORA_OP_MX_BWD_DROPOUT
            ws = _mx_workspace(op, M, w, r, X)
        _lib.check(_lib.load().qlora_mx_linear_bwd(cw, x, dy, M, a, b, r, alpha, dr, t, dX.data_ptr(),
                                                   _ptr(dA), _ptr(dB), *_scratch(ws, dev), s),
                   "qlora_mx_linear_bwd")
    return dX, dA, dB


def qlora_mx_linear_bwd(w: MXTensor, X, dY, A, B, alpha: float, dX, dA, dB, T=None,
                        p: float = 0.0, seed: int = 0, ws=None, stream=None):
    """Its backward (A = B = dA = dB = None: dX alone)."""
    if dX is None:
        raise ValueError("dX is missing")
    _mx_bwd(w, X, dY, A, B, alpha, dX, dA, dB, T, p, seed, ws, stream)


def _like(t, X, what: str):
    """(address, row stride) of a tensor with X's device, type and shape."""
    if t is None:
        return None, 0
    if t.get_device() != X.get_device() or t.dtype is not X.dtype or t.shape != X.shape:
        raise ValueError(f"{what}: expected {X.dtype} {tuple(X.shape)} on {X.device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr(), _rows_of(t, what)


def _dropout(X, p, seed, Y, residual, first, stream, where):
    ldx, dev = _rows_of(X, "X"), X.get_device()
    r, ldr = _like(residual, X, "residual")
    with _On(dev, stream) as s:
        if Y is None:
            Y = X.new_empty(X.shape)
            y, ldy = Y.data_ptr(), X.shape[1]
        else:
            y, ldy = _like(Y, X, "output")
        dr, (n, k), lib = C.byref(_lib.Dropout(float(p), 0, int(seed))), X.shape, _lib.load()
        if where == "qlora_dropout_fwd":
            st = lib.qlora_dropout_fwd(X.data_ptr(), ldx, r, ldr, _float_type(X), n, k, dr, int(first),
                                       y, ldy, s)
        else:
            st = lib.qlora_dropout_bwd(X.data_ptr(), ldx, _float_type(X), n, k, dr, int(first), y, ldy,
                                       s)
        _lib.check(st, where)
    return Y


def qlora_dropout_fwd(X, p: float, seed: int, Y, residual=None, first: int = 0, stream=None):
    """Y = dropout(X) + residual with the layer's mask; element (i, j) has
    number first + i * cols + j.  Y may be X or residual."""
    if Y is None:
        raise ValueError("Y is missing")
    _dropout(X, p, seed, Y, residual, first, stream, "qlora_dropout_fwd")


def qlora_dropout_bwd(dY, p: float, seed: int, dX, first: int = 0, stream=None):
    """dX = D c dY with the forward's mask, regenerated."""
    if dX is None:
        raise ValueError("dX is missing")
    _dropout(dY, p, seed, dX, None, first, stream, "qlora_dropout_bwd")


def qlora_check_status(stream=None) -> int:
    """Synchronise the stream; return and clear the device status word."""
    return int(_lib.load().qlora_check_status(_stream(stream)))


def code_table(quant_type: int = _lib.QLORA_QUANT_NF4) -> list[float]:
    buf = (C.c_float * 16)()
    _lib.check(_lib.load().qlora_code_table(int(quant_type), buf), "qlora_code_table")
    return list(buf)


def code_thresholds(quant_type: int = _lib.QLORA_QUANT_NF4) -> list[float]:
    buf = (C.c_float * 15)()
    cnt = C.c_int(0)
    _lib.check(_lib.load().qlora_code_thresholds(int(quant_type), buf, C.byref(cnt)),
               "qlora_code_thresholds")
    return list(buf)[:cnt.value]


# ---------------------------------------------------------------------------
# Conveniences
# ---------------------------------------------------------------------------

def empty_quantized(rows: int, cols: int, device, double_quant: int = 1,
                    quant_type: int = _lib.QLORA_QUANT_NF4) -> NF4Tensor:
    """Buffers of a quantised [rows, cols] weight (absmax is kept either way:
    the quantise pass writes it)."""
    n = rows * cols
    na = n // BLOCKSIZE
    t = NF4Tensor(torch.empty(n // 2, dtype=torch.uint8, device=device), rows, cols,
                  torch.empty(na, dtype=torch.float32, device=device), None, None, None,
                  int(double_quant), quant_type)
    if double_quant:
        t.qabsmax = torch.empty(na, dtype=torch.int8, device=device)
        t.dq_scale = torch.empty((na + DQ_BLOCKSIZE - 1) // DQ_BLOCKSIZE, dtype=torch.float32,
                                 device=device)
        t.dq_mean = torch.empty(4, dtype=torch.float32, device=device)[:1]
    return t


def quantize(W: torch.Tensor, double_quant: int = 1, quant_type: int = _lib.QLORA_QUANT_NF4,
             stream=None) -> NF4Tensor:
    """Quantise W.  double_quant: 0 (or False) keeps fp32 block scales, 1 (or
    True) int8 codes, 2 E4M3 codes; the mean's histogram is built in the
    quantise pass and one more pass writes the 8-bit scales."""
    rows, cols = W.shape
    dq = int(double_quant)
    q = empty_quantized(rows, cols, W.device, dq, quant_type)
    if not dq:
        qlora_quantize_4bit(W, q.packed, q.absmax, quant_type, None, stream)
        return q
    hist = torch.empty(256, dtype=torch.int64, device=W.device)
    qlora_quantize_4bit(W, q.packed, q.absmax, quant_type, hist, stream)
    nf4_double_quantize_hist(q.absmax, hist, q.absmax.numel(), q.qabsmax, q.dq_scale, q.dq_mean,
                             stream, dq_type=dq)
    return q


def dequantize(w: NF4Tensor, stream=None) -> torch.Tensor:
    out = torch.empty(w.rows, w.cols, dtype=torch.bfloat16, device=w.packed.device)
    nf4_dequantize(w, out, stream)
    return out


def merge(w: NF4Tensor, A, B, alpha: float, stream=None) -> torch.Tensor:
    out = torch.empty(w.rows, w.cols, dtype=torch.bfloat16, device=w.packed.device)
    qlora_merge(w, A, B, alpha, out, stream)
    return out


def linear_fwd(w: NF4Tensor, X, A, B, alpha: float, save_T: bool = True, stream=None):
    M, r = X.shape[0], A.shape[0]
    Y = torch.empty(M, w.rows, dtype=torch.bfloat16, device=X.device)
    T = torch.empty(M, r, dtype=torch.bfloat16, device=X.device) if save_T else None
    qlora_linear_fwd(w, X, A, B, alpha, Y, T, stream=stream)
    return Y, T


def linear_fwd_dropout(w: NF4Tensor, X, A, B, alpha: float, p: float, seed: int,
                       save_T: bool = True, stream=None):
    M, r = X.shape[0], A.shape[0]
    Y = torch.empty(M, w.rows, dtype=torch.bfloat16, device=X.device)
    T = torch.empty(M, r, dtype=torch.bfloat16, device=X.device) if save_T else None
    qlora_linear_fwd_dropout(w, X, A, B, alpha, p, seed, Y, T, stream=stream)
    return Y, T


def linear_bwd_dropout(w: NF4Tensor, X, dY, A, B, alpha: float, p: float, seed: int, T=None,
                       stream=None):
    dX = torch.empty_like(X)
    dA = torch.empty_like(A)
    dB = torch.empty_like(B)
    qlora_linear_bwd_dropout(w, X, dY, A, B, alpha, p, seed, dX, dA, dB, T=T, stream=stream)
    return dX, dA, dB


def linear_bwd(w: NF4Tensor, X, dY, A, B, alpha: float, T=None, stream=None):
    dX = torch.empty_like(X)
    dA = torch.empty_like(A)
    dB = torch.empty_like(B)
    qlora_linear_bwd(w, X, dY, A, B, alpha, dX, dA, dB, T=T, stream=stream)
    return dX, dA, dB


def mx_empty(rows: int, cols: int, device, format: int = _lib.QLORA_NVFP4) -> MXTensor:
    """Buffers of a microscaled [rows, cols] matrix."""
    nv = format == _lib.QLORA_NVFP4
    return MXTensor(torch.empty(rows * cols // 2, dtype=torch.uint8, device=device),
                    torch.empty(mx_scale_bytes(format, rows, cols), dtype=torch.uint8, device=device),
                    torch.empty(rows, dtype=torch.float32, device=device) if nv else None,
                    rows, cols, int(format))


def mx_quantize(X: torch.Tensor, format: int = _lib.QLORA_NVFP4, stream=None) -> MXTensor:
    """Quantise a weight or activations: format 0 MXFP4, 1 NVFP4."""
    return _mx_quantize(X, None, int(format), stream)


def mx_dequantize(t: MXTensor, stream=None) -> torch.Tensor:
    return _mx_dequantize(t, None, stream)


def mx_matmul(x: MXTensor, w: MXTensor, stream=None) -> torch.Tensor:
    return _mx_matmul(x, w, None, stream)


def mx_linear_fwd(w: MXTensor, X, A=None, B=None, alpha: float = 0.0, p: float = 0.0, seed: int = 0,
                  save_T: bool = True, stream=None):
    """(Y, T) of the layer on a microscaled base; T is None without an adapter."""
    return _mx_fwd(w, X, A, B, alpha, None, None, save_T, p, seed, None, stream)


def mx_linear_bwd(w: MXTensor, X, dY, A=None, B=None, alpha: float = 0.0, p: float = 0.0,
                  seed: int = 0, T=None, stream=None):
    """(dX, dA, dB); dA and dB are None without an adapter."""
    return _mx_bwd(w, X, dY, A, B, alpha, None, None, None, T, p, seed, None, stream)


def dropout_fwd(X, p: float, seed: int, residual=None, first: int = 0, stream=None) -> torch.Tensor:
    """dropout(X) (+ residual) with the mask of the layer's dropout."""
    return _dropout(X, p, seed, None, residual, first, stream, "qlora_dropout_fwd")


def dropout_bwd(dY, p: float, seed: int, first: int = 0, stream=None) -> torch.Tensor:
    return _dropout(dY, p, seed, None, None, first, stream, "qlora_dropout_bwd")
