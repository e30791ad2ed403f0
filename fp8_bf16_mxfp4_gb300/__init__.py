"""GB300 grouped microscaled (MX) GEMM library -- Python binding.

Argument marshalling only: every computation runs in libmxg.so (CUDA kernels
for sm_103a) through its C ABI (include/mxg.h).  PyTorch provides device
memory and the current stream.  There is no CPU fallback: without the built
library or a GPU these functions raise.

Layouts (row-major, K-major operands):
  * E2M1 codes: uint8 [rows, cols/2], element 2j in the low nibble.
  * E4M3 codes: uint8 [rows, cols].
  * UE8M0 scales: uint8 [rows, cols/32] (one per 32 elements along cols).
"""

from __future__ import annotations

import ctypes
import functools
import threading
from dataclasses import dataclass

import torch
from torch.autograd.graph import increment_version

from . import _lib

__all__ = [
    "MXOperand", "MXGError", "mx_quantize_rowwise", "mx_quantize_colwise_segment_padded",
    "mx_quantize_rowwise_packed", "mx_packed_scale_bytes", "mx_packed_colwise_scale_bytes",
    "mx_quantize_dual_segment_padded",
    "grouped_gemm_fwd", "grouped_gemm_dgrad", "grouped_gemm_wgrad", "gemm_workspace_size", "mx_gemm_dense",
    "mx_padded_rows_capacity", "check_status", "status_tensor", "set_wait_timeout_ns", "set_gemm_cta_group",
    "library_path", "BWOperand", "bw_quantize_1x128", "bw_quantize_128x128",
    "bw_quantize_colwise_padded", "bw_grouped_gemm_fwd", "bw_grouped_gemm_dgrad",
    "bw_grouped_gemm_wgrad", "bw_quantize_1x128_pow2", "bw_quantize_128x128_pow2",
    "bw_quantize_colwise_padded_pow2", "bw_quantize_dual_padded",
    "moe_route", "moe_experts", "moe_experts_workspace_size", "lora_add", "lora_add_workspace_size",
    "moe_sort", "moe_sort_workspace_size", "moe_gather", "moe_combine", "moe_combine_backward", "moe_route_backward",
    "Int8Operand", "int8_quantize_rowwise", "int8_grouped_gemm_fwd", "int8_gemm_dense", "int8_gemm_workspace_size",
]

ELEM = {"e2m1": 1, "e4m3": 2}
SCALE_LAYOUT = {"plain": 0, "packed": 1}
PASS = {"fwd": 0, "dgrad": 1, "wgrad": 2}
_OUT = {torch.bfloat16: 1, torch.float32: 2}

library_path = _lib.LIB_PATH


class MXGError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        msg = _lib.load().mxg_status_string(code).decode()
        super().__init__(f"{what}: {msg} (status {code})")


def _ok(code: int, what: str):
    if code != 0:
        raise MXGError(code, what)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(dev) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("libmxg operates on CUDA tensors only")


@dataclass
class MXOperand:
    """A quantized K-major operand: codes, UE8M0 scales, element format and
    logical column count (the contraction length).  ``scale_layout`` "plain"
    means scales [rows, cols/32]; "packed" means the tensor-core staging order
    of ``mx_quantize_rowwise_packed`` (a flat uint8 tensor)."""
    data: torch.Tensor
    scale: torch.Tensor
    elem: str
    cols: int
    scale_layout: str = "plain"

    @property
    def rows(self) -> int:
        return self.data.shape[0]

    def c(self) -> _lib.MxOperandC:
        packed = self.scale_layout == "packed"
        return _lib.MxOperandC(self.data.data_ptr(), self.scale.data_ptr(), self.rows, self.cols,
                               _ld(self.data, _codes_cols(self.elem, self.cols)),
                               0 if packed else _ld(self.scale, self.cols // 32), ELEM[self.elem],
                               SCALE_LAYOUT[self.scale_layout])


def _ld(t: torch.Tensor, row_elems: int) -> int:
    """Row stride in elements.  Zero-size tensors and tensors with a single
    row report arbitrary strides (the stride is never used for them), so their
    logical contiguous stride is passed instead."""
    if t.numel() == 0 or t.shape[0] <= 1:
        return max(row_elems, 16)
    return t.stride(0)


_status = {}


def status_tensor(device) -> torch.Tensor:
    """Per-device int32 status word used when the caller passes none."""
    d = torch.device(device)
    idx = d.index if d.index is not None else torch.cuda.current_device()
    if idx not in _status:
        _status[idx] = torch.zeros(1, dtype=torch.int32, device=f"cuda:{idx}")
    return _status[idx]


def check_status(status: torch.Tensor | None = None, device=None) -> int:
    """Synchronise, read and clear the device status word; raise on error."""
    st = status if status is not None else status_tensor(device or torch.cuda.current_device())
    code = _lib.load().mxg_check_status(_ptr(st), _stream(st.device))
    _ok(code, "device-side check")
    return code


def set_wait_timeout_ns(ns: int):
    _lib.load().mxg_set_wait_timeout_ns(int(ns))


def set_gemm_cta_group(n: int) -> int:
    """Choose the MX GEMM kernel: 2 = CTA pairs sharing each 256x256 tile
    (the default), 1 = the one-SM kernel.  Returns the previous choice."""
    lib = _lib.load()
    prev = int(lib.mxg_get_gemm_cta_group())
    _ok(lib.mxg_set_gemm_cta_group(int(n)), "set_gemm_cta_group")
    return prev


def mx_padded_rows_capacity(rows: int, G: int, pad: int) -> int:
    return int(_lib.load().mx_padded_rows_capacity(rows, G, pad))


def _codes_cols(elem: str, cols: int) -> int:
    return cols // 2 if elem == "e2m1" else cols


SCALE_RULES = {"ocp": 0, "round_up": 0x100}  # MXG_SCALE_ROUND_UP


def _quant_elem(elem: str, rule: str) -> int:
    """The quantizers' elem argument: format code with the scale-rule flag."""
    if rule not in SCALE_RULES:
        raise ValueError(f"unknown scale rule {rule!r} (ocp or round_up)")
    return ELEM[elem] | SCALE_RULES[rule]


def mx_quantize_rowwise(x: torch.Tensor, elem: str, q: torch.Tensor | None = None,
                        s: torch.Tensor | None = None, rule: str = "ocp") -> MXOperand:
    """BF16 [rows, cols] -> MX operand quantized along cols."""
    _need_cuda(x)
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    rows, cols = x.shape
    if q is None:
        q = torch.empty((rows, _codes_cols(elem, cols)), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty((rows, cols // 32), dtype=torch.uint8, device=x.device)
    lib = _lib.load()
    _ok(lib.mx_quantize_rowwise(_ptr(x), rows, cols, _ld(x, cols), _quant_elem(elem, rule), _ptr(q),
                                _ld(q, _codes_cols(elem, cols)), _ptr(s), _ld(s, cols // 32),
                                _stream(x.device)), "mx_quantize_rowwise")
    return MXOperand(q, s, elem, cols)


def mx_packed_scale_bytes(rows: int, cols: int, G: int) -> int:
    """Bytes of packed scales for `rows` x `cols` cut into G segments (an upper
    bound over every split)."""
    return int(_lib.load().mx_packed_scale_bytes(rows, cols, G))


def mx_packed_colwise_scale_bytes(cols: int, capacity: int, G: int) -> int:
    """Bytes of packed scales of a column-wise operand with `cols` channels and
    `capacity` padded positions over G experts (an upper bound over splits)."""
    return int(_lib.load().mx_packed_colwise_scale_bytes(cols, capacity, G))


def mx_quantize_rowwise_packed(x: torch.Tensor, elem: str, m_splits: torch.Tensor | None = None,
                               groups: int | None = None, status: torch.Tensor | None = None,
                               check: bool = False, rule: str = "ocp") -> MXOperand:
    """BF16 [rows, cols] -> MX operand whose scales are already in the grouped
    GEMM's tensor-core staging order (no repacking pass in the GEMM).  Rows
    are cut into segments by the device ``m_splits`` (activations and
    gradients), or into ``groups`` equal segments (forward weights: G experts
    of N rows).  The GEMM call must use the same segments."""
    _need_cuda(x, m_splits)
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    if (m_splits is None) == (groups is None):
        raise ValueError("give exactly one of m_splits and groups")
    rows, cols = x.shape
    G = m_splits.numel() if m_splits is not None else int(groups)
    if m_splits is not None and m_splits.dtype != torch.int32:
        raise ValueError("m_splits must be int32")
    nbytes = mx_packed_scale_bytes(rows, cols, G)
    if nbytes < 0:
        raise ValueError("invalid shape for packed scales")
    q = torch.empty((rows, _codes_cols(elem, cols)), dtype=torch.uint8, device=x.device)
    s = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=x.device)
    st = status if status is not None else status_tensor(x.device)
    lib = _lib.load()
    _ok(lib.mx_quantize_rowwise_packed(_ptr(x), rows, cols, _ld(x, cols), _quant_elem(elem, rule), _ptr(q),
                                       _ld(q, _codes_cols(elem, cols)), _ptr(s), s.numel(),
                                       _ptr(m_splits), G, _ptr(st),
                                       _stream(x.device)), "mx_quantize_rowwise_packed")
    if check:
        check_status(st)
    return MXOperand(q, s, elem, cols, "packed")


def mx_quantize_colwise_segment_padded(x: torch.Tensor, m_splits: torch.Tensor, pad_multiple: int,
                                       elem: str, capacity: int | None = None,
                                       status: torch.Tensor | None = None, check: bool = False,
                                       rule: str = "ocp", packed: bool = False):
    """BF16 [S, C] with experts' rows concatenated -> (operand [C, capacity],
    int64 padded offsets [G+1]).  Columns beyond the last expert's padded end
    are left uninitialised.  With ``packed`` the scales are written in the
    grouped GEMM's staging order (a flat uint8 tensor; the GEMM call must use
    the same splits and pad)."""
    _need_cuda(x, m_splits)
    S, C = x.shape
    G = m_splits.numel()
    if capacity is None:
        capacity = mx_padded_rows_capacity(S, G, pad_multiple)
    qT = torch.empty((C, _codes_cols(elem, capacity)), dtype=torch.uint8, device=x.device)
    poff = torch.empty(G + 1, dtype=torch.int64, device=x.device)
    st = status if status is not None else status_tensor(x.device)
    lib = _lib.load()
    if packed:
        nbytes = mx_packed_colwise_scale_bytes(C, capacity, G)
        if nbytes < 0:
            raise ValueError("invalid shape for packed scales")
        sp = torch.empty((max(nbytes, 16),), dtype=torch.uint8, device=x.device)
        _ok(lib.mx_quantize_colwise_segment_padded_packed(
            _ptr(x), S, C, _ld(x, C), _ptr(m_splits), G, pad_multiple, _quant_elem(elem, rule), _ptr(qT),
            _ld(qT, _codes_cols(elem, capacity)), _ptr(sp), sp.numel(), capacity, _ptr(poff), _ptr(st),
            _stream(x.device)), "mx_quantize_colwise_segment_padded_packed")
        if check:
            check_status(st)
        return MXOperand(qT, sp, elem, capacity, "packed"), poff
    sT = torch.empty((C, capacity // 32), dtype=torch.uint8, device=x.device)
    _ok(lib.mx_quantize_colwise_segment_padded(
        _ptr(x), S, C, _ld(x, C), _ptr(m_splits), G, pad_multiple, _quant_elem(elem, rule), _ptr(qT),
        _ld(qT, _codes_cols(elem, capacity)), _ptr(sT), _ld(sT, capacity // 32), capacity,
        _ptr(poff), _ptr(st), _stream(x.device)),
        "mx_quantize_colwise_segment_padded")
    if check:
        check_status(st)
    return MXOperand(qT, sT, elem, capacity), poff


def mx_quantize_dual_segment_padded(x: torch.Tensor, m_splits: torch.Tensor, pad_multiple: int,
                                    elem: str, capacity: int | None = None,
                                    q: torch.Tensor | None = None, s: torch.Tensor | None = None,
                                    status: torch.Tensor | None = None, check: bool = False,
                                    rule: str = "ocp"):
    """BF16 [S, C] -> (row-wise operand [S, C], column-wise operand
    [C, capacity], int64 padded offsets [G+1]) from one read of x; the same
    bytes as mx_quantize_rowwise plus mx_quantize_colwise_segment_padded."""
    _need_cuda(x, m_splits)
    if x.dtype != torch.bfloat16 or x.dim() != 2:
        raise ValueError("x must be a 2-D bfloat16 tensor")
    S, C = x.shape
    G = m_splits.numel()
    if capacity is None:
        capacity = mx_padded_rows_capacity(S, G, pad_multiple)
    if q is None:
        q = torch.empty((S, _codes_cols(elem, C)), dtype=torch.uint8, device=x.device)
    if s is None:
        s = torch.empty((S, C // 32), dtype=torch.uint8, device=x.device)
    qT = torch.empty((C, _codes_cols(elem, capacity)), dtype=torch.uint8, device=x.device)
    sT = torch.empty((C, capacity // 32), dtype=torch.uint8, device=x.device)
    poff = torch.empty(G + 1, dtype=torch.int64, device=x.device)
    st = status if status is not None else status_tensor(x.device)
    lib = _lib.load()
    _ok(lib.mx_quantize_dual_segment_padded(
        _ptr(x), S, C, _ld(x, C), _ptr(m_splits), G, pad_multiple, _quant_elem(elem, rule), _ptr(q),
        _ld(q, _codes_cols(elem, C)), _ptr(s), _ld(s, C // 32), _ptr(qT),
        _ld(qT, _codes_cols(elem, capacity)), _ptr(sT), _ld(sT, capacity // 32), capacity,
        _ptr(poff), _ptr(st), _stream(x.device)),
        "mx_quantize_dual_segment_padded")
    if check:
        check_status(st)
    return MXOperand(q, s, elem, C), MXOperand(qT, sT, elem, capacity), poff


def gemm_workspace_size(pass_: str, G: int, S: int, N: int, K: int, pad: int = 32) -> int:
    return int(_lib.load().mxg_gemm_workspace_size(PASS[pass_], G, S, N, K, pad))


def _workspace(nbytes: int, device, ws: torch.Tensor | None):
    if ws is not None:
        return ws
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def grouped_gemm_fwd(A: MXOperand, W: MXOperand, m_splits: torch.Tensor, N: int,
                     out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                     check: bool = False) -> torch.Tensor:
    """Y[off_g+i, :] = A[off_g+i, :] @ W[g*N:(g+1)*N, :]^T for every expert g."""
    _need_cuda(A.data, W.data, m_splits)
    G = m_splits.numel()
    dev = A.data.device
    if out is None:
        out = torch.empty((A.rows, N), dtype=out_dtype, device=dev)
    need = gemm_workspace_size("fwd", G, A.rows, N, A.cols)
    ws = _workspace(need, dev, workspace)
    st = status if status is not None else status_tensor(dev)
    a, w = A.c(), W.c()
    _ok(_lib.load().grouped_gemm_fwd(ctypes.byref(a), ctypes.byref(w), _ptr(m_splits), G, N,
                                     _ptr(out), _ld(out, N), _OUT[out.dtype], _ptr(ws),
                                     ws.numel(), _ptr(st), _stream(dev)), "grouped_gemm_fwd")
    if check:
        check_status(st)
    return out


def mx_gemm_dense(A: MXOperand, B: MXOperand, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                  check: bool = False) -> torch.Tensor:
    """C[M, N] = A[M, K] @ B[N, K]^T, both MX operands quantized along K (no
    experts, no m_splits)."""
    _need_cuda(A.data, B.data)
    dev = A.data.device
    N = B.rows
    if out is None:
        out = torch.empty((A.rows, N), dtype=out_dtype, device=dev)
    need = gemm_workspace_size("fwd", 1, A.rows, N, A.cols)
    ws = _workspace(need, dev, workspace)
    st = status if status is not None else status_tensor(dev)
    a, b = A.c(), B.c()
    _ok(_lib.load().mx_gemm_dense(ctypes.byref(a), ctypes.byref(b), _ptr(out), _ld(out, N), _OUT[out.dtype],
                                  _ptr(ws), ws.numel(), _ptr(st), _stream(dev)), "mx_gemm_dense")
    if check:
        check_status(st)
    return out


def grouped_gemm_dgrad(dY: MXOperand, Wt: MXOperand, m_splits: torch.Tensor,
                       out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                       check: bool = False) -> torch.Tensor:
    """dX[off_g+i, :] = dY[off_g+i, :] @ Wt[:, g*N:(g+1)*N]^T (Wt = W^T quantized along N)."""
    _need_cuda(dY.data, Wt.data, m_splits)
    G = m_splits.numel()
    dev = dY.data.device
    K = Wt.rows
    if out is None:
        out = torch.empty((dY.rows, K), dtype=out_dtype, device=dev)
    need = gemm_workspace_size("dgrad", G, dY.rows, dY.cols, K)
    ws = _workspace(need, dev, workspace)
    st = status if status is not None else status_tensor(dev)
    a, b = dY.c(), Wt.c()
    _ok(_lib.load().grouped_gemm_dgrad(ctypes.byref(a), ctypes.byref(b), _ptr(m_splits), G,
                                       _ptr(out), _ld(out, K), _OUT[out.dtype], _ptr(ws),
                                       ws.numel(), _ptr(st), _stream(dev)), "grouped_gemm_dgrad")
    if check:
        check_status(st)
    return out


def grouped_gemm_wgrad(dYt: MXOperand, Xt: MXOperand, m_splits: torch.Tensor, total_rows: int,
                       pad_multiple: int, out: torch.Tensor | None = None,
                       out_dtype=torch.float32, accumulate: bool = False,
                       workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                       check: bool = False) -> torch.Tensor:
    """dW[g] (+)= dYt[:, seg_g] @ Xt[:, seg_g]^T over expert g's padded token
    segment; out is [G, N, K]."""
    _need_cuda(dYt.data, Xt.data, m_splits)
    G = m_splits.numel()
    dev = dYt.data.device
    N, K = dYt.rows, Xt.rows
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an existing out tensor")
        out = torch.empty((G, N, K), dtype=out_dtype, device=dev)
    need = gemm_workspace_size("wgrad", G, dYt.cols, N, K, pad_multiple)
    ws = _workspace(need, dev, workspace)
    st = status if status is not None else status_tensor(dev)
    a, b = dYt.c(), Xt.c()
    _ok(_lib.load().grouped_gemm_wgrad(ctypes.byref(a), ctypes.byref(b), _ptr(m_splits), G,
                                       total_rows, pad_multiple, _ptr(out), _OUT[out.dtype],
                                       1 if accumulate else 0, _ptr(ws), ws.numel(), _ptr(st),
                                       _stream(dev)), "grouped_gemm_wgrad")
    if check:
        check_status(st)
    return out


# ----------------------------------------------------------------------------- blockwise FP8


@dataclass
class BWOperand:
    """Blockwise-FP8 K-major operand: E4M3 codes [rows, cols] and fp32 scales
    (activation-type [cols/128, >= rows] or weight-type [rows/128, cols/128])."""
    data: torch.Tensor
    scale: torch.Tensor

    @property
    def rows(self) -> int:
        return self.data.shape[0]

    @property
    def cols(self) -> int:
        return self.data.shape[1]

    def c(self) -> _lib.BwOperandC:
        return _lib.BwOperandC(self.data.data_ptr(), self.scale.data_ptr(), self.rows, self.cols,
                               _ld(self.data, self.cols), _ld(self.scale, self.scale.shape[-1]),
                               0, 0)


def bw_quantize_1x128(x: torch.Tensor) -> BWOperand:
    """BF16 [rows, cols] -> E4M3 [rows, cols] + activation-type scales [cols/128, rows]."""
    _need_cuda(x)
    R, C = x.shape
    q = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    s = torch.empty((C // 128, R), dtype=torch.float32, device=x.device)
    _ok(_lib.load().bw_quantize_1x128(_ptr(x), R, C, _ld(x, C), _ptr(q), _ld(q, C), _ptr(s),
                                      _ld(s, R), _stream(x.device)), "bw_quantize_1x128")
    return BWOperand(q, s)


def bw_quantize_128x128(w: torch.Tensor, transposed: bool = True):
    """BF16 weights [rows, cols] -> (operand with weight-type scales, and when
    `transposed` the dgrad copy [cols, rows] with its scales)."""
    _need_cuda(w)
    R, C = w.shape
    dev = w.device
    q = torch.empty((R, C), dtype=torch.uint8, device=dev)
    s = torch.empty((R // 128, C // 128), dtype=torch.float32, device=dev)
    qT = torch.empty((C, R), dtype=torch.uint8, device=dev) if transposed else None
    sT = torch.empty((C // 128, R // 128), dtype=torch.float32, device=dev) if transposed else None
    _ok(_lib.load().bw_quantize_128x128(_ptr(w), R, C, _ld(w, C), _ptr(q), _ld(q, C), _ptr(s),
                                        _ptr(qT), _ld(qT, R) if transposed else 0, _ptr(sT),
                                        _stream(dev)), "bw_quantize_128x128")
    return BWOperand(q, s), (BWOperand(qT, sT) if transposed else None)


def bw_quantize_colwise_padded(x: torch.Tensor, m_splits: torch.Tensor, capacity: int | None = None,
                               status: torch.Tensor | None = None, check: bool = False):
    """BF16 [S, C] -> (operand [C, capacity] with activation-type scales
    [capacity/128, C], int64 padded offsets [G+1]); segments padded to 128."""
    _need_cuda(x, m_splits)
    S, C = x.shape
    G = m_splits.numel()
    if capacity is None:
        capacity = mx_padded_rows_capacity(S, G, 128)
    qT = torch.empty((C, capacity), dtype=torch.uint8, device=x.device)
    sT = torch.empty((capacity // 128, C), dtype=torch.float32, device=x.device)
    poff = torch.empty(G + 1, dtype=torch.int64, device=x.device)
    st = status if status is not None else status_tensor(x.device)
    _ok(_lib.load().bw_quantize_colwise_padded(
        _ptr(x), S, C, _ld(x, C), _ptr(m_splits), G, _ptr(qT), _ld(qT, capacity), _ptr(sT),
        _ld(sT, C), capacity, _ptr(poff), _ptr(st), _stream(x.device)), "bw_quantize_colwise_padded")
    if check:
        check_status(st)
    return BWOperand(qT, sT), poff


def bw_quantize_1x128_pow2(x: torch.Tensor) -> MXOperand:
    """BF16 [rows, cols] -> blockwise FP8 (1x128, power-of-two scales) as an
    MXFP8 operand: E4M3 [rows, cols] + UE8M0 [rows, cols/32]."""
    _need_cuda(x)
    R, C = x.shape
    q = torch.empty((R, C), dtype=torch.uint8, device=x.device)
    s = torch.empty((R, C // 32), dtype=torch.uint8, device=x.device)
    _ok(_lib.load().bw_quantize_1x128_pow2(_ptr(x), R, C, _ld(x, C), _ptr(q), _ld(q, C), _ptr(s),
                                           _ld(s, C // 32), _stream(x.device)), "bw_quantize_1x128_pow2")
    return MXOperand(q, s, "e4m3", C)


def bw_quantize_128x128_pow2(w: torch.Tensor, transposed: bool = True):
    """BF16 weights [rows, cols] -> (MXFP8 operand with 128x128 power-of-two
    scales, and when `transposed` the dgrad copy [cols, rows])."""
    _need_cuda(w)
    R, C = w.shape
    dev = w.device
    q = torch.empty((R, C), dtype=torch.uint8, device=dev)
    s = torch.empty((R, C // 32), dtype=torch.uint8, device=dev)
    qT = torch.empty((C, R), dtype=torch.uint8, device=dev) if transposed else None
    sT = torch.empty((C, R // 32), dtype=torch.uint8, device=dev) if transposed else None
    _ok(_lib.load().bw_quantize_128x128_pow2(
        _ptr(w), R, C, _ld(w, C), _ptr(q), _ld(q, C), _ptr(s), _ld(s, C // 32), _ptr(qT),
        _ld(qT, R) if transposed else 0, _ptr(sT), _ld(sT, R // 32) if transposed else 0, _stream(dev)),
        "bw_quantize_128x128_pow2")
    return MXOperand(q, s, "e4m3", C), (MXOperand(qT, sT, "e4m3", R) if transposed else None)


def bw_quantize_colwise_padded_pow2(x: torch.Tensor, m_splits: torch.Tensor, capacity: int | None = None,
                                    status: torch.Tensor | None = None, check: bool = False):
    """BF16 [S, C] -> (MXFP8 operand [C, capacity], segments padded to 128,
    power-of-two 1x128 scales as UE8M0 [C, capacity/32]; int64 padded offsets)."""
    _need_cuda(x, m_splits)
    S, C = x.shape
    G = m_splits.numel()
    if capacity is None:
        capacity = mx_padded_rows_capacity(S, G, 128)
    qT = torch.empty((C, capacity), dtype=torch.uint8, device=x.device)
    sT = torch.empty((C, capacity // 32), dtype=torch.uint8, device=x.device)
    poff = torch.empty(G + 1, dtype=torch.int64, device=x.device)
    st = status if status is not None else status_tensor(x.device)
    _ok(_lib.load().bw_quantize_colwise_padded_pow2(
        _ptr(x), S, C, _ld(x, C), _ptr(m_splits), G, _ptr(qT), _ld(qT, capacity), _ptr(sT),
        _ld(sT, capacity // 32), capacity, _ptr(poff), _ptr(st), _stream(x.device)),
        "bw_quantize_colwise_padded_pow2")
    if check:
        check_status(st)
    return MXOperand(qT, sT, "e4m3", capacity), poff


def bw_quantize_dual_padded(x: torch.Tensor, m_splits: torch.Tensor, capacity: int | None = None,
                            pow2: bool = False, status: torch.Tensor | None = None, check: bool = False):
    """One read of BF16 x [S, C] -> (row-wise 1x128 operand, column-wise
    operand [C, capacity] with segments padded to 128, int64 padded offsets):
    the same bytes as the separate row-wise and column-wise quantizers.  With
    pow2 both are MXFP8 operands (UE8M0 power-of-two scales); otherwise
    BWOperands with fp32 activation-type scales."""
    _need_cuda(x, m_splits)
    S, C = x.shape
    G = m_splits.numel()
    dev = x.device
    if capacity is None:
        capacity = mx_padded_rows_capacity(S, G, 128)
    q = torch.empty((S, C), dtype=torch.uint8, device=dev)
    qT = torch.empty((C, capacity), dtype=torch.uint8, device=dev)
    if pow2:
        s = torch.empty((S, C // 32), dtype=torch.uint8, device=dev)
        sT = torch.empty((C, capacity // 32), dtype=torch.uint8, device=dev)
        ld_s, ld_sT = _ld(s, C // 32), _ld(sT, capacity // 32)
    else:
        s = torch.empty((C // 128, S), dtype=torch.float32, device=dev)
        sT = torch.empty((capacity // 128, C), dtype=torch.float32, device=dev)
        ld_s, ld_sT = _ld(s, S), _ld(sT, C)
    poff = torch.empty(G + 1, dtype=torch.int64, device=dev)
    st = status if status is not None else status_tensor(dev)
    fn = _lib.load().bw_quantize_dual_padded_pow2 if pow2 else _lib.load().bw_quantize_dual_padded
    _ok(fn(_ptr(x), S, C, _ld(x, C), _ptr(m_splits), G, _ptr(q), _ld(q, C), _ptr(s), ld_s, _ptr(qT),
           _ld(qT, capacity), _ptr(sT), ld_sT, capacity, _ptr(poff), _ptr(st), _stream(dev)),
        "bw_quantize_dual_padded")
    if check:
        check_status(st)
    if pow2:
        return MXOperand(q, s, "e4m3", C), MXOperand(qT, sT, "e4m3", capacity), poff
    return BWOperand(q, s), BWOperand(qT, sT), poff


def _bw_ws(G, device, ws):
    if ws is not None:
        return ws
    return torch.empty(max(int(_lib.load().bw_gemm_workspace_size(G)), 256), dtype=torch.uint8,
                       device=device)


def bw_grouped_gemm_fwd(A: BWOperand, W: BWOperand, m_splits: torch.Tensor, N: int,
                        out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                        check: bool = False) -> torch.Tensor:
    _need_cuda(A.data, W.data, m_splits)
    G = m_splits.numel()
    dev = A.data.device
    if out is None:
        out = torch.empty((A.rows, N), dtype=out_dtype, device=dev)
    ws = _bw_ws(G, dev, workspace)
    st = status if status is not None else status_tensor(dev)
    a, w = A.c(), W.c()
    _ok(_lib.load().bw_grouped_gemm_fwd(ctypes.byref(a), ctypes.byref(w), _ptr(m_splits), G, N,
                                        _ptr(out), _ld(out, N), _OUT[out.dtype], _ptr(ws),
                                        ws.numel(), _ptr(st), _stream(dev)), "bw_grouped_gemm_fwd")
    if check:
        check_status(st)
    return out


def bw_grouped_gemm_dgrad(dY: BWOperand, Wt: BWOperand, m_splits: torch.Tensor,
                          out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                          check: bool = False) -> torch.Tensor:
    _need_cuda(dY.data, Wt.data, m_splits)
    G = m_splits.numel()
    dev = dY.data.device
    K = Wt.rows
    if out is None:
        out = torch.empty((dY.rows, K), dtype=out_dtype, device=dev)
    ws = _bw_ws(G, dev, workspace)
    st = status if status is not None else status_tensor(dev)
    a, b = dY.c(), Wt.c()
    _ok(_lib.load().bw_grouped_gemm_dgrad(ctypes.byref(a), ctypes.byref(b), _ptr(m_splits), G,
                                          _ptr(out), _ld(out, K), _OUT[out.dtype], _ptr(ws),
                                          ws.numel(), _ptr(st), _stream(dev)), "bw_grouped_gemm_dgrad")
    if check:
        check_status(st)
    return out


def bw_grouped_gemm_wgrad(dYt: BWOperand, Xt: BWOperand, m_splits: torch.Tensor, total_rows: int,
                          out: torch.Tensor | None = None, out_dtype=torch.float32,
                          accumulate: bool = False, workspace: torch.Tensor | None = None,
                          status: torch.Tensor | None = None, check: bool = False) -> torch.Tensor:
    _need_cuda(dYt.data, Xt.data, m_splits)
    G = m_splits.numel()
    dev = dYt.data.device
    N, K = dYt.rows, Xt.rows
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs an existing out tensor")
        out = torch.empty((G, N, K), dtype=out_dtype, device=dev)
    ws = _bw_ws(G, dev, workspace)
    st = status if status is not None else status_tensor(dev)
    a, b = dYt.c(), Xt.c()
    _ok(_lib.load().bw_grouped_gemm_wgrad(ctypes.byref(a), ctypes.byref(b), _ptr(m_splits), G,
                                          total_rows, _ptr(out), _OUT[out.dtype],
                                          1 if accumulate else 0, _ptr(ws), ws.numel(), _ptr(st),
                                          _stream(dev)), "bw_grouped_gemm_wgrad")
    if check:
        check_status(st)
    return out


# ----------------------------------------------------------------------------- serving
#
# These calls take microseconds on the device, so their checks are single
# comparisons on the way through; what is wrong is worked out only on failure.


def _raw_stream(dev) -> int:
    return torch._C._cuda_getCurrentRawStream(dev.index)


class _Scratch(threading.local):
    def __init__(self):
        self.buffers = {}


_scratch_kept = _Scratch()
_SCRATCH_KEEP = 64 << 20


def _scratch(nbytes: int, dev, stream: int) -> torch.Tensor:
    """A call's workspace when the caller gives none.  An allocation costs as
    much host time as the launches, so each thread keeps one buffer of up to
    64 MiB for each stream (a thread's calls on a stream are ordered, and each
    writes what it reads; calls of two threads interleave); a captured graph
    gets memory of its own pool."""
    if nbytes <= _SCRATCH_KEEP and not torch._C._cuda_isCurrentStreamCapturing():
        kept = _scratch_kept.buffers
        key = (dev.index, stream)
        buf = kept.get(key)
        if buf is None or buf.numel() < nbytes:
            buf = kept[key] = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=dev)
        return buf
    return torch.empty(nbytes, dtype=torch.uint8, device=dev)


def _status_ptr(status, dev) -> int:
    if status is not None:
        if status.dtype != torch.int32:
            raise ValueError("status must be int32")
        return status.data_ptr()
    st = _status.get(dev.index)
    return (st if st is not None else status_tensor(dev)).data_ptr()


def _row_ld(t: torch.Tensor, cols: int) -> int:
    """Row stride of a 2-D tensor; its rows must be contiguous.  A tensor of at
    most one row reports arbitrary strides: its width, rounded up to 8."""
    rows = t.shape[0]
    if rows > 0 and cols > 1 and t.stride(1) != 1:
        raise ValueError("elements of a row must be contiguous")
    return t.stride(0) if rows > 1 else (cols + 7) & ~7


def _refuse(**named):
    """Raise for the first argument that is not what it has to be: name =
    (tensor, shape, dtype or dtypes, contiguous)."""
    for name, (t, shape, dtypes, contiguous) in named.items():
        if t is None:
            continue
        dtypes = dtypes if isinstance(dtypes, (tuple, dict)) else (dtypes,)
        if not t.is_cuda:
            raise ValueError("libmxg operates on CUDA tensors only")
        if tuple(t.shape) != tuple(shape) or t.dtype not in dtypes:
            raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)} of shape {list(shape)}, "
                             f"got {t.dtype} of shape {list(t.shape)}")
        if contiguous and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    raise ValueError("arguments do not fit together")


def _refuse_grad(name: str):
    """No gradient goes through these calls: an input that asks for one is refused instead of being detached."""
    if torch.is_grad_enabled():
        raise ValueError(f"{name} is forward only and an input requires grad: detach it, or call under torch.no_grad()")


def _written(t: torch.Tensor):
    """Tell autograd that the caller's tensor was written, as torch's in-place operations do."""
    if not t.is_inference():
        increment_version(t)


def moe_route(logits: torch.Tensor, top_k: int, renormalize: bool = True, ids: torch.Tensor | None = None,
              weights: torch.Tensor | None = None):
    """Router logits [T, E] (BF16 or FP32) -> (int32 ids [T, top_k], FP32
    weights [T, top_k]): each token's top_k experts, largest logit first and
    equal logits in index order, with their softmax weights -- over the chosen
    experts (``renormalize``) or over all of them.  Experts whose logit is -inf
    or NaN are never chosen; slots left over have id -1 and weight 0.
    Forward only."""
    if logits.dim() != 2:
        raise ValueError("logits must be [tokens, experts]")
    if logits.requires_grad or (weights is not None and weights.requires_grad):
        _refuse_grad("moe_route")
    T, E = logits.shape
    dtype = _OUT.get(logits.dtype)
    dev = logits.device
    if dtype is None or not logits.is_cuda:
        _refuse(logits=(logits, (T, E), _OUT, False))
    ids_given, weights_given = ids, weights
    if ids is None:
        ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    elif ids.shape != (T, top_k) or ids.dtype != torch.int32 or not ids.is_contiguous() or not ids.is_cuda:
        _refuse(ids=(ids, (T, top_k), torch.int32, True))
    if weights is None:
        weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    elif (weights.shape != (T, top_k) or weights.dtype != torch.float32 or not weights.is_contiguous()
          or not weights.is_cuda):
        _refuse(weights=(weights, (T, top_k), torch.float32, True))
    code = _lib.load().moe_route(logits.data_ptr(), T, E, _row_ld(logits, E), dtype, top_k, renormalize,
                                 ids.data_ptr(), weights.data_ptr(), _raw_stream(dev))
    if code:
        raise MXGError(code, "moe_route")
    if ids_given is not None:
        _written(ids)
    if weights_given is not None:
        _written(weights)
    return ids, weights


@functools.lru_cache(maxsize=1024)
def moe_experts_workspace_size(tokens: int, top_k: int, experts: int, hidden: int, inter: int) -> int:
    return int(_lib.load().moe_experts_workspace_size(tokens, top_k, experts, hidden, inter))


def _expert_weights(w: MXOperand) -> _lib.MxOperandC:
    """The C form of one expert weight matrix: rows of codes, and a packed byte
    for every 32 weights (rows and columns are multiples of 128)."""
    data, scale, cols = w.data, w.scale, w.cols
    rows, ld = data.shape[0], data.stride(0)
    if w.scale_layout != "packed":
        raise ValueError("W13 and W2 need packed scales (mx_quantize_rowwise_packed with groups=experts)")
    if data.shape[1:] != (_codes_cols(w.elem, cols),) or data.stride(-1) != 1:
        raise ValueError("codes of W13 and W2 must be rows of their columns, contiguous in a row")
    if scale.numel() < rows * (cols // 32) or not scale.is_contiguous():
        raise ValueError("packed scales must be contiguous and as many as the weights need")
    if not (data.is_cuda and scale.is_cuda):
        raise ValueError("libmxg operates on CUDA tensors only")
    return _lib.MxOperandC(data.data_ptr(), scale.data_ptr(), rows, cols, ld, cols // 32, ELEM[w.elem], 1)


def moe_experts(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, W13: MXOperand, W2: MXOperand,
                out_dtype=torch.bfloat16, out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                status: torch.Tensor | None = None, check: bool = False) -> torch.Tensor:
    """The expert layer of a few tokens over MX-quantized weights (decode):
    out[t] = sum_j weights[t, j] * W2[e] silu_mul(W13[e] x[t]), e = ids[t, j].

    ``x`` BF16 [T, H]; ``ids`` / ``weights`` [T, top_k] as from ``moe_route``
    (a negative id is an empty slot); ``W13`` [E * 2I, H] (each expert's I gate
    rows, then its I up rows) and ``W2`` [E * H, I] from
    ``mx_quantize_rowwise_packed(..., groups=E)``, both "e2m1" or both "e4m3".
    Activations are rounded to MXFP8 in front of each product, as the grouped
    GEMMs of the same operands take them.  T * top_k <= 4096.  Forward only."""
    if ids.dim() != 2 or x.dim() != 2:
        raise ValueError("x must be [tokens, hidden] and ids [tokens, top_k]")
    if x.requires_grad or weights.requires_grad or (out is not None and out.requires_grad):
        _refuse_grad("moe_experts")
    T, k = ids.shape
    H, I, dev = W13.cols, W2.cols, x.device
    if (x.shape != (T, H) or x.dtype != torch.bfloat16 or weights.shape != (T, k) or ids.dtype != torch.int32
            or weights.dtype != torch.float32 or not ids.is_contiguous() or not weights.is_contiguous()
            or not (x.is_cuda and ids.is_cuda and weights.is_cuda)):
        _refuse(x=(x, (T, H), torch.bfloat16, False), ids=(ids, (T, k), torch.int32, True),
                weights=(weights, (T, k), torch.float32, True))
    a, b = _expert_weights(W13), _expert_weights(W2)
    E = b.rows // H
    if b.rows != E * H or a.rows != E * 2 * I:
        raise ValueError("W13 must be [E * 2I, H] and W2 [E * H, I]")
    lib = _lib.load()
    given = out
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=dev)
    if out.shape != (T, H) or out.dtype not in _OUT or not out.is_cuda:
        _refuse(out=(out, (T, H), _OUT, False))
    stream = _raw_stream(dev)
    if workspace is None:
        workspace = _scratch(moe_experts_workspace_size(T, k, E, H, I), dev, stream)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous uint8")
    code = lib.moe_experts(x.data_ptr(), T, _row_ld(x, H), ids.data_ptr(), weights.data_ptr(), k, E, ctypes.byref(a),
                           ctypes.byref(b), out.data_ptr(), _row_ld(out, H), _OUT[out.dtype], workspace.data_ptr(),
                           workspace.numel(), _status_ptr(status, dev), stream)
    if code:
        raise MXGError(code, "moe_experts")
    if given is not None:
        _written(out)
    if check:
        check_status(status, dev)
    return out


@functools.lru_cache(maxsize=1024)
def lora_add_workspace_size(tokens: int, K: int, rank: int) -> int:
    return int(_lib.load().lora_add_workspace_size(tokens, K, rank))


def lora_add(y: torch.Tensor, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, ids: torch.Tensor,
             scale: torch.Tensor | None = None, out: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
             check: bool = False) -> torch.Tensor:
    """Low-rank adapters of many requests beside a shared projection:
    out[t] = y[t] + scale[a] * B[a] (A[a] x[t]) with a = ids[t]; out[t] = y[t]
    for a negative id.

    ``y`` [T, N] BF16 or FP32, the projection's output; ``x`` BF16 [T, K];
    ``A`` BF16 [adapters, rank, K]; ``B`` BF16 [adapters, N, rank]; ``ids``
    int32 [T]; ``scale`` FP32 [adapters] (None: 1).  ``out=y`` updates in
    place.  rank is a multiple of 8 up to 128.  Forward only."""
    if y.dim() != 2 or A.dim() != 3:
        raise ValueError("y must be [tokens, N] and A [adapters, rank, K]")
    if (y.requires_grad or x.requires_grad or A.requires_grad or B.requires_grad
            or (scale is not None and scale.requires_grad) or (out is not None and out.requires_grad)):
        _refuse_grad("lora_add")
    T, N = y.shape
    n, R, K = A.shape
    bf16 = torch.bfloat16
    dtype = _OUT.get(y.dtype)
    if (x.shape != (T, K) or B.shape != (n, N, R) or ids.shape != (T,) or dtype is None or x.dtype != bf16
            or A.dtype != bf16 or B.dtype != bf16 or ids.dtype != torch.int32 or not A.is_contiguous()
            or not B.is_contiguous() or not ids.is_contiguous()
            or not (y.is_cuda and x.is_cuda and A.is_cuda and B.is_cuda and ids.is_cuda)):
        _refuse(y=(y, (T, N), _OUT, False), x=(x, (T, K), bf16, False), A=(A, (n, R, K), bf16, True),
                B=(B, (n, N, R), bf16, True), ids=(ids, (T,), torch.int32, True))
    if scale is not None and (scale.shape != (n,) or scale.dtype != torch.float32 or not scale.is_contiguous()
                              or not scale.is_cuda):
        _refuse(scale=(scale, (n,), torch.float32, True))
    dev = y.device
    lib = _lib.load()
    given = out
    if out is None:
        out = torch.empty((T, N), dtype=y.dtype, device=dev)
    elif out.shape != (T, N) or out.dtype != y.dtype or not out.is_cuda:
        _refuse(out=(out, (T, N), y.dtype, False))
    stream = _raw_stream(dev)
    if workspace is None:
        workspace = _scratch(lora_add_workspace_size(T, K, R), dev, stream)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous uint8")
    code = lib.lora_add(y.data_ptr(), _row_ld(y, N), x.data_ptr(), _row_ld(x, K), A.data_ptr(), B.data_ptr(),
                        ids.data_ptr(), None if scale is None else scale.data_ptr(), T, N, K, R, n, dtype,
                        out.data_ptr(), _row_ld(out, N), workspace.data_ptr(), workspace.numel(),
                        _status_ptr(status, dev), stream)
    if code:
        raise MXGError(code, "lora_add")
    if given is not None:
        _written(out)
    if check:
        check_status(status, dev)
    return out


# ----------------------------------------------------------------------------- tokens to the experts and back


@functools.lru_cache(maxsize=1024)
def moe_sort_workspace_size(tokens: int, top_k: int, experts: int) -> int:
    return int(_lib.load().moe_sort_workspace_size(tokens, top_k, experts))


def _given_workspace(workspace: torch.Tensor):
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous uint8")


def moe_sort(ids: torch.Tensor, experts: int, m_splits: torch.Tensor | None = None, rows: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, status: torch.Tensor | None = None, check: bool = False):
    """Expert ids [T, top_k] (int32, as from ``moe_route``) -> (m_splits int32
    [experts], rows int32 [T, top_k]): every slot's row in expert order, slots of
    one expert in the order of their index.  An empty slot (negative id) owns a
    row r behind all others and has the entry -1 - r; the last expert's split
    counts these rows (zeros in the calls below), so that the splits add up to
    T * top_k, as the grouped GEMMs and quantizers ask."""
    if ids.dim() != 2:
        raise ValueError("ids must be [tokens, top_k]")
    T, k = ids.shape
    i32, dev = torch.int32, ids.device
    if ids.dtype != i32 or not ids.is_contiguous() or not ids.is_cuda:
        _refuse(ids=(ids, (T, k), i32, True))
    m_given, r_given = m_splits, rows
    if m_splits is None:
        m_splits = torch.empty((experts,), dtype=i32, device=dev)
    elif m_splits.shape != (experts,) or m_splits.dtype != i32 or not m_splits.is_contiguous() or not m_splits.is_cuda:
        _refuse(m_splits=(m_splits, (experts,), i32, True))
    if rows is None:
        rows = torch.empty((T, k), dtype=i32, device=dev)
    elif rows.shape != (T, k) or rows.dtype != i32 or not rows.is_contiguous() or not rows.is_cuda:
        _refuse(rows=(rows, (T, k), i32, True))
    stream = _raw_stream(dev)
    if workspace is None:
        workspace = _scratch(moe_sort_workspace_size(T, k, experts), dev, stream)
    else:
        _given_workspace(workspace)
    code = _lib.load().moe_sort(ids.data_ptr(), T, k, experts, m_splits.data_ptr(), rows.data_ptr(), workspace.data_ptr(),
                                workspace.numel(), _status_ptr(status, dev), stream)
    if code:
        raise MXGError(code, "moe_sort")
    if m_given is not None:
        _written(m_splits)
    if r_given is not None:
        _written(rows)
    if check:
        check_status(status, dev)
    return m_splits, rows


def _refuse_rows(rows: torch.Tensor):
    raise ValueError(f"rows must be contiguous int32 [tokens, top_k] on the GPU (from moe_sort), got {rows.dtype} of "
                     f"shape {list(rows.shape)}")


def moe_gather(x: torch.Tensor, rows: torch.Tensor, out: torch.Tensor | None = None, status: torch.Tensor | None = None,
               check: bool = False) -> torch.Tensor:
    """x [T, H] (BF16 or FP32) -> [T * top_k, H] in expert order: out[rows[t, j]] =
    x[t], zeros in the rows of empty slots.  ``rows`` from ``moe_sort``.  The
    gradient is ``moe_combine(dout, rows)``.  H is a multiple of 8 (FP32: 4)."""
    if rows.dim() != 2 or rows.dtype != torch.int32 or not rows.is_contiguous() or not rows.is_cuda:
        _refuse_rows(rows)
    T, k = rows.shape
    dtype = _OUT.get(x.dtype)
    if x.dim() != 2 or x.shape[0] != T or dtype is None or not x.is_cuda:
        _refuse(x=(x, (T, *x.shape[-1:]), _OUT, False))
    if x.requires_grad or (out is not None and out.requires_grad):
        _refuse_grad("moe_gather")
    H, dev, given = x.shape[1], x.device, out
    if out is None:
        out = torch.empty((T * k, H), dtype=x.dtype, device=dev)
    elif out.shape != (T * k, H) or out.dtype != x.dtype or not out.is_cuda:
        _refuse(out=(out, (T * k, H), x.dtype, False))
    code = _lib.load().moe_gather(x.data_ptr(), H if x.is_contiguous() else _row_ld(x, H), rows.data_ptr(), T, k, H, dtype,
                                  out.data_ptr(), H if given is None else _row_ld(out, H), _status_ptr(status, dev),
                                  _raw_stream(dev))
    if code:
        raise MXGError(code, "moe_gather")
    if given is not None:
        _written(out)
    if check:
        check_status(status, dev)
    return out


def moe_combine(y: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor | None = None, out: torch.Tensor | None = None,
                status: torch.Tensor | None = None, check: bool = False) -> torch.Tensor:
    """Rows in expert order back to their tokens: out[t] = sum_j weights[t, j] *
    y[rows[t, j]] (``weights`` None: 1), empty slots adding nothing.  ``y`` BF16 or
    FP32 [rows, H]; ``weights`` FP32 [T, top_k] as from ``moe_route``.  Sums in FP32,
    in the order of the slots, rounded once."""
    if rows.dim() != 2 or rows.dtype != torch.int32 or not rows.is_contiguous() or not rows.is_cuda:
        _refuse_rows(rows)
    shape = rows.shape
    T, k = shape
    dtype = _OUT.get(y.dtype)
    if y.dim() != 2 or dtype is None or not y.is_cuda:
        _refuse(y=(y, (T * k, *y.shape[-1:]), _OUT, False))
    if weights is not None and (weights.shape != shape or weights.dtype != torch.float32 or not weights.is_contiguous()
                                or not weights.is_cuda):
        _refuse(weights=(weights, shape, torch.float32, True))
    if y.requires_grad or (weights is not None and weights.requires_grad) or (out is not None and out.requires_grad):
        _refuse_grad("moe_combine")
    n, H = y.shape
    dev, given = y.device, out
    if out is None:
        out = torch.empty((T, H), dtype=y.dtype, device=dev)
    elif out.shape != (T, H) or out.dtype != y.dtype or not out.is_cuda:
        _refuse(out=(out, (T, H), y.dtype, False))
    code = _lib.load().moe_combine(y.data_ptr(), H if y.is_contiguous() else _row_ld(y, H), n, rows.data_ptr(),
                                   None if weights is None else weights.data_ptr(), T, k, H, dtype, out.data_ptr(),
                                   H if given is None else _row_ld(out, H), _status_ptr(status, dev), _raw_stream(dev))
    if code:
        raise MXGError(code, "moe_combine")
    if given is not None:
        _written(out)
    if check:
        check_status(status, dev)
    return out


def moe_combine_backward(dout: torch.Tensor, y: torch.Tensor, rows: torch.Tensor, weights: torch.Tensor,
                         dy: torch.Tensor | None = None, dweights: torch.Tensor | None = None,
                         status: torch.Tensor | None = None, check: bool = False):
    """Gradients of ``moe_combine(y, rows, weights)`` -> (dy, dweights):
    dy[rows[t, j]] = weights[t, j] * dout[t] (zeros in the rows of empty slots) and
    dweights[t, j] = <dout[t], y[rows[t, j]]> (0 for an empty slot), FP32 sums.
    ``dout`` [T, H] and ``y`` [T * top_k, H] of one type.  ``dy=y`` writes over y."""
    if rows.dim() != 2 or rows.dtype != torch.int32 or not rows.is_contiguous() or not rows.is_cuda:
        _refuse_rows(rows)
    shape = rows.shape
    T, k = shape
    f32, dt = torch.float32, y.dtype
    dtype = _OUT.get(dt)
    if y.dim() != 2 or y.shape[0] != T * k or dtype is None or not y.is_cuda:
        _refuse(y=(y, (T * k, *y.shape[-1:]), _OUT, False))
    H, dev = y.shape[1], y.device
    if (dout.shape != (T, H) or dout.dtype != dt or not dout.is_cuda or weights.shape != shape or weights.dtype != f32
            or not weights.is_contiguous() or not weights.is_cuda):
        _refuse(dout=(dout, (T, H), dt, False), weights=(weights, shape, f32, True))
    if (dout.requires_grad or y.requires_grad or weights.requires_grad or (dy is not None and dy.requires_grad)
            or (dweights is not None and dweights.requires_grad)):
        _refuse_grad("moe_combine_backward")
    dy_given, dw_given = dy, dweights
    if dy is None:
        dy = torch.empty((T * k, H), dtype=dt, device=dev)
    elif dy.shape != (T * k, H) or dy.dtype != dt or not dy.is_cuda:
        _refuse(dy=(dy, (T * k, H), dt, False))
    if dweights is None:
        dweights = torch.empty(shape, dtype=f32, device=dev)
    elif dweights.shape != shape or dweights.dtype != f32 or not dweights.is_contiguous() or not dweights.is_cuda:
        _refuse(dweights=(dweights, shape, f32, True))
    code = _lib.load().moe_combine_backward(
        dout.data_ptr(), H if dout.is_contiguous() else _row_ld(dout, H), y.data_ptr(),
        H if y.is_contiguous() else _row_ld(y, H), rows.data_ptr(), weights.data_ptr(), T, k, H, dtype, dy.data_ptr(),
        H if dy.is_contiguous() else _row_ld(dy, H), dweights.data_ptr(), _status_ptr(status, dev), _raw_stream(dev))
    if code:
        raise MXGError(code, "moe_combine_backward")
    if dy_given is not None:
        _written(dy)
    if dw_given is not None:
        _written(dweights)
    if check:
        check_status(status, dev)
    return dy, dweights


def moe_route_backward(dweights: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, logits: torch.Tensor,
                       renormalize: bool = True, dlogits: torch.Tensor | None = None,
                       status: torch.Tensor | None = None, check: bool = False) -> torch.Tensor:
    """Gradient of ``moe_route``'s weights for its logits: with s = sum_j weights_j
    dweights_j over a token's slots, dlogits[id_j] = weights_j (dweights_j - s) and
    zeros elsewhere (``renormalize``), or [e = id_j] weights_j dweights_j - p_e s with
    p = softmax(logits).  ``ids`` and ``weights`` as ``moe_route`` returned them for
    these ``logits`` [T, E] and this ``renormalize``; the result has the logits' type."""
    if logits.dim() != 2 or ids.dim() != 2:
        raise ValueError("logits must be [tokens, experts] and ids [tokens, top_k]")
    T, E = logits.shape
    shape, dev, dt, f32 = ids.shape, logits.device, logits.dtype, torch.float32
    dtype = _OUT.get(dt)
    if (dtype is None or not logits.is_cuda or shape[0] != T or ids.dtype != torch.int32 or not ids.is_contiguous()
            or not ids.is_cuda or dweights.shape != shape or dweights.dtype != f32 or not dweights.is_contiguous()
            or not dweights.is_cuda or weights.shape != shape or weights.dtype != f32 or not weights.is_contiguous()
            or not weights.is_cuda):
        want = (T, shape[1])
        _refuse(logits=(logits, (T, E), _OUT, False), ids=(ids, want, torch.int32, True),
                dweights=(dweights, want, f32, True), weights=(weights, want, f32, True))
    if (dweights.requires_grad or weights.requires_grad or logits.requires_grad
            or (dlogits is not None and dlogits.requires_grad)):
        _refuse_grad("moe_route_backward")
    given = dlogits
    if dlogits is None:
        dlogits = torch.empty((T, E), dtype=dt, device=dev)
    elif dlogits.shape != (T, E) or dlogits.dtype != dt or not dlogits.is_cuda:
        _refuse(dlogits=(dlogits, (T, E), dt, False))
    code = _lib.load().moe_route_backward(dweights.data_ptr(), ids.data_ptr(), weights.data_ptr(), logits.data_ptr(),
                                          E if logits.is_contiguous() else _row_ld(logits, E), T, E, shape[1], renormalize,
                                          dtype, dlogits.data_ptr(), E if given is None else _row_ld(dlogits, E),
                                          _status_ptr(status, dev), _raw_stream(dev))
    if code:
        raise MXGError(code, "moe_route_backward")
    if given is not None:
        _written(dlogits)
    if check:
        check_status(status, dev)
    return dlogits


# ----------------------------------------------------------------------------- 8-bit integers

_CODES = {"int8": torch.int8, "f16": torch.float16}
_CODE_KIND = {torch.int8: 1, torch.float16: 2}  # and a code's bytes


@dataclass
class Int8Operand:
    """A K-major operand of 8-bit integers with one FP32 scale per row (token or
    channel): codes [rows, cols] as int8, or as FP16 tensors of the same integers
    (activations, the form the tensor core takes)."""
    data: torch.Tensor
    scale: torch.Tensor

    @property
    def rows(self) -> int:
        return self.data.shape[0]

    @property
    def cols(self) -> int:
        return self.data.shape[1]

    def c(self) -> _lib.Int8OperandC:
        data, scale = self.data, self.scale
        kind = _CODE_KIND.get(data.dtype)
        if data.dim() != 2 or kind is None or not data.is_cuda:
            _refuse(codes=(data, (*data.shape[:1], *data.shape[1:][-1:]), _CODE_KIND, False))
        rows, cols = data.shape
        if scale.shape != (rows,) or scale.dtype != torch.float32 or not scale.is_contiguous() or not scale.is_cuda:
            _refuse(scale=(scale, (rows,), torch.float32, True))
        ld = cols * kind if data.is_contiguous() else _code_ld(data, cols, kind)
        return _lib.Int8OperandC(data.data_ptr(), scale.data_ptr(), rows, cols, ld, kind, 0)


def _code_ld(t: torch.Tensor, cols: int, kind: int) -> int:
    """Row stride of codes in bytes; their rows must be contiguous."""
    if t.shape[0] > 0 and cols > 1 and t.stride(1) != 1:
        raise ValueError("codes of a row must be contiguous")
    return (t.stride(0) if t.shape[0] > 1 else (cols + 15) & ~15) * kind


def int8_quantize_rowwise(x: torch.Tensor, rows: torch.Tensor | None = None, codes: str = "int8",
                          q: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                          status: torch.Tensor | None = None, check: bool = False) -> Int8Operand:
    """BF16 [T, cols] -> 8-bit integers with a scale per row: scale = max(max |x|,
    2^-100) / 127, codes to the nearest integer.  For activations, and for weights
    per channel.  With ``rows`` (from ``moe_sort``) the rows come out in expert order
    [T * top_k, cols], as from quantizing ``moe_gather(x, rows)``, from one read of
    x.  ``codes="f16"`` writes the integers as FP16 values, which the GEMMs take
    without widening them first.  A row with a NaN or an infinity gets the scale NaN."""
    dtype = _CODES.get(codes)
    if dtype is None:
        raise ValueError(f"unknown codes {codes!r} (int8 or f16)")
    if x.dim() != 2 or x.dtype != torch.bfloat16 or not x.is_cuda:
        _refuse(x=(x, (*x.shape[:1], *x.shape[1:][-1:]), torch.bfloat16, False))
    if x.requires_grad or (scale is not None and scale.requires_grad) or (q is not None and q.requires_grad):
        _refuse_grad("int8_quantize_rowwise")
    T, K = x.shape
    n, k, dev, kind = T, 1, x.device, _CODE_KIND[dtype]
    if rows is not None:
        if rows.dim() != 2 or rows.dtype != torch.int32 or not rows.is_contiguous() or not rows.is_cuda:
            _refuse_rows(rows)
        if rows.shape[0] != T:
            raise ValueError("rows must have a row for every token of x")
        k = rows.shape[1]
        n = T * k
    q_given, s_given = q, scale
    if q is None:
        q = torch.empty((n, K), dtype=dtype, device=dev)
    elif q.shape != (n, K) or q.dtype != dtype or not q.is_cuda:
        _refuse(q=(q, (n, K), dtype, False))
    if scale is None:
        scale = torch.empty((n,), dtype=torch.float32, device=dev)
    elif scale.shape != (n,) or scale.dtype != torch.float32 or not scale.is_contiguous() or not scale.is_cuda:
        _refuse(scale=(scale, (n,), torch.float32, True))
    code = _lib.load().int8_quantize_rowwise(x.data_ptr(), K if x.is_contiguous() else _row_ld(x, K),
                                             None if rows is None else rows.data_ptr(), T, k, K, kind, q.data_ptr(),
                                             K * kind if q_given is None else _code_ld(q, K, kind), scale.data_ptr(),
                                             _status_ptr(status, dev), _raw_stream(dev))
    if code:
        raise MXGError(code, "int8_quantize_rowwise")
    if q_given is not None:
        _written(q)
    if s_given is not None:
        _written(scale)
    if check:
        check_status(status, dev)
    return Int8Operand(q, scale)


@functools.lru_cache(maxsize=1024)
def int8_gemm_workspace_size(G: int, S: int, N: int, K: int, codes: str = "int8") -> int:
    return int(_lib.load().int8_gemm_workspace_size(G, S, N, K, _CODE_KIND[_CODES[codes]]))


def _int8_gemm(name, fn, A, W, splits, G, N, out_dtype, out, workspace, status, check):
    a, w = A.c(), W.c()
    if A.scale.requires_grad or W.scale.requires_grad or A.data.requires_grad or (out is not None and out.requires_grad):
        _refuse_grad(name)
    dev, given, S = A.data.device, out, a.rows
    if out is None:
        out = torch.empty((S, N), dtype=out_dtype, device=dev)
    dtype = _OUT.get(out.dtype)
    if out.shape != (S, N) or dtype is None or not out.is_cuda:
        _refuse(out=(out, (S, N), _OUT, False))
    stream = _raw_stream(dev)
    if workspace is None:
        workspace = _scratch(int8_gemm_workspace_size(G, S, N, a.cols, "int8" if a.codes == 1 else "f16"), dev, stream)
    else:
        _given_workspace(workspace)
    code = fn(ctypes.byref(a), ctypes.byref(w), *splits, out.data_ptr(), N if given is None else _row_ld(out, N), dtype,
              workspace.data_ptr(), workspace.numel(), _status_ptr(status, dev), stream)
    if code:
        raise MXGError(code, name)
    if given is not None:
        _written(out)
    if check:
        check_status(status, dev)
    return out


def int8_grouped_gemm_fwd(A: Int8Operand, W: Int8Operand, m_splits: torch.Tensor, N: int, out_dtype=torch.bfloat16,
                          out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                          status: torch.Tensor | None = None, check: bool = False) -> torch.Tensor:
    """Y[off_g+i, :] = A[off_g+i, :] @ W[g*N:(g+1)*N, :]^T for every expert g, both
    operands standing for scale * codes; ``W`` int8 [G * N, K].  Codes' products are
    exact and their sums in FP32: exact below 2^24, above within 2^-23 of the largest
    partial sum for every 16 elements.  Forward only."""
    if m_splits.dim() != 1 or m_splits.dtype != torch.int32 or not m_splits.is_contiguous() or not m_splits.is_cuda:
        _refuse(m_splits=(m_splits, (m_splits.numel(),), torch.int32, True))
    G = m_splits.numel()
    return _int8_gemm("int8_grouped_gemm_fwd", _lib.load().int8_grouped_gemm_fwd, A, W, (m_splits.data_ptr(), G, N), G, N,
                      out_dtype, out, workspace, status, check)


def int8_gemm_dense(A: Int8Operand, B: Int8Operand, out_dtype=torch.bfloat16, out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
                    check: bool = False) -> torch.Tensor:
    """C[M, N] = A[M, K] @ B[N, K]^T of two 8-bit integer operands (``B`` int8)."""
    return _int8_gemm("int8_gemm_dense", _lib.load().int8_gemm_dense, A, B, (), 1, B.rows, out_dtype, out, workspace,
                      status, check)
