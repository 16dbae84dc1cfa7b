"""torch-facing helpers over the libpgq C ABI.

torch provides device memory and the current HIP stream; every step of the quantizer
runs in libpgq's kernels.  Outputs that are fp16 / bf16 bit patterns are returned as
int16 tensors (reinterpret with .view(torch.float16) / .view(torch.bfloat16)).
"""
from __future__ import annotations

import ctypes
import struct
import warnings
from dataclasses import dataclass
from typing import Dict, List, Optional, Sequence, Tuple

import torch

from . import pgq

DEFAULT_INT8_PATTERNS = ("tok_emb.weight", "lm_head.weight")


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


# The current stream's handle of GPU `index`: what torch.cuda.current_stream(index).cuda_stream gives, without
# building the Stream object (2.8 us a call against 0.1).
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.float32:
        return pgq.PGQ_F32
    if dt == torch.bfloat16:
        return pgq.PGQ_BF16
    if dt == torch.float16:
        return pgq.PGQ_F16
    raise TypeError(f"unsupported dtype {dt}")


def _rows_view(t: torch.Tensor) -> Tuple[int, int, int]:
    """(rows, cols, ld) of a tensor seen as [shape0, prod(rest)] (1-D: one row)."""
    if t.dim() == 0:
        return 1, 1, 1
    if t.dim() == 1:
        assert t.stride(0) == 1 or t.numel() <= 1, "1-D tensors must be contiguous"
        return 1, t.numel(), t.numel()
    if t.dim() > 2:
        t = t.reshape(t.shape[0], -1)
    assert t.stride(1) == 1 or t.shape[1] <= 1, "rows must be contiguous"
    return t.shape[0], t.shape[1], (t.stride(0) if t.shape[0] > 1 else t.shape[1])


def new_status(device=None) -> torch.Tensor:
    return torch.zeros(1, dtype=torch.int32, device=device or "cuda")


def qparams(bits: int, pct: Tuple[int, int] = (1, 1)) -> pgq.pgq_qparams:
    return pgq.pgq_qparams(bits, pct[0], pct[1])


def quantize_rows(w: torch.Tensor, bits: int = 6, pct: Tuple[int, int] = (1, 1),
                  awq_s: Optional[torch.Tensor] = None, want_codes: bool = True,
                  dq_dtype: Optional[torch.dtype] = torch.float32,
                  status: Optional[torch.Tensor] = None, out: Optional[dict] = None) -> dict:
    """Per-row quantization of one matrix (fp32, bf16 or fp16, rows contiguous)."""
    rows, cols, ld = _rows_view(w)
    dev = w.device
    if out is None:
        out = {}
        out["scales"] = torch.empty(rows, dtype=torch.int16, device=dev)
        if want_codes:
            out["codes"] = torch.empty(rows, cols, dtype=torch.int8, device=dev)
        if dq_dtype is not None:
            out["dq"] = torch.empty(rows, cols, dtype=dq_dtype, device=dev)
        if awq_s is not None:
            out["awq"] = torch.empty(cols, dtype=torch.int16, device=dev)
    st = status if status is not None else new_status(dev)
    dq = out.get("dq")
    rc = pgq.pgq_quantize_rows(_p(w), _dtype_code(w.dtype), rows, cols, ld, qparams(bits, pct), _p(awq_s),
                               _p(out.get("awq")), _p(out.get("codes")), _p(out["scales"]), _p(dq),
                               _dtype_code(dq.dtype) if dq is not None else pgq.PGQ_F32, _p(st), _stream())
    pgq.check(rc, "pgq_quantize_rows")
    out["status"] = st
    return out


class FakeQuant:
    """STE fake quantization of a fixed list of bf16 weight matrices (grouped launches).

    Buffers for dq, scales, mask and grad_out are allocated once; each call re-runs the
    kernels on the same buffers, reusing the uploaded descriptor table."""

    def __init__(self, weights: Sequence[torch.Tensor], bits: int = 6, pct: Tuple[int, int] = (1, 1),
                 want_codes: bool = False):
        self.weights = list(weights)
        self.qp = qparams(bits, pct)
        dev = self.weights[0].device
        self.dq, self.scales, self.mask, self.codes, self.grad_out = [], [], [], [], []
        for w in self.weights:
            assert w.dtype == torch.bfloat16 and w.dim() == 2 and w.stride(1) == 1
            r, c = w.shape
            self.dq.append(torch.empty(r, c, dtype=torch.bfloat16, device=dev))
            self.scales.append(torch.empty(r, dtype=torch.int16, device=dev))
            self.mask.append(torch.empty(r, (c + 7) // 8, dtype=torch.uint8, device=dev))
            self.codes.append(torch.empty(r, c, dtype=torch.int8, device=dev) if want_codes else None)
            self.grad_out.append(torch.empty(r, c, dtype=torch.bfloat16, device=dev))
        self.status = new_status(dev)
        self._tables = {}

    def _descs(self, grads):
        n = len(self.weights)
        arr = (pgq.pgq_fq_tensor * n)()
        for i, w in enumerate(self.weights):
            g = None if grads is None else grads[i]
            if g is not None:
                assert g.shape == w.shape and g.dtype == torch.bfloat16 and g.is_contiguous()
            arr[i] = pgq.pgq_fq_tensor(w.data_ptr(), w.shape[0], w.shape[1], w.stride(0),
                                       self.dq[i].data_ptr(), self.scales[i].data_ptr(), self.mask[i].data_ptr(),
                                       0 if g is None else g.data_ptr(), self.grad_out[i].data_ptr(),
                                       0 if self.codes[i] is None else self.codes[i].data_ptr())
        return arr

    def run(self, mode: int, grads: Optional[Sequence[torch.Tensor]] = None, reuse_table: bool = True):
        """Enqueue one grouped launch.  The descriptor array and the workspace holding its
        uploaded table are kept per (mode, gradient buffers), so repeated steps over the same
        buffers only re-enqueue the kernel."""
        n = len(self.weights)
        key = (mode, tuple(0 if grads is None else g.data_ptr() for g in (grads or [])))
        cached = self._tables.get(key)
        flags = 0
        if cached is not None and reuse_table:
            arr, ws = cached
            flags = pgq.PGQ_TABLE_RESIDENT
        else:
            arr = self._descs(grads)
            need = ctypes.c_size_t(0)
            pgq.check(pgq.pgq_fakequant_workspace(arr, n, ctypes.byref(need)), "pgq_fakequant_workspace")
            ws = torch.empty(max(need.value, 64), dtype=torch.uint8, device=self.weights[0].device)
            self._tables[key] = (arr, ws)
        rc = pgq.pgq_fakequant_fwd_bwd(mode, arr, n, self.qp, _p(ws), ws.numel(), flags, _p(self.status), _stream())
        pgq.check(rc, "pgq_fakequant_fwd_bwd")


@dataclass
class ExportTensor:
    name: str
    w: torch.Tensor
    awq_s: Optional[torch.Tensor] = None


def _tensor_in_array(tensors: Sequence[ExportTensor]):
    n = len(tensors)
    arr = (pgq.pgq_tensor_in * n)()
    keep = []
    for i, t in enumerate(tensors):
        rows, cols, ld = _rows_view(t.w)
        nm = t.name.encode()
        keep.append(nm)
        arr[i] = pgq.pgq_tensor_in(nm, t.w.data_ptr() if t.w.numel() else 0, _dtype_code(t.w.dtype), 0,
                                   rows, cols, ld, 0 if t.awq_s is None else t.awq_s.data_ptr())
    return arr, keep


def make_policy(int8_patterns=DEFAULT_INT8_PATTERNS, passthrough_below: int = 65536,
                q_default=(6, 9999, 10000), q_sensitive=(8, 1, 1), per_tensor: bool = False,
                pack6: bool = False):
    pats = [p.encode() for p in int8_patterns]
    parr = (ctypes.c_char_p * max(1, len(pats)))(*pats)
    pol = pgq.pgq_policy(ctypes.cast(parr, ctypes.POINTER(ctypes.c_char_p)), len(pats), 1 if per_tensor else 0,
                         passthrough_below,
                         pgq.pgq_qparams(*q_default), pgq.pgq_qparams(*q_sensitive), 1 if pack6 else 0, 0)
    pol._keep = (pats, parr)
    return pol


class Exporter:
    """Whole-model export: plan once, then one grouped launch per call."""

    def __init__(self, tensors: Sequence[ExportTensor], policy=None, want_dq: bool = False):
        self.tensors = list(tensors)
        self.policy = policy if policy is not None else make_policy()
        n = len(self.tensors)
        self.n = n
        self.arr, self._keep = _tensor_in_array(self.tensors)
        self.plan = (pgq.pgq_tensor_plan * max(n, 1))()
        ab, wb = ctypes.c_size_t(0), ctypes.c_size_t(0)
        pgq.check(pgq.pgq_export_plan(self.arr, n, ctypes.byref(self.policy), self.plan, ctypes.byref(ab),
                                      ctypes.byref(wb)), "pgq_export_plan")
        dev = self.tensors[0].w.device
        self.arena = torch.empty(ab.value, dtype=torch.uint8, device=dev)
        self.workspace = torch.empty(max(wb.value, 64), dtype=torch.uint8, device=dev)
        self.dq = None
        self.dq_ptrs = None
        if want_dq:
            self.dq = [torch.empty(t.w.shape, dtype=torch.float32, device=dev) for t in self.tensors]
            self.dq_ptrs = (ctypes.c_void_p * n)(*[d.data_ptr() for d in self.dq])
        self.status = new_status(dev)
        self._uploaded = False

    def run(self, reuse_table: bool = True):
        flags = pgq.PGQ_TABLE_RESIDENT if (reuse_table and self._uploaded) else 0
        rc = pgq.pgq_export_model(self.arr, self.n, self.plan, _p(self.arena), self.dq_ptrs, _p(self.workspace),
                                  self.workspace.numel(), flags, _p(self.status), _stream())
        pgq.check(rc, "pgq_export_model")
        self._uploaded = True

    def decode(self, out: Optional[List[torch.Tensor]] = None, reuse_table: bool = True) -> List[torch.Tensor]:
        """fp32 weights from the arena (the stored artifact), every tensor in one launch."""
        dev = self.arena.device
        if out is None:
            out = [torch.empty(t.w.shape, dtype=torch.float32, device=dev) for t in self.tensors]
        key = tuple(o.data_ptr() for o in out)
        cached = getattr(self, "_decode_table", None)
        flags = 0
        if cached is not None and cached[0] == key and reuse_table:
            ptrs, ws = cached[1], cached[2]
            flags = pgq.PGQ_TABLE_RESIDENT
        else:
            ptrs = (ctypes.c_void_p * self.n)(*[o.data_ptr() for o in out])
            ws = torch.empty(self.workspace.numel(), dtype=torch.uint8, device=dev)
            self._decode_table = (key, ptrs, ws)
        rc = pgq.pgq_dequant_model(self.arr, self.n, self.plan, _p(self.arena), ptrs, _p(ws), ws.numel(), flags,
                                   _p(self.status), _stream())
        pgq.check(rc, "pgq_dequant_model")
        return out

    def kinds(self) -> List[int]:
        return [self.plan[i].kind for i in range(self.n)]

    def outputs(self) -> List[dict]:
        """Per-tensor views into the arena: codes [rows, cols] int8, scales [rows] int16,
        f16 [shape] int16, awq [cols] int16."""
        res = []
        for i, t in enumerate(self.tensors):
            p = self.plan[i]
            rows, cols, _ = _rows_view(t.w)
            rec = {"name": t.name, "kind": p.kind}
            if p.kind == pgq.PGQ_KIND_F16:
                rec["f16"] = self.arena[p.f16_off:p.f16_off + 2 * rows * cols].view(torch.int16).view(t.w.shape)
            else:
                if p.packed:
                    rb = 3 * ((cols + 3) // 4)
                    rec["packed"] = self.arena[p.codes_off:p.codes_off + rows * rb].view(rows, rb)
                else:
                    rec["codes"] = self.arena[p.codes_off:p.codes_off + rows * cols].view(torch.int8).view(rows, cols)
                ns = 1 if p.per_tensor else rows
                rec["scales"] = self.arena[p.scales_off:p.scales_off + 2 * ns].view(torch.int16)
                if p.has_awq:
                    rec["awq"] = self.arena[p.awq_off:p.awq_off + 2 * cols].view(torch.int16)
            if self.dq is not None:
                rec["dq"] = self.dq[i]
            res.append(rec)
        return res


class Sqwa:
    """Running mean of quantize-dequantize snapshots, then export of the mean."""

    def __init__(self, tensors: Sequence[ExportTensor], policy=None):
        self.policy = policy if policy is not None else make_policy(int8_patterns=())
        self.exporter_template = list(tensors)
        dev = tensors[0].w.device
        self.means = [torch.empty(t.w.shape, dtype=torch.float32, device=dev) for t in tensors]
        self.mean_ptrs = (ctypes.c_void_p * len(tensors))(*[m.data_ptr() for m in self.means])
        self.n = len(tensors)
        arr, keep = _tensor_in_array(tensors)
        self.plan = (pgq.pgq_tensor_plan * max(self.n, 1))()
        ab, wb = ctypes.c_size_t(0), ctypes.c_size_t(0)
        pgq.check(pgq.pgq_export_plan(arr, self.n, ctypes.byref(self.policy), self.plan, ctypes.byref(ab),
                                      ctypes.byref(wb)), "pgq_export_plan")
        self.workspace_bytes = max(wb.value, 64)
        self.status = new_status(dev)
        self._tables: Dict[tuple, tuple] = {}

    def accumulate(self, snapshot: Sequence[torch.Tensor], k: int, reuse_table: bool = True):
        """Fold snapshot k (1-based) into the means.  The tensor array and the workspace with
        its uploaded table are kept per snapshot buffer set (k is a kernel argument, not part
        of the table), so repeated runs over resident snapshots only re-enqueue the kernel."""
        key = tuple(w.data_ptr() for w in snapshot)
        cached = self._tables.get(key)
        flags = 0
        if cached is not None and reuse_table:
            arr, keep, ws = cached
            flags = pgq.PGQ_TABLE_RESIDENT
        else:
            tensors = [ExportTensor(t.name, w, t.awq_s) for t, w in zip(self.exporter_template, snapshot)]
            arr, keep = _tensor_in_array(tensors)
            ws = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.means[0].device)
            self._tables[key] = (arr, keep, ws)
        rc = pgq.pgq_sqwa_accumulate(arr, self.n, self.plan, self.mean_ptrs, k, _p(ws), ws.numel(), flags,
                                     _p(self.status), _stream())
        pgq.check(rc, "pgq_sqwa_accumulate")

    def exporter(self, want_dq: bool = False) -> Exporter:
        return Exporter([ExportTensor(t.name, m, t.awq_s) for t, m in zip(self.exporter_template, self.means)],
                        self.policy, want_dq=want_dq)


class _Averager:
    """fp32 averages of a fixed list of weight tensors (fp32, bf16 or fp16, rows contiguous), updated
    in place by one grouped launch per call.  The tensor array and the workspace holding the
    uploaded descriptor table are kept per weight buffer set, so calls over resident weights
    only re-enqueue the kernel."""

    def __init__(self, like: Sequence[torch.Tensor]):
        like = list(like)
        self.n = len(like)
        dev = like[0].device
        self.avg = [torch.empty(w.shape, dtype=torch.float32, device=dev) for w in like]
        self.avg_ptrs = (ctypes.c_void_p * self.n)(*[a.data_ptr() for a in self.avg])
        self.status = new_status(dev)
        self._tables: Dict[tuple, tuple] = {}

    def _table(self, weights: Sequence[torch.Tensor], reuse_table: bool):
        key = tuple(w.data_ptr() for w in weights)
        cached = self._tables.get(key)
        if cached is not None and reuse_table:
            return cached + (pgq.PGQ_TABLE_RESIDENT,)
        assert len(weights) == self.n
        arr, keep = _tensor_in_array([ExportTensor("", w) for w in weights])
        wb = ctypes.c_size_t(0)
        pgq.check(pgq.pgq_average_workspace(arr, self.n, ctypes.byref(wb)), "pgq_average_workspace")
        ws = torch.empty(max(wb.value, 64), dtype=torch.uint8, device=self.avg[0].device)
        self._tables[key] = (arr, keep, ws)
        return arr, keep, ws, 0


class Ema(_Averager):
    """Exponential moving average of the weights (decay 0.997 by default)."""

    def __init__(self, like: Sequence[torch.Tensor], decay: float = 0.997):
        super().__init__(like)
        self.decay = decay

    def update(self, weights: Sequence[torch.Tensor], init: bool = False, reuse_table: bool = True):
        arr, _, ws, flags = self._table(weights, reuse_table)
        rc = pgq.pgq_ema_update(arr, self.n, self.avg_ptrs, self.decay, 1 if init else 0, _p(ws), ws.numel(),
                                flags, _p(self.status), _stream())
        pgq.check(rc, "pgq_ema_update")


class Swa(_Averager):
    """Running mean of weight checkpoints k = 1, 2, ... (stochastic weight averaging)."""

    def accumulate(self, weights: Sequence[torch.Tensor], k: int, reuse_table: bool = True):
        arr, _, ws, flags = self._table(weights, reuse_table)
        rc = pgq.pgq_swa_accumulate(arr, self.n, self.avg_ptrs, k, _p(ws), ws.numel(), flags, _p(self.status),
                                    _stream())
        pgq.check(rc, "pgq_swa_accumulate")


def dequant_codes(codes: torch.Tensor, scales: torch.Tensor, cols: int, packed: bool = False,
                  per_tensor: bool = False, awq: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """fp32 weights from stored codes (int8 [rows, cols], or packed uint8 [rows, 3 ceil(cols/4)])
    and fp16 scales (int16 bit patterns); awq: cols fp16 multipliers (int16 bit patterns)."""
    rows = codes.shape[0]
    assert codes.is_contiguous() and scales.is_contiguous()
    if out is None:
        out = torch.empty(rows, cols, dtype=torch.float32, device=codes.device)
    rc = pgq.pgq_dequant_codes(_p(codes), 1 if packed else 0, rows, cols, _p(scales), 1 if per_tensor else 0,
                               _p(awq), _p(out), None, _stream())
    pgq.check(rc, "pgq_dequant_codes")
    return out


def qgemm(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, out: Optional[torch.Tensor] = None,
          out_dtype: torch.dtype = torch.float32) -> torch.Tensor:
    """Y = X What^T with What = bf16(code * s) formed inside the GEMM.  x: bf16 [M, K] (rows
    contiguous), codes: int8 [N, K], scales: fp16 bit patterns [N] (int16); returns Y [M, N] in
    out_dtype: fp32, or bf16 (each element bf16 of the fp32 result, the same accumulation)."""
    assert x.dtype == torch.bfloat16 and x.dim() == 2 and x.stride(1) == 1
    assert codes.dtype == torch.int8 and codes.dim() == 2 and codes.stride(1) == 1
    assert out_dtype in (torch.float32, torch.bfloat16)
    M, K = x.shape
    N = codes.shape[0]
    assert codes.shape[1] == K and scales.numel() == N and scales.is_contiguous()
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=x.device)
    assert out.dtype == out_dtype and out.dim() == 2 and out.shape == (M, N) and out.stride(1) == 1
    fn, name = ((pgq.pgq_qgemm_bf16, "pgq_qgemm_bf16") if out_dtype == torch.float32
                else (pgq.pgq_qgemm_bf16_ybf16, "pgq_qgemm_bf16_ybf16"))
    rc = fn(_p(x), M, K, x.stride(0) if M > 1 else K, _p(codes), codes.stride(0) if N > 1 else K,
            _p(scales), N, _p(out), out.stride(0) if M > 1 else N, _stream())
    pgq.check(rc, name)
    return out


ACTS = {"none": pgq.PGQ_ACT_NONE, "relu": pgq.PGQ_ACT_RELU, "relu2": pgq.PGQ_ACT_RELU2, "silu": pgq.PGQ_ACT_SILU}


# One call per layer and token: the wrappers below keep their own cost to a few microseconds -- plain
# comparisons, the descriptor packed in one go, scratch only when the call asks for it.
_FWD = struct.Struct("15q4ifi")         # pgq_linear_fwd
_BWD = struct.Struct("18q4ifi")        # pgq_linear_bwd
_B16 = (torch.bfloat16,)
_B16_F32 = (torch.bfloat16, torch.float32)
_I8 = (torch.int8,)
_U8 = (torch.uint8,)
_SCALE_TYPES = (torch.float16, torch.int16)


def _matrix(name: str, t: torch.Tensor, rows: int, cols: int, dtypes, index: int) -> int:
    """The row stride of a matrix argument whose rows are contiguous."""
    shape = t.shape
    if len(shape) != 2 or shape[0] != rows or shape[1] != cols:
        raise ValueError(f"{name}: shape {tuple(shape)}, expected {(rows, cols)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected GPU {index}")
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{name}: rows must be contiguous")
    if rows <= 1:
        return cols
    if ld < cols:
        raise ValueError(f"{name}: rows overlap (row stride {ld} < {cols})")
    return ld


def _vector(name: str, t: torch.Tensor, n: int, dtypes, index: int) -> int:
    """The address of an argument of n contiguous values."""
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: {n} contiguous values expected")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected GPU {index}")
    return t.data_ptr()


def _gpu_of(name: str, t: torch.Tensor) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} is on {t.device}, not on a GPU")
    return index


def _launch_linear(fn, size_fn, name: str, desc: bytes, index: int) -> None:
    """One call of a linear-layer entry point on GPU `index`: the scratch, when the call asks for any,
    comes from torch's allocator (ordered with the current stream, private to a graph under capture)."""
    if index != torch.cuda.current_device():
        with torch.cuda.device(index):
            return _launch_linear(fn, size_fn, name, desc, index)
    stream = _stream_of(index)
    rc = fn(desc, None, 0, stream)          # (refused at once, with nothing enqueued, when it needs scratch)
    if rc == pgq.PGQ_ERR_WORKSPACE:
        need = ctypes.c_size_t(0)
        pgq.check(size_fn(desc, ctypes.byref(need)), name)
        ws = torch.empty(need.value, dtype=torch.uint8, device=torch.device("cuda", index))
        rc = fn(desc, ws.data_ptr(), need.value, stream)
    if rc != pgq.PGQ_OK:
        pgq.check(rc, name)


def qlinear(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, bias: Optional[torch.Tensor] = None,
            act: str = "none", slope: float = 0.0, residual: Optional[torch.Tensor] = None, want_z: bool = False,
            out: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16):
    """Y = act(X What^T + b) + R with What = bf16(code * s).

    x: bf16 [M, K]; codes: int8 [N, K]; scales: fp16 [N] (or int16 bit patterns); bias: fp32 or bf16
    [N]; residual: fp32 or bf16 [M, N], which may be `out` itself; act: "none", "relu", "relu2" (both
    with a leaky slope) or "silu".  Returns Y [M, N] in out_dtype (bf16 or fp32), or (Y, Z) with the
    bf16 pre-activation Z that qlinear_backward takes when want_z.  No gradient is recorded (a warning
    says so where one would be expected): call qlinear_backward."""
    if x.dim() != 2 or codes.dim() != 2:
        raise ValueError("x and codes must be matrices")
    (M, K), N, dev = x.shape, codes.shape[0], _gpu_of("x", x)
    ldx, ldc = _matrix("x", x, M, K, _B16, dev), _matrix("codes", codes, N, K, _I8, dev)
    pb = bt = pr = ldr = rt = pz = 0
    if torch.is_grad_enabled() and (x.requires_grad or (bias is not None and bias.requires_grad)
                                    or (residual is not None and residual.requires_grad)):
        warnings.warn("qlinear records no gradient for its arguments: call qlinear_backward, or torch.no_grad() around it",
                      stacklevel=2)
    if bias is not None:
        pb, bt = _vector("bias", bias, N, _B16_F32, dev), _dtype_code(bias.dtype)
    if residual is not None:
        ldr = _matrix("residual", residual, M, N, _B16_F32, dev)
        pr, rt = residual.data_ptr(), _dtype_code(residual.dtype)
    if out_dtype not in _B16_F32:
        raise TypeError(f"unsupported out_dtype {out_dtype}")
    if out is None:
        out = torch.empty(M, N, dtype=out_dtype, device=x.device)
        ldy = N
    else:
        ldy = _matrix("out", out, M, N, (out_dtype,), dev)
    z = None
    if want_z:
        z = torch.empty(M, N, dtype=torch.bfloat16, device=x.device)
        pz = z.data_ptr()
    desc = _FWD.pack(M, N, K, x.data_ptr(), ldx, codes.data_ptr(), ldc, _vector("scales", scales, N, _SCALE_TYPES, dev),
                     pb, pr, ldr, pz, N, out.data_ptr(), ldy, bt, rt, _dtype_code(out_dtype), ACTS[act], slope, 0)
    _launch_linear(pgq._lib.pgq_linear_forward, pgq._lib.pgq_linear_forward_workspace, "pgq_linear_forward", desc, dev)
    return (out, z) if want_z else out


def qlinear_backward(dy: torch.Tensor, codes: Optional[torch.Tensor], scales: Optional[torch.Tensor],
                     x: Optional[torch.Tensor] = None, z: Optional[torch.Tensor] = None, act: str = "none",
                     slope: float = 0.0, mask: Optional[torch.Tensor] = None, want_dx: bool = True,
                     want_dw: bool = True, want_dbias: bool = False, dx_dtype: torch.dtype = torch.bfloat16,
                     dw_dtype: torch.dtype = torch.bfloat16) -> Dict[str, torch.Tensor]:
    """Gradients of qlinear: "dx" [M, K], "dw" [N, K] (of the bf16 weights, zeroed where the fake-quant
    mask bit is 0) and "dbias" fp32 [N], each when wanted; the residual's gradient is dy itself.

    dy: bf16 or fp32 [M, N]; z: the bf16 pre-activation of the forward call (not for act "none"); x:
    bf16 [M, K] (for dw); codes, scales: as in qlinear (for dx); mask: uint8 [N, ceil(K / 8)].  dZ = dy act'(z)
    is an fp32 value that enters the products in two bf16 parts (at most 2^-14 of it is lost) for a bf16 gradient and
    in three (nothing is) for an fp32 one; one is enough, and takes about half as long, where it is a bf16 value:
    a bf16 dy with act "none", or with "relu" and a slope of 0 or a power of two."""
    if dy.dim() != 2:
        raise ValueError("dy must be a matrix")
    (M, N), dev = dy.shape, _gpu_of("dy", dy)
    if want_dx and (codes is None or scales is None):
        raise ValueError("dx needs codes and scales")
    if want_dw and x is None:
        raise ValueError("dw needs x")
    if act != "none" and z is None:
        raise ValueError(f"act {act!r} needs z")
    for t in (codes, x):
        if t is not None and t.dim() != 2:
            raise ValueError("codes and x must be matrices")
    if dx_dtype not in _B16_F32 or dw_dtype not in _B16_F32:
        raise TypeError(f"unsupported gradient types {dx_dtype}, {dw_dtype}")
    K = codes.shape[1] if codes is not None else x.shape[1] if x is not None else 0
    lddy = _matrix("dy", dy, M, N, _B16_F32, dev)
    pz = ldz = px = ldx = pc = ldc = ps = pm = pdx = pdw = pdb = 0
    if act != "none":
        pz, ldz = z.data_ptr(), _matrix("z", z, M, N, _B16, dev)
    res = {}
    if want_dx:
        pc, ldc = codes.data_ptr(), _matrix("codes", codes, N, K, _I8, dev)
        ps = _vector("scales", scales, N, _SCALE_TYPES, dev)
        res["dx"] = torch.empty(M, K, dtype=dx_dtype, device=dy.device)
        pdx = res["dx"].data_ptr()
    if want_dw:
        px, ldx = x.data_ptr(), _matrix("x", x, M, K, _B16, dev)
        res["dw"] = torch.empty(N, K, dtype=dw_dtype, device=dy.device)
        pdw = res["dw"].data_ptr()
        if mask is not None:
            if tuple(mask.shape) != (N, (K + 7) // 8):
                raise ValueError(f"mask: shape {tuple(mask.shape)}, expected {(N, (K + 7) // 8)}")
            pm = _vector("mask", mask, mask.numel(), _U8, dev)
    if want_dbias:
        res["dbias"] = torch.empty(N, dtype=torch.float32, device=dy.device)
        pdb = res["dbias"].data_ptr()
    desc = _BWD.pack(M, N, K, dy.data_ptr(), lddy, pz, ldz, px, ldx, pc, ldc, ps, pm, pdx, K, pdw, K, pdb,
                     _dtype_code(dy.dtype), _dtype_code(dx_dtype), _dtype_code(dw_dtype), ACTS[act], slope, 0)
    _launch_linear(pgq._lib.pgq_linear_backward, pgq._lib.pgq_linear_backward_workspace, "pgq_linear_backward", desc, dev)
    return res


def _same_device(tensors: Sequence[Optional[torch.Tensor]], device) -> None:
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"a tensor is on {t.device}, expected {device}")


def _separate(tensors: Sequence[Optional[torch.Tensor]]) -> None:
    """Tensors that one launch writes: dense, and no two of them in the same memory."""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in tensors if t is not None and t.numel())
    for (_, end), (start, _) in zip(spans, spans[1:]):
        if start < end:
            raise ValueError("two of the weights, copies and states share memory")


def _dense(name: str, t: torch.Tensor, numel: int, dtypes) -> None:
    if t.numel() != numel or not t.is_contiguous():
        raise ValueError(f"{name}: {numel} dense values expected")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: unsupported dtype {t.dtype}")


class AdamW:
    """AdamW over a fixed list of weight tensors (fp32 or bf16, dense), one grouped launch a step.

    lr_scale, weight_decay: one number, or one per tensor.  state_bits: 32 (fp32 m and v) or 8 (codes
    of m and sqrt(v) with a scale byte for every 64 elements).  copies: bf16 tensors (or None each)
    that receive the updated fp32 weights.  states: existing state tensors to go on from -- per tensor
    (m, v), or (m, v, m_scale, v_scale) for 8 bits; zero states are made when it is None.  The
    first step (or decode) uploads the descriptor table, so it cannot be the captured one; the steps
    after it take only the gradients."""

    def __init__(self, weights: Sequence[torch.Tensor], lr: float = 1e-3, betas: Tuple[float, float] = (0.9, 0.999),
                 eps: float = 1e-8, weight_decay=0.01, lr_scale=1.0, state_bits: int = 32, states=None, copies=None,
                 step_count: int = 0, seed: int = 0):
        self.weights = list(weights)
        self.n = n = len(self.weights)
        if n == 0:
            raise ValueError("no weights")
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        self.lr, self.betas, self.eps, self.state_bits = lr, betas, eps, state_bits
        self.step_count, self.seed = step_count, seed
        self.device = self.weights[0].device
        self.copies = list(copies) if copies is not None else [None] * n
        per = [[x] * n if isinstance(x, (int, float)) else list(x) for x in (lr_scale, weight_decay)]
        if states is None:
            states = [self._zero_state(w.numel()) for w in self.weights]
        self.states = [tuple(s) for s in states]
        if any(len(x) != n for x in (self.copies, self.states, *per)):
            raise ValueError(f"{n} tensors: copies, states, lr_scale and weight_decay must have as many entries")
        self._arr = (pgq.pgq_adamw_tensor * n)()
        for i, (w, c, s) in enumerate(zip(self.weights, self.copies, self.states)):
            k = w.numel()
            _dense("weight", w, k, _B16_F32)
            _same_device((w, c, *s), self.device)
            kinds = (torch.float32,) if state_bits == 32 else (torch.uint8,)
            if len(s) != (2 if state_bits == 32 else 4):
                raise ValueError(f"{state_bits}-bit states: {2 if state_bits == 32 else 4} tensors each")
            for name, t, m in zip(("m", "v", "m_scale", "v_scale"), s, (k, k, (k + 63) // 64, (k + 63) // 64)):
                _dense(name, t, m, kinds)
            if c is not None:
                _dense("copy", c, k, (torch.bfloat16,))
            self._arr[i] = pgq.pgq_adamw_tensor(
                w.data_ptr(), 0 if c is None else c.data_ptr(), s[0].data_ptr(), s[1].data_ptr(),
                s[2].data_ptr() if state_bits == 8 else 0, s[3].data_ptr() if state_bits == 8 else 0, k,
                _dtype_code(w.dtype), pgq.PGQ_F32, per[0][i], per[1][i])
        _separate([*self.weights, *self.copies, *(t for s in self.states for t in s)])
        need = ctypes.c_size_t(0)
        pgq.check(pgq.pgq_adamw_workspace(self._arr, n, ctypes.byref(need)), "pgq_adamw_workspace")
        self.workspace = torch.empty(max(need.value, 64), dtype=torch.uint8, device=self.device)
        self.status = new_status(self.device)
        self.hyper = torch.zeros(10, dtype=torch.int32, device=self.device)
        self._uploaded = self._loaded = False
        self._index = _gpu_of("weight", self.weights[0])
        self._numel = [w.numel() for w in self.weights]
        self._ptrs = (ctypes.c_void_p * n)()
        self._g_dtypes = [torch.float32] * n
        self._ws_ptr, self._ws_bytes, self._status_ptr = self.workspace.data_ptr(), self.workspace.numel(), self.status.data_ptr()

    def _zero_state(self, k: int):
        if self.state_bits == 32:
            return tuple(torch.zeros(k, dtype=torch.float32, device=self.device) for _ in range(2))
        return tuple(torch.zeros(m, dtype=torch.uint8, device=self.device) for m in (k, k, (k + 63) // 64, (k + 63) // 64))

    def _hyper(self, lr, grad_scale: float, count: int) -> pgq.pgq_adamw_hyper:
        """The constants of step number `count`."""
        h = pgq.pgq_adamw_hyper()
        pgq.check(pgq.pgq_adamw_hyper_at(self.lr if lr is None else lr, self.betas[0], self.betas[1], self.eps,
                                         count, grad_scale, (self.seed + count) & 0xFFFFFFFF,
                                         ctypes.byref(h)), "pgq_adamw_hyper_at")
        return h

    def load_hyper(self, lr: Optional[float] = None, grad_scale: float = 1.0) -> None:
        """Count a step and write its constants to device memory, for a step that reads them there
        (device_hyper=True): before each replay of a graph that holds such a step.  A replay before the first
        load_hyper changes nothing and sets PGQ_DEV_NO_HYPER in `status`."""
        h = self._hyper(lr, grad_scale, self.step_count + 1)
        self.hyper.copy_(torch.frombuffer(bytearray(bytes(h)), dtype=torch.int32))
        self.step_count += 1
        self._loaded = True

    def step(self, grads: Sequence[torch.Tensor], lr: Optional[float] = None, grad_scale: float = 1.0,
             device_hyper: bool = False) -> None:
        """One update from the gradients (fp32, bf16 or fp16, dense, in memory of their own).  device_hyper: take the constants that
        load_hyper wrote instead of counting this step here; a captured step needs it, since a graph would
        repeat one step's constants."""
        if len(grads) != self.n:
            raise ValueError(f"{len(grads)} gradients for {self.n} weights")
        if not device_hyper and torch.cuda.is_current_stream_capturing():
            raise pgq.PgqError(pgq.PGQ_ERR_PARAM, "a captured step takes its constants from the device (device_hyper=True)")
        if device_hyper and not self._loaded and not torch.cuda.is_current_stream_capturing():
            raise pgq.PgqError(pgq.PGQ_ERR_PARAM, "device_hyper: load_hyper has not written any constants")
        ptrs, numel, types, index = self._ptrs, self._numel, self._g_dtypes, self._index
        for i, g in enumerate(grads):
            if g.numel() != numel[i] or not g.is_contiguous():
                raise ValueError(f"gradient {i}: {numel[i]} dense values expected")
            if g.get_device() != index:
                raise ValueError(f"gradient {i} is on {g.device}, expected GPU {index}")
            ptrs[i] = g.data_ptr()
            if g.dtype is not types[i]:
                self._arr[i].g_dtype = _dtype_code(g.dtype)
                types[i] = g.dtype
        h = None if device_hyper else self._hyper(lr, grad_scale, self.step_count + 1)
        self._on_device(self._enqueue_step, h, ptrs)
        if not device_hyper:
            self.step_count += 1
        self._uploaded = True

    def _enqueue_step(self, h, ptrs) -> None:
        rc = pgq._lib.pgq_adamw_step(self._arr, self.n, self.state_bits, ptrs, h, None if h is not None else _p(self.hyper),
                                     self._ws_ptr, self._ws_bytes, self._table_flags(), self._status_ptr, _stream_of(self._index))
        if rc != pgq.PGQ_OK:
            pgq.check(rc, "pgq_adamw_step")

    def _on_device(self, call, *args):
        """call(*args) with this optimizer's GPU current."""
        if self._index == torch.cuda.current_device():
            return call(*args)
        with torch.cuda.device(self._index):
            return call(*args)

    def _table_flags(self) -> int:
        return pgq.PGQ_TABLE_RESIDENT if self._uploaded else 0

    def decode_states(self, m_out: Optional[Sequence[torch.Tensor]] = None,
                      r_out: Optional[Sequence[torch.Tensor]] = None):
        """The values that 8-bit states hold: lists of bf16 tensors m and r = sqrt(v) (exact), in the given tensors
        (which share no memory) or in new ones."""
        if self.state_bits != 8:
            raise ValueError("32-bit states are held as values")
        outs = []
        for given in (m_out, r_out):
            if given is None:
                given = [torch.empty(w.numel(), dtype=torch.bfloat16, device=self.device) for w in self.weights]
            if len(given) != self.n:
                raise ValueError(f"{len(given)} outputs for {self.n} weights")
            _same_device(given, self.device)
            for t, w in zip(given, self.weights):
                _dense("output", t, w.numel(), (torch.bfloat16,))
            outs.append(given)
        ptrs = [(ctypes.c_void_p * self.n)(*[t.data_ptr() for t in o]) for o in outs]
        self._on_device(self._enqueue_decode, ptrs[0], ptrs[1])
        self._uploaded = True
        return outs[0], outs[1]

    def _enqueue_decode(self, m_ptrs, r_ptrs) -> None:
        pgq.check(pgq.pgq_adamw_decode(self._arr, self.n, m_ptrs, r_ptrs, self._ws_ptr, self._ws_bytes, self._table_flags(),
                                       self._status_ptr, _stream_of(self._index)), "pgq_adamw_decode")
