"""Thin Python binding of libzdmmv.so (the C ABI declared in include/zdmmv.h).

Argument marshalling only: every function passes device pointers
(``tensor.data_ptr()``), sizes and the current CUDA stream to the C entry point
of the same name and raises ``ZdmmvError`` on a non-OK status. All arithmetic
runs in the CUDA kernels; there is no CPU fallback, and loading fails loudly if
the library cannot be built or found.

torch is used only for device memory and streams.
"""
from __future__ import annotations

import ctypes
import re
import struct
import threading

import torch

from . import _build

Q4_0 = 2
Q8_0 = 8
GGUF = 0
REPACKED = 1
QK = 32
MAX_BATCH = 8
BLOCK_BYTES = {Q4_0: 18, Q8_0: 34}
FAULT_WAIT_TIMEOUT = 1
FAULT_SMEM_ALIGN = 2
ARGMAX_WORKSPACE_BYTES = 16384
ROPE_PAIRS = 0
ROPE_HALVES = 1
KV_SLAB = 16

STATUS = {0: "ok", 1: "null pointer", 2: "bad shape", 3: "misaligned pointer or stride",
          4: "unknown layout", 5: "unknown block format", 6: "buffer too small",
          7: "CUDA runtime error", 8: "device fault reported"}


class ZdmmvError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {STATUS.get(code, 'unknown')} (status {code})")
        self.code = code


_lock = threading.Lock()
_lib = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int

# The argument structs of the attention half's entry points, packed field by field (native alignment, as the C
# compiler lays them out); a bytes object passes as a pointer.
_RMSNORM_ARGS = struct.Struct("@6P4qf4x")
_KV_CACHE = struct.Struct("@2Pq5i4x")
_KV_APPEND_ARGS = struct.Struct("@10P4q4i")
_ATTN_ARGS = struct.Struct("@6PNq5if")
_ATTN_TREE = struct.Struct("@2Pi4x")
_ATTN_WEIGHTS_ARGS = struct.Struct("@9PN3q6i2f")
_KV_EVICT_ARGS = struct.Struct("@6P2q4i")
_KV_ACCEPT_ARGS = struct.Struct("@6P2qi4x")
_SIGS = {
    "zdmmv_status_str": ([_int], ctypes.c_char_p),
    "zdmmv_version": ([], ctypes.c_char_p),
    "zdmmv_block_bytes": ([_int], ctypes.c_size_t),
    "zdmmv_quantize_act_q8_0": ([_vp, _i64, _vp, _vp], _int),
    "zdmmv_q8_0": ([_vp, _int, _i64, _i64, _vp, _vp, _vp], _int),
    "zdmmv_q4_0": ([_vp, _int, _i64, _i64, _vp, _vp, _vp], _int),
    "zdmmv_q8_0_batched": ([_vp, _int, _i64, _i64, _vp, _int, _vp, _vp], _int),
    "zdmmv_q4_0_batched": ([_vp, _int, _i64, _i64, _vp, _int, _vp, _vp], _int),
    "zdmmv_dmmv_f32": ([_int, _vp, _int, _i64, _i64, _vp, _int, _vp, _vp], _int),
    "zdmmv_dmmv_xf32": ([_int, _vp, _int, _i64, _i64, _vp, _int, _vp, _vp], _int),
    "zdmmv_dmmv_acc": ([_int, _vp, _int, _i64, _i64, _vp, _vp, _vp, _vp], _int),
    "zdmmv_dmmv_argmax": ([_int, _vp, _int, _i64, _i64, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp], _int),
    "zdmmv_dmmv_argmax_noalloc": ([_int, _vp, _int, _i64, _i64, _vp, _vp, _vp, _vp], _int),
    "zdmmv_expert_gather": ([_int, _vp, _i64, _int, _i64, _i64, _vp, _int, _int, _vp, _i64, _vp, _vp, _vp],
                            _int),
    "zdmmv_expert_gather_ready": ([_int, _vp, _i64, _int, _i64, _i64, _vp, _int, _int, _vp, _i64, _vp, _vp,
                                   _vp], _int),
    "zdmmv_expert_gather_f32": ([_int, _vp, _i64, _int, _i64, _i64, _vp, _int, _int, _vp, _i64, _vp, _vp,
                                 _int, _vp], _int),
    "zdmmv_expert_gather2": ([_int, _vp, _vp, _i64, _int, _i64, _i64, _vp, _int, _int, _vp, _i64, _vp, _vp,
                              _vp, _vp], _int),
    "zdmmv_expert_swiglu": ([_int, _vp, _vp, _i64, _int, _i64, _i64, _vp, _int, _int, _vp, _i64, _vp, _vp,
                             _vp], _int),
    "zdmmv_expert_ffn_workspace_bytes": ([_int, _i64], ctypes.c_size_t),
    "zdmmv_expert_ffn": ([_int, _vp, _vp, _i64, _int, _vp, _i64, _i64, _i64, _vp, _int, _int, _vp, _vp, _vp,
                          ctypes.c_size_t, _vp, _vp], _int),
    "zdmmv_repacked_bytes": ([_int, _i64, _i64], ctypes.c_size_t),
    "zdmmv_repack": ([_int, _vp, _i64, _i64, _vp, ctypes.c_size_t, _vp], _int),
    "zdmmv_host_step_workspace_bytes": ([_i64, _i64, _int], ctypes.c_size_t),
    "zdmmv_host_step": ([_int, _vp, _int, _i64, _i64, _vp, _int, _vp, _vp, ctypes.c_size_t, _vp], _int),
    "zdmmv_debug_block_sums": ([_int, _vp, _int, _i64, _i64, _vp, _vp, _vp], _int),
    "zdmmv_selftest_dp4a": ([_vp, _vp, _vp, _vp, _int, _vp], _int),
    "zdmmv_selftest_wait_timeout": ([_vp, _vp], _int),
    "zdmmv_device_status": ([ctypes.POINTER(ctypes.c_uint32), _int], _int),
    "zdmmv_add_rmsnorm_q8_0": ([_vp, _vp], _int),
    "zdmmv_kv_page_bytes": ([_int, _int, _int], ctypes.c_size_t),
    "zdmmv_kv_append_q4_0": ([_vp, _vp, _vp], _int),
    "zdmmv_attn_q4_0_workspace_bytes": ([_vp, _int, _int, _int], ctypes.c_size_t),
    "zdmmv_attn_q4_0": ([_vp, _vp, _vp], _int),
    "zdmmv_kv_append_at_q4_0": ([_vp, _vp, _vp, _vp], _int),
    "zdmmv_attn_tree_q4_0": ([_vp, _vp, _vp, _vp], _int),
    "zdmmv_attn_weights_q4_0_workspace_bytes": ([_vp, _int, _int, _int], ctypes.c_size_t),
    "zdmmv_attn_weights_q4_0": ([_vp, _vp, _vp], _int),
    "zdmmv_kv_evict_q4_0": ([_vp, _vp, _vp, _vp], _int),
    "zdmmv_kv_accept_q4_0": ([_vp, _vp, _vp], _int),
}


def library_path() -> str:
    return _build.LIB


def lib(build: bool = True) -> ctypes.CDLL:
    """Load libzdmmv.so (building it first if it is stale) and declare its ABI."""
    global _lib
    with _lock:
        if _lib is None:
            path = _build.build() if build else _build.LIB
            L = ctypes.CDLL(path)
            for name, (args, res) in _SIGS.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = res
            _lib = L
    return _lib


def header_functions() -> list[str]:
    """Names of the functions declared in include/zdmmv.h."""
    import os
    hdr = os.path.join(_build.INCLUDE, "zdmmv.h")
    text = open(hdr).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(zdmmv_[a-z0-9_]+)\s*\(", text)))


def _call(name: str, *args):
    rc = getattr(lib(), name)(*args)
    if rc != 0:
        raise ZdmmvError(name, rc)


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("zdmmv: expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("zdmmv: expected a contiguous tensor")
    return t.data_ptr()


def _nbytes(t: torch.Tensor) -> int:
    return t.numel() * t.element_size()


# ---------------------------------------------------------------- entry points
def quantize_act_q8_0(x: torch.Tensor, xq: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 activations (any shape, numel % 32 == 0) -> uint8 Q8_0 blocks."""
    k = x.numel()
    if x.dtype != torch.float32:
        raise ValueError("quantize_act_q8_0: x must be float32")
    if xq is None:
        xq = torch.empty(k // QK * 34, dtype=torch.uint8, device=x.device)
    elif _nbytes(xq) < k // QK * 34:
        raise ValueError("quantize_act_q8_0: xq too small")
    _call("zdmmv_quantize_act_q8_0", _ptr(x), k, _ptr(xq), _stream(stream))
    return xq


def _out(y, shape, device):
    if y is None:
        return torch.empty(shape, dtype=torch.float32, device=device)
    if y.dtype != torch.float32 or y.numel() < int(torch.tensor(shape).prod()):
        raise ValueError("output must be float32 with enough elements")
    return y


def q8_0(w, rows: int, cols: int, xq, y=None, layout: int = GGUF, stream=None):
    y = _out(y, (rows,), w.device)
    _call("zdmmv_q8_0", _ptr(w), layout, rows, cols, _ptr(xq), _ptr(y), _stream(stream))
    return y


def q4_0(w, rows: int, cols: int, xq, y=None, layout: int = GGUF, stream=None):
    y = _out(y, (rows,), w.device)
    _call("zdmmv_q4_0", _ptr(w), layout, rows, cols, _ptr(xq), _ptr(y), _stream(stream))
    return y


def q8_0_batched(w, rows: int, cols: int, xq, batch: int, y=None, layout: int = GGUF, stream=None):
    y = _out(y, (batch, rows), w.device)
    _call("zdmmv_q8_0_batched", _ptr(w), layout, rows, cols, _ptr(xq), batch, _ptr(y), _stream(stream))
    return y


def q4_0_batched(w, rows: int, cols: int, xq, batch: int, y=None, layout: int = GGUF, stream=None):
    y = _out(y, (batch, rows), w.device)
    _call("zdmmv_q4_0_batched", _ptr(w), layout, rows, cols, _ptr(xq), batch, _ptr(y), _stream(stream))
    return y


def dmmv(fmt: int, w, rows: int, cols: int, xq, y=None, layout: int = GGUF, stream=None):
    return (q8_0 if fmt == Q8_0 else q4_0)(w, rows, cols, xq, y=y, layout=layout, stream=stream)


def dmmv_batched(fmt: int, w, rows: int, cols: int, xq, batch: int, y=None, layout: int = GGUF, stream=None):
    f = q8_0_batched if fmt == Q8_0 else q4_0_batched
    return f(w, rows, cols, xq, batch, y=y, layout=layout, stream=stream)


def dmmv_f32(fmt: int, w, rows: int, cols: int, x, batch: int = 1, y=None, layout: int = GGUF,
             stream=None):
    """Fused decode step: quantize the fp32 activation x ([batch][cols]) and run
    the DMMV in one launch; identical to quantize_act_q8_0 followed by dmmv."""
    if x.dtype != torch.float32 or x.numel() != batch * cols:
        raise ValueError("dmmv_f32: x must be float32 [batch][cols]")
    y = _out(y, (batch, rows) if batch > 1 else (rows,), w.device)
    _call("zdmmv_dmmv_f32", fmt, _ptr(w), layout, rows, cols, _ptr(x), batch, _ptr(y), _stream(stream))
    return y


def dmmv_xf32(fmt: int, w, rows: int, cols: int, x, batch: int = 1, y=None, layout: int = GGUF, stream=None):
    """W.x with the fp32 activation taken as is (no quantization); x fp32 [batch][cols]."""
    if x.dtype != torch.float32:
        raise ValueError("dmmv_xf32: x must be float32")
    y = _out(y, (batch, rows) if batch > 1 else (rows,), w.device)
    _call("zdmmv_dmmv_xf32", fmt, _ptr(w), layout, rows, cols, _ptr(x), batch, _ptr(y), _stream(stream))
    return y


def dmmv_acc(fmt: int, w, rows: int, cols: int, xq, y, gate=None, layout: int = GGUF, stream=None):
    """y += s * W.x in place, s = sigmoid(gate[0]) for a device gate scalar, else 1."""
    _call("zdmmv_dmmv_acc", fmt, _ptr(w), layout, rows, cols, _ptr(xq), _ptr(gate), _ptr(y), _stream(stream))
    return y


def dmmv_argmax(fmt: int, w, rows: int, cols: int, xq, workspace=None, out=None, max_out=None,
                layout: int = GGUF, stream=None):
    """Index (int32 device tensor [1]) of the largest of W.x, without writing W.x."""
    if workspace is None:
        workspace = torch.empty(ARGMAX_WORKSPACE_BYTES, dtype=torch.uint8, device=w.device)
    if out is None:
        out = torch.empty(1, dtype=torch.int32, device=w.device)
    _call("zdmmv_dmmv_argmax", fmt, _ptr(w), layout, rows, cols, _ptr(xq), _ptr(out), _ptr(max_out),
          _ptr(workspace), _nbytes(workspace), _stream(stream))
    return out


def dmmv_argmax_noalloc(fmt: int, w, rows: int, cols: int, xq, out=None, max_out=None, layout: int = GGUF,
                        stream=None):
    """The argmax DMMV without a workspace: for callers that cannot allocate
    device memory (see include/zdmmv.h). Overlapping calls race."""
    if out is None:
        out = torch.empty(1, dtype=torch.int32, device=w.device)
    _call("zdmmv_dmmv_argmax_noalloc", fmt, _ptr(w), layout, rows, cols, _ptr(xq), _ptr(out), _ptr(max_out),
          _stream(stream))
    return out


def expert_gather(fmt: int, w_stack, expert_stride: int, rows: int, cols: int, idx, n_experts: int, xq,
                  xq_stride: int, y=None, status=None, layout: int = GGUF, stream=None, idx_ready: bool = False):
    """idx_ready=True calls zdmmv_expert_gather_ready: an earlier expert call on
    the stream has read the same final index list (see include/zdmmv.h)."""
    n = idx.numel()
    if idx.dtype != torch.int32:
        raise ValueError("expert_gather: idx must be int32")
    y = _out(y, (n, rows), w_stack.device)
    _call("zdmmv_expert_gather_ready" if idx_ready else "zdmmv_expert_gather", fmt, _ptr(w_stack), expert_stride,
          layout, rows, cols, _ptr(idx), n, n_experts, _ptr(xq), xq_stride, _ptr(y), _ptr(status), _stream(stream))
    return y


def expert_gather_f32(fmt: int, w_stack, expert_stride: int, rows: int, cols: int, idx, n_experts: int, x,
                      x_stride: int, y=None, status=None, layout: int = GGUF, stream=None, idx_ready: bool = False):
    """Gather over fp32 activations (slot k: x + k*x_stride floats), quantized in the launch."""
    n = idx.numel()
    if idx.dtype != torch.int32:
        raise ValueError("expert_gather_f32: idx must be int32")
    if x.dtype != torch.float32:
        raise ValueError("expert_gather_f32: x must be float32")
    y = _out(y, (n, rows), w_stack.device)
    _call("zdmmv_expert_gather_f32", fmt, _ptr(w_stack), expert_stride, layout, rows, cols, _ptr(idx), n,
          n_experts, _ptr(x), x_stride, _ptr(y), _ptr(status), 1 if idx_ready else 0, _stream(stream))
    return y


def expert_gather2(fmt: int, w_stack_a, w_stack_b, expert_stride: int, rows: int, cols: int, idx,
                   n_experts: int, xq, xq_stride: int, y_a=None, y_b=None, status=None, layout: int = GGUF,
                   stream=None):
    """Two same-shaped expert stacks (e.g. gate and up) in one launch."""
    n = idx.numel()
    if idx.dtype != torch.int32:
        raise ValueError("expert_gather2: idx must be int32")
    y_a = _out(y_a, (n, rows), w_stack_a.device)
    y_b = _out(y_b, (n, rows), w_stack_a.device)
    _call("zdmmv_expert_gather2", fmt, _ptr(w_stack_a), _ptr(w_stack_b), expert_stride, layout, rows, cols,
          _ptr(idx), n, n_experts, _ptr(xq), xq_stride, _ptr(y_a), _ptr(y_b), _ptr(status), _stream(stream))
    return y_a, y_b


def expert_swiglu(fmt: int, w_gate, w_up, rows: int, cols: int, xq, idx=None, expert_stride: int = 0,
                  n_experts: int = 0, xq_stride: int = 0, h=None, status=None, layout: int = GGUF, stream=None):
    """h[k] = silu(G_idx[k] . x_k) * (U_idx[k] . x_k) in one launch; idx=None: one gate/up pair."""
    if idx is not None and idx.dtype != torch.int32:
        raise ValueError("expert_swiglu: idx must be int32")
    n = 1 if idx is None else idx.numel()
    h = _out(h, (n, rows), w_gate.device)
    _call("zdmmv_expert_swiglu", fmt, _ptr(w_gate), _ptr(w_up), expert_stride, layout, rows, cols, _ptr(idx), n,
          n_experts, _ptr(xq), xq_stride, _ptr(h), _ptr(status), _stream(stream))
    return h


def expert_ffn_workspace(n: int, ffn: int, device="cuda"):
    """A zero-filled workspace for expert_ffn (reusable across calls on one stream)."""
    nbytes = lib().zdmmv_expert_ffn_workspace_bytes(n, ffn)
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def expert_ffn(fmt_gate_up: int, w_gate, w_up, gate_up_stride: int, fmt_down: int, w_down, down_stride: int,
               hidden: int, ffn: int, idx, n_experts: int, xq, y=None, workspace=None, status=None, stream=None):
    """The selected experts' gate/up DMMVs, SwiGLU and down DMMV in one launch:
    y[k] = D_idx[k] . q8_0(silu(G_idx[k] . x) * (U_idx[k] . x)). Returns (y, h)."""
    if idx.dtype != torch.int32:
        raise ValueError("expert_ffn: idx must be int32")
    n = idx.numel()
    y = _out(y, (n, hidden), w_gate.device)
    if workspace is None:
        workspace = expert_ffn_workspace(n, ffn, w_gate.device)
    _call("zdmmv_expert_ffn", fmt_gate_up, _ptr(w_gate), _ptr(w_up), gate_up_stride, fmt_down, _ptr(w_down),
          down_stride, hidden, ffn, _ptr(idx), n, n_experts, _ptr(xq), _ptr(y), _ptr(workspace),
          _nbytes(workspace), _ptr(status), _stream(stream))
    h = workspace[: 4 * n * ffn].view(torch.float32).view(n, ffn)
    return y, h


def repacked_bytes(fmt: int, rows: int, cols: int) -> int:
    return int(lib().zdmmv_repacked_bytes(fmt, rows, cols))


def repack(fmt: int, src, rows: int, cols: int, dst=None, stream=None):
    need = repacked_bytes(fmt, rows, cols)
    if dst is None:
        dst = torch.empty(need, dtype=torch.uint8, device=src.device)
    _call("zdmmv_repack", fmt, _ptr(src), rows, cols, _ptr(dst), _nbytes(dst), _stream(stream))
    return dst


def host_step_workspace_bytes(rows: int, cols: int, batch: int = 1) -> int:
    return int(lib().zdmmv_host_step_workspace_bytes(rows, cols, batch))


def host_step(fmt: int, w, rows: int, cols: int, x_host: torch.Tensor, y_host: torch.Tensor, workspace,
              batch: int = 1, layout: int = GGUF, stream=None):
    """One decode step from host activations to host outputs (asynchronous on
    the stream; synchronize before reading y_host)."""
    if x_host.is_cuda or y_host.is_cuda:
        raise ValueError("host_step: x_host and y_host must be host tensors")
    _call("zdmmv_host_step", fmt, _ptr(w), layout, rows, cols, x_host.data_ptr(), batch, y_host.data_ptr(),
          _ptr(workspace), _nbytes(workspace), _stream(stream))
    return y_host


def debug_block_sums(fmt: int, w, rows: int, cols: int, xq, sums=None, layout: int = GGUF, stream=None):
    if sums is None:
        sums = torch.empty((rows, cols // QK), dtype=torch.int32, device=w.device)
    _call("zdmmv_debug_block_sums", fmt, _ptr(w), layout, rows, cols, _ptr(xq), _ptr(sums), _stream(stream))
    return sums


def selftest_dp4a(a, b, c, out=None, stream=None):
    if out is None:
        out = torch.empty_like(a)
    _call("zdmmv_selftest_dp4a", _ptr(a), _ptr(b), _ptr(c), _ptr(out), a.numel(), _stream(stream))
    return out


def selftest_wait_timeout(result=None, stream=None):
    """Run the failure-path self-test (a wait that can never complete, bounded)."""
    if result is None:
        result = torch.zeros(1, dtype=torch.int32, device="cuda")
    _call("zdmmv_selftest_wait_timeout", _ptr(result), _stream(stream))
    return result


def device_status(clear: bool = False) -> int:
    v = ctypes.c_uint32(0)
    _call("zdmmv_device_status", ctypes.byref(v), 1 if clear else 0)
    return int(v.value)


# ------------------------------------------- the attention half of a decode layer
# These calls are a few microseconds on the device: the arguments are checked with as few tensor queries as will do.
_F32, _F16, _U8, _I32 = torch.float32, torch.float16, torch.uint8, torch.int32
_entries: dict = {}


def _entry(name: str):
    fn = _entries.get(name)
    return _entries.setdefault(name, getattr(lib(), name)) if fn is None else fn


def _enter(name: str, *args):
    fn = _entries.get(name)
    if fn is None:
        fn = _entry(name)
    rc = fn(*args)
    if rc != 0:
        raise ZdmmvError(name, rc)


def _raw_stream(stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _bad(what: str):
    raise ValueError(what)


def _rows(t: torch.Tensor, what: str) -> tuple[int, int, int, int]:
    """(data pointer, rows, values of a row, floats between rows) of a float32 CUDA tensor [rows][values] or
    [rows][heads][values of a head]; rows may be any distance apart, the values of a row lie side by side."""
    if t.dtype is not _F32 or not t.is_cuda:
        _bad(f"{what}: expected a float32 CUDA tensor")
    shape, st = t.shape, t.stride()
    if len(shape) == 2:
        rows, width = shape
        side_by_side = st[1] == 1 or width == 1
    elif len(shape) == 3:
        rows, width = shape[0], shape[1] * shape[2]
        side_by_side = (st[2] == 1 or shape[2] == 1) and (st[1] == shape[2] or shape[1] == 1)
    else:
        _bad(f"{what}: expected [rows][values] or [rows][heads][values]")
    if not side_by_side:
        _bad(f"{what}: the values of a row have to lie side by side")
    return t.data_ptr(), rows, width, st[0] if rows > 1 else width


def _whole(t: torch.Tensor, dtype, n: int, what: str) -> int:
    """Data pointer of a contiguous CUDA tensor of at least n values."""
    if t.dtype is not dtype or not t.is_cuda or not t.is_contiguous() or t.numel() < n:
        _bad(f"{what}: expected a contiguous CUDA tensor of {dtype} with {n} values")
    return t.data_ptr()


def _make(shape, dtype, device, stream, how=torch.empty):
    """A tensor for a call on `stream`: of that stream's memory, so that it is not
    handed out again while the call may still be using it."""
    if stream is None:
        return how(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return how(shape, dtype=dtype, device=device)


def add_rmsnorm_q8_0(x, weight, eps: float, residual=None, out=None, xq=None, y=None, stream=None):
    """s = x + residual; the Q8_0 blocks (uint8 tensor, returned) of s / sqrt(mean(s^2) + eps) * weight, per row of
    x (fp32 [rows][cols]; rows may be strided). out: s (may be x or residual); y: fp16, the blocks' values."""
    px, rows, cols, sx = _rows(x, "x")
    pr = sr = pw = po = py = 0
    if residual is not None:
        pr, rrows, rcols, sr = _rows(residual, "residual")
        if rrows != rows or rcols != cols:
            _bad("add_rmsnorm_q8_0: residual must have x's shape")
    if weight is not None:
        pw = _whole(weight, _F32, cols, "weight")
    if out is not None:
        po = _whole(out, _F32, rows * cols, "out")
    nbytes = rows * (cols // QK) * 34
    if xq is None:
        xq = _make(nbytes, _U8, x.device, stream)
    pq = _whole(xq, _U8, nbytes, "xq")
    if y is not None:
        py = _whole(y, _F16, rows * cols, "y")
    _enter("zdmmv_add_rmsnorm_q8_0", _RMSNORM_ARGS.pack(px, pr, pw, po, pq, py, rows, cols, sx, sr, eps),
           _raw_stream(stream))
    return xq


def kv_page_bytes(page_tokens: int, n_kv_heads: int, head_dim: int) -> int:
    return int(lib().zdmmv_kv_page_bytes(page_tokens, n_kv_heads, head_dim))


class KVCache:
    """A paged key/value cache in Q4_0 (zdmmv_kv_cache): `pages` is a uint8 tensor of whole pages (see
    kv_page_bytes), `page_table` int32 [sequences][pages of a sequence]. Both stay the caller's: the table's
    contents may change between calls."""

    def __init__(self, pages, page_tokens: int, n_kv_heads: int, head_dim: int, page_table):
        per = kv_page_bytes(page_tokens, n_kv_heads, head_dim)
        if per == 0:
            _bad("KVCache: page_tokens must be a multiple of 16 up to 1024, head_dim 64, 96, 128, 192 or 256")
        if page_table.dim() != 2:
            _bad("KVCache: page_table must be int32 [n_seq][max_pages]")
        self.pages, self.page_table = pages, page_table
        self.page_tokens, self.n_kv_heads, self.head_dim = page_tokens, n_kv_heads, head_dim
        self.n_pages, (self.n_seq, self.max_pages) = _nbytes(pages) // per, page_table.shape
        self.c = _KV_CACHE.pack(_whole(pages, _U8, 0, "pages"), _whole(page_table, _I32, 0, "page_table"), self.n_pages,
                                self.n_seq, self.max_pages, page_tokens, n_kv_heads, head_dim)


def kv_append_q4_0(cache: KVCache, k, v, seq, pos, q=None, q_out=None, rope=None, rope_style: int = ROPE_HALVES,
                   k_val=None, v_val=None, status=None, stream=None, rope_pos=None):
    """Append tokens (fp32 k and v, [n_tok][heads * head_dim] or [n_tok][heads][head_dim], tokens may be strided) to
    their sequences' pages, rotated by rope (fp32 [positions][rot_dim]: cosines, then sines) and quantized to Q4_0.
    With q, returns it rotated (q_out). k_val, v_val: fp16, the values the cache then holds. rope_pos: int32 [n_tok], the
    rows of rope where they are not pos (drafted trees, a cache that was cut back)."""
    dim = cache.head_dim
    kv = cache.n_kv_heads * dim
    pk, n_tok, wk, sk = _rows(k, "k")
    pv, nv, wv, sv = _rows(v, "v")
    if wk != kv or wv != kv or nv != n_tok:
        _bad(f"kv_append_q4_0: k and v must be [n_tok][{kv}]")
    pq = po = heads = sq = pr = rot = positions = pkv = pvv = ps = 0
    if q is not None:
        pq, nq, wq, sq = _rows(q, "q")
        heads = wq // dim
        if nq != n_tok or heads * dim != wq:
            _bad("kv_append_q4_0: q must be [n_tok][heads * head_dim]")
        if q_out is None:
            q_out = _make((n_tok, heads, dim), _F32, q.device, stream)
        po = _whole(q_out, _F32, n_tok * wq, "q_out")
    if rope is not None:
        positions, rot = rope.shape
        pr = _whole(rope, _F32, 0, "rope")
    if k_val is not None:
        pkv = _whole(k_val, _F16, n_tok * kv, "k_val")
    if v_val is not None:
        pvv = _whole(v_val, _F16, n_tok * kv, "v_val")
    if status is not None:
        ps = _whole(status, _I32, 1, "status")
    args = _KV_APPEND_ARGS.pack(pk, pv, pq, _whole(seq, _I32, n_tok, "seq"), _whole(pos, _I32, n_tok, "pos"), pr, po, pkv,
                                pvv, ps, sk, sv, sq, positions, n_tok, heads, rot, rope_style)
    if rope_pos is None:
        _enter("zdmmv_kv_append_q4_0", cache.c, args, _raw_stream(stream))
    else:
        _enter("zdmmv_kv_append_at_q4_0", cache.c, args, _whole(rope_pos, _I32, n_tok, "rope_pos"), _raw_stream(stream))
    return q_out


def attn_q4_0_workspace_bytes(cache: KVCache, n_q_heads: int, max_q_len: int, max_kv_len: int) -> int:
    return int(lib().zdmmv_attn_q4_0_workspace_bytes(cache.c, n_q_heads, max_q_len, max_kv_len))


def attn_q4_0_workspace(cache: KVCache, n_q_heads: int, max_q_len: int, max_kv_len: int):
    """A workspace for attn_q4_0 calls of these bounds or smaller ones, one in flight at a time (zeros: its counters
    start at zero, and every call leaves them so)."""
    n = attn_q4_0_workspace_bytes(cache, n_q_heads, max_q_len, max_kv_len)
    return torch.zeros(n, dtype=_U8, device=cache.pages.device)


def attn_q4_0(cache: KVCache, q, q_start, kv_len, max_q_len: int, max_kv_len: int, scale: float | None = None,
              window: int = 0, out=None, workspace=None, status=None, stream=None):
    """Attention of the new tokens q (fp32 [n_tok][heads][head_dim] or [n_tok][heads * head_dim]) over the cache;
    sequence s has the rows q_start[s] .. q_start[s+1]-1 and kv_len[s] tokens in the cache. scale: default
    1/sqrt(head_dim). Returns out, fp32 [n_tok][heads][head_dim]."""
    args, out, _, _ = _attn_args("attn_q4_0", cache, q, q_start, kv_len, max_q_len, max_kv_len, scale, window, out, workspace,
                                 status, stream)
    _enter("zdmmv_attn_q4_0", cache.c, args, _raw_stream(stream))
    return out


def _attn_args(who, cache, q, q_start, kv_len, max_q_len, max_kv_len, scale, window, out, workspace, status, stream):
    """(packed zdmmv_attn_args, out, tokens, query heads)."""
    dim, n_seq = cache.head_dim, cache.n_seq
    pq, n_tok, width, sq = _rows(q, "q")
    heads = width // dim
    if heads * dim != width:
        _bad(f"{who}: q must be [n_tok][heads * head_dim]")
    if out is None:
        out = _make((n_tok, heads, dim), _F32, q.device, stream)
    if workspace is None:
        workspace = _make(attn_q4_0_workspace_bytes(cache, heads, max_q_len, max_kv_len), _U8, q.device, stream, torch.zeros)
    args = _ATTN_ARGS.pack(pq, _whole(q_start, _I32, n_seq + 1, "q_start"), _whole(kv_len, _I32, n_seq, "kv_len"),
                           _whole(out, _F32, n_tok * width, "out"), _whole(workspace, _U8, 0, "workspace"),
                           0 if status is None else _whole(status, _I32, 1, "status"), workspace.numel(), sq, n_tok, heads,
                           max_q_len, max_kv_len, window, dim ** -0.5 if scale is None else scale)
    return args, out, n_tok, heads


def attn_tree_q4_0(cache: KVCache, q, q_start, kv_len, max_q_len: int, max_kv_len: int, seen=None, lse=None,
                   scale: float | None = None, window: int = 0, out=None, workspace=None, status=None, stream=None):
    """attn_q4_0 where the new tokens see one another as `seen` says (int32 [n_tok][words], bit j%32 of word j/32 of token
    i's row: it sees the sequence's new token j; None: those before it and itself). lse: fp32 [n_tok][heads], filled
    with the logarithms of the rows' sums of exp(score), for attn_weights_q4_0 or to join parts. Returns out."""
    args, out, n_tok, heads = _attn_args("attn_tree_q4_0", cache, q, q_start, kv_len, max_q_len, max_kv_len, scale, window, out,
                                         workspace, status, stream)
    ps, words = _seen(seen, n_tok)
    tree = _ATTN_TREE.pack(ps, 0 if lse is None else _whole(lse, _F32, n_tok * heads, "lse"), words)
    _enter("zdmmv_attn_tree_q4_0", cache.c, args, tree, _raw_stream(stream))
    return out


def _seen(seen, n_tok: int) -> tuple[int, int]:
    """(data pointer, words of a row) of a tree's bits; (0, 0) for none."""
    if seen is None:
        return 0, 0
    shape = seen.shape
    if len(shape) != 2 or shape[0] < n_tok:
        _bad(f"seen: expected int32 [n_tok][words] with {n_tok} rows")
    return _whole(seen, _I32, 0, "seen"), shape[1]


def _per_head(t: torch.Tensor, cache: KVCache, n: int, what: str) -> tuple[int, int]:
    """(data pointer, floats between kv heads) of a float32 CUDA tensor [n_seq][n_kv_heads][n or more]."""
    shape, n_seq, kv = t.shape, cache.n_seq, cache.n_kv_heads
    if t.dtype is not _F32 or not t.is_cuda or len(shape) != 3 or shape[0] != n_seq or shape[1] != kv or shape[2] < n:
        _bad(f"{what}: expected float32 CUDA [{n_seq}][{kv}][{n} or more]")
    s0, s1, s2 = t.stride()
    if kv == 1:
        s1 = s0 if n_seq > 1 else shape[2]
    if s2 != 1 and shape[2] > 1 or n_seq > 1 and s0 != s1 * kv:
        _bad(f"{what}: kv heads have to lie evenly apart, their values side by side")
    return t.data_ptr(), s1


_FEW_COLUMNS = 24  # rows times heads of a kv head up to which attn_weights_q4_0 needs no workspace (a call spared each step)


def attn_weights_q4_0_workspace_bytes(cache: KVCache, n_q_heads: int, n_tok: int, max_q_len: int) -> int:
    return _entry("zdmmv_attn_weights_q4_0_workspace_bytes")(cache.c, n_q_heads, n_tok, max_q_len)


def attn_weights_q4_0(cache: KVCache, q, q_start, kv_len, lse, max_q_len: int, max_kv_len: int, seen=None,
                      scale: float | None = None, window: int = 0, sums=None, out=None, keep: float = 1.0, workspace=None, status=None,
                      stream=None):
    """What the rows of an attention call gave each cached token: keep * sums + the sum of exp(score - lse) over the rows
    of a kv head that see it (without sums for the new tokens), fp32 [n_seq][n_kv_heads][max_kv_len or more]. lse: as
    attn_tree_q4_0 wrote it for the same q, seen, scale and window. out: where it goes (may be sums; None: a new tensor
    of zeros behind the sequences' ends). workspace: uint8, of attn_weights_q4_0_workspace_bytes (None: a new one where
    one is needed). Returns out."""
    dim, n_seq = cache.head_dim, cache.n_seq
    pq, n_tok, width, sq = _rows(q, "q")
    heads = width // dim
    if heads * dim != width:
        _bad("attn_weights_q4_0: q must be [n_tok][heads * head_dim]")
    if out is None:
        out = _make((n_seq, cache.n_kv_heads, max_kv_len), _F32, q.device, stream, torch.zeros)
    po, so = _per_head(out, cache, max_kv_len, "out")
    pb, sb = (0, 0) if sums is None else _per_head(sums, cache, max_kv_len, "sums")
    ps, words = _seen(seen, n_tok)
    pw = nw = 0
    if workspace is None and heads * min(n_tok, max_q_len) > _FEW_COLUMNS * cache.n_kv_heads:
        workspace = _make(attn_weights_q4_0_workspace_bytes(cache, heads, n_tok, max_q_len), _U8, q.device, stream)
    if workspace is not None:
        pw, nw = _whole(workspace, _U8, 0, "workspace"), workspace.numel()
    args = _ATTN_WEIGHTS_ARGS.pack(pq, _whole(q_start, _I32, n_seq + 1, "q_start"), _whole(kv_len, _I32, n_seq, "kv_len"),
                                   _whole(lse, _F32, n_tok * heads, "lse"), ps, pb, po, pw,
                                   0 if status is None else _whole(status, _I32, 1, "status"), nw, sq, sb, so, n_tok, heads, max_q_len,
                                   max_kv_len, window, words, dim ** -0.5 if scale is None else scale, keep)
    _enter("zdmmv_attn_weights_q4_0", cache.c, args, _raw_stream(stream))
    return out


def kv_evict_q4_0(cache: KVCache, to: KVCache, kv_len, sums, budget: int, max_kv_len: int, sinks: int = 0, recent: int = 0, index=None,
                  sums_out=None, len_out=None, status=None, stream=None):
    """Keep `budget` tokens of each kv head of a longer sequence: the first `sinks`, the last `recent` and those with the
    largest sums (fp32 [n_seq][n_kv_heads][max_kv_len or more]), in their order in the pages of `to`, which are no pages
    of `cache`. Returns index, int32 [n_seq][n_kv_heads][budget]: the kept tokens' positions, -1 behind the last.
    sums_out: the kept tokens' sums; len_out: int32 [n_seq], the new lengths (may be kv_len itself)."""
    n_seq, kv = cache.n_seq, cache.n_kv_heads
    if index is None:
        index = _make((n_seq, kv, budget), _I32, cache.pages.device, stream)
    ps, ss = _per_head(sums, cache, max_kv_len, "sums")
    po, so = (0, 0) if sums_out is None else _per_head(sums_out, cache, budget, "sums_out")
    args = _KV_EVICT_ARGS.pack(_whole(kv_len, _I32, n_seq, "kv_len"), ps, _whole(index, _I32, n_seq * kv * budget, "index"), po,
                               0 if len_out is None else _whole(len_out, _I32, n_seq, "len_out"),
                               0 if status is None else _whole(status, _I32, 1, "status"), ss, so, max_kv_len, budget, sinks, recent)
    _enter("zdmmv_kv_evict_q4_0", cache.c, to.c, args, _raw_stream(stream))
    return index


def kv_accept_q4_0(cache: KVCache, base, path, n_path, sums=None, len_out=None, status=None, stream=None):
    """The accepted path of a drafted tree: of the tokens behind the first base[s] of sequence s, number path[s][j] moves to
    position base[s] + j (j < n_path[s], path rising), and so do sums (fp32 [n_seq][n_kv_heads][tokens], nullable).
    Returns len_out, int32 [n_seq]: the new lengths (it may not be base: its old ones are read until the end)."""
    n_seq, shape = cache.n_seq, path.shape
    if len(shape) != 2 or shape[0] != n_seq:
        _bad("kv_accept_q4_0: path must be int32 [n_seq][max_path]")
    if len_out is None:
        len_out = _make((n_seq,), _I32, path.device, stream)
    args = _KV_ACCEPT_ARGS.pack(_whole(base, _I32, n_seq, "base"), _whole(path, _I32, 0, "path"), _whole(n_path, _I32, n_seq, "n_path"),
                                _whole(len_out, _I32, n_seq, "len_out"), 0 if status is None else _whole(status, _I32, 1, "status"),
                                *((0, 0, 0) if sums is None else (*_per_head(sums, cache, 0, "sums"), sums.shape[2])), shape[1])
    _enter("zdmmv_kv_accept_q4_0", cache.c, args, _raw_stream(stream))
    return len_out
