"""q4_quantized_speech_amd -- GGUF Q4_0 hot path for AMD Instinct MI355X (gfx950).

A thin ctypes binding over the C ABI of ``libq4mi.so`` (declared in
``include/q4.h``).  PyTorch supplies device memory and the current HIP stream;
every computation runs in the library's HIP kernels.  There is no CPU
fallback: if the library is not built, every entry point raises.

Entry points (same names as the C ABI, minus the ``q4_`` prefix):
    matvec(w_q4, x, out=None)                    y = deq(W) x          (M <= 8)
    matmul(w_q4, x, out=None, workspace=True)    Y = X deq(W)^T        (matrix cores)
    matmul_residual(w_q4, x, r, out=None, ...)   Y = R + X deq(W)^T   (fused epilogue)
    embed_rows(table_q4, ids, out=None)          rows of deq(T)
    lmhead_argmax(w_q4, x, workspace=None, ...)  argmax_n (deq(T) x)_n
    quantize(w, out=None, check=True)            float32 -> Q4_0 bytes
    matmul_dx(w_q4, dy, out=None, ...)           dX = dY deq(W): the gradient through a projection
    lmhead_xent(w_q4, x, targets, grad=False)    cross entropy of the head, and its gradient
    lora(x, a, b, ids, scale=None, r=None, ...)  y = r + s_a B_a (A_a x), a = ids[row]
    lora_grad(x, dy, a, b, ids, ...)             its gradient: dx, da, db
    gated_ffn(w_gate, w_up, x, act, r, ...)      h = act(g) u, the gated block's projections
    gated_ffn_grad(w_gate, w_up, z, dh, ...)     its gradient: dx, dz
    lmhead_distill(w_q4, x, top_ids, ...)        loss of the head against a teacher's best logits
    verify_draft(logits, draft, u, probs, ...)   drafted tokens that stand, and the next one

Q4_0 tensors are ``torch.uint8`` of shape [N, 18*K/32] (rows of 32-weight
blocks: binary16 scale + 16 bytes of nibbles, as stored in GGUF).
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq4mi.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "q4.h")

QK = 32
BLOCK_BYTES = 18

(Q4_OK, Q4_ERR_NULL, Q4_ERR_SHAPE, Q4_ERR_ALIGN, Q4_ERR_WORKSPACE, Q4_ERR_HIP, Q4_ERR_FORMAT,
 Q4_ERR_IO, Q4_ERR_NOT_FOUND) = range(9)


class Q4Error(RuntimeError):
    def __init__(self, status: int, where: str, hip_error: int = 0):
        msg = f"{where}: {status_string(status)} (status {status}"
        if status == Q4_ERR_HIP:
            msg += f", hipError {hip_error}"
        super().__init__(msg + ")")
        self.status = status
        self.hip_error = hip_error


_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_SIGS = {
    "q4_abi_version": ([], ctypes.c_int),
    "q4_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "q4_last_hip_error": ([], ctypes.c_int),
    "q4_row_bytes": ([_I64], _SZ),
    "q4_matvec": ([_P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "q4_matmul_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "q4_matmul": ([_P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], ctypes.c_int),
    "q4_matmul_residual_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "q4_matmul_residual": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], ctypes.c_int),
    "q4_embed_rows": ([_P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "q4_lmhead_argmax_workspace_bytes": ([_I64, _I64, _I64], _SZ),
    "q4_lmhead_argmax": ([_P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P], ctypes.c_int),
    "q4_quantize": ([_P, _P, _I64, _I64, _P, _P], ctypes.c_int),
    "q4_lmhead_argmax_noalloc": ([_P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "q4_decode_chain": ([_P, _I64, _P, _I64, _I64, _P, _P, _P, _P, _P, _SZ, _P], ctypes.c_int),
    "q4_matmul_route": ([_I64, _I64, _I64, _SZ, _P], ctypes.c_char_p),
    "q4_matvec_route": ([_I64, _I64, ctypes.c_int32], ctypes.c_char_p),
    "q4_matmul_dx_workspace_bytes": ([ctypes.c_int32, _I64, _I64, _I64], _SZ),
    "q4_matmul_dx": ([_P] * 3 + [ctypes.c_int32] + [_I64] * 3 + [_P, _SZ, _P], ctypes.c_int),
    "q4_lmhead_xent_workspace_bytes": ([ctypes.c_int32] * 2 + [_I64] * 3, _SZ),
    "q4_lmhead_xent": ([_P] * 7 + [ctypes.c_int32] + [_I64] * 3 + [_P, _SZ, _P], ctypes.c_int),
    "q4_lora_workspace_bytes": ([_I64, _I64, _I64, _I64], _SZ),
    "q4_lora": ([_P] * 7 + [ctypes.c_int32] * 2 + [_I64] * 5 + [_P, _SZ, _P], ctypes.c_int),
    "q4_lora_grad_workspace_bytes": ([_I64, _I64, _I64, _I64], _SZ),
    "q4_lora_grad": ([_P] * 10 + [ctypes.c_int32] * 2 + [_I64] * 5 + [_P, _SZ, _P], ctypes.c_int),
    "q4_gated_ffn_workspace_bytes": ([ctypes.c_int32] + [_I64] * 3, _SZ),
    "q4_gated_ffn": ([_P] * 6 + [ctypes.c_int32] * 2 + [_I64] * 3 + [_P, _SZ, _P], ctypes.c_int),
    "q4_gated_ffn_grad_workspace_bytes": ([ctypes.c_int32] + [_I64] * 3, _SZ),
    "q4_gated_ffn_grad": ([_P] * 6 + [ctypes.c_int32] * 2 + [_I64] * 3 + [_P, _SZ, _P], ctypes.c_int),
    "q4_lmhead_distill_workspace_bytes": ([ctypes.c_int32] * 2 + [_I64] * 4, _SZ),
    "q4_lmhead_distill": ([_P] * 4 + [ctypes.c_double] + [_P] * 4 + [ctypes.c_int32] + [_I64] * 4
                          + [_P, _SZ, _P], ctypes.c_int),
    "q4_verify_draft_workspace_bytes": ([_I64] * 3, _SZ),
    "q4_verify_draft": ([_P] * 5 + [ctypes.c_double] + [_P] * 2 + [ctypes.c_int32] + [_I64] * 3
                        + [_P, _SZ, _P], ctypes.c_int),
    "q4_gguf_open": ([_P, _I64, _P], ctypes.c_int),
    "q4_gguf_close": ([_P], None),
    "q4_gguf_version": ([_P], ctypes.c_uint32),
    "q4_gguf_alignment": ([_P], ctypes.c_uint64),
    "q4_gguf_data_offset": ([_P], ctypes.c_uint64),
    "q4_gguf_tensor_count": ([_P], _I64),
    "q4_gguf_metadata_count": ([_P], _I64),
    "q4_gguf_tensor_info": ([_P, _I64, _P, _P, _P, _P, _P, _P], ctypes.c_int),
    "q4_gguf_find_tensor": ([_P, ctypes.c_char_p], _I64),
    "q4_gguf_read_tensor": ([_P, _I64, _P, ctypes.c_uint64], ctypes.c_int),
    "q4_gguf_metadata_key": ([_P, _I64, _P, _P], ctypes.c_int),
    "q4_gguf_metadata_int": ([_P, ctypes.c_char_p, _P], ctypes.c_int),
    "q4_gguf_metadata_float": ([_P, ctypes.c_char_p, _P], ctypes.c_int),
    "q4_gguf_metadata_string": ([_P, ctypes.c_char_p, _P, _P], ctypes.c_int),
    "q4_gguf_metadata_array": ([_P, ctypes.c_char_p, _P, _P], ctypes.c_int),
}


def lib() -> ctypes.CDLL:
    """Load libq4mi.so (built in-tree by q4_quantized_speech_amd.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built: run `python -m q4_quantized_speech_amd.build` "
                "(there is no CPU fallback)")
        handle = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGS.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def status_string(status: int) -> str:
    return lib().q4_status_string(status).decode()


def _check(status: int, where: str) -> None:
    if status != Q4_OK:
        raise Q4Error(status, where, lib().q4_last_hip_error() if status == Q4_ERR_HIP else 0)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _on(stream):
    """Context in which tensors this module allocates (outputs, workspaces,
    flags) come from ``stream``'s pool and their fills run on ``stream``: the
    library's kernel runs there, so nothing else orders them before it, and
    a buffer freed back to another stream's pool could be reused by that
    stream while the kernel still writes it.  The caller orders its own
    inputs with ``stream``."""
    import contextlib
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must live on the GPU")


def q4_shape(w_q4: torch.Tensor):
    """(N, K) of a Q4_0 tensor of shape [N, 18*K/32]."""
    if w_q4.dtype != torch.uint8 or w_q4.dim() != 2 or not w_q4.is_contiguous():
        raise ValueError("Q4_0 weights must be a contiguous uint8 tensor [N, 18*K/32]")
    n, rb = w_q4.shape
    if rb % BLOCK_BYTES:
        raise ValueError(f"row length {rb} is not a multiple of {BLOCK_BYTES}")
    return n, rb // BLOCK_BYTES * QK


def row_bytes(k: int) -> int:
    return int(lib().q4_row_bytes(k))


def _as_2d_f32(x: torch.Tensor, k: int) -> torch.Tensor:
    if x.dtype != torch.float32 or not x.is_contiguous():
        raise ValueError("activations must be contiguous float32")
    if x.dim() == 1:
        x = x.view(1, -1)
    if x.dim() != 2 or x.shape[1] != k:
        raise ValueError(f"activations must be [M, {k}]")
    return x


def matvec(w_q4: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    """y[m, n] = sum_k deq(W)[n, k] x[m, k] (float32 FMA path); x is [K] or [M, K]."""
    n, k = q4_shape(w_q4)
    squeeze = x.dim() == 1
    x2 = _as_2d_f32(x, k)
    m = x2.shape[0]
    with _on(stream):
        if out is None:
            out = torch.empty((m, n), dtype=torch.float32, device=x.device)
        _need_cuda(w_q4, x2, out)
        _check(lib().q4_matvec(_ptr(w_q4), _ptr(x2), _ptr(out), m, n, k, _stream(stream)),
               "q4_matvec")
    return out.view(n) if squeeze else out


def matmul_workspace(m: int, n: int, k: int, device) -> torch.Tensor | None:
    """A workspace for matmul's K split on the current device (None if no split is planned)."""
    nbytes = int(lib().q4_matmul_workspace_bytes(m, n, k))
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def matmul(w_q4: torch.Tensor, x: torch.Tensor, out: torch.Tensor | None = None,
           workspace: torch.Tensor | None | bool = True, stream=None):
    """Y = X deq(W)^T.  M >= 5: on the matrix cores with binary16 operands and
    float32 accumulation.  M <= 4: q4_matvec's bound, either through the matvec
    kernel (rows of x in pairs) or with exact weights and a two-part x on the
    matrix cores.

    ``workspace``: a uint8 device tensor for the K split, ``True`` to allocate the
    planned size here, or ``None``/``False`` for no split."""
    n, k = q4_shape(w_q4)
    x2 = _as_2d_f32(x, k)
    m = x2.shape[0]
    with _on(stream):
        if out is None:
            out = torch.empty((m, n), dtype=torch.float32, device=x.device)
        if workspace is True:
            workspace = matmul_workspace(m, n, k, x.device)
        elif workspace is False:
            workspace = None
        _need_cuda(w_q4, x2, out, workspace)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(lib().q4_matmul(_ptr(w_q4), _ptr(x2), _ptr(out), m, n, k, _ptr(workspace), ws_bytes,
                               _stream(stream)), "q4_matmul")
    return out


def matmul_residual_workspace(m: int, n: int, k: int, device) -> torch.Tensor | None:
    """A workspace that covers matmul_residual for the shape on the current
    device, in place or not (None if none is needed)."""
    nbytes = int(lib().q4_matmul_residual_workspace_bytes(m, n, k))
    if nbytes == 0:
        return None
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def matmul_residual(w_q4: torch.Tensor, x: torch.Tensor, r: torch.Tensor,
                    out: torch.Tensor | None = None,
                    workspace: torch.Tensor | None | bool = True, stream=None):
    """Y = R + X deq(W)^T, the add fused into the product's epilogue where
    the route allows (bit for bit R + matmul(...) in float32).  ``out`` may be
    ``r`` itself (in place).  ``workspace`` as for matmul; ``True`` allocates
    what the shape needs, in place included."""
    n, k = q4_shape(w_q4)
    x2 = _as_2d_f32(x, k)
    m = x2.shape[0]
    if r.dtype != torch.float32 or tuple(r.shape) != (m, n) or not r.is_contiguous():
        raise ValueError(f"r must be a contiguous float32 [{m}, {n}] tensor")
    with _on(stream):
        if out is None:
            out = torch.empty((m, n), dtype=torch.float32, device=x.device)
        if workspace is True:
            workspace = matmul_residual_workspace(m, n, k, x.device)
        elif workspace is False:
            workspace = None
        _need_cuda(w_q4, x2, r, out, workspace)
        ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
        _check(lib().q4_matmul_residual(_ptr(w_q4), _ptr(x2), _ptr(r), _ptr(out), m, n, k,
                                        _ptr(workspace), ws_bytes, _stream(stream)),
               "q4_matmul_residual")
    return out


def matmul_route(m: int, n: int, k: int, ws_bytes: int = 0):
    """(kernel name, K splits) q4_matmul takes for the shape and workspace size."""
    sp = ctypes.c_int32(0)
    r = lib().q4_matmul_route(m, n, k, ws_bytes, ctypes.byref(sp))
    if r is None:
        raise ValueError(f"q4_matmul rejects M={m} N={n} K={k}")
    return r.decode(), int(sp.value)


def matvec_route(n: int, k: int, argmax: bool = False) -> str:
    """Kernel variant q4_matvec (or q4_lmhead_argmax) takes for an N x K matrix."""
    r = lib().q4_matvec_route(n, k, 1 if argmax else 0)
    if r is None:
        raise ValueError(f"rejected shape N={n} K={k}")
    return r.decode()


def embed_rows(table_q4: torch.Tensor, ids: torch.Tensor, out: torch.Tensor | None = None,
               stream=None):
    """out[i, :] = deq(T)[ids[i], :]; ids outside [0, N) give zero rows."""
    n, k = q4_shape(table_q4)
    if ids.dtype != torch.int32 or ids.dim() != 1 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 vector")
    m = ids.shape[0]
    with _on(stream):
        if out is None:
            out = torch.empty((m, k), dtype=torch.float32, device=ids.device)
        _need_cuda(table_q4, ids, out)
        _check(lib().q4_embed_rows(_ptr(table_q4), _ptr(ids), _ptr(out), m, n, k, _stream(stream)),
               "q4_embed_rows")
    return out


def lmhead_workspace(m: int, device) -> torch.Tensor:
    """A zeroed workspace for lmhead_argmax; each call leaves it zeroed, so it
    can be reused by calls ordered on one stream."""
    nbytes = int(lib().q4_lmhead_argmax_workspace_bytes(m, 0, 0))
    if nbytes == 0:
        raise ValueError("M out of range for lmhead_argmax")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def lmhead_argmax(w_q4: torch.Tensor, x: torch.Tensor, workspace: torch.Tensor | None = None,
                  out_idx: torch.Tensor | None = None, out_val: torch.Tensor | None = None,
                  stream=None):
    """(idx, val): per row of x, the lowest n maximising (deq(T) x)_n and that maximum."""
    n, k = q4_shape(w_q4)
    x2 = _as_2d_f32(x, k)
    m = x2.shape[0]
    with _on(stream):
        if workspace is None:
            workspace = lmhead_workspace(m, x.device)   # zero-filled on `stream`
        if out_idx is None:
            out_idx = torch.empty(m, dtype=torch.int32, device=x.device)
        if out_val is None:
            out_val = torch.empty(m, dtype=torch.float32, device=x.device)
        _need_cuda(w_q4, x2, workspace, out_idx, out_val)
        _check(lib().q4_lmhead_argmax(_ptr(w_q4), _ptr(x2), _ptr(out_idx), _ptr(out_val), m, n, k,
                                      _ptr(workspace), workspace.numel(), _stream(stream)),
               "q4_lmhead_argmax")
    return out_idx, out_val


class _Step(ctypes.Structure):
    _fields_ = [("w_q4", ctypes.c_void_p), ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64)]


def decode_chain(steps, table_q4: torch.Tensor | None = None, head_x: torch.Tensor | None = None,
                 out_idx: torch.Tensor | None = None, out_val: torch.Tensor | None = None,
                 out_embed: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None):
    """One decode step's Q4_0 work in order on one stream: ``steps`` is a list
    of (w_q4, x, y) matvecs at M = 1 (x may be a view into an earlier y), then,
    with ``table_q4``, the argmax over deq(T) head_x and, with ``out_embed``,
    the chosen token's decoded row.  Returns (out_idx, out_val, out_embed)."""
    arr = (_Step * max(1, len(steps)))()
    keep = []
    for i, (w, x, y) in enumerate(steps):
        n, k = q4_shape(w)
        if x.dtype != torch.float32 or x.dim() != 1 or x.shape[0] != k or not x.is_contiguous():
            raise ValueError(f"step {i}: x must be a contiguous float32 vector of {k}")
        if y.dtype != torch.float32 or y.dim() != 1 or y.shape[0] != n or not y.is_contiguous():
            raise ValueError(f"step {i}: y must be a contiguous float32 vector of {n}")
        _need_cuda(w, x, y)
        arr[i] = _Step(w.data_ptr(), x.data_ptr(), y.data_ptr(), n, k)
        keep.append((w, x, y))
    vocab = dim = 0
    with _on(stream):
        if table_q4 is not None:
            vocab, dim = q4_shape(table_q4)
            if head_x is None or head_x.dtype != torch.float32 or head_x.numel() != dim \
                    or not head_x.is_contiguous():
                raise ValueError(f"head_x must be a contiguous float32 vector of {dim}")
            if workspace is None:
                workspace = lmhead_workspace(1, head_x.device)
            if out_idx is None:
                out_idx = torch.empty(1, dtype=torch.int32, device=head_x.device)
            _need_cuda(table_q4, head_x, out_idx, out_val, out_embed, workspace)
        ws_bytes = 0 if workspace is None else workspace.numel()
        _check(lib().q4_decode_chain(ctypes.cast(arr, ctypes.c_void_p), len(steps), _ptr(table_q4),
                                     vocab, dim, _ptr(head_x), _ptr(out_idx), _ptr(out_val),
                                     _ptr(out_embed), _ptr(workspace), ws_bytes, _stream(stream)),
               "q4_decode_chain")
    return out_idx, out_val, out_embed


def lmhead_argmax_noalloc(w_q4: torch.Tensor, x: torch.Tensor, out_idx: torch.Tensor,
                          out_val: torch.Tensor | None = None, stream=None):
    """lmhead_argmax with the library's own scratch: the caller passes the
    outputs, nothing is allocated (M <= 64; calls on one GPU must be ordered)."""
    n, k = q4_shape(w_q4)
    x2 = _as_2d_f32(x, k)
    m = x2.shape[0]
    _need_cuda(w_q4, x2, out_idx, out_val)
    if out_idx.dtype != torch.int32 or out_idx.numel() < m or not out_idx.is_contiguous():
        raise ValueError("out_idx must be a contiguous int32 tensor of at least M entries")
    if out_val is not None and (out_val.dtype != torch.float32 or out_val.numel() < m
                                or not out_val.is_contiguous()):
        raise ValueError("out_val must be a contiguous float32 tensor of at least M entries")
    _check(lib().q4_lmhead_argmax_noalloc(_ptr(w_q4), _ptr(x2), _ptr(out_idx), _ptr(out_val), m,
                                          n, k, _stream(stream)), "q4_lmhead_argmax_noalloc")
    return out_idx, out_val


def quantize(w: torch.Tensor, out: torch.Tensor | None = None, check: bool = True, stream=None):
    """GGUF Q4_0 encoding of a float32 [N, K] tensor on the GPU."""
    if w.dtype != torch.float32 or w.dim() != 2 or not w.is_contiguous():
        raise ValueError("w must be a contiguous float32 [N, K] tensor")
    n, k = w.shape
    if k % QK:
        raise ValueError("K must be a multiple of 32")
    with _on(stream):
        if out is None:
            out = torch.empty((n, k // QK * BLOCK_BYTES), dtype=torch.uint8, device=w.device)
        flag = torch.zeros(4, dtype=torch.int32, device=w.device) if check else None
        _need_cuda(w, out, flag)
        _check(lib().q4_quantize(_ptr(w), _ptr(out), n, k, _ptr(flag), _stream(stream)),
               "q4_quantize")
        # the copy behind item() runs on `stream`, after the kernel
        bad = check and int(flag[0].item()) != 0
    if bad:
        raise ValueError("q4_quantize: non-finite input or a scale overflowing binary16")
    return out


# Element types of the operators that adapt a frozen model (Q4_TYPE_* of the ABI).
_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 30}


def _addr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _matrix(t: torch.Tensor, name: str, shape, dtype) -> None:
    """A contiguous tensor of `shape` and `dtype`."""
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)}, "
                         f"got {t.dtype} {list(t.shape)}")


def _activations(t: torch.Tensor, name: str) -> int:
    """The type code of a contiguous activation matrix."""
    code = _TYPES.get(t.dtype)
    if code is None or t.dim() != 2 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous matrix of float32, float16 or bfloat16")
    return code


def _gpu(first, *rest) -> int:
    """The GPU all tensors live on, which has to be the current one (the library
    launches on the current device)."""
    dev = first.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        raise ValueError("tensors must live on the current GPU")
    for t in rest:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors must live on the current GPU")
    return dev


@functools.lru_cache(maxsize=4096)
def _scratch_bytes(query: str, dev: int, *args) -> int:
    """A workspace size (it depends on the sizes and the device's CUs alone)."""
    return int(getattr(lib(), query)(*args))


def _scratch(workspace, query: str, dev: int, *args):
    """The caller's uint8 workspace, or one from the current stream's pool."""
    if workspace is None:
        return torch.empty(_scratch_bytes(query, dev, *args), dtype=torch.uint8,
                           device=torch.device("cuda", dev))
    if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.get_device() != dev:
        raise ValueError("workspace must be a contiguous uint8 tensor on the same GPU")
    return workspace


def _realigned(status: int, *vectors):
    """After a call refused for its alignment: the vectors it reads, copied on the current
    stream where they start inside a 16-byte word (as the targets tokens[1:] do), or None if
    none does and the call stays refused."""
    if status != Q4_ERR_ALIGN or not any(v is not None and v.data_ptr() % 16 for v in vectors):
        return None
    return [v.clone() if v is not None and v.data_ptr() % 16 else v for v in vectors]


def _raw_stream(dev: int) -> int:
    """The current stream's handle."""
    return torch._C._cuda_getCurrentRawStream(dev)


def matmul_dx(w_q4: torch.Tensor, dy: torch.Tensor, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None):
    """dX = dY deq(W), the gradient of ``matmul`` with respect to x: dy is [M, N] of float32,
    float16 or bfloat16, the result [M, K] of its type.  Without ``workspace`` one is
    allocated: dy's operands and, for split sums, float32 copies of the result (42 MB for
    375 x 18432 x 3072 in float32); very many rows of a small matrix also keep the
    decoded weights."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return matmul_dx(w_q4, dy, out, workspace)
    n, k = q4_shape(w_q4)
    t = _activations(dy, "dy")
    m, n2 = dy.shape
    if n2 != n:
        raise ValueError(f"dy must be [M, {n}]")
    if out is not None:
        _matrix(out, "out", (m, k), dy.dtype)
    dev = _gpu(w_q4, dy, out)
    if out is None:
        out = torch.empty((m, k), dtype=dy.dtype, device=dy.device)
    ws = _scratch(workspace, "q4_matmul_dx_workspace_bytes", dev, t, m, n, k)
    _check(lib().q4_matmul_dx(w_q4.data_ptr(), dy.data_ptr(), out.data_ptr(), t, m, n, k,
                              ws.data_ptr(), ws.numel(), _raw_stream(dev)), "q4_matmul_dx")
    return out


def lmhead_xent(w_q4: torch.Tensor, x: torch.Tensor, targets: torch.Tensor, grad: bool = False,
                dloss: torch.Tensor | None = None, loss: torch.Tensor | None = None,
                lse: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                workspace: torch.Tensor | None = None, stream=None):
    """(loss, lse, dx): per row of x, lse = logsumexp(deq(T) x), loss = lse - the target's
    logit (float32), and with ``grad`` (or a ``dx`` to write) the gradient of
    sum(dloss * loss) with respect to x, in x's type; dx is None otherwise.  Rows whose
    target is outside [0, N) have loss 0 and dx 0.  Logits are kept in pieces of the
    vocabulary, at most 256 MiB of them (512 MiB for more than 32768 rows)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return lmhead_xent(w_q4, x, targets, grad, dloss, loss, lse, dx, workspace)
    n, k = q4_shape(w_q4)
    t = _activations(x, "x")
    m, k2 = x.shape
    if k2 != k:
        raise ValueError(f"x must be [M, {k}]")
    _matrix(targets, "targets", (m,), torch.int32)
    for v, name in ((dloss, "dloss"), (loss, "loss"), (lse, "lse")):
        if v is not None:
            _matrix(v, name, (m,), torch.float32)
    if dx is not None:
        _matrix(dx, "dx", (m, k), x.dtype)
        grad = True
    dev = _gpu(w_q4, x, targets, dloss, loss, lse, dx)
    if loss is None:
        loss = torch.empty(m, dtype=torch.float32, device=x.device)
    if lse is None:
        lse = torch.empty(m, dtype=torch.float32, device=x.device)
    if grad and dx is None:
        dx = torch.empty((m, k), dtype=x.dtype, device=x.device)
    ws = _scratch(workspace, "q4_lmhead_xent_workspace_bytes", dev, t, int(bool(grad)), m, n, k)
    status = lib().q4_lmhead_xent(w_q4.data_ptr(), x.data_ptr(), targets.data_ptr(), _addr(dloss),
                                  loss.data_ptr(), lse.data_ptr(), _addr(dx), t, m, n, k,
                                  ws.data_ptr(), ws.numel(), _raw_stream(dev))
    again = _realigned(status, targets, dloss)
    if again:
        return lmhead_xent(w_q4, x, again[0], grad, again[1], loss, lse, dx, ws)
    _check(status, "q4_lmhead_xent")
    return loss, lse, dx


def _adapters(x, a, b, ids, scale):
    """(type code, adapters' type code, M, N, K, R, adapters) of a low-rank adapter call."""
    t = _activations(x, "x")
    m, k = x.shape
    if a.dim() != 3 or b.dim() != 3:
        raise ValueError("a must be [adapters, R, K] and b [adapters, N, R]")
    na, rank, ka = a.shape
    nb, n, rb = b.shape
    if ka != k or nb != na or rb != rank or not a.is_contiguous() or not b.is_contiguous():
        raise ValueError(f"a and b must be contiguous [adapters, R, {k}] and [adapters, N, R], "
                         f"got {list(a.shape)} and {list(b.shape)}")
    ta = _TYPES.get(a.dtype)
    if ta is None or b.dtype != a.dtype:
        raise ValueError("a and b must both be float32, float16 or bfloat16")
    _matrix(ids, "ids", (m,), torch.int32)
    if scale is not None:
        _matrix(scale, "scale", (na,), torch.float32)
    return t, ta, m, n, k, rank, na


def lora(x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, ids: torch.Tensor,
         scale: torch.Tensor | None = None, r: torch.Tensor | None = None,
         out: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """y[m] = r[m] + scale[i] B_i (A_i x[m]) with i = ids[m]: low-rank adapters of many
    requests at once.  x is [M, K] (float32, float16 or bfloat16), a [adapters, R, K] and
    b [adapters, N, R] (x's type, or float32; with a float32 x any of the three), ids int32
    [M]; an id outside [0, adapters) leaves y = r.  r (zeros if None) may be ``out``.
    With ``matmul_residual(w, x, y, out=y)`` after it, which takes float32, y is the
    adapted projection."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return lora(x, a, b, ids, scale, r, out, workspace)
    t, ta, m, n, k, rank, na = _adapters(x, a, b, ids, scale)
    if r is not None:
        _matrix(r, "r", (m, n), x.dtype)
    if out is not None:
        _matrix(out, "out", (m, n), x.dtype)
    dev = _gpu(x, a, b, ids, scale, r, out)
    if out is None:
        out = torch.empty((m, n), dtype=x.dtype, device=x.device)
    ws = _scratch(workspace, "q4_lora_workspace_bytes", dev, m, n, k, rank)
    status = lib().q4_lora(x.data_ptr(), a.data_ptr(), b.data_ptr(), _addr(scale), ids.data_ptr(),
                           _addr(r), out.data_ptr(), t, ta, m, n, k, rank, na, ws.data_ptr(),
                           ws.numel(), _raw_stream(dev))
    again = _realigned(status, ids, scale)
    if again:
        return lora(x, a, b, again[0], again[1], r, out, ws)
    _check(status, "q4_lora")
    return out


def lora_grad(x: torch.Tensor, dy: torch.Tensor, a: torch.Tensor, b: torch.Tensor,
              ids: torch.Tensor, scale: torch.Tensor | None = None, r: torch.Tensor | None = None,
              dx: torch.Tensor | None = None, da: torch.Tensor | None = None,
              db: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """(dx, da, db): the gradient of ``lora`` for dy [M, N], the gradient of its y.
    dx = r + scale A^T B^T dy row by row (x's type; r zeros if None, or the gradient
    through the projection itself, may be ``dx``); da and db are float32, summed over
    the rows of each adapter, zeros for one without rows."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return lora_grad(x, dy, a, b, ids, scale, r, dx, da, db, workspace)
    t, ta, m, n, k, rank, na = _adapters(x, a, b, ids, scale)
    _matrix(dy, "dy", (m, n), x.dtype)
    if r is not None:
        _matrix(r, "r", (m, k), x.dtype)
    if dx is not None:
        _matrix(dx, "dx", (m, k), x.dtype)
    if da is not None:
        _matrix(da, "da", (na, rank, k), torch.float32)
    if db is not None:
        _matrix(db, "db", (na, n, rank), torch.float32)
    dev = _gpu(x, dy, a, b, ids, scale, r, dx, da, db)
    if dx is None:
        dx = torch.empty((m, k), dtype=x.dtype, device=x.device)
    if da is None:
        da = torch.empty((na, rank, k), dtype=torch.float32, device=x.device)
    if db is None:
        db = torch.empty((na, n, rank), dtype=torch.float32, device=x.device)
    ws = _scratch(workspace, "q4_lora_grad_workspace_bytes", dev, m, n, k, rank)
    status = lib().q4_lora_grad(x.data_ptr(), dy.data_ptr(), a.data_ptr(), b.data_ptr(),
                                _addr(scale), ids.data_ptr(), _addr(r), dx.data_ptr(),
                                da.data_ptr(), db.data_ptr(), t, ta, m, n, k, rank, na,
                                ws.data_ptr(), ws.numel(), _raw_stream(dev))
    again = _realigned(status, ids, scale)
    if again:
        return lora_grad(x, dy, a, b, again[0], again[1], r, dx, da, db, ws)
    _check(status, "q4_lora_grad")
    return dx, da, db


# Activations of the gated block (Q4_ACT_* of the ABI).
_ACTS = {"silu": 0, "gelu": 1}


def _gated(w_gate: torch.Tensor, w_up: torch.Tensor, act: str):
    """(activation code, N, K) of a gated block's projections."""
    if act not in _ACTS:
        raise ValueError(f"act must be one of {', '.join(map(repr, _ACTS))}, got {act!r}")
    n, k = q4_shape(w_gate)
    if q4_shape(w_up) != (n, k):
        raise ValueError("w_gate and w_up must have the same shape")
    return _ACTS[act], n, k


def gated_ffn(w_gate: torch.Tensor, w_up: torch.Tensor, x: torch.Tensor, act: str = "silu",
              r: torch.Tensor | None = None, keep: bool = False, out: torch.Tensor | None = None,
              z: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """(h, z): h = act(g) u with (g, u) = r + x (deq(Wg), deq(Wu))^T, the first half of a gated
    feed-forward block.  x is [M, K] of float32, float16 or bfloat16, the others of its type:
    r [M, 2 N] (zeros if None) what adapters add to the two projections, as
    ``lora(x, a, b, ids)`` with b of 2 N rows gives it; h [M, N]; z [M, 2 N], with ``keep`` (or
    a ``z`` to write, which may be r), (g, u) for ``gated_ffn_grad``, else None.  act is "silu"
    or "gelu" (its tanh form).  Above 64 rows the workspace holds the unpacked codes of both
    projections, 2 bytes each (113 MB for 9216 x 3072)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_ffn(w_gate, w_up, x, act, r, keep, out, z, workspace)
    code, n, k = _gated(w_gate, w_up, act)
    t = _activations(x, "x")
    m, k2 = x.shape
    if k2 != k:
        raise ValueError(f"x must be [M, {k}]")
    for v, name, width in ((r, "r", 2 * n), (out, "out", n), (z, "z", 2 * n)):
        if v is not None:
            _matrix(v, name, (m, width), x.dtype)
    dev = _gpu(w_gate, w_up, x, r, out, z)
    if out is None:
        out = torch.empty((m, n), dtype=x.dtype, device=x.device)
    if keep and z is None:
        z = torch.empty((m, 2 * n), dtype=x.dtype, device=x.device)
    ws = _scratch(workspace, "q4_gated_ffn_workspace_bytes", dev, t, m, n, k)
    _check(lib().q4_gated_ffn(w_gate.data_ptr(), w_up.data_ptr(), x.data_ptr(), _addr(r),
                              out.data_ptr(), _addr(z), code, t, m, n, k, ws.data_ptr(), ws.numel(),
                              _raw_stream(dev)), "q4_gated_ffn")
    return out, z


def gated_ffn_grad(w_gate: torch.Tensor, w_up: torch.Tensor, z: torch.Tensor, dh: torch.Tensor,
                   act: str = "silu", keep: bool = False, dx: torch.Tensor | None = None,
                   dz: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                   stream=None, need_dx: bool = True):
    """(dx, dz): the gradient of ``gated_ffn`` for dh [M, N], the gradient of its h, from the z
    it kept.  dx is [M, K]; dz [M, 2 N], with ``keep`` (or a ``dz`` to write, which may be z),
    the gradient of r and the dy of ``lora_grad`` for adapters beside the projections, else
    None.  Without ``need_dx`` (the model's first block) dx is None, and dz alone is computed,
    without its products and without a workspace."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return gated_ffn_grad(w_gate, w_up, z, dh, act, keep, dx, dz, workspace, None, need_dx)
    if not need_dx and (dx is not None or not (keep or dz is not None)):
        raise ValueError("without need_dx there is no dx to write, and dz is needed (keep, or a dz to write)")
    code, n, k = _gated(w_gate, w_up, act)
    t = _activations(z, "z")
    m, n2 = z.shape
    if n2 != 2 * n:
        raise ValueError(f"z must be [M, {2 * n}]")
    for v, name, width in ((dh, "dh", n), (dx, "dx", k), (dz, "dz", 2 * n)):
        if v is not None:
            _matrix(v, name, (m, width), z.dtype)
    dev = _gpu(w_gate, w_up, z, dh, dx, dz)
    ws = None
    if need_dx:
        if dx is None:
            dx = torch.empty((m, k), dtype=z.dtype, device=z.device)
        ws = _scratch(workspace, "q4_gated_ffn_grad_workspace_bytes", dev, t, m, n, k)
    if keep and dz is None:
        dz = torch.empty((m, 2 * n), dtype=z.dtype, device=z.device)
    _check(lib().q4_gated_ffn_grad(w_gate.data_ptr(), w_up.data_ptr(), z.data_ptr(), dh.data_ptr(),
                                   _addr(dx), _addr(dz), code, t, m, n, k, _addr(ws),
                                   ws.numel() if need_dx else 0, _raw_stream(dev)), "q4_gated_ffn_grad")
    return dx, dz


def lmhead_distill(w_q4: torch.Tensor, x: torch.Tensor, top_ids: torch.Tensor,
                   top_logits: torch.Tensor, temperature: float = 1.0, grad: bool = False,
                   dloss: torch.Tensor | None = None, loss: torch.Tensor | None = None,
                   lse: torch.Tensor | None = None, dx: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None, stream=None):
    """(loss, lse, dx): per row of x, temperature^2 times the divergence of the student's
    p = softmax(deq(T) x / temperature) from the teacher's q, the softmax of the row's
    top_logits / temperature (float32 [M, top], 1 to 256) at the tokens top_ids (int32
    [M, top]): sum q (log q - log p); lse = logsumexp(deq(T) x / temperature); and with
    ``grad`` (or a ``dx`` to write) the gradient of sum(dloss * loss) with respect to x, in
    x's type; dx is None otherwise.  Entries whose token is outside [0, N) are absent, those of
    one token add up; rows without any have loss 0 and dx 0.  Memory as for ``lmhead_xent``."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return lmhead_distill(w_q4, x, top_ids, top_logits, temperature, grad, dloss, loss, lse,
                                  dx, workspace)
    n, k = q4_shape(w_q4)
    t = _activations(x, "x")
    m, k2 = x.shape
    if k2 != k:
        raise ValueError(f"x must be [M, {k}]")
    if top_ids.dim() != 2:
        raise ValueError("top_ids must be [M, top]")
    top = top_ids.shape[1]
    _matrix(top_ids, "top_ids", (m, top), torch.int32)
    _matrix(top_logits, "top_logits", (m, top), torch.float32)
    for v, name in ((dloss, "dloss"), (loss, "loss"), (lse, "lse")):
        if v is not None:
            _matrix(v, name, (m,), torch.float32)
    if dx is not None:
        _matrix(dx, "dx", (m, k), x.dtype)
        grad = True
    dev = _gpu(w_q4, x, top_ids, top_logits, dloss, loss, lse, dx)
    if loss is None:
        loss = torch.empty(m, dtype=torch.float32, device=x.device)
    if lse is None:
        lse = torch.empty(m, dtype=torch.float32, device=x.device)
    if grad and dx is None:
        dx = torch.empty((m, k), dtype=x.dtype, device=x.device)
    ws = _scratch(workspace, "q4_lmhead_distill_workspace_bytes", dev, t, int(bool(grad)), m, n, k,
                  top)
    status = lib().q4_lmhead_distill(w_q4.data_ptr(), x.data_ptr(), top_ids.data_ptr(),
                                     top_logits.data_ptr(), temperature, _addr(dloss),
                                     loss.data_ptr(), lse.data_ptr(), _addr(dx), t, m, n, k, top,
                                     ws.data_ptr(), ws.numel(), _raw_stream(dev))
    again = _realigned(status, top_ids, top_logits, dloss)
    if again:
        return lmhead_distill(w_q4, x, again[0], again[1], temperature, grad, again[2], loss, lse,
                              dx, ws)
    _check(status, "q4_lmhead_distill")
    return loss, lse, dx


def verify_draft(logits: torch.Tensor, draft: torch.Tensor, u: torch.Tensor,
                 probs: torch.Tensor | None = None, lens: torch.Tensor | None = None,
                 temperature: float = 1.0, tokens: torch.Tensor | None = None,
                 accepted: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 stream=None):
    """(tokens, accepted): for each of S sequences, how many of its drafted tokens stand
    (int32 [S]), and those tokens, the one after them and -1s (int32 [S, D + 1]).  logits is
    [S, D + 1, N] (float32, float16 or bfloat16), the large model's after 0 .. D drafted tokens,
    as ``matmul`` with the head gives them; draft int32 [S, D]; probs [S, D, N] of logits' type
    the draft's probabilities, or None: it was certain of its tokens; u float32 [S, D + 1] in
    [0, 1), column i for drafted token i and the last for the draw; lens int32 [S], drafted
    tokens of each sequence (D if None); temperature 0 is greedy."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return verify_draft(logits, draft, u, probs, lens, temperature, tokens, accepted,
                                workspace)
    t = _TYPES.get(logits.dtype)
    if t is None or logits.dim() != 3 or not logits.is_contiguous() or logits.shape[1] < 1:
        raise ValueError("logits must be a contiguous [S, D + 1, N] tensor of float32, float16 or "
                         "bfloat16")
    s, d, n = logits.shape[0], logits.shape[1] - 1, logits.shape[2]
    _matrix(draft, "draft", (s, d), torch.int32)
    _matrix(u, "u", (s, d + 1), torch.float32)
    if probs is not None:
        _matrix(probs, "probs", (s, d, n), logits.dtype)
    if lens is not None:
        _matrix(lens, "lens", (s,), torch.int32)
    if tokens is not None:
        _matrix(tokens, "tokens", (s, d + 1), torch.int32)
    if accepted is not None:
        _matrix(accepted, "accepted", (s,), torch.int32)
    dev = _gpu(logits, draft, u, probs, lens, tokens, accepted)
    if tokens is None:
        tokens = torch.empty((s, d + 1), dtype=torch.int32, device=logits.device)
    if accepted is None:
        accepted = torch.empty(s, dtype=torch.int32, device=logits.device)
    ws = _scratch(workspace, "q4_verify_draft_workspace_bytes", dev, s, d, n)
    status = lib().q4_verify_draft(logits.data_ptr(), draft.data_ptr(), _addr(probs), u.data_ptr(),
                                   _addr(lens), temperature, tokens.data_ptr(), accepted.data_ptr(),
                                   t, s, d, n, ws.data_ptr(), ws.numel(), _raw_stream(dev))
    again = _realigned(status, draft, u, lens)
    if again:
        return verify_draft(logits, again[0], again[1], probs, again[2], temperature, tokens,
                            accepted, ws)
    _check(status, "q4_verify_draft")
    return tokens, accepted


GGUF_F32, GGUF_F16, GGUF_Q4_0, GGUF_Q8_0, GGUF_BF16 = 0, 1, 2, 8, 30


class Gguf:
    """A GGUF file (or the ordered byte pieces of one) opened with the
    library's reader.  ``tensors`` maps name -> (type, dims, offset, nbytes)
    with dims innermost first; ``read(name)`` returns the tensor's bytes as a
    numpy uint8 array (a Q4_0 weight of N rows of K as [N, 18*K/32])."""

    def __init__(self, paths):
        if isinstance(paths, (str, os.PathLike)):
            paths = [paths]
        enc = [os.fsencode(p) for p in paths]
        arr = (ctypes.c_char_p * len(enc))(*enc)
        h = ctypes.c_void_p()
        _check(lib().q4_gguf_open(ctypes.cast(arr, ctypes.c_void_p), len(enc), ctypes.byref(h)),
               "q4_gguf_open")
        self._h = h
        self.version = int(lib().q4_gguf_version(h))
        self.alignment = int(lib().q4_gguf_alignment(h))
        self.data_offset = int(lib().q4_gguf_data_offset(h))
        self.tensors = {}
        for i in range(int(lib().q4_gguf_tensor_count(h))):
            name, typ, nd = ctypes.c_char_p(), ctypes.c_uint32(), ctypes.c_uint32()
            dims, off, nb = (ctypes.c_int64 * 4)(), ctypes.c_uint64(), ctypes.c_uint64()
            _check(lib().q4_gguf_tensor_info(h, i, ctypes.byref(name), ctypes.byref(typ),
                                             ctypes.byref(nd), dims, ctypes.byref(off),
                                             ctypes.byref(nb)), "q4_gguf_tensor_info")
            self.tensors[name.value.decode()] = (int(typ.value), tuple(dims[: nd.value]),
                                                 int(off.value), int(nb.value))
        self.metadata = []
        for i in range(int(lib().q4_gguf_metadata_count(h))):
            key, vt = ctypes.c_char_p(), ctypes.c_uint32()
            _check(lib().q4_gguf_metadata_key(h, i, ctypes.byref(key), ctypes.byref(vt)),
                   "q4_gguf_metadata_key")
            self.metadata.append((key.value.decode(), int(vt.value)))

    def close(self):
        if self._h:
            lib().q4_gguf_close(self._h)
            self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:  # pragma: no cover - interpreter shutdown
            pass

    def read(self, name: str):
        import numpy as np
        i = int(lib().q4_gguf_find_tensor(self._h, name.encode()))
        if i < 0:
            raise KeyError(name)
        typ, dims, _, nbytes = self.tensors[name]
        out = np.empty(nbytes, dtype=np.uint8)
        _check(lib().q4_gguf_read_tensor(self._h, i, out.ctypes.data_as(ctypes.c_void_p), nbytes),
               "q4_gguf_read_tensor")
        if typ == GGUF_Q4_0 and len(dims) == 2:
            return out.reshape(dims[1], dims[0] // QK * BLOCK_BYTES)
        return out

    def meta_int(self, key: str) -> int:
        v = ctypes.c_int64()
        _check(lib().q4_gguf_metadata_int(self._h, key.encode(), ctypes.byref(v)), "q4_gguf_metadata_int")
        return int(v.value)

    def meta_float(self, key: str) -> float:
        v = ctypes.c_double()
        _check(lib().q4_gguf_metadata_float(self._h, key.encode(), ctypes.byref(v)), "q4_gguf_metadata_float")
        return float(v.value)

    def meta_string(self, key: str) -> str:
        v, n = ctypes.c_char_p(), ctypes.c_uint64()
        _check(lib().q4_gguf_metadata_string(self._h, key.encode(), ctypes.byref(v), ctypes.byref(n)),
               "q4_gguf_metadata_string")
        return ctypes.string_at(v, n.value).decode()

    def meta_array(self, key: str):
        t, n = ctypes.c_uint32(), ctypes.c_uint64()
        _check(lib().q4_gguf_metadata_array(self._h, key.encode(), ctypes.byref(t), ctypes.byref(n)),
               "q4_gguf_metadata_array")
        return int(t.value), int(n.value)


def declared_symbols(header: str = HEADER):
    """Function names declared in include/q4.h."""
    import re
    with open(header) as fh:
        text = fh.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(q4_[a-z0-9_]+)\s*\(", text)))
