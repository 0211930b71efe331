"""Python binding of the operators around the FFN (include/twell_lm.h): token
embedding, residual addition + RMS norm, 8-bit product, distillation loss.

Argument marshalling only, as in the package's top module, under the ABI's
names.  Tensors are checked before the call: the element type (TWELL_ERR_DTYPE),
the number of elements, contiguity and a CUDA device (TWELL_ERR_ARG); raw
integer device pointers are passed as they are.
"""
from __future__ import annotations

import torch

from . import TWELL_BF16, TWELL_F32, TWELL_OK, TwellError, load

_TORCH = {TWELL_F32: torch.float32, TWELL_BF16: torch.bfloat16}
_ARG, _DTYPE = -1, -3


def _arg(a, dtype, count, where):
    """The device pointer of an operand of `count` elements."""
    if a is None or isinstance(a, int):
        return a
    if a.dtype is dtype and a.numel() == count and a.is_contiguous() and a.is_cuda:
        return a.data_ptr()
    raise TwellError(_ARG if a.dtype is dtype else _DTYPE, where)


def _pitched(a, dtype, rows, cols, pitch, where):
    """The same for a [rows][cols] operand with a row pitch (elements)."""
    if a is None or isinstance(a, int):
        return a
    if a.dtype is not dtype:
        raise TwellError(_DTYPE, where)
    if (not a.is_cuda or a.dim() != 2 or a.shape[0] != rows or a.shape[1] not in (cols, pitch)
            or (a.shape[1] > 1 and a.stride(1) != 1) or (rows > 1 and a.stride(0) != pitch)):
        raise TwellError(_ARG, where)
    return a.data_ptr()


def _elem(dtype, where):
    t = _TORCH.get(dtype)
    if t is None:
        raise TwellError(_DTYPE, where)
    return t


def _tokens(tokens, T, where):
    """(pointer, bytes of a token); a raw pointer holds int32."""
    if tokens is None or isinstance(tokens, int):
        return tokens, 4
    if tokens.dtype is torch.int64:
        return _arg(tokens, torch.int64, T, where), 8
    return _arg(tokens, torch.int32, T, where), 4


def _scratch(workspace, nbytes, where):
    if workspace is None or isinstance(workspace, int):
        return workspace
    if not workspace.is_cuda or workspace.numel() * workspace.element_size() < nbytes:
        raise TwellError(-8, where)
    return workspace.data_ptr()


def _stream(stream):
    """Raw handle of a stream; None: the current one (as a handle, without the stream object that
    torch.cuda.current_stream() makes, which takes as long as a launch)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _run(where, fn, *args):
    code = fn(*args)
    if code != TWELL_OK:
        raise TwellError(code, where)


def twell_read_status(status, stream=None) -> int:
    """The status word, read and cleared; synchronises the stream."""
    where = "twell_read_status"
    n = status.numel() if hasattr(status, "numel") else 1
    return int(load().twell_read_status(_arg(status, torch.int32, n, where), _stream(stream)))


def twell_embed_workspace_size(T: int, V: int, D: int) -> int:
    return int(load().twell_embed_workspace_size(T, V, D))


def twell_embed_forward(tokens, table, T: int, V: int, D: int, dtype: int, scale: float,
                        pad_id: int, out, status, stream=None) -> None:
    where = "twell_embed_forward"
    t = _elem(dtype, where)
    tok, nb = _tokens(tokens, T, where)
    _run(where, load().twell_embed_forward, tok, nb, _arg(table, t, V * D, where), T, V, D, dtype,
         scale, pad_id, _arg(out, t, T * D, where), _arg(status, torch.int32, 1, where),
         _stream(stream))


def twell_embed_backward(tokens, dy, T: int, V: int, D: int, dtype: int, scale: float, pad_id: int,
                         dtable, status, workspace, workspace_bytes: int, stream=None) -> None:
    where = "twell_embed_backward"
    t = _elem(dtype, where)
    tok, nb = _tokens(tokens, T, where)
    _run(where, load().twell_embed_backward, tok, nb, _arg(dy, t, T * D, where), T, V, D, dtype,
         scale, pad_id, _arg(dtable, torch.float32, V * D, where),
         _arg(status, torch.int32, 1, where), _scratch(workspace, workspace_bytes, where),
         workspace_bytes, _stream(stream))


def twell_add_rmsnorm_workspace_size(T: int, D: int) -> int:
    return int(load().twell_add_rmsnorm_workspace_size(T, D))


def twell_add_rmsnorm_forward(x, residual, weight, T: int, D: int, dtype: int, eps: float, s, y, q,
                              qscale, rstd, stream=None) -> None:
    where = "twell_add_rmsnorm_forward"
    t, f32 = _elem(dtype, where), torch.float32
    _run(where, load().twell_add_rmsnorm_forward, _arg(x, t, T * D, where),
         _arg(residual, t, T * D, where), _arg(weight, f32, D, where), T, D, dtype, eps,
         _arg(s, t, T * D, where), _arg(y, t, T * D, where), _arg(q, torch.int8, T * D, where),
         _arg(qscale, f32, T, where), _arg(rstd, f32, T, where), _stream(stream))


def twell_add_rmsnorm_backward(s, weight, rstd, dy, ds, T: int, D: int, dtype: int, dx, dweight,
                               workspace, workspace_bytes: int, stream=None) -> None:
    where = "twell_add_rmsnorm_backward"
    t, f32 = _elem(dtype, where), torch.float32
    _run(where, load().twell_add_rmsnorm_backward, _arg(s, t, T * D, where),
         _arg(weight, f32, D, where), _arg(rstd, f32, T, where), _arg(dy, t, T * D, where),
         _arg(ds, t, T * D, where), T, D, dtype, _arg(dx, t, T * D, where),
         _arg(dweight, f32, D, where), _scratch(workspace, workspace_bytes, where),
         workspace_bytes, _stream(stream))


def twell_q8_quantize(a, rows: int, cols: int, dtype: int, q, scale, stream=None) -> None:
    where = "twell_q8_quantize"
    _run(where, load().twell_q8_quantize, _arg(a, _elem(dtype, where), rows * cols, where), rows,
         cols, dtype, _arg(q, torch.int8, rows * cols, where),
         _arg(scale, torch.float32, rows, where), _stream(stream))


def twell_q8_workspace_size(M: int, N: int, K: int) -> int:
    return int(load().twell_q8_workspace_size(M, N, K))


def twell_q8_matmul(aq, ascale, wq, wscale, bias, M: int, N: int, K: int, dtype: int, y, status,
                    workspace, workspace_bytes: int, stream=None) -> None:
    where = "twell_q8_matmul"
    i8, f32 = torch.int8, torch.float32
    _run(where, load().twell_q8_matmul, _arg(aq, i8, M * K, where), _arg(ascale, f32, M, where),
         _arg(wq, i8, N * K, where), _arg(wscale, f32, N, where), _arg(bias, f32, N, where), M, N,
         K, dtype, _arg(y, _elem(dtype, where), M * N, where),
         _arg(status, torch.int32, 1, where), _scratch(workspace, workspace_bytes, where),
         workspace_bytes, _stream(stream))


def twell_distill_forward(z, ldz: int, ids, teacher, row_weight, T: int, V: int, k: int,
                          dtype: int, tau: float, loss, stats, dz, status, stream=None) -> None:
    where = "twell_distill_forward"
    t, f32 = _elem(dtype, where), torch.float32
    _run(where, load().twell_distill_forward, _pitched(z, t, T, V, ldz, where), ldz,
         _arg(ids, torch.int32, T * k, where), _arg(teacher, f32, T * k, where),
         _arg(row_weight, f32, T, where), T, V, k, dtype, tau, _arg(loss, f32, T, where),
         _arg(stats, f32, 2 * T, where), _pitched(dz, t, T, V, ldz, where),
         _arg(status, torch.int32, 1, where), _stream(stream))


def twell_distill_backward(z, ldz: int, ids, teacher, stats, row_grad, T: int, V: int, k: int,
                           dtype: int, tau: float, dz, status, stream=None) -> None:
    where = "twell_distill_backward"
    t, f32 = _elem(dtype, where), torch.float32
    _run(where, load().twell_distill_backward, _pitched(z, t, T, V, ldz, where), ldz,
         _arg(ids, torch.int32, T * k, where), _arg(teacher, f32, T * k, where),
         _arg(stats, f32, 2 * T, where), _arg(row_grad, f32, T, where), T, V, k, dtype, tau,
         _pitched(dz, t, T, V, ldz, where), _arg(status, torch.int32, 1, where), _stream(stream))
