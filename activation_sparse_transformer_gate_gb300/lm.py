"""Python binding of the operators around the FFN (include/twell_lm.h): token
embedding, residual addition + RMS norm, 8-bit product, distillation loss.

Argument marshalling only, under the ABI's names.  Tensors are checked before
the call: the element type (TWELL_ERR_DTYPE), the number of elements,
contiguity and a CUDA device (TWELL_ERR_ARG), a workspace's size
(TWELL_ERR_WORKSPACE); integers are passed as raw device pointers, None as NULL.
Tokens are int32 or int64 tensors.  ``stream`` is None (the current one), a raw
handle or a torch stream.  The checks and the call are compiled (_lm.so, built
with libtwell.so): through ctypes they took as long as a small call's kernels.
"""
from __future__ import annotations

import ctypes

import torch  # noqa: F401  (its libraries, which _lm.so uses)

from . import TWELL_OK, TwellError, _build, load

try:
    from . import _lm
except ImportError as e:
    raise ImportError(f"{_build.BINDING} is not built ({e}); run __graft_entry__.build()") from e


def _check(code: int, where: str) -> None:
    if code != TWELL_OK:
        raise TwellError(code, where)


def twell_read_status(status, stream=None) -> int:
    """The status word, read and cleared; synchronises the stream."""
    if stream is None:
        stream = torch.cuda.current_stream()
    if not isinstance(status, int):
        if status.dtype is not torch.int32 or not status.is_cuda:
            raise TwellError(-1, "twell_read_status")
        status = status.data_ptr()
    return int(load().twell_read_status(ctypes.c_void_p(status),
                                        getattr(stream, "cuda_stream", stream)))


def twell_embed_workspace_size(T: int, V: int, D: int) -> int:
    return int(load().twell_embed_workspace_size(T, V, D))


def twell_embed_forward(tokens, table, T: int, V: int, D: int, dtype: int, scale: float,
                        pad_id: int, out, status, stream=None) -> None:
    _check(_lm.embed_forward(tokens, table, T, V, D, dtype, scale, pad_id, out, status, stream),
           "twell_embed_forward")


def twell_embed_backward(tokens, dy, T: int, V: int, D: int, dtype: int, scale: float, pad_id: int,
                         dtable, status, workspace, workspace_bytes: int, stream=None) -> None:
    _check(_lm.embed_backward(tokens, dy, T, V, D, dtype, scale, pad_id, dtable, status, workspace,
                              workspace_bytes, stream), "twell_embed_backward")


def twell_add_rmsnorm_workspace_size(T: int, D: int) -> int:
    return int(load().twell_add_rmsnorm_workspace_size(T, D))


def twell_add_rmsnorm_forward(x, residual, weight, T: int, D: int, dtype: int, eps: float, s, y, q,
                              qscale, rstd, stream=None) -> None:
    _check(_lm.add_rmsnorm_forward(x, residual, weight, T, D, dtype, eps, s, y, q, qscale, rstd,
                                   stream), "twell_add_rmsnorm_forward")


def twell_add_rmsnorm_backward(s, weight, rstd, dy, ds, T: int, D: int, dtype: int, dx, dweight,
                               workspace, workspace_bytes: int, stream=None) -> None:
    _check(_lm.add_rmsnorm_backward(s, weight, rstd, dy, ds, T, D, dtype, dx, dweight, workspace,
                                    workspace_bytes, stream), "twell_add_rmsnorm_backward")


def twell_q8_quantize(a, rows: int, cols: int, dtype: int, q, scale, stream=None) -> None:
    _check(_lm.q8_quantize(a, rows, cols, dtype, q, scale, stream), "twell_q8_quantize")


def twell_q8_workspace_size(M: int, N: int, K: int) -> int:
    return int(load().twell_q8_workspace_size(M, N, K))


def twell_q8_matmul(aq, ascale, wq, wscale, bias, M: int, N: int, K: int, dtype: int, y, status,
                    workspace, workspace_bytes: int, stream=None) -> None:
    _check(_lm.q8_matmul(aq, ascale, wq, wscale, bias, M, N, K, dtype, y, status, workspace,
                         workspace_bytes, stream), "twell_q8_matmul")


def twell_distill_forward(z, ldz: int, ids, teacher, row_weight, T: int, V: int, k: int,
                          dtype: int, tau: float, loss, stats, dz, status, stream=None) -> None:
    _check(_lm.distill_forward(z, ldz, ids, teacher, row_weight, T, V, k, dtype, tau, loss, stats,
                               dz, status, stream), "twell_distill_forward")


def twell_distill_backward(z, ldz: int, ids, teacher, stats, row_grad, T: int, V: int, k: int,
                           dtype: int, tau: float, dz, status, stream=None) -> None:
    _check(_lm.distill_backward(z, ldz, ids, teacher, stats, row_grad, T, V, k, dtype, tau, dz,
                                status, stream), "twell_distill_backward")
