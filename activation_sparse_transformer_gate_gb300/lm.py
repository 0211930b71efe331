"""Python binding of the operators around the FFN (include/twell_lm.h): token
embedding, residual addition + RMS norm, gated recurrence, 8-bit product,
distillation and policy loss, AdamW step.

Argument marshalling only, under the ABI's names.  Tensors are checked before
the call: the element type (TWELL_ERR_DTYPE), the number of elements,
contiguity and a CUDA device (TWELL_ERR_ARG), a workspace's size
(TWELL_ERR_WORKSPACE); integers are passed as raw device pointers, None as NULL.
Tokens are int32 or int64 tensors.  ``stream`` is None (the current one), a raw
handle or a torch stream.  The checks and the call are compiled (_lm.so, built
with libtwell.so): through ctypes they took as long as a small call's kernels.
"""
from __future__ import annotations

import bisect
import ctypes
import struct

import torch  # (and its libraries, which _lm.so uses)

from . import TWELL_BF16, TWELL_F32, TWELL_OK, TwellError, _build, load

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


def twell_recur_states(T: int) -> int:
    return int(load().twell_recur_states(T))


def twell_recur_forward(x, gate, ld: int, bias, starts, B: int, h0, T: int, D: int, dtype: int, h,
                        hT, states, status, stream=None) -> None:
    _check(_lm.recur_forward(x, gate, ld, bias, starts, B, h0, T, D, dtype, h, hT, states, status,
                             stream), "twell_recur_forward")


def twell_recur_backward(x, gate, ld: int, bias, starts, B: int, h0, states, dh, dhT, T: int, D: int,
                         dtype: int, dx, dgate, dbias, dh0, status, stream=None) -> None:
    _check(_lm.recur_backward(x, gate, ld, bias, starts, B, h0, states, dh, dhT, T, D, dtype, dx,
                              dgate, dbias, dh0, status, stream), "twell_recur_backward")


def twell_policy_forward(z, ldz: int, tokens, old_logp, ref_logp, advantage, row_weight, T: int,
                         V: int, dtype: int, tau: float, clip_low: float, clip_high: float,
                         beta: float, loss, logp, stats, dz, status, stream=None) -> None:
    _check(_lm.policy_forward(z, ldz, tokens, old_logp, ref_logp, advantage, row_weight, T, V, dtype,
                              tau, clip_low, clip_high, beta, loss, logp, stats, dz, status, stream),
           "twell_policy_forward")


def twell_policy_backward(z, ldz: int, tokens, old_logp, ref_logp, advantage, logp, stats, row_grad,
                          T: int, V: int, dtype: int, tau: float, clip_low: float, clip_high: float,
                          beta: float, dz, status, stream=None) -> None:
    _check(_lm.policy_backward(z, ldz, tokens, old_logp, ref_logp, advantage, logp, stats, row_grad,
                               T, V, dtype, tau, clip_low, clip_high, beta, dz, status, stream),
           "twell_policy_backward")


class twell_adamw_tensor(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("param", "grad", "m", "v", "mscale", "vscale",
                                               "copy")]
    _fields_ += [("n", ctypes.c_longlong), ("first", ctypes.c_longlong), ("decay", ctypes.c_float)]


class AdamWTensors:
    """The tensors of a twell_adamw_step, kept by a program beside them: ``add`` each once, then
    step as often as wanted.  The tensors are held, and checked when they are added: types
    (TWELL_ERR_DTYPE), elements, place and contiguity (TWELL_ERR_ARG); before the first step, that
    nothing that it writes overlaps with anything else (TWELL_ERR_ARG).  A step goes to the memory
    that they had then: it is refused (the same codes) once one of them has been given other memory
    or another shape or type, as by ``p.data = ...``; a list is then built anew.  A gradient is the
    tensor that was added, not what ``p.grad`` is later; a captured step has its addresses, and
    needs the list to be kept.  ``state_bits`` 8: m and v are float8_e4m3fn codes with fp32 scales
    for each 256 elements."""

    def __init__(self, state_bits: int = 32):
        if state_bits not in (8, 32):
            raise TwellError(-3, "AdamWTensors")
        self.state_bits, self.grad_dtype = state_bits, None
        self.held, self.rows, self.written, self.read, self.array = [], [], [], [], None

    def add(self, param, grad, m, v, mscale=None, vscale=None, copy=None, decay: float = 0.0,
            first: int = 0) -> None:
        n = param.numel()
        small = self.state_bits == 8
        state = torch.float8_e4m3fn if small else torch.float32
        blocks = -(-n // 256)
        wanted = [(param, torch.float32, n), (m, state, n), (v, state, n)]
        if small:
            wanted += [(mscale, torch.float32, blocks), (vscale, torch.float32, blocks)]
        elif mscale is not None or vscale is not None:
            raise TwellError(-1, "AdamWTensors.add")
        if copy is not None:
            wanted.append((copy, torch.bfloat16, n))
        dtype = {torch.float32: TWELL_F32, torch.bfloat16: TWELL_BF16}.get(grad.dtype)
        if dtype is None or self.grad_dtype not in (None, dtype):
            raise TwellError(-3, "AdamWTensors.add")
        every = wanted + [(grad, grad.dtype, n)]
        if any(t is None for t, _, _ in every):
            raise TwellError(-1, "AdamWTensors.add")
        if any(t.dtype is not kind for t, kind, _ in every):
            raise TwellError(-3, "AdamWTensors.add")
        if any(t.numel() != k or not t.is_cuda or not t.is_contiguous() for t, _, k in every):
            raise TwellError(-1, "AdamWTensors.add")
        span = lambda t: (t.data_ptr(), t.data_ptr() + t.nbytes)  # noqa: E731
        self.written += [span(t) for t, _, k in wanted if k]
        if n:
            self.read.append(span(grad))
        self.grad_dtype, self.array = dtype, None
        self.held.append((param, grad, m, v, mscale, vscale, copy))
        self.rows.append([None if t is None else t.data_ptr() for t in self.held[-1]]
                         + [n, int(first), float(decay)])

    def table(self):
        """The address of the C array, and how many it has."""
        if self.array is None:
            # (gradients may be shared: they are compared with what is written alone)
            both = sorted(self.written)
            ends = [b for _, b in both]
            if any(a[1] > b[0] for a, b in zip(both, both[1:])):
                raise TwellError(-1, "AdamWTensors")
            for lo, hi in self.read:
                i = bisect.bisect_right(ends, lo)
                if i < len(both) and both[i][0] < hi:
                    raise TwellError(-1, "AdamWTensors")
            array = (twell_adamw_tensor * max(1, len(self.rows)))(*map(tuple, self.rows))
            self.address = ctypes.addressof(array)
            self.list = _lm.adamw_list(tuple(t for row in self.held for t in row), self.address,
                                       len(self.rows))
            if self.list is None:   # (a tensor has got other memory since it was added)
                raise TwellError(-1, "AdamWTensors")
            self.array = array
        return self.address, len(self.rows)


def adamw_dynamic(lr: float, beta1: float, beta2: float, step: int, seed: int = 0):
    """A twell_adamw_dynamic as an int32 tensor of 4 in host memory, to be copied to the device
    before a captured step is replayed."""
    b1, b2 = (struct.unpack("f", struct.pack("f", b))[0] for b in (beta1, beta2))
    data = struct.pack("fffI", lr, 1.0 - b1 ** step, 1.0 - b2 ** step, seed & 0xFFFFFFFF)
    return torch.frombuffer(bytearray(data), dtype=torch.int32)


def twell_adamw_step(tensors: AdamWTensors, lr: float, beta1: float, beta2: float, eps: float,
                     step: int, seed: int = 0, grad_scale=None, dynamic=None, stream=None) -> None:
    if tensors.array is None:
        tensors.table()
    _check(_lm.adamw_step(tensors.list, tensors.address, len(tensors.rows), tensors.grad_dtype or 0,
                          tensors.state_bits, lr, beta1, beta2, eps, step, seed, grad_scale, dynamic,
                          stream), "twell_adamw_step")
