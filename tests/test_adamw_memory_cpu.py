"""The check of a list's tensors against its rows, without a GPU: one that does not stand where its row
says, now or since the list was made, is refused before anything is launched."""
import ctypes

import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from activation_sparse_transformer_gate_gb300 import _build
from activation_sparse_transformer_gate_gb300.lm import twell_adamw_tensor

ARG, DTYPE = -1, -3
NAMES = ("param", "grad", "m", "v")
NONE = (None, None, None)


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()
    tw.load()


def made(x, flat=None, **change):
    from activation_sparse_transformer_gate_gb300 import _lm
    row = dict(zip(NAMES, (t.data_ptr() for t in x)), n=300) | change
    array = (twell_adamw_tensor * 1)(twell_adamw_tensor(**row))
    address = ctypes.addressof(array)
    return array, _lm.adamw_list((*x, *NONE) if flat is None else flat, address, 1)


def code(array, lst, lr=1e-3):
    from activation_sparse_transformer_gate_gb300 import _lm
    return _lm.adamw_step(lst, ctypes.addressof(array), 1, 0, 32, lr, 0.9, 0.99, 1e-8, 1, 0, None, None, 0)


def tensors():
    whole = torch.zeros(4, 304)             # (16-byte boundaries)
    return [whole[i, :300] for i in range(4)]


def test_rows_that_are_not_their_tensors():
    x = tensors()
    assert made(x, n=299)[1] is None
    assert made(x, m=x[0].data_ptr())[1] is None
    assert made(x, copy=x[0].data_ptr())[1] is None                         # a row without its tensor
    assert made(x, flat=(*x[:3], None, *NONE))[1] is None
    for wrong in ([*x, *NONE], (*x, None), ("x", *x[1:], *NONE)):
        with pytest.raises(TypeError):
            made(x, flat=wrong)


@pytest.mark.parametrize("which", range(4))
def test_other_memory_since(which):
    """(a step with lr NaN is refused by itself, after the tensors: nothing is ever launched here)"""
    x = tensors()
    array, lst = made(x)
    assert code(array, lst, float("nan")) == ARG
    old = x[which].detach()
    for new, want in ((torch.zeros(300), ARG), (old[:299], ARG), (old.view(torch.int32), DTYPE),
                      (torch.empty(0), ARG), (old.view(150, 2).t(), ARG)):
        x[which].data = new
        assert code(array, lst) == want, want
    with pytest.raises(ValueError):                                         # (no list)
        code(array, (*x, *NONE))
