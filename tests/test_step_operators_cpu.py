"""What the recurrence, the policy loss and the AdamW step refuse: host-detectable errors return
their code before a pointer is read or a launch made (so these run without a GPU), and the
Python binding's checks."""
import ctypes

import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from activation_sparse_transformer_gate_gb300 import _build
from activation_sparse_transformer_gate_gb300.lm import twell_adamw_tensor

ARG, ALIGN, DTYPE = -1, -2, -3
A = 1 << 40          # fake, aligned "device" addresses
OFF, ODD = A + 8, A + 2
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return tw.load()


def refused(fn, good, changes):
    for pos, value, code in changes:
        args = list(good)
        args[pos] = value
        assert fn(*args) == code, (fn.__name__, pos, value)


def test_recurrence(lib):
    good = [A, A, 128, A, A, 4, A, 64, 128, 1, A, A, A, A, None]
    common = [(0, None, ARG), (0, OFF, ALIGN), (1, None, ARG), (1, OFF, ALIGN), (2, 127, ARG),
              (2, 132, ALIGN), (2, 1 << 41, ARG), (3, OFF, ALIGN), (4, ODD, ALIGN), (5, 0, ARG),
              (5, (1 << 30) + 1, ARG), (6, OFF, ALIGN)]
    refused(lib.twell_recur_forward, good, common + [
        (7, 0, ARG), (7, (1 << 30) + 1, ARG), (8, 0, ARG), (8, 100, ALIGN), (8, 1 << 17, ARG),
        (9, 2, DTYPE), (10, None, ARG), (10, OFF, ALIGN), (11, OFF, ALIGN), (12, OFF, ALIGN),
        (13, None, ARG), (13, ODD, ALIGN)])
    assert lib.twell_recur_forward(A, A, 128, A, None, 5, A, 64, 128, 1, A, A, A, A, None) == ARG
    good = [A, A, 128, A, A, 4, A, A, A, A, 64, 128, 1, A, A, A, A, A, None]
    refused(lib.twell_recur_backward, good, common + [
        (7, None, ARG), (7, OFF, ALIGN), (8, None, ARG), (8, OFF, ALIGN), (9, OFF, ALIGN),
        (10, 0, ARG), (11, 4, ALIGN), (12, 9, DTYPE), (13, None, ARG), (13, OFF, ALIGN),
        (14, None, ARG), (14, OFF, ALIGN), (15, OFF, ALIGN), (16, OFF, ALIGN), (17, None, ARG)])
    assert lib.twell_recur_forward(A, A, (1 << 34) + 64, A, A, 5, A, 64, 128, 1, A, A, A, A, None) == ARG
    assert [lib.twell_recur_states(t) for t in (0, -3, 1, 64, 65, (1 << 30) + 1)] == [0, 0, 1, 1, 2, 0]


def test_policy(lib):
    good = [A, 512, A, 8, A, A, A, A, 4, 500, 1, 1.0, 0.2, 0.3, 0.1, A, A, A, A, A, None]
    common = [(0, None, ARG), (0, OFF, ALIGN), (1, 499, ARG), (2, None, ARG), (2, A + 4, ALIGN),
              (3, 2, DTYPE), (4, ODD, ALIGN), (5, ODD, ALIGN), (6, ODD, ALIGN)]
    refused(lib.twell_policy_forward, good, common + [
        (7, ODD, ALIGN), (8, 0, ARG), (8, (1 << 30) + 1, ARG), (9, 0, ARG), (10, 4, DTYPE),
        (11, 0.0, ARG), (11, NAN, ARG), (11, INF, ARG), (12, -0.1, ARG), (12, 1.5, ARG),
        (12, NAN, ARG), (13, -0.1, ARG), (13, INF, ARG), (14, -1.0, ARG), (14, NAN, ARG),
        (15, None, ARG), (15, ODD, ALIGN), (16, None, ARG), (17, None, ARG), (17, A + 4, ALIGN),
        (18, OFF, ALIGN), (19, None, ARG)])
    # the log-probabilities alone have neither loss nor gradient
    for loss, dz in ((A, None), (None, A), (A, A)):
        args = list(good)
        args[6], args[15], args[18] = None, loss, dz
        assert lib.twell_policy_forward(*args) == ARG
    good = [A, 512, A, 4, A, A, A, A, A, A, 4, 500, 1, 1.0, 0.2, 0.3, 0.1, A, A, None]
    refused(lib.twell_policy_backward, good, [
        (0, None, ARG), (1, 10, ARG), (2, ODD, ALIGN), (3, 1, DTYPE), (6, None, ARG), (7, None, ARG),
        (8, None, ARG), (9, None, ARG), (9, ODD, ALIGN), (10, 0, ARG), (13, 1e-5, ARG),
        (14, 2.0, ARG), (17, None, ARG), (17, OFF, ALIGN), (18, None, ARG)])


def test_adamw(lib):
    def call(bits=32, gt=0, count=1, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, step=1, scale=None, dyn=None,
             **change):
        t = dict(param=A, grad=A, m=A, v=A, mscale=A, vscale=A, copy=A, n=10, first=0, decay=0.0)
        t.update(change)
        row = (twell_adamw_tensor * 1)(twell_adamw_tensor(**t))
        return lib.twell_adamw_step(ctypes.addressof(row), count, gt, bits, lr, b1, b2, eps, step, 0,
                                    scale, dyn, None)

    for code, kw in ((DTYPE, dict(bits=16)), (DTYPE, dict(gt=3)), (ARG, dict(count=0)),
                     (ARG, dict(count=-1)), (ARG, dict(lr=NAN)), (ARG, dict(lr=INF)),
                     (ARG, dict(b1=1.0)), (ARG, dict(b1=-0.1)), (ARG, dict(b2=1.0)),
                     (ARG, dict(b2=NAN)), (ARG, dict(eps=-1.0)), (ARG, dict(eps=INF)),
                     (ARG, dict(step=0)), (ALIGN, dict(scale=ODD)), (ALIGN, dict(dyn=OFF)),
                     (ARG, dict(n=-1)), (ARG, dict(n=(1 << 39) + 1)), (ARG, dict(first=-1)),
                     (ARG, dict(decay=INF)), (ARG, dict(param=None)), (ARG, dict(grad=None)),
                     (ARG, dict(m=None)), (ARG, dict(v=None)), (ARG, dict(bits=8, mscale=None)),
                     (ARG, dict(bits=8, vscale=None)), (ALIGN, dict(param=OFF)),
                     (ALIGN, dict(grad=OFF)), (ALIGN, dict(m=OFF)), (ALIGN, dict(v=OFF)),
                     (ALIGN, dict(copy=OFF)), (ALIGN, dict(bits=8, mscale=ODD))):
        assert call(**kw) == code, kw
    assert lib.twell_adamw_step(None, 1, 0, 32, 1e-3, 0.9, 0.99, 1e-8, 1, 0, None, None, None) == ARG


def test_binding(lib):
    def code(fn, *args):
        with pytest.raises(tw.TwellError) as e:
            fn(*args, stream=0)
        return e.value.code

    x = torch.zeros(64, 128)
    rest = (128, None, None, 4, None, 64, 128, 0, A, None, None, A)
    assert code(tw.twell_recur_forward, x, A, *rest) == ARG                   # not on the GPU
    assert code(tw.twell_recur_forward, x.bfloat16(), A, *rest) == DTYPE
    assert code(tw.twell_recur_forward, A, A, 128, None, torch.zeros(5), 4, None, 64, 128, 0, A, None,
                None, A) == DTYPE                                             # starts in int32
    z = torch.zeros(4, 512)
    tail = (A, A, A, A, 4, 500, 0, 1.0, 0.2, 0.2, 0.0, A, A, A, A, A)
    assert code(tw.twell_policy_forward, z[:, :500], 512, A, *tail) == ARG
    assert code(tw.twell_policy_forward, A, 512, torch.zeros(4, dtype=torch.int16), *tail) == DTYPE
    with pytest.raises(TypeError):
        tw.twell_policy_forward("z", 512, A, *tail, stream=0)


def test_list_of_tensors():
    """A list takes tensors of the right types and sizes on the GPU."""
    def code(lst, *args, **kw):
        with pytest.raises(tw.TwellError) as e:
            lst.add(*args, **kw)
        return e.value.code

    with pytest.raises(tw.TwellError):
        tw.AdamWTensors(16)
    x = torch.zeros(300)
    assert code(tw.AdamWTensors(), x, x, x, x) == ARG                         # not on the GPU
    assert code(tw.AdamWTensors(), x.half(), x, x, x) == DTYPE
    assert code(tw.AdamWTensors(), x, x.half(), x, x) == DTYPE
    assert code(tw.AdamWTensors(8), x, x, x, x, x, x) == DTYPE                # codes are e4m3
    assert code(tw.AdamWTensors(), x, x, x, x, x, x) == ARG                   # no scales in 32 bits
    lst = tw.AdamWTensors()
    assert lst.table()[1] == 0
    with pytest.raises(tw.TwellError):
        tw.twell_adamw_step(lst, 1e-3, 0.9, 0.99, 1e-8, 1, stream=0)          # nothing in it


def test_dynamic_scalars():
    d = tw.adamw_dynamic(0.5, 0.9, 0.5, 3, seed=2 ** 32 - 1)
    lr, c1, c2 = d[:3].view(torch.float32).tolist()
    assert lr == 0.5 and abs(c1 - 0.271) < 1e-6 and c2 == 0.875 and d[3].item() == -1
