"""A list of AdamW whose tensors have been given other memory is refused before anything is launched:
its rows would still hold what was freed."""
import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import gen, setup

pytestmark = pytest.mark.gpu
ARG, DTYPE = -1, -3
NAMES = ("param", "grad", "m", "v", "mscale", "vscale", "copy")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


def tensors(bits, n=700):
    code = torch.float8_e4m3fn if bits == 8 else torch.float32
    rand = lambda k: torch.randn(k, generator=gen(k)).cuda()  # noqa: E731
    t = [rand(n), rand(n), torch.zeros(n, device="cuda").to(code), torch.zeros(n, device="cuda").to(code)]
    t += [torch.zeros(-(-n // 256), device="cuda") for _ in range(2)] if bits == 8 else [None, None]
    return t + [torch.zeros(n, dtype=torch.bfloat16, device="cuda")]


def step(lst, code=None):
    if code is None:
        return tw.twell_adamw_step(lst, 1e-3, 0.9, 0.99, 1e-8, 1)
    with pytest.raises(tw.TwellError) as e:
        tw.twell_adamw_step(lst, 1e-3, 0.9, 0.99, 1e-8, 1)
    assert e.value.code == code


def bits_of(ts):
    return [t.clone().view(torch.uint8) for t in ts if t is not None]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("which", range(7))
def test_other_memory(which, bits):
    first, ts = tensors(bits, 300), tensors(bits)
    if ts[which] is None:
        pytest.skip("32 bits have no scales")
    lst = tw.AdamWTensors(bits)
    for row in (first, ts):
        lst.add(*row[:6], copy=row[6])
    step(lst)
    old = ts[which].detach()                # (keeps the memory; another tensor object)
    new = ts[which].clone()
    before = bits_of(first + ts + [new])
    ts[which].data = new
    step(lst, ARG)
    ts[which].data = old[:-1]               # fewer elements from the same place on
    step(lst, ARG)
    ts[which].data = old.view(torch.uint8 if old.element_size() == 1 else
                              torch.int16 if old.element_size() == 2 else torch.int32)
    step(lst, DTYPE)
    ts[which].data = torch.empty(0, dtype=old.dtype, device="cuda")
    step(lst, ARG)
    torch.cuda.synchronize()
    ts[which].data = old
    after = bits_of(first + ts + [new])
    assert all(bool((a == b).all()) for a, b in zip(before, after))
    step(lst)                               # the memory that it had
    ts[which].data = new                    # and a list built anew
    lst = tw.AdamWTensors(bits)
    lst.add(*ts[:6], copy=ts[6])
    step(lst)
    if which == 0:                          # (the others' codes may well be the same again)
        assert not bool((new.view(torch.uint8) == before[-1]).all())


def test_a_tensor_in_host_memory():
    ts = tensors(32)
    lst = tw.AdamWTensors(32)
    lst.add(*ts[:4])
    step(lst)
    old = ts[0].detach()
    ts[0].data = ts[0].cpu()
    step(lst, ARG)
    assert old.is_cuda
