"""A batch padded with a few hundred empty sequences: the bits of the batch without them, wherever
they stand."""
import pytest
import torch

from lm_testlib import setup
from test_recur_gpu import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D", [(5000, 1536), (5000, 2560), (5000, 264), (300, 2048)])
def test_empty_sequences_change_nothing(T, D, dtype):
    cut, end = T // 3, T - 7
    plain = Case(T, D, [0, cut, end], dtype)
    want = plain.run()
    for starts, which in (([0, cut, end] + [end] * 300, [0, 1]), ([0] * 90 + [0, cut, cut, cut, end], [90, 93])):
        c = Case(T, D, starts, dtype)
        for n in ("x", "gate", "dh"):
            setattr(c, n, getattr(plain, n))
        c.bias = plain.bias
        for n in ("h0", "dhT"):
            getattr(c, n)[which] = getattr(plain, n)
        got = c.run()
        for n in ("h", "dx", "dgate"):
            assert torch.equal(got[n][:end], want[n][:end]), n
        assert torch.equal(got["dbias"], want["dbias"])
        for n, passed in (("hT", c.h0), ("dh0", c.dhT)):
            assert torch.equal(got[n][which], want[n]), n
            rest = [i for i in range(c.B) if i not in which]
            assert torch.equal(got[n].cpu()[rest], passed[rest]), n
