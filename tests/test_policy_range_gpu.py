"""The policy loss where its KL term leaves fp32's range: a token that the policy gives no
probability, or one too small beside the reference's.

With d = ref - logp, exp(d) is beyond fp32: the loss is infinite by the formula, and the KL term
of the slope is held at -2^126, beside which the other one is nothing (r < 2^-100).  So dz is
-w 2^126 (1 - q) at the token, and w 2^126 q elsewhere to the exponentials' and their sum's
roundings, (8 s + 80 + V / 4096) 2^-24 of itself with s = max |z|, and 64 for those below 2^-120,
which may be flushed to 0."""
import pytest
import torch

from lm_testlib import U, check, gen, setup
from test_policy_gpu import Case

pytestmark = pytest.mark.gpu
HELD = 2.0 ** 126


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


def far(T, V, dtype):
    """Rows 0 and 1 sample what has no logit, row 2 what lies 150 below the others."""
    c = Case(T, V, dtype)
    c.w = 0.5 + 0.5 * torch.rand(T, generator=gen(T + V))
    c.tok[0], c.tok[1], c.tok[2] = 3, V - 1, V // 2
    c.z[0, 3] = c.z[1, V - 1] = -float("inf")
    c.z[0, V // 2::2] = -float("inf")
    c.z[2, V // 2] = -150.0
    return c


@pytest.mark.parametrize("V", [300, 5000, 50001, 131072])
@pytest.mark.parametrize("T", [8, 310])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_token_without_probability(T, V, dtype):
    if T * V > 2 ** 24:
        pytest.skip("long on the host")
    c = far(T, V, dtype)
    c.ref[:3] = -0.5
    c.old[:3] = -2.0
    plain = Case(T, V, dtype)
    plain.w = c.w
    z = c.z[:3].double()
    q = torch.softmax(z, 1)
    hot = torch.zeros_like(q).scatter_(1, c.tok[:3, None], 1.0).bool()
    want = c.w[:3, None].double() * torch.where(hot, -HELD * (1 - q), HELD * q)
    s = torch.where(torch.isinf(z), torch.zeros_like(z), z).abs().amax(1, keepdim=True)
    bound = want.abs() * (8 * s + 80 + V / 4096) * U + torch.where((q > 0) & (q < 2.0 ** -120), 64.0, 0.0)
    for two in (False, True):
        for in_place in (False, True):
            base = plain.run(two=two, in_place=in_place)
            got = c.run(two=two, in_place=in_place)
            assert (got["logp"][:2] == -float("inf")).all() and got["logp"][2] < -140
            assert (got["loss"][:3] == float("inf")).all()
            check(got["dz"][:3], want, bound, dtype, "dz")
            assert (got["dz"][:3].cpu()[(q == 0) & ~hot] == 0).all()
            for n in ("loss", "logp", "dz"):
                assert torch.equal(got[n][3:], base[n][3:]), n


@pytest.mark.parametrize("V", [300, 50001])
def test_both_terms_out_of_range(V):
    """r and exp(d) beyond fp32 at once: no NaN from their difference."""
    c = Case(8, V, "f32")
    c.z[2, V // 2], c.tok[2], c.adv[2] = -150.0, V // 2, -1.0
    c.old[2], c.ref[2] = -300.0, 0.0
    for two in (False, True):
        got = c.run(two=two)
        assert got["loss"][2] == float("inf") and got["dz"][2].isfinite().all()


def test_no_reference_or_no_beta():
    """Without a KL term such a token has a finite loss."""
    for beta, ref in ((0.0, True), (0.04, False)):
        c = far(8, 700, "f32")
        c.beta, c.ref = beta, c.ref if ref else None
        c.old[:3] = -2.0
        got = c.run()
        assert got["loss"].isfinite().all() and got["dz"].isfinite().all()
