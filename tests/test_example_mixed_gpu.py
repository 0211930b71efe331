"""The example model with its recurrence, under both losses: gradients against
automatic differentiation of the same model in 64 bits, its optimizer against the
formula, serving token by token, and its command.

As for the model without the recurrence, the reference goes on from what the model
stored at each place (with the gradient of the identity).  A gradient passes about 25
roundings of 2^-9 relative in a chain of 2 layers (15 without the recurrences), each of
them random, so all are compared in the 2-norm with 25^(1/2) 2^-9 times 4 (0.04)."""
import os
import subprocess
import sys

import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
import distill_student as ex  # noqa: E402

pytestmark = pytest.mark.gpu
OFF = 0.04


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw._build.build()
    tw.load()


def model(T=384, V=300, k=16, **kw):
    starts = torch.tensor([0, 100, 101, 250, 250, T], dtype=torch.int32, device="cuda")
    return ex.Student(T, V, 256, 512, layers=2, k=k, tau=1.5, lam=1e-6, mix=True, starts=starts, **kw)


def recurrence(x, f, bounds):
    a, c = torch.sigmoid(f), torch.sigmoid(-f)
    rows = []
    for lo, hi in zip(bounds, bounds[1:]):
        h = torch.zeros_like(x[0])
        for t in range(lo, hi):
            h = a[t] * h + c[t] * x[t]
            rows.append(h)
    return torch.stack(rows)


def reference(st, tokens, loss_of):
    """loss_of(log-softmax of the logits / tau) -> the rows' losses; (losses, gradients)."""
    p = {n: v.double().requires_grad_(True) for n, v in st.p.items()}
    bounds = st.starts.tolist()

    def norm(s, weight):
        return s / torch.sqrt((s * s).mean(1, keepdim=True) + ex.EPS) * weight

    def stored(x, actual):
        actual = actual.double()
        assert (x.detach() - actual).norm() <= OFF * actual.norm()
        return x + (actual - x.detach())

    s, l1, y = p["embed"][tokens] * st.scale, 0.0, None
    for i in range(st.L):
        s = stored(s if y is None else s + y, st.s_mix[i])
        n = stored(norm(s, p[f"norm_mix{i}"]), st.n_mix[i])
        xg = stored(n @ p[f"mix{i}"].t(), st.xg[i])
        h = recurrence(xg[:, :st.D], xg[:, st.D:] + p[f"bias_mix{i}"], bounds)
        s = stored(s + stored(h, st.h[i]), st.s[i])
        n = stored(norm(s, p[f"norm{i}"]), st.n[i])
        u = torch.relu(n @ p[f"gate{i}"].t() + p[f"bias{i}"]) * (n @ p[f"up{i}"].t())
        l1 = l1 + st.lam * u.abs().sum()
        y = u @ p[f"down{i}"]
    n = stored(norm(stored(s + y, st.s[st.L]), p["norm_out"]), st.n[st.L])
    loss = loss_of(torch.log_softmax((n @ p["out"].t()) / st.tau, 1))
    (loss.sum() + l1).backward()
    return loss, {n: v.grad for n, v in p.items()}


def compare(st, loss, want, grad):
    assert (loss - want).norm() <= OFF * want.norm()
    for n, g in grad.items():
        off = ((st.grad[n].double() - g).norm() / g.norm()).item()
        assert off <= OFF, (n, off)


def test_distillation_gradients():
    st = model()
    tokens = torch.randint(0, st.V, (st.T,), device="cuda")
    ids, logits = ex.Teacher(st.V, st.k).of(tokens)
    w = torch.full((st.T,), 1.0 / st.T, device="cuda")
    w[::7] = 0
    loss = st.loss_and_gradients(tokens, ids, logits, w).clone()
    st.check()
    pt, logp = (f(logits.double() / st.tau, 1) for f in (torch.softmax, torch.log_softmax))

    def loss_of(lq):
        return w.double() * st.tau ** 2 * (pt * (logp - lq.gather(1, ids.long()))).sum(1)

    compare(st, loss, *reference(st, tokens, loss_of))


def test_policy_gradients():
    st = model()
    tokens, sampled = (torch.randint(0, st.V, (st.T,), device="cuda") for _ in range(2))
    w = torch.full((st.T,), 1.0 / st.T, device="cuda")
    w[5::9] = 0
    now = st.log_probabilities(tokens, sampled, w)
    old, ref = now - 0.1 * torch.randn_like(now), now + 0.3 * torch.randn_like(now)
    adv = torch.randn_like(now)
    # (rows near the clip's borders stay out: a rounding decides there)
    r = torch.exp(now - old)
    w[((r - 0.8).abs() < 0.02) | ((r - 1.2).abs() < 0.02)] = 0
    loss = st.policy_and_gradients(tokens, sampled, old, ref, adv, w).clone()
    st.check()

    def loss_of(lq):
        lp = lq.gather(1, sampled[:, None])[:, 0]
        r, d = torch.exp(lp - old.double()), ref.double() - lp
        gain = torch.minimum(r * adv.double(), r.clamp(0.8, 1.2) * adv.double())
        return w.double() * (0.05 * (torch.exp(d) - d - 1) - gain)

    compare(st, loss, *reference(st, tokens, loss_of))


@pytest.mark.parametrize("bits", [32, 8])
def test_update(bits):
    """The first step of every weight by the formula (averages that start from zero: in 8 bits
    rounded only behind it), and the copies that the next forward reads."""
    st = model(bits=bits)
    tokens = torch.randint(0, st.V, (st.T,), device="cuda")
    w = torch.full((st.T,), 1.0 / st.T, device="cuda")
    st.loss_and_gradients(tokens, *ex.Teacher(st.V, st.k).of(tokens), w)
    before = {n: p.clone() for n, p in st.master.items()}
    st.update(lr=1e-2)
    for n, p in st.master.items():
        g = st.grad[n].double()
        want = before[n].double() - 1e-2 * g / (g.abs() + 1e-8)
        # (the step is off by about 10 roundings, of 2^-24 of it each, and beta in fp32 by 2^-24 / 0.01)
        assert (p.double() - want).abs().max() <= 1e-2 * 2 ** -16 + 2 ** -23 * before[n].abs().max(), n
        copy = st.p[n]
        assert torch.equal(copy, p.bfloat16() if p.dim() == 2 else p), n


def test_serving_goes_on_from_the_state():
    """Logits token by token, in 8 bits, are those of the whole sequences' forward up to the
    rounding of q, and of the states and activations that the two round apart."""
    B, L, V = 3, 20, 200
    st = ex.Student(B * L, V, 128, 256, layers=2, k=8, mix=True,
                    starts=torch.arange(0, B * L + 1, L, dtype=torch.int32, device="cuda"))
    tokens = torch.randint(0, V, (B, L), device="cuda")
    want = (st.forward(tokens.view(-1)) @ st.p["out"].t()).float().view(B, L, V)
    srv = ex.Server(st, B)
    for t in range(L):
        z = srv.logits(tokens[:, t].contiguous()).float()
        assert (z - want[:, t]).norm() <= OFF * want[:, t].norm(), t
    st.check()


@pytest.mark.parametrize("args", [["--mix", "--tune", "3"], ["--bits", "8"]])
def test_command(args):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "distill_student.py"),
                        "--steps", "3"] + args, capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "served" in r.stdout.splitlines()[-1]
