"""The example model (examples/distill_student.py), which runs the operators
around the FFN together with it: its gradients against automatic
differentiation of the same model in 64 bits, and that it learns and serves.

The reference goes on, at each place where the model stores an activation, from
what the model stored there (with the gradient of the identity), after comparing
the two: rounded apart, a thousandth of the ReLUs would be on the other side of
zero, which alone is 3% of a gradient in the 2-norm.  What is left are the
roundings of one layer's activations, and those of the gradients, each 2^-9
relative; a gradient passes about 15 of them in a chain of 2 layers, each of
them random, so all are compared in the 2-norm with 15^(1/2) 2^-9 times 4
(0.03)."""
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


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw._build.build()
    tw.load()


def reference(st, tokens, ids, teacher, w):
    """Losses and gradients of the student's bf16 weights, by autograd in 64 bits."""
    p = {n: v.double().requires_grad_(True) for n, v in st.p.items()}

    def norm(s, weight):
        return s / torch.sqrt((s * s).mean(1, keepdim=True) + ex.EPS) * weight

    def stored(x, actual):
        actual = actual.double()
        assert (x.detach() - actual).norm() <= 0.03 * actual.norm()
        return x + (actual - x.detach())

    s = p["embed"][tokens] * st.scale
    l1, y = 0.0, None
    for i in range(st.L):
        s = stored(s if y is None else s + y, st.s[i])
        n = stored(norm(s, p[f"norm{i}"]), st.n[i])
        h = torch.relu(n @ p[f"gate{i}"].t() + p[f"bias{i}"]) * (n @ p[f"up{i}"].t())
        l1 = l1 + st.lam * h.abs().sum()
        y = h @ p[f"down{i}"]
    n = stored(norm(stored(s + y, st.s[st.L]), p["norm_out"]), st.n[st.L])
    z = (n @ p["out"].t()) / st.tau
    pt = torch.softmax(teacher.double() / st.tau, 1)
    logp = torch.log_softmax(teacher.double() / st.tau, 1)
    logq = torch.log_softmax(z, 1).gather(1, ids.long())
    loss = w.double() * st.tau ** 2 * (pt * (logp - logq)).sum(1)
    (loss.sum() + l1).backward()
    return loss, {n: v.grad for n, v in p.items()}


def test_gradients_against_autograd():
    T, V, k = 384, 300, 16
    teacher = ex.Teacher(V, k)
    st = ex.Student(T, V, 256, 512, layers=2, k=k, tau=1.5, lam=1e-6)
    tokens = torch.randint(0, V, (T,), device="cuda")
    ids, logits = teacher.of(tokens)
    w = torch.full((T,), 1.0 / T, device="cuda")
    w[::7] = 0
    loss = st.loss_and_gradients(tokens, ids, logits, w).clone()
    st.check()
    ref, grad = reference(st, tokens, ids, logits, w)
    assert (loss - ref).norm() <= 0.03 * ref.norm()
    assert (loss[::7] == 0).all()
    for n, g in grad.items():
        off = ((st.grad[n].double() - g).norm() / g.norm()).item()
        assert off <= 0.03, (n, off)


def test_it_learns_and_serves():
    """Steps lower the loss, and the 8-bit logits are the bf16 ones up to the rounding of q (a
    127th of a row's largest value, uniform: 1 / (127 * 12^(1/2)) of it, twice)."""
    T, V, k = 2048, 400, 32
    teacher, st = ex.Teacher(V, k), ex.Student(2048, V, 128, 512, layers=2, k=k)
    w = torch.full((T,), 1.0 / T, device="cuda")
    losses = []
    for step in range(60):
        tokens = torch.randint(0, V, (T,), device="cuda")
        losses.append(st.loss_and_gradients(tokens, *teacher.of(tokens), w).sum().item())
        st.update(lr=3e-3)
    st.check()
    assert losses[-1] < 0.5 * losses[0], losses[::10]
    for n in (1, 13, 300):
        tokens = torch.arange(n, device="cuda")
        z = ex.Server(st, n).logits(tokens).float()
        full = torch.zeros(T, dtype=torch.long, device="cuda")
        full[:n] = tokens
        want = st.forward(full)[:n].float() @ st.p["out"].float().t()
        assert (z - want).norm() <= 0.03 * want.norm(), n
    st.check()


def test_command():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "distill_student.py"),
                        "--steps", "41"], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    lines = r.stdout.splitlines()
    first, last = (float(ln.split()[-1]) for ln in (lines[0], lines[2]))
    assert last < first and "served" in lines[-1]
