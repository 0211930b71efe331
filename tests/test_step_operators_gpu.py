"""The recurrence, the policy loss and the AdamW step as a program has them: call after call with
nothing waited for in between, two at once on two streams, captured before any of them has run in
the process, and one captured step replayed while others run."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import setup, status

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF16 = tw.TWELL_BF16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


class Step:
    """A training step's tail on its own buffers: x -> recurrence -> logits (a product in torch) ->
    policy loss and gradient -> back -> AdamW of the product's weights and the recurrence's bias."""

    def __init__(self, T, D, V, seed, bits=8):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        r = lambda *s, dt=torch.float32: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
        e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        self.T, self.D, self.V, self.no = T, D, V, 0
        self.xg, self.starts = r(T, 2 * D, dt=torch.bfloat16), torch.tensor(
            [0, T // 3, T // 3, T // 2 + 1, T - 2], dtype=torch.int32, device="cuda")
        self.w, self.bias = r(V, D) * D ** -0.5, torch.linspace(0, 4, D, device="cuda")
        self.tok, self.adv = torch.randint(0, V, (T,), generator=g, device="cuda"), r(T)
        self.weight = torch.full((T,), 1.0 / T, device="cuda")
        self.h, self.dxg, self.dw, self.db = e(T, D), e(T, 2 * D), e(V, D, dt=torch.float32), e(D, dt=torch.float32)
        self.kept = e(tw.twell_recur_states(T), D, dt=torch.float32)
        self.z, self.copy, self.dh = e(T, V), self.w.bfloat16(), e(T, D)
        self.loss, self.logp, self.stats = e(T, dt=torch.float32), e(T, dt=torch.float32), e(T, 2, dt=torch.float32)
        self.status, self.list = status(), tw.AdamWTensors(bits)
        self.state, first = [], 0
        for p, d, c in ((self.w, self.dw, self.copy), (self.bias, self.db, None)):
            kind = torch.float8_e4m3fn if bits == 8 else torch.float32
            st = [torch.zeros_like(p, dtype=kind) for _ in range(2)]
            sc = [e(-(-p.numel() // 256), dt=torch.float32) for _ in range(2)] if bits == 8 else []
            self.list.add(p, d, *st, *sc, copy=c, first=first, decay=0.01)
            self.state += st + sc
            first += -(-p.numel() // 256) * 256
        self.dyn = torch.zeros(4, dtype=torch.int32, device="cuda")
        torch.cuda.synchronize()

    def run(self, dynamic=False):
        T, D, V = self.T, self.D, self.V
        x, gate, dx, dg = self.xg[:, :D], self.xg[:, D:], self.dxg[:, :D], self.dxg[:, D:]
        self.no += 1
        tw.twell_recur_forward(x, gate, 2 * D, self.bias, self.starts, 4, None, T, D, BF16, self.h, None,
                               self.kept, self.status)
        torch.matmul(self.h, self.copy.t(), out=self.z)
        tw.twell_policy_forward(self.z, V, self.tok, None, None, self.adv, self.weight, T, V, BF16, 1.0,
                                0.2, 0.2, 0.0, self.loss, self.logp, self.stats, self.z, self.status)
        self.dw.copy_(self.z.t() @ self.h)
        torch.matmul(self.z, self.copy, out=self.dh)
        tw.twell_recur_backward(x, gate, 2 * D, self.bias, self.starts, 4, None, self.kept, self.dh, None,
                                T, D, BF16, dx, dg, self.db, None, self.status)
        tw.twell_adamw_step(self.list, 1e-2, 0.9, 0.99, 1e-8, self.no, seed=self.no,
                            dynamic=self.dyn if dynamic else None)

    def all(self):
        return [self.h, self.kept, self.loss, self.logp, self.stats, self.dxg, self.db, self.dw, self.w,
                self.bias, self.copy] + self.state


def same(a, b):
    return all(torch.equal(x.contiguous().view(torch.uint8), y.contiguous().view(torch.uint8))
               for x, y in zip(a.all(), b.all()))


SIZES = [(500, 192, 700), (65, 64, 5001), (1500, 2048, 300)]


@pytest.mark.parametrize("T,D,V", SIZES)
@pytest.mark.parametrize("bits", [8, 32])
def test_steps_back_to_back(T, D, V, bits):
    a, b = Step(T, D, V, 1, bits), Step(T, D, V, 1, bits)
    for _ in range(12):
        a.run()
    for _ in range(12):
        b.run()
        torch.cuda.synchronize()
    assert same(a, b) and tw.twell_read_status(a.status) == 0
    assert torch.isfinite(a.w).all() and a.loss.abs().sum() > 0


@pytest.mark.parametrize("T,D,V", SIZES)
def test_two_at_once(T, D, V):
    """On two streams, interleaved: what each gives alone."""
    alone = [Step(T, D, V, s) for s in (1, 2)]
    for m in alone:
        for _ in range(8):
            m.run()
    both, streams = [Step(T, D, V, s) for s in (1, 2)], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(8):
        for m, s in zip(both, streams):
            with torch.cuda.stream(s):
                m.run()
    torch.cuda.synchronize()
    for m, n in zip(both, alone):
        assert same(m, n) and tw.twell_read_status(m.status) == 0


def test_a_replayed_step_beside_others():
    """Steps captured once, replayed with their scalars from device memory, while another model's run
    on a second stream: the bits of the same steps called one by one."""
    want, got, other = Step(500, 192, 700, 1), Step(500, 192, 700, 1), Step(500, 192, 700, 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got.run(dynamic=True)
    for n in range(1, 7):
        for m in (want, got):
            m.dyn.copy_(tw.adamw_dynamic(1e-2, 0.9, 0.99, n, seed=n))
        want.run(dynamic=True)
        graph.replay()
        with torch.cuda.stream(s):
            other.run()
    torch.cuda.synchronize()
    assert same(want, got) and not same(want, other)
    assert tw.twell_read_status(got.status) == 0 and tw.twell_read_status(other.status) == 0


CHILD = textwrap.dedent(r"""
    import sys
    sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
    import torch
    import test_step_operators_gpu as t

    a = t.Step(500, 192, 700, 1)
    torch.matmul(a.h, a.copy.t(), out=a.z)     # (the library of the products is up)
    a.dw.copy_(a.z.t() @ a.h)
    torch.matmul(a.z, a.copy, out=a.dh)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        a.run()
    graph.replay()
    torch.cuda.synchronize()
    b = t.Step(500, 192, 700, 1)
    b.run()
    torch.cuda.synchronize()
    assert t.same(a, b)
    print("DONE")
""")


def test_the_first_calls_of_a_process_are_captured():
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, timeout=300,
                       cwd=ROOT)
    assert r.returncode == 0 and "DONE" in r.stdout, r.stdout[-500:] + r.stderr[-3000:]
