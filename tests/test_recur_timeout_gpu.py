"""The recurrence's waits for the other CTAs of a cluster with a limit of 1 ns: calls return,
what was on its way has come in (the outputs are the product library's), nothing but the status
word tells, and the context stays usable."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = textwrap.dedent(r"""
    import sys
    import torch
    sys.path.insert(0, sys.argv[1])
    import activation_sparse_transformer_gate_gb300 as tw
    from activation_sparse_transformer_gate_gb300 import _build

    T, D, B = 3000, 512, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, gate, dh = (torch.randn(T, D, generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    starts = torch.tensor([0, 1234, T], dtype=torch.int32, device="cuda")

    def run(lib):
        h, dx, dg = (torch.zeros_like(x) for _ in range(3))
        kept = torch.zeros(lib.twell_recur_states(T), D, device="cuda")
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        s = torch.cuda.current_stream().cuda_stream
        P = lambda t: None if t is None else t.data_ptr()
        rc = lib.twell_recur_forward(P(x), P(gate), D, None, P(starts), B, None, T, D, 1, P(h), None,
                                     P(kept), P(st), s)
        rc2 = lib.twell_recur_backward(P(x), P(gate), D, None, P(starts), B, None, P(kept), P(dh), None,
                                       T, D, 1, P(dx), P(dg), None, None, P(st), s)
        torch.cuda.synchronize()
        return rc, rc2, lib.twell_read_status(P(st), s), (h, dx, dg)

    good = run(tw.load())
    late = run(tw.load(_build.lib_path("timeout")))
    again = run(tw.load())
    assert good[:3] == (0, 0, 0) and again[:3] == (0, 0, 0), (good[:3], again[:3])
    assert late[:2] == (0, 0) and late[2] in (0, -6), late[:3]
    for a, b, c in zip(good[3], late[3], again[3]):
        assert torch.equal(a, b) and torch.equal(a, c)
    print("DONE", late[2])
""")


def test_waits_that_run_out():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw._build.build(variants=("", "timeout"))
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, timeout=300,
                       cwd=ROOT)
    assert r.returncode == 0, r.stdout[-1000:] + r.stderr[-3000:]
    assert "DONE" in r.stdout
