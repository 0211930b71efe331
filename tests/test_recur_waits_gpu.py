"""The recurrence's waits with a limit of 1 ns, each direction with a status word of its own: both
report waits that ran out, of every width of their kernels, what was on its way has come in (the
outputs have the bits of the product library's), and the context stays usable."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TIMEOUT = -6

CHILD = textwrap.dedent(r"""
    import sys
    import torch
    sys.path.insert(0, sys.argv[1])
    import activation_sparse_transformer_gate_gb300 as tw
    from activation_sparse_transformer_gate_gb300 import _build

    P = lambda t: None if t is None else t.data_ptr()

    def run(lib, T, D, dt, x, gate, dh, starts):
        h, dx, dg = (torch.zeros_like(x) for _ in range(3))
        kept = torch.zeros(lib.twell_recur_states(T), D, device="cuda")
        st = torch.zeros(2, dtype=torch.int32, device="cuda")
        s = torch.cuda.current_stream().cuda_stream
        rc = lib.twell_recur_forward(P(x), P(gate), D, None, P(starts), 2, None, T, D, dt, P(h), None,
                                     P(kept), P(st[:1]), s)
        rc2 = lib.twell_recur_backward(P(x), P(gate), D, None, P(starts), 2, None, P(kept), P(dh),
                                       None, T, D, dt, P(dx), P(dg), None, None, P(st[1:]), s)
        torch.cuda.synchronize()
        assert rc == rc2 == 0
        return tuple(st.tolist()), (h, dx, dg)

    good, late = tw.load(), tw.load(_build.lib_path("timeout"))
    for T, D, dt in ((3000, 512, 1), (6000, 512, 1), (3000, 1536, 1), (6000, 2560, 1), (6000, 512, 0)):
        g = torch.Generator(device="cuda")
        g.manual_seed(T + D)
        kind = torch.bfloat16 if dt else torch.float32
        x, gate, dh = (torch.randn(T, D, generator=g, device="cuda", dtype=kind) for _ in range(3))
        starts = torch.tensor([0, 1234, T], dtype=torch.int32, device="cuda")
        args = (T, D, dt, x, gate, dh, starts)
        codes, want = run(good, *args)
        assert codes == (0, 0), codes
        seen = set()
        for _ in range(20):
            codes, got = run(late, *args)
            assert all(c in (0, -6) for c in codes), codes
            assert all(torch.equal(a, b) for a, b in zip(want, got))
            seen |= {(i, c) for i, c in enumerate(codes)}
        assert (0, -6) in seen and (1, -6) in seen, (T, D, dt, seen)
        codes, again = run(good, *args)
        assert codes == (0, 0) and all(torch.equal(a, b) for a, b in zip(want, again))
    print("DONE")
""")


def test_both_directions_report():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    tw._build.build(variants=("", "timeout"))
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT], capture_output=True, text=True, timeout=300,
                       cwd=ROOT)
    assert r.returncode == 0, r.stdout[-1000:] + r.stderr[-3000:]
    assert "DONE" in r.stdout
