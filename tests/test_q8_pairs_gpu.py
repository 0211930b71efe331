"""CTA pairs of the 8-bit product end only after every commit of the leader's has arrived in both
CTAs: each looks at its own barriers as it leaves (test-only builds), where the product comes to its
end and where its waits run out at once."""
import os
import subprocess
import sys

import pytest

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import setup

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = """
import ctypes, sys
import torch
sys.path.insert(0, sys.argv[1])
import activation_sparse_transformer_gate_gb300 as tw
from activation_sparse_transformer_gate_gb300 import _build
lib = tw.load(_build.lib_path(sys.argv[2]))
ended, early = ctypes.c_uint(), ctypes.c_uint()
sh = torch.cuda.current_stream().cuda_stream
P = lambda t: t.data_ptr()
for M, N, K in ((129, 64, 16), (200, 300, 320), (256, 20000, 256), (700, 2000, 1024),
                (1000, 20000, 4096), (513, 129, 8208)):
    a = torch.ones(M, K, dtype=torch.int8, device="cuda")
    w = torch.ones(N, K, dtype=torch.int8, device="cuda")
    sa, sw = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    y, st = torch.zeros(M, N, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    n = lib.twell_q8_workspace_size(M, N, K)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    for _ in range(5):
        assert lib.twell_q8_matmul(P(a), P(sa), P(w), P(sw), None, M, N, K, 0, P(y), P(st), P(ws),
                                   n, sh) == 0
    code = lib.twell_read_status(P(st), sh)
    assert lib.twell_test_q8_pairs(ctypes.byref(ended), ctypes.byref(early)) == 0
    print("RESULT", code, int((y == K).all()), ended.value, early.value)
"""


@pytest.mark.parametrize("variant", ["hooks", "timeout"])
def test_pairs_leave_after_the_last_arrival(variant):
    setup()
    tw._build.build(variants=(variant,))
    r = subprocess.run([sys.executable, "-c", CHILD, ROOT, variant], capture_output=True, text=True,
                       timeout=300, cwd=ROOT)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    got = [[int(v) for v in ln.split()[1:]] for ln in r.stdout.splitlines()
           if ln.startswith("RESULT")]
    assert len(got) == 6
    for code, right, ended, early in got:
        assert ended >= 10 and ended % 10 == 0, got     # five calls, pairs
        assert early == 0, got
        assert (code == 0 and right) or (variant == "timeout" and code == -6), got
    if variant == "timeout":
        assert any(g[0] == -6 for g in got), got
