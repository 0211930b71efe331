"""The 8-bit product against exact integer sums.

Bounds, with u = 2^-24: for K <= 1024 every partial sum is an integer below
2^24, so the accumulator is exact and the result has three fp32 roundings
(two scales, the bias): 3 u of |sum sa sw| + |bias| in total, and its storage.
Beyond, each of the at most K / 8 additions into the fp32 accumulator loses
at most 2 u (rounding towards zero) of a partial sum of magnitude at most
sum |a w|, and nothing where that stays below 2^24."""
import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import DT, U, check, empty, gen, scratch, setup, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


def run(a, w, sa, sw, bias, dtype):
    (M, K), N = a.shape, w.shape[0]
    tdt, dt = DT[dtype]
    y, st = empty(M, N, dtype=tdt), status()
    ws, n = scratch(tw.twell_q8_workspace_size(M, N, K))
    tw.twell_q8_matmul(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(),
                       None if bias is None else bias.cuda(), M, N, K, dt, y, st, ws, n)
    assert tw.twell_read_status(st) == 0
    return y


def verify(a, w, sa, sw, bias, dtype):
    y = run(a, w, sa, sw, bias, dtype)
    acc = a.cuda().double() @ w.cuda().double().t()        # integers, exact in 64 bits
    mag = a.cuda().double().abs() @ w.cuda().double().abs().t()
    K = a.shape[1]
    eacc = torch.where(mag < 2.0 ** 24, 0.0, K / 8 * 2 * U * mag)
    scale = sa.cuda().double()[:, None] * sw.cuda().double()
    ref = acc * scale
    bound = eacc * scale.abs() + 3 * U * ref.abs()
    if bias is not None:
        ref = ref + bias.cuda().double()
        bound = bound + 3 * U * bias.cuda().double().abs()
    check(y, ref.cpu(), bound.cpu(), dtype, "y")
    assert torch.equal(run(a, w, sa, sw, bias, dtype), y)
    return y


def inputs(M, N, K, seed, lo=-127):
    g = gen(seed)
    a = torch.randint(lo, 128, (M, K), generator=g, dtype=torch.int8)
    w = torch.randint(lo, 128, (N, K), generator=g, dtype=torch.int8)
    return (a, w, torch.rand(M, generator=g) + 0.01, torch.rand(N, generator=g) + 0.01,
            torch.randn(N, generator=g) * 100)


SHAPES = [(1, 1, 16), (1, 64, 128), (1, 8192, 2048), (1, 50001, 512), (2, 33, 48), (3, 1000, 4096),
          (4, 129, 8192), (5, 77, 1040), (8, 14336, 256), (9, 300, 2064), (16, 128, 64),
          (17, 255, 1024), (31, 257, 528), (37, 4096, 1008), (64, 513, 2048), (65, 100, 80),
          (100, 3001, 1024), (127, 128, 4096), (128, 256, 64), (129, 130, 144), (250, 1001, 768),
          (256, 512, 128), (300, 2000, 2000), (513, 129, 16), (1001, 5001, 2048), (1500, 64, 7008),
          (4096, 2048, 512)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype,bias", [("bf16", False), ("f32", True)])
def test_against_exact_sums(M, N, K, dtype, bias):
    a, w, sa, sw, b = inputs(M, N, K, M + N + K)
    verify(a, w, sa, sw, b if bias else None, dtype)


@pytest.mark.parametrize("M,N,K", [(1, 200, 65536), (20, 130, 16384), (300, 300, 16384)])
def test_largest_sums(M, N, K):
    """All entries -128: the sums are the largest there can be."""
    a = torch.full((M, K), -128, dtype=torch.int8)
    w = torch.full((N, K), -128, dtype=torch.int8)
    w[::2] = 127
    w[1, K // 2:] = 127
    verify(a, w, torch.ones(M), torch.ones(N), None, "f32")


@pytest.mark.parametrize("M", [1, 7, 40, 300])
def test_every_value_and_lane(M):
    """Row m of a picks out column m's bytes: each product is a single entry of w, over all 256
    values."""
    K, N = 512, 300
    w = (torch.arange(N * K) % 256 - 128).to(torch.int8).reshape(N, K)
    a = torch.zeros(M, K, dtype=torch.int8)
    at = torch.arange(M) * 37 % K
    a[torch.arange(M), at] = 1
    y = run(a, w, torch.ones(M), torch.ones(N), None, "f32")
    assert torch.equal(y.cpu(), w.float().t()[at])


@pytest.mark.parametrize("M", [1, 6, 50, 200])
def test_scales_at_the_edges(M):
    """Scales of zero, infinity and NaN reach their row or column only."""
    a, w, sa, sw, _ = inputs(M, 140, 256, M)
    sw[3], sw[70] = 0.0, float("nan")
    sa[0] = float("nan")
    y = run(a, w, sa, sw, None, "f32").cpu()
    bad = torch.zeros(M, 140, dtype=torch.bool)
    bad[0] = True
    bad[:, 70] = True
    assert torch.equal(torch.isnan(y), bad)
    assert (y[1:, 3] == 0).all()


def test_norm_feeds_the_product():
    """The norm's 8-bit output through the product against the 64-bit chain: the rounding of q
    (half a step, uniform) is the error that remains; 6 standard deviations of its sum."""
    g = gen(77)
    T, D, N = 50, 1024, 700
    x = torch.randn(T, D, generator=g).bfloat16().cuda()
    wn = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    W = (torch.randn(N, D, generator=g) / 32).bfloat16().cuda()
    q, qs = empty(T, D, dtype=torch.int8), empty(T)
    wq, ws_ = empty(N, D, dtype=torch.int8), empty(N)
    tw.twell_add_rmsnorm_forward(x, None, wn, T, D, tw.TWELL_BF16, 1e-6, None, None, q, qs, None)
    tw.twell_q8_quantize(W, N, D, tw.TWELL_BF16, wq, ws_)
    y = run(q.cpu(), wq.cpu(), qs.cpu(), ws_.cpu(), None, "f32").double()
    xd = x.double()
    h = xd / torch.sqrt((xd * xd).mean(1, keepdim=True) + 1e-6) * wn.double()
    ref = h @ W.double().t()
    sd = torch.sqrt((qs.double()[:, None] ** 2 / 12) * (W.double() ** 2).sum(1)
                    + (ws_.double() ** 2 / 12) * (h ** 2).sum(1)[:, None])
    assert ((y - ref).abs() <= 6 * sd).all()


def test_other_stream_and_graph():
    for M in (1, 200):
        a, w, sa, sw, b = inputs(M, 600, 1024, 5)
        want = run(a, w, sa, sw, b, "bf16")
        a, w, sa, sw, b = (t.cuda() for t in (a, w, sa, sw, b))
        y, st = empty(M, 600, dtype=torch.bfloat16), status()
        ws, n = scratch(tw.twell_q8_workspace_size(M, 600, 1024))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            tw.twell_q8_matmul(a, sa, w, sw, b, M, 600, 1024, tw.TWELL_BF16, y, st, ws, n)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


@pytest.mark.parametrize("M,N,K", [(128, 50000, 4096), (40, 30001, 4112), (100, 20000, 8192),
                                   (300, 40001, 4096), (700, 9000, 8208)])
def test_many_tiles(M, N, K):
    """Several tiles a CTA or pair, every ring of stages used many times over."""
    a, w, sa, sw, _ = inputs(M, N, K, M + N + K)
    for _ in range(3):
        verify(a, w, sa, sw, None, "bf16")


@pytest.mark.parametrize("M,N,K", [(5, 14336, 4096), (9, 25001, 2064), (16, 50000, 1040),
                                   (33, 1, 16), (40, 129, 4112), (97, 1030, 2064),
                                   (128, 2048, 8192), (128, 4104, 528)])
@pytest.mark.parametrize("dtype,bias", [("bf16", True), ("f32", True), ("bf16", False)])
def test_few_rows(M, N, K, dtype, bias):
    """Up to 128 rows: MMAs as wide as the rows, tiles alone or shared by a cluster, columns that
    end inside a tile, a warp or a vector of eight."""
    a, w, sa, sw, b = inputs(M, N, K, M + N + K)
    verify(a, w, sa, sw, b if bias else None, dtype)


@pytest.mark.parametrize("M,N,K", [(33, 1000, 1024), (48, 4096, 2048), (49, 301, 2064),
                                   (63, 4095, 1040), (64, 128, 64), (64, 4097, 528)])
def test_fragments_of_many_rows(M, N, K):
    """33 to 64 rows of small weights, up to where they leave the fragments."""
    a, w, sa, sw, b = inputs(M, N, K, M + N + K)
    verify(a, w, sa, sw, b, "bf16")


@pytest.mark.parametrize("M,N,K", [(5, 130, 16384), (16, 257, 8208), (17, 1000, 8192),
                                   (33, 128, 4112), (48, 300, 16384), (49, 1000, 2064),
                                   (64, 1024, 8192), (64, 100, 65536)])
def test_long_sums_of_few_columns(M, N, K):
    """Where few columns leave the fragments for their long k."""
    a, w, sa, sw, b = inputs(M, N, K, M + N + K)
    verify(a, w, sa, sw, b, "f32")


TIMEOUT_CHILD = """
import sys
import torch
sys.path.insert(0, sys.argv[1])
import activation_sparse_transformer_gate_gb300 as tw
from activation_sparse_transformer_gate_gb300 import _build
lib = tw.load(_build.lib_path("timeout"))
sh = torch.cuda.current_stream().cuda_stream
for M, N, K in ((100, 2000, 1024), (700, 2000, 1024), (100, 20000, 8192), (128, 50000, 4096),
                (1000, 20000, 4096)):
    a = torch.ones(M, K, dtype=torch.int8, device="cuda")
    w = torch.ones(N, K, dtype=torch.int8, device="cuda")
    sa, sw = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
    y = torch.zeros(M, N, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    n = lib.twell_q8_workspace_size(M, N, K)
    ws = torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda")
    P = lambda t: t.data_ptr()
    rc = lib.twell_q8_matmul(P(a), P(sa), P(w), P(sw), None, M, N, K, 0, P(y), P(st), P(ws), n, sh)
    print("RESULT", rc, lib.twell_read_status(P(st), sh), lib.twell_read_status(P(st), sh),
          int((a.float().sum(1) == K).all()), int((y == K).all()))
"""


def test_waits_that_run_out():
    """With the waits' limit at 1 ns (the test-only build) both tensor-core kernels return, record
    TWELL_ERR_TIMEOUT and leave the context usable.  (A wait whose first try lasts until it is
    satisfied does not run out: a call may also come through, and is then right.)"""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    tw._build.build(variants=("timeout",))
    r = subprocess.run([sys.executable, "-c", TIMEOUT_CHILD, root], capture_output=True, text=True,
                       timeout=300, cwd=root)
    assert r.returncode == 0, r.stdout[-2000:] + r.stderr[-2000:]
    got = [ln.split()[1:] for ln in r.stdout.splitlines() if ln.startswith("RESULT")]
    assert len(got) == 5
    for rc, first, second, usable, right in got:
        assert rc == "0" and second == "0" and usable == "1", got
        assert first == "-6" or (first == "0" and right == "1"), got
    ran_out = [g[1] == "-6" for g in got]
    assert ran_out[0] or ran_out[2] or ran_out[3], got      # up to 128 rows
    assert ran_out[1] or ran_out[4], got                    # CTA pairs
