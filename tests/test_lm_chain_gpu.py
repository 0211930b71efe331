"""The norm's 8-bit output and the product behind it, call after call through the same q, qscale and
workspace with nothing waited for in between, on a stream and in a graph: the product starts while
the kernel that widens its rows still runs, and must neither read what the call before left nor
widen over rows that are still read.  The results have the bits of calls that stand alone."""
import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import empty, gen, scratch, setup, status

pytestmark = pytest.mark.gpu
BF16 = tw.TWELL_BF16

# rows of a, columns of y, k: few rows with a CTA a tile, with shared tiles, pairs, fragments, rows
SHAPES = [(37, 14336, 4096), (100, 2048, 2048), (128, 130, 1040), (300, 2000, 2048),
          (129, 14336, 1024), (40, 1000, 1024), (3, 8192, 2048)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


class Chain:
    def __init__(self, M, N, K, sets=3):
        g = gen(M + N + K)
        self.size = M, N, K
        self.x = [(torch.randn(M, K, generator=g) * (1 + i)).bfloat16().cuda() for i in range(sets)]
        self.wn = (1 + 0.1 * torch.randn(K, generator=g)).cuda()
        self.w = torch.randint(-127, 128, (N, K), generator=g, dtype=torch.int8).cuda()
        self.sw = (torch.rand(N, generator=g) + 0.1).cuda()
        self.y = [empty(M, N, dtype=torch.bfloat16) for _ in range(sets)]
        self.q, self.qs, self.st = empty(M, K, dtype=torch.int8), empty(M), status()
        self.ws, self.n = scratch(tw.twell_q8_workspace_size(M, N, K))
        torch.cuda.synchronize()

    def call(self, i):
        M, N, K = self.size
        tw.twell_add_rmsnorm_forward(self.x[i], None, self.wn, M, K, BF16, 1e-6, None, None, self.q,
                                     self.qs, None)
        tw.twell_q8_matmul(self.q, self.qs, self.w, self.sw, None, M, N, K, BF16, self.y[i], self.st,
                           self.ws, self.n)

    def alone(self):
        want = []
        for i in range(len(self.x)):
            self.call(i)
            torch.cuda.synchronize()
            acc = self.q.double() @ self.w.double().t()     # (below 2^24 at these K: exact)
            assert acc.abs().max() < 2 ** 24
            ref = (acc.float() * self.qs[:, None] * self.sw).bfloat16()
            assert torch.equal(self.y[i], ref)
            want.append(ref)
        assert not torch.equal(want[0], want[1])
        return want

    def compare(self, want):
        torch.cuda.synchronize()
        for y, w in zip(self.y, want):
            assert torch.equal(y, w)
            y.fill_(float("nan"))
        assert tw.twell_read_status(self.st) == 0


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_calls_back_to_back(M, N, K):
    c = Chain(M, N, K)
    want = c.alone()
    for order in ((0, 1, 2), (2, 0, 1), (1, 1, 0, 2, 2, 0, 1), (0, 2, 1) * 8):
        for i in order:
            c.call(i)
        c.compare(want)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_calls_back_to_back_in_a_graph(M, N, K):
    c = Chain(M, N, K)
    want = c.alone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        for i in (0, 1, 2, 2, 1, 0):
            c.call(i)
    for _ in range(3):
        graph.replay()
        graph.replay()
        c.compare(want)


@pytest.mark.parametrize("M,N,K", SHAPES[:5])
def test_what_follows_reads_all_of_it(M, N, K):
    """The rows that the next kernel of the stream reads are the product's: y feeds a norm at once."""
    if N % 16 or N > 8192:
        N = 2048
    c = Chain(M, N, K)
    want = c.alone()
    ones = torch.ones(N, device="cuda")
    q2, qs2 = empty(M, N, dtype=torch.int8), empty(M)
    for i in (0, 1, 2, 0, 1, 2):
        c.call(i)
        tw.twell_add_rmsnorm_forward(c.y[i], None, ones, M, N, BF16, 1e-6, None, None, q2, qs2, None)
        c.y[i].fill_(float("nan"))                     # (behind the norm on the stream)
    q3, qs3 = empty(M, N, dtype=torch.int8), empty(M)
    torch.cuda.synchronize()
    tw.twell_add_rmsnorm_forward(want[2], None, ones, M, N, BF16, 1e-6, None, None, q3, qs3, None)
    torch.cuda.synchronize()
    assert torch.equal(q2, q3) and torch.equal(qs2, qs3)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_weights_written_right_before(M, N, K):
    """Weights quantised on the stream just before the product that reads them."""
    c = Chain(M, N, K, sets=1)
    g = gen(K)
    W = [torch.randn(N, K, generator=g).bfloat16().cuda() for _ in range(2)]
    c.call(0)
    want = []
    for w in W:
        tw.twell_q8_quantize(w, N, K, BF16, c.w, c.sw)
        torch.cuda.synchronize()
        want.append(((c.q.double() @ c.w.double().t()).float() * c.qs[:, None] * c.sw).bfloat16())
    y = [torch.empty_like(c.y[0]) for _ in range(6)]
    for i in range(6):
        tw.twell_q8_quantize(W[i & 1], N, K, BF16, c.w, c.sw)
        tw.twell_q8_matmul(c.q, c.qs, c.w, c.sw, None, M, N, K, BF16, y[i], c.st, c.ws, c.n)
    for i in range(6):
        assert torch.equal(y[i], want[i & 1])
