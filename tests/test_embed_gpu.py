"""Token embedding and its gradient by sorted tokens against 64-bit sums.

Bounds: the forward is one fp32 product rounded once (bit-exact against the
same two roundings); a gradient entry is an fp32 sum of n values and one
product, so it is within (n + 1) 2^-24 scale sum|dy| of the exact one in any
order of summation."""
import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import DT, U, check, empty, gen, scratch, setup, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


def run(tok, table, dy, V, D, dtype, scale, pad_id):
    T = tok.numel()
    tdt, dt = DT[dtype]
    st = status()
    out, dtable = empty(T, D, dtype=tdt), empty(V, D)
    ws, n = scratch(tw.twell_embed_workspace_size(T, V, D))
    tok, table, dy = tok.cuda(), table.cuda(), dy.cuda()
    tw.twell_embed_forward(tok, table, T, V, D, dt, scale, pad_id, out, st)
    tw.twell_embed_backward(tok, dy, T, V, D, dt, scale, pad_id, dtable, st, ws, n)
    return out, dtable, tw.twell_read_status(st)


def reference(tok, table, dy, V, scale, pad_id):
    live = (tok != pad_id) & (tok >= 0) & (tok < V)
    at = torch.where(live, tok, 0).long()
    prod = table.float()[at] * torch.tensor(scale, dtype=torch.float32)
    out = torch.where(live[:, None], prod, 0.0).to(table.dtype)
    s32 = float(torch.tensor(scale, dtype=torch.float32))
    d = dy[live].double()
    grad = torch.zeros(V, dy.shape[1], dtype=torch.float64).index_add_(0, at[live], d) * s32
    mag = torch.zeros_like(grad).index_add_(0, at[live], d.abs()) * abs(s32)
    n = torch.zeros(V, dtype=torch.float64).index_add_(0, at[live], torch.ones_like(d[:, 0]))
    return out, grad, (n[:, None] + 1) * U * mag * 1.001


def tokens_of(kind, T, V, g):
    if kind == "zipf":
        return (torch.exp(torch.rand(T, generator=g) * torch.log(torch.tensor(V + 1.0))) - 1) \
            .long().clamp_(0, V - 1)
    if kind == "same":
        return torch.full((T,), V // 2)
    if kind == "distinct":
        return torch.randperm(V, generator=g)[:T]
    return torch.randint(0, V, (T,), generator=g)


CASES = [  # kind, T, V, D, dtype, token type
    ("uniform", 1, 1, 8, "bf16", torch.int64),
    ("uniform", 1, 50001, 2048, "bf16", torch.int32),
    ("zipf", 33, 512, 128, "f32", torch.int64),
    ("zipf", 64, 512, 128, "f32", torch.int32),
    ("zipf", 1000, 777, 2056, "bf16", torch.int64),
    ("zipf", 4097, 50001, 264, "bf16", torch.int32),
    ("same", 16, 9, 64, "bf16", torch.int64),
    ("same", 5003, 300, 72, "bf16", torch.int64),
    ("same", 40000, 100, 4, "f32", torch.int32),
    ("distinct", 1024, 1024, 40, "f32", torch.int64),
    ("distinct", 3001, 131072, 8, "bf16", torch.int64),
    ("uniform", 20000, 300000, 8, "bf16", torch.int32),   # three sort passes
    ("uniform", 70001, 300, 16, "bf16", torch.int64),
    ("uniform", 2000, 100, 4096, "f32", torch.int64),
    ("same", 512, 3, 40, "bf16", torch.int32),            # the most tokens of the one-launch form
    ("zipf", 512, 70001, 8, "bf16", torch.int64),
    ("uniform", 511, 20, 1032, "f32", torch.int64),
    ("zipf", 513, 300, 136, "bf16", torch.int64),         # the fewest of the sort
]


@pytest.mark.parametrize("kind,T,V,D,dtype,itype", CASES)
def test_against_64_bits(kind, T, V, D, dtype, itype):
    g = gen(T + V + D)
    tok = tokens_of(kind, T, V, g).to(itype)
    table = torch.randn(V, D, generator=g).to(DT[dtype][0])
    dy = torch.randn(T, D, generator=g).to(DT[dtype][0])
    scale = D ** 0.5
    out, dtable, code = run(tok, table, dy, V, D, dtype, scale, -1)
    assert code == 0
    ref, grad, bound = reference(tok, table, dy, V, scale, -1)
    assert torch.equal(out.cpu(), ref)
    check(dtable, grad, bound, "f32", "dtable")
    again = run(tok, table, dy, V, D, dtype, scale, -1)[1]
    assert torch.equal(again, dtable)  # the same bits


@pytest.mark.parametrize("kind,T,V,D", [
    ("uniform", 600, 5, 16), ("zipf", 2047, 511, 72), ("uniform", 2048, 512, 16),
    ("same", 2048, 40000, 8), ("distinct", 2048, 262143, 8), ("zipf", 2049, 50001, 24),
    ("uniform", 700, 262144, 8), ("zipf", 1537, 9000, 520)])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_sort_forms(kind, T, V, D, itype):
    """One, two and three passes, by one CTA (up to 2048 tokens below 2^18) and by the cluster;
    some tokens are padding, some out of range."""
    g = gen(T + V)
    tok = tokens_of(kind, T, V, g).to(itype)
    tok[5::11] = -7
    tok[9::17] = V
    table = torch.randn(V, D, generator=g).bfloat16()
    dy = torch.randn(T, D, generator=g).bfloat16()
    out, dtable, code = run(tok, table, dy, V, D, "bf16", 1.5, -7)
    assert code == -5
    ref, grad, bound = reference(tok, table, dy, V, 1.5, -7)
    assert torch.equal(out.cpu(), ref)
    check(dtable, grad, bound, "f32", "dtable")
    assert torch.equal(run(tok, table, dy, V, D, "bf16", 1.5, -7)[1], dtable)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_padding_and_out_of_range(dtype):
    """Padded positions give zero rows and take no gradient, whatever dy holds there; a token
    outside the vocabulary does the same and is recorded."""
    g = gen(5)
    T, V, D = 700, 97, 136
    tok = torch.randint(0, V, (T,), generator=g)
    tok[::3] = 7
    table = torch.randn(V, D, generator=g).to(DT[dtype][0])
    dy = torch.randn(T, D, generator=g).to(DT[dtype][0])
    dy[::3] = float("nan")
    out, dtable, code = run(tok, table, dy, V, D, dtype, 0.5, 7)
    assert code == 0
    ref, grad, bound = reference(tok, table, dy, V, 0.5, 7)
    assert torch.equal(out.cpu(), ref)
    check(dtable, grad, bound, "f32", "dtable")
    assert (dtable[7] == 0).all() and (out[::3] == 0).all()
    tok[5], tok[10], tok[11] = -4, V, 1 << 40
    dy[5], dy[10], dy[11] = float("inf"), float("nan"), float("nan")
    out, dtable, code = run(tok, table, dy, V, D, dtype, 0.5, 7)
    assert code == -5
    ref, grad, bound = reference(tok, table, dy, V, 0.5, 7)
    assert torch.equal(out.cpu(), ref)
    check(dtable, grad, bound, "f32", "dtable")


def test_all_padding():
    tok = torch.full((100,), -1)
    out, dtable, code = run(tok, torch.ones(11, 8), torch.full((100, 8), float("nan")), 11, 8, "f32",
                            1.0, -1)
    assert code == 0 and (out == 0).all() and (dtable == 0).all()


def test_gradient_against_differences():
    """The embedding is linear: <dtable, E> = L(table + E) - L(table) for L = <dy, out>."""
    g = gen(9)
    T, V, D, scale = 300, 50, 64, 1.75
    tok = tokens_of("zipf", T, V, g)
    table, step = torch.randn(V, D, generator=g), torch.randn(V, D, generator=g)
    dy = torch.randn(T, D, generator=g)
    _, dtable, _ = run(tok, table, dy, V, D, "f32", scale, -1)

    def loss(tab):
        return (dy.double() * tab.double()[tok] * scale).sum()

    want = loss(table.double() + step.double()) - loss(table)
    _, _, bound = reference(tok, table, dy, V, scale, -1)
    got = (dtable.double().cpu() * step.double()).sum()
    assert abs(got - want) <= (bound * step.abs()).sum() + 1e-10 * abs(want)


def test_other_stream_and_graph():
    """A step on a side stream, captured and replayed, gives the eager bits."""
    g = gen(3)
    T, V, D = 600, 400, 128
    tok = tokens_of("zipf", T, V, g).cuda()
    table, dy = torch.randn(V, D, generator=g).cuda(), torch.randn(T, D, generator=g).cuda()
    want = run(tok, table, dy, V, D, "f32", 2.0, -1)
    st, out, dtable = status(), empty(T, D), empty(V, D)
    ws, n = scratch(tw.twell_embed_workspace_size(T, V, D))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tw.twell_embed_forward(tok, table, T, V, D, tw.TWELL_F32, 2.0, -1, out, st)
        tw.twell_embed_backward(tok, dy, T, V, D, tw.TWELL_F32, 2.0, -1, dtable, st, ws, n)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(dtable, want[1])
