"""The operators around the FFN where element offsets pass 32 bits: more than
2^31 elements in an operand, checked at its first and last rows.  Bounds as in
the operators' own tests."""
import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import U, check, scratch, setup, status
from test_distill_gpu import reference as distill_reference
from test_rmsnorm_gpu import ref_norm

pytestmark = pytest.mark.gpu
BF16 = tw.TWELL_BF16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()
    yield
    torch.cuda.empty_cache()


def rand(*shape, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


@pytest.mark.parametrize("T", [300, 3000])
def test_embedding_table(T):
    V, D = 600001, 4096
    tok = torch.randint(0, V, (T,), device="cuda")
    tok[:3], tok[-2:] = V - 1, torch.tensor([0, V - 2], device="cuda")
    table, dy = rand(V, D), rand(T, D, seed=1)
    out, dtable, st = empty(T, D), empty(V, D, dtype=torch.float32).fill_(7.0), status()
    ws, n = scratch(tw.twell_embed_workspace_size(T, V, D))
    tw.twell_embed_forward(tok, table, T, V, D, BF16, 1.0, -1, out, st)
    tw.twell_embed_backward(tok, dy, T, V, D, BF16, 1.0, -1, dtable, st, ws, n)
    assert tw.twell_read_status(st) == 0
    assert torch.equal(out, table[tok])
    want = torch.zeros(D, dtype=torch.float64, device="cuda")
    mag = torch.zeros_like(want)
    for t in range(3):
        want += dy[t].double()
        mag += dy[t].double().abs()
    check(dtable[V - 1], want.cpu(), 4 * U * mag.cpu(), "f32", "last row")
    assert torch.equal(dtable[V - 2], dy[T - 1].float()) and torch.equal(dtable[0], dy[T - 2].float())
    named = torch.zeros(V, dtype=torch.bool, device="cuda")
    named[tok] = True
    assert (dtable.abs().amax(dim=1)[~named] == 0).all()


def test_embedding_rows():
    T, V, D = 530000, 1000, 4096
    tok = torch.randint(0, V, (T,), device="cuda")
    table, dy = rand(V, D), rand(T, D, seed=1)
    out, dtable, st = empty(T, D), empty(V, D, dtype=torch.float32), status()
    ws, n = scratch(tw.twell_embed_workspace_size(T, V, D))
    tw.twell_embed_forward(tok, table, T, V, D, BF16, 1.0, -1, out, st)
    tw.twell_embed_backward(tok, dy, T, V, D, BF16, 1.0, -1, dtable, st, ws, n)
    assert tw.twell_read_status(st) == 0
    assert torch.equal(out[-1000:], table[tok[-1000:]]) and torch.equal(out[:9], table[tok[:9]])
    for v in (0, 517, V - 1):
        rows = dy[tok == v].double()
        check(dtable[v], rows.sum(0).cpu(), ((len(rows) + 1) * U * rows.abs().sum(0)).cpu(), "f32",
              f"row {v}")


def test_norm():
    T, D = 530000, 4096
    x, res = rand(T, D), rand(T, D, seed=1)
    w = torch.ones(D, device="cuda")
    s, y, rstd = empty(T, D), empty(T, D), empty(T, dtype=torch.float32)
    q, qs = empty(T, D, dtype=torch.int8), empty(T, dtype=torch.float32)
    tw.twell_add_rmsnorm_forward(x, res, w, T, D, BF16, 1e-6, s, y, q, qs, rstd)
    for r in (slice(0, 5), slice(T - 5, T)):
        want = (x[r].float() + res[r].float()).bfloat16()
        assert torch.equal(s[r], want)
        ref = ref_norm(want, w)[1].cpu()
        check(y[r], ref, 32 * U * ref.abs(), "bf16", "y")
        top = ref.abs().amax(1, keepdim=True)
        assert (q[r].double().cpu() - ref * 127 / top).abs().max() <= 0.5 + 127 * 128 * U
    dw = empty(D, dtype=torch.float32)
    ws, n = scratch(tw.twell_add_rmsnorm_workspace_size(T, D))
    tw.twell_add_rmsnorm_backward(s, w, rstd, y, None, T, D, BF16, x, dw, ws, n)
    # dy = y: the gradient of sum(xhat^2) / 2 is zero but for y's rounding (2^-9 of |y| <= 7, twice)
    assert (x[-5:].float().abs() <= 2 ** -7 * 7 * rstd[-5:, None]).all()
    exact = (y.float() * s.float() * rstd[:, None]).sum(dim=0, dtype=torch.float64)
    assert ((dw - exact).abs() <= (T + 64) * U * 1.1 * exact).all()


def test_product():
    M, N, K = 45000, 50001, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    a = torch.randint(-127, 128, (M, K), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-127, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    sa, sw = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
    y, st = empty(M, N), status()
    ws, n = scratch(tw.twell_q8_workspace_size(M, N, K))
    tw.twell_q8_matmul(a, sa, w, sw, None, M, N, K, BF16, y, st, ws, n)
    assert tw.twell_read_status(st) == 0
    for r in (slice(0, 300), slice(M - 300, M)):
        ref = (a[r].double() @ w.double().t()) * sa[r].double()[:, None] * sw.double()
        check(y[r], ref.cpu(), 3 * U * ref.abs().cpu(), "bf16", "y")


def test_distillation():
    T, V, k = 17000, 131073, 5
    z = rand(T, V)
    ids = torch.randint(0, V, (T, k), device="cuda", dtype=torch.int32)
    ids[-1, 0], ids[-1, 1] = V - 1, 0
    t = torch.randn(T, k, device="cuda")
    loss, stats = empty(T, dtype=torch.float32), empty(T, 2, dtype=torch.float32)
    dz, st = torch.empty_like(z), status()
    args = (T, V, k, BF16, 1.0)
    tw.twell_distill_forward(z, V, ids, t, None, *args, loss, stats, dz, st)
    for r in (slice(0, 2), slice(T - 3, T)):
        ref = distill_reference(z[r].cpu(), ids[r].cpu(), t[r].cpu(), None, 1.0, V)
        check(loss[r], ref[0], ref[3], "f32", "loss")
        check(dz[r], ref[2], ref[4], "bf16", "dz")
    again, loss2 = dz, empty(T, dtype=torch.float32)
    tw.twell_distill_forward(z, V, ids, t, None, *args, loss2, stats, None, st)
    assert torch.equal(loss, loss2)
    ones = torch.ones(T, device="cuda")
    tw.twell_distill_backward(z, V, ids, t, stats, ones, *args, z, st)     # in place
    assert tw.twell_read_status(st) == 0
    for r in (slice(0, 2), slice(T - 3, T)):
        assert ((z[r].float() - again[r].float()).abs() <= 2 ** -7 * again[r].float().abs() + 1e-9).all()
