"""Residual addition + RMS norm (output in the row's type or in 8 bits) and
its backward against 64 bits.

Bounds, with u = 2^-24.  s: the fp32 sum rounded once, bit-exact.  The sum of
squares is at most 32 additions in a lane, 5 shuffles and 8 warps deep, so
rstd is within (45 / 2 + 4) u of exact and y (two products more) within 32 u,
before its rounding.  q: |q - y / scale| <= 1/2 plus 127 times the relative
errors of y and scale (2 * 64 u).  dx: 64 u of the magnitudes of its terms.
dw: (T + 64) u sum |dy xhat|."""
import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import DT, U, check, empty, gen, scratch, setup

pytestmark = pytest.mark.gpu
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


def forward(x, res, w, dtype, eps=EPS, want="yqr", in_place=False):
    T, D = x.shape
    tdt, dt = DT[dtype]
    x, w = x.cuda(), w.cuda()
    res = None if res is None else res.cuda()
    s = (res if res is not None else x) if in_place else empty(T, D, dtype=tdt)
    y = empty(T, D, dtype=tdt) if "y" in want else None
    q = empty(T, D, dtype=torch.int8) if "q" in want else None
    qs = empty(T) if "q" in want else None
    r = empty(T) if "r" in want else None
    tw.twell_add_rmsnorm_forward(x, res, w, T, D, dt, eps, s, y, q, qs, r)
    return s, y, q, qs, r


def backward(s, w, rstd, dy, ds, dtype, in_place=False):
    T, D = s.shape
    dt = DT[dtype][1]
    s, w, rstd, dy = s.cuda(), w.cuda(), rstd.cuda(), dy.cuda()
    ds = None if ds is None else ds.cuda()
    dx = ds if in_place else empty(T, D, dtype=DT[dtype][0])
    dw = empty(D)
    ws, n = scratch(tw.twell_add_rmsnorm_workspace_size(T, D))
    tw.twell_add_rmsnorm_backward(s, w, rstd, dy, ds, T, D, dt, dx, dw, ws, n)
    return dx, dw


def ref_norm(s, w, eps=EPS):
    s, w = s.double(), w.double()
    rstd = 1.0 / torch.sqrt((s * s).mean(1, keepdim=True) + eps)
    return rstd, s * rstd * w


SHAPES = [(1, 16), (3, 16), (1, 2048), (64, 128), (37, 4096), (5, 272), (2000, 528), (513, 2048),
          (9, 1040), (301, 4080)]


@pytest.mark.parametrize("T,D", SHAPES + [(4, 8192), (70, 6000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_forward(T, D, dtype):
    if dtype == "f32" and D > 4096:
        pytest.skip("beyond 16 KB a row")
    g = gen(T * D)
    tdt = DT[dtype][0]
    scale = torch.exp(torch.randn(T, 1, generator=g))
    x, res = (torch.randn(T, D, generator=g) * scale).to(tdt), torch.randn(T, D, generator=g).to(tdt)
    w = 1 + 0.2 * torch.randn(D, generator=g)
    s, y, q, qs, r = forward(x, res, w, dtype)
    want = (x.float() + res.float()).to(tdt)
    assert torch.equal(s.cpu(), want)
    rstd, yr = ref_norm(want, w)
    check(r, rstd[:, 0], 32 * U * rstd[:, 0], "f32", "rstd")
    check(y, yr, 32 * U * yr.abs(), dtype, "y")
    top = yr.abs().amax(1)
    check(qs, top / 127, 64 * U * top / 127, "f32", "qscale")
    off = (q.double().cpu() - yr * 127 / top[:, None]).abs().max().item()
    assert off <= 0.5 + 127 * 128 * U, off
    assert q.abs().amax(1).min().item() == 127 and q.min().item() >= -127
    # outputs by themselves, without a residual, and in place
    _, y1, _, _, r1 = forward(x, res, w, dtype, want="yr")
    _, _, q1, qs1, _ = forward(x, res, w, dtype, want="q")
    s2, y2, _, _, _ = forward(x, res, w, dtype, want="y", in_place=True)
    assert torch.equal(y1, y) and torch.equal(r1, r) and torch.equal(q1, q)
    assert torch.equal(qs1, qs) and torch.equal(y2, y) and torch.equal(s2, s)
    s3, y3, _, _, _ = forward(want, None, w, dtype)
    assert torch.equal(y3, y) and torch.equal(s3, s)


@pytest.mark.parametrize("T,D", [(2, 8), (11, 1032)])
def test_forward_width_not_a_multiple_of_16(T, D):
    """The output in the row's type takes any row of whole 16-byte vectors."""
    g = gen(D)
    x = torch.randn(T, D, generator=g)
    w = torch.ones(D)
    for dtype in ("bf16", "f32"):
        xd = x.to(DT[dtype][0])
        _, y, _, _, _ = forward(xd, None, w, dtype, want="y")
        _, yr = ref_norm(xd, w)
        check(y, yr, 32 * U * yr.abs(), dtype, "y")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_at_the_edges(dtype):
    """Zero rows, tiny and huge rows, and rows with infinities or NaN; no row disturbs another."""
    tdt = DT[dtype][0]
    D = 256
    x = torch.randn(9, D, generator=gen(1))
    x[1] = 0
    x[2] *= 1e-30
    x[3] *= 1e15
    x[4, 17] = float("inf")
    x[5, 200] = float("nan")
    x[6] = 0
    x[6, 3] = 1e-38
    x[7, 0] = -float("inf")
    x = x.to(tdt)
    w = 1 + 0.2 * torch.randn(D, generator=gen(2))
    for eps in (EPS, 0.0):
        _, y, q, qs, _ = forward(x, None, w, dtype, eps=eps)
        ok = [0, 3, 8] + ([1, 2, 6] if eps else [])  # (eps 0: their squares underflow, 0 * inf)
        _, yr = ref_norm(x, w, eps)
        check(y[ok], yr[ok], 32 * U * yr[ok].abs(), dtype, "y")
        top = yr[ok].abs().amax(1)
        check(qs[ok], top / 127, 64 * U * top / 127 + 2.0 ** -149, "f32", "qscale")
        for i, t in zip(ok, top):
            if t > 0:
                off = (q[i].double().cpu() - yr[i] * 127 / t).abs().max().item()
                assert off <= 0.5 + 127 * 128 * U, (i, off)
            else:
                assert (q[i] == 0).all() and qs[i] == 0
        for i in (4, 5, 7):
            assert torch.isnan(qs[i]) and (q[i] == 0).all()


@pytest.mark.parametrize("T,D", SHAPES + [(4, 8192), (70, 6000)])
@pytest.mark.parametrize("dtype,with_ds", [("bf16", True), ("bf16", False), ("f32", True)])
def test_backward(T, D, dtype, with_ds):
    if dtype == "f32" and D > 4096:
        pytest.skip("beyond 16 KB a row")
    g = gen(T + D)
    tdt = DT[dtype][0]
    s, dy = torch.randn(T, D, generator=g).to(tdt), torch.randn(T, D, generator=g).to(tdt)
    ds = torch.randn(T, D, generator=g).to(tdt) if with_ds else None
    w = 1 + 0.2 * torch.randn(D, generator=g)
    rstd = ref_norm(s, w)[0][:, 0].float()
    dx, dw = backward(s, w, rstd, dy, ds, dtype)
    r, x64, g64 = rstd.double()[:, None], s.double(), dy.double()
    hat, wg = x64 * r, g64 * w.double()
    d0 = ds.double() if with_ds else torch.zeros_like(x64)
    mean = (wg * hat).mean(1, keepdim=True)
    ref = d0 + r * (wg - hat * mean)
    mag = d0.abs() + r * (wg.abs() + hat.abs() * (wg * hat).abs().mean(1, keepdim=True))
    check(dx, ref, 64 * U * mag, dtype, "dx")
    check(dw, (g64 * hat).sum(0), (T + 64) * U * (g64 * hat).abs().sum(0), "f32", "dw")
    dx2, dw2 = backward(s, w, rstd, dy, ds, dtype, in_place=with_ds)
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_gradients_against_differences():
    """Central differences of L = <y, dy> + <s, ds> in 64 bits, step h: error h^2 times the third
    derivative (bounded here by 1e2 in these units) and the kernels' fp32 bound."""
    T, D, h = 5, 64, 1e-4
    g = gen(4)
    s, dy, ds = (torch.randn(T, D, generator=g) for _ in range(3))
    w = 1 + 0.2 * torch.randn(D, generator=g)
    rstd = forward(s, None, w, "f32", want="yr")[4]
    dx, dw = backward(s, w, rstd, dy, ds, "f32")

    def loss(s64, w64):
        return (ref_norm(s64, w64)[1] * dy.double()).sum() + (s64 * ds.double()).sum()

    for name, got, at in (("dx", dx, 0), ("dw", dw, 1)):
        arg = [s.double(), w.double()]
        flat = arg[at].reshape(-1)
        for i in range(0, flat.numel(), 7):
            keep = flat[i].item()
            flat[i] = keep + h
            up = loss(*arg)
            flat[i] = keep - h
            down = loss(*arg)
            flat[i] = keep
            want = ((up - down) / (2 * h)).item()
            assert abs(got.reshape(-1)[i].item() - want) <= 100 * h * h + 2e-5, (name, i)


@pytest.mark.parametrize("rows,cols", [(1, 16), (300, 2048), (7, 20000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize(rows, cols, dtype):
    g = gen(rows)
    a = (torch.randn(rows, cols, generator=g)).to(DT[dtype][0])
    if rows > 5:
        a[1], a[2, 5], a[3, 7] = 0, float("nan"), float("inf")
        a[4] *= 1e-32
    q, sc = empty(rows, cols, dtype=torch.int8), empty(rows)
    tw.twell_q8_quantize(a.cuda(), rows, cols, DT[dtype][1], q, sc)
    top = a.double().abs().amax(1)
    for i in range(rows):
        if not torch.isfinite(top[i]):
            assert torch.isnan(sc[i]) and (q[i] == 0).all()
        elif top[i] == 0:
            assert sc[i] == 0 and (q[i] == 0).all()
        else:
            # one division, and a division and two products: 4 u of at most 127
            assert abs(sc[i].item() - top[i].item() / 127) <= 2 * U * top[i].item() / 127 + 2.0 ** -149
            off = (q[i].double().cpu() - a[i].double() * 127 / top[i]).abs().max().item()
            assert off <= 0.5 + 127 * 4 * U, (i, off)


@pytest.mark.parametrize("D", [64, 2048, 4096])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_that_leave_the_range(dtype, D):
    """Zeros and values whose squares vanish, with eps 0, and values whose squares overflow: rstd, y,
    q and qscale are 0, the gradient is what reaches the sum past the norm, and the row leaves no
    trace in the weight's gradient; the rows beside them are as ever."""
    tdt = DT[dtype][0]
    x = torch.randn(7, D, generator=gen(D))
    x[1] = 0
    x[2] *= 1e-30
    x[3] = 0
    x[3, 3] = 1e-38
    x[4] = 2e19                    # (squares beyond fp32)
    x[6] = -0.0
    x = x.to(tdt)
    w = 1 + 0.2 * torch.randn(D, generator=gen(2))
    gone, ok = [1, 2, 3, 4, 6], [0, 5]
    s, y, q, qs, r = forward(x, None, w, dtype, eps=0.0)
    for v in (y, q, qs, r):
        assert (v[gone] == 0).all()
    rstd, yr = ref_norm(x, w, 0.0)
    check(y[ok], yr[ok], 32 * U * yr[ok].abs(), dtype, "y")
    check(r[ok], rstd[ok][:, 0], 32 * U * rstd[ok][:, 0], "f32", "rstd")
    dy, ds = torch.randn(7, D, generator=gen(3)).to(tdt), torch.randn(7, D, generator=gen(4)).to(tdt)
    dx, dw = backward(s, w, r, dy, ds, dtype)
    assert torch.equal(dx.cpu()[gone], ds[gone])
    # (dw: the sums of the two rows, in whatever order the zeros are added)
    hat = x[ok].double() * r.double().cpu()[ok][:, None]
    check(dw, (dy[ok].double() * hat).sum(0), (7 + 64) * U * (dy[ok].double() * hat).abs().sum(0),
          "f32", "dw")
    # with eps, zeros are zeros and the small rows count
    _, y, q, qs, r = forward(x, None, w, dtype)
    rstd, yr = ref_norm(x, w)
    some = [0, 1, 2, 3, 5, 6]
    check(y[some], yr[some], 32 * U * yr[some].abs(), dtype, "y")
    assert (y[4] == 0).all() and qs[4] == 0 and qs[1] == 0 and (q[1] == 0).all()
