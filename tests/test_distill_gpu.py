"""Distillation from a teacher's top logits against 64 bits.

Bounds, with u = 2^-24, x = (z - max z) / tau and n the additions behind a
row's sum of exponentials (a thread's V / 256 and 64 more): an exponential is
within 4 u (ex2) + 3 u (1 + 1.5 |x|) (its argument) of exact, the row's sum
within that of its largest terms and n u, so e_q = q u (16 + 6 |x| + n); p
alike over at most 256 entries.  dz: |w| tau (e_q + e_p) + 2 u of its terms.
loss: the same p, and logs within 4 u of the magnitudes they are formed from.
What is below 2^-126 in fp32 is flushed to zero."""
import math

import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import DT, U, check, empty, gen, setup, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


def inputs(T, V, k, dtype, seed, scale=3.0, ragged=False):
    g = gen(seed)
    z = (torch.randn(T, V, generator=g) * scale).to(DT[dtype][0])
    ids = torch.stack([torch.randperm(V, generator=g)[:k] for _ in range(T)]).int() if V < 5000 else \
        torch.randint(0, V, (T, k), generator=g).int()
    if ragged:
        n = torch.randint(0, k + 1, (T, 1), generator=g)
        ids = torch.where(torch.arange(k) < n, ids, -1).int()
    t = torch.randn(T, k, generator=g) * 3
    return z, ids, t, torch.rand(T, generator=g) + 0.1


def run(z, ids, t, w, tau, dtype, ldz=None, fused=True, in_place=False, fill=float("nan")):
    T, V = z.shape
    k = ids.shape[1]
    tdt, dt = DT[dtype]
    ldz = V if ldz is None else ldz
    zp = torch.full((T, ldz), fill, dtype=tdt, device="cuda")
    zp[:, :V] = z.cuda()
    dz = zp if in_place else torch.full((T, ldz), 7.0, dtype=tdt, device="cuda")
    ids, t = ids.cuda(), t.cuda()
    w = None if w is None else w.cuda()
    loss, stats, st = empty(T), empty(T, 2), status()
    tw.twell_distill_forward(zp, ldz, ids, t, w, T, V, k, dt, tau, loss, stats,
                             dz if fused else None, st)
    if not fused:
        tw.twell_distill_backward(zp, ldz, ids, t, stats,
                                  torch.ones(T, device="cuda") if w is None else w, T, V, k, dt, tau,
                                  dz, st)
    if not in_place:
        assert (dz[:, V:] == 7.0).all()  # the pitch's tail is not the operator's
    return loss, stats, dz[:, :V], tw.twell_read_status(st)


def reference(z, ids, t, w, tau, V):
    """(loss, stats, dz, bound of loss, bound of dz), row by row in 64 bits."""
    T, k = ids.shape
    w = torch.ones(T) if w is None else w
    tau = float(torch.tensor(tau, dtype=torch.float32))
    loss, stats = torch.zeros(T, dtype=torch.float64), torch.zeros(T, 2, dtype=torch.float64)
    dz = torch.zeros(T, V, dtype=torch.float64)
    eloss, edz = torch.zeros_like(loss), torch.zeros_like(dz)
    n = V / 256 + 64
    for r in range(T):
        wr = w[r].item()
        if wr == 0:
            continue
        zr = z[r].double()
        top = zr.max()
        x = (zr - top) / tau
        lnl = torch.log(torch.exp(x).sum())
        stats[r, 0], stats[r, 1] = top, lnl
        use = (ids[r] >= 0) & (ids[r] < V) & (t[r] != -math.inf)
        if not use.any():
            continue
        at = ids[r][use].long()
        tt = t[r][use].double() / tau
        p = torch.softmax(tt, 0)
        logp = torch.log_softmax(tt, 0)
        q = torch.exp(x - lnl)
        eq = q * U * (16 + 6 * torch.where(q > 0, x.abs(), 0.0) + n) + 2.0 ** -126
        ep = p * U * (320 + 6 * (tt - tt.max()).abs()) + 2.0 ** -126
        full = torch.zeros(V, dtype=torch.float64).index_add_(0, at, p)
        efull = torch.zeros(V, dtype=torch.float64).index_add_(0, at, ep)
        dz[r] = wr * tau * (q - full)
        edz[r] = abs(wr) * tau * (eq + efull + 2 * U * (q + full))
        diff = logp - (x[at] - lnl)
        keep = p > 0
        loss[r] = wr * tau * tau * (p * diff)[keep].sum()
        mag = logp.abs() + x[at].abs() + lnl.abs() + (tt - tt.max()).abs() + 1
        eloss[r] = abs(wr) * tau * tau * (ep * diff.abs() + p * mag * U * (16 + n))[keep].sum()
    return loss, stats, dz, eloss, edz


def verify(z, ids, t, w, tau, dtype, **kw):
    V = z.shape[1]
    ref = reference(z, ids, t, w, tau, V)
    n = V / 256 + 64
    for fused in (True, False):
        loss, stats, dz, code = run(z, ids, t, w, tau, dtype, fused=fused, **kw)
        check(loss, ref[0], ref[3], "f32", f"loss fused={fused}")
        check(stats[:, 0], ref[1][:, 0], torch.zeros(len(z), dtype=torch.float64), "f32", "max")
        check(stats[:, 1], ref[1][:, 1], U * (16 + n) * (1 + ref[1][:, 1].abs()), "f32", "log sum")
        check(dz, ref[2], ref[4], dtype, f"dz fused={fused}")
    return code


@pytest.mark.parametrize("T,V,k,dtype,tau", [
    (1, 1, 1, "bf16", 1.0), (3, 2, 2, "f32", 1.0), (64, 512, 8, "f32", 2.0),
    (5, 513, 256, "bf16", 1.0), (7, 1000, 17, "bf16", 0.7), (2, 4099, 33, "f32", 3.0),
    (1, 50001, 64, "bf16", 2.0), (9, 50001, 64, "bf16", 1.0), (1, 131072, 128, "bf16", 1.0),
    (3, 100003, 5, "f32", 2.0), (400, 9001, 3, "bf16", 1.0), (2, 900001, 20, "bf16", 1.0),
    (1, 450001, 20, "f32", 1.0)])
def test_against_64_bits(T, V, k, dtype, tau):
    z, ids, t, w = inputs(T, V, k, dtype, T * V + k)
    assert verify(z, ids, t, w, tau, dtype) == 0


def test_many_rows_share_an_sm():
    """Slices of one CTA a row at the size that lets two of them share an SM."""
    z, ids, t, w = inputs(330, 40007, 16, "bf16", 8)
    assert verify(z, ids, t, w, 1.0, "bf16") == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pitch_ragged_lists_and_masked_rows(dtype):
    """A padded vocabulary (NaN in the tail), lists cut short (some empty), rows of weight 0 whose
    logits are NaN: what is masked leaves no trace."""
    T, V = 61, 1003
    z, ids, t, w = inputs(T, V, 12, dtype, 3, ragged=True)
    ids[4] = -1
    w[::5] = 0
    z[::5] = float("nan")
    assert verify(z, ids, t, w, 1.5, dtype, ldz=1024) == 0
    assert verify(z, ids, t, w, 1.5, dtype, ldz=1009) == 0
    loss, stats, dz, _ = run(z, ids, t, w, 1.5, dtype)
    assert (dz[::5] == 0).all() and (loss[::5] == 0).all() and (stats[::5] == 0).all()
    assert (dz[4] == 0).all() and loss[4] == 0


@pytest.mark.parametrize("V,dtype", [(70003, "bf16"), (5003, "f32"), (3001, "f32"), (20011, "bf16")])
def test_a_cta_a_row(V, dtype):
    """Enough rows for a CTA each, in every width of that kernel: ragged lists, masked rows of NaN,
    and the gradient in place of the logits, the same bits as beside them."""
    z, ids, t, w = inputs(308, V, 9, dtype, V, ragged=True)
    w[::5] = 0
    z[::5] = float("nan")
    assert verify(z, ids, t, w, 1.5, dtype) == 0
    for fused in (True, False):
        a = run(z, ids, t, w, 1.5, dtype, fused=fused)
        b = run(z, ids, t, w, 1.5, dtype, fused=fused, in_place=True)
        for u, v in zip(a[:3], b[:3]):
            assert torch.equal(u, v)


@pytest.mark.parametrize("T,V", [(40, 777), (9, 40001), (1, 131075)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("fused", [True, False])
def test_in_place(dtype, fused, T, V):
    z, ids, t, w = inputs(T, V, 9, dtype, 6)
    a = run(z, ids, t, w, 1.0, dtype, fused=fused)
    b = run(z, ids, t, w, 1.0, dtype, fused=fused, in_place=True)
    for u, v in zip(a[:3], b[:3]):
        assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,rows", [(300, 8), (30011, 8), (6007, 312)])
def test_masked_logits(dtype, V, rows):
    """Vocabulary masked with -inf or with the type's lowest value, also in a row of nothing
    else; large logits; a teacher entry that the student excludes has infinite loss."""
    tdt = DT[dtype][0]
    z, ids, t, _ = inputs(rows, V, 6, dtype, 12)
    low = torch.finfo(tdt).min
    z[0, ::2] = -math.inf
    z[1, ::2] = low
    z[2] = low
    z[3] = z[3] * 1e4
    z[4] = 3e38
    z[5, 5:] = -math.inf
    z[5, 77] = -math.inf
    for r in (0, 1):  # keep the teacher on what is left
        ids[r] = ids[r] // 2 * 2 + 1
        ids[r][ids[r] >= V] = 1
    ids[5] = torch.tensor([0, 1, 2, 3, 4, 77])   # 77 is excluded
    t[6, 3] = -math.inf                            # the teacher excludes an entry
    assert verify(z, ids, t, None, 1.0, dtype) == 0
    loss = run(z, ids, t, None, 1.0, dtype)[0]
    assert loss[5] == math.inf


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("V", [400, 20011])
def test_bad_rows_stay_alone(bad, V):
    """A row with NaN or +inf has NaN outputs; the others are untouched."""
    z, ids, t, w = inputs(6, V, 5, "f32", 2)
    z[2, 31] = bad
    z[4] = -math.inf
    for fused in (True, False):
        loss, _, dz, code = run(z, ids, t, w, 1.0, "f32", fused=fused)
        assert code == 0
        for r in (2, 4):
            assert torch.isnan(loss[r]) and torch.isnan(dz[r]).all()
        ok = [0, 1, 3, 5]
        ref = reference(z[ok], ids[ok], t[ok], w[ok], 1.0, V)
        check(loss[ok], ref[0], ref[3], "f32", "loss")
        check(dz[ok], ref[2], ref[4], "f32", "dz")


def test_repeated_and_out_of_range_ids():
    z, ids, t, w = inputs(5, 200, 8, "f32", 21)
    ids[0, 3] = ids[0, 0]
    ids[0, 7] = ids[0, 0]
    ids[1] = 17
    assert verify(z, ids, t, w, 1.0, "f32") == 0
    ids[2, 1], ids[2, 2], ids[3] = 200, 1 << 30, 200
    assert verify(z, ids, t, w, 1.0, "f32") == -5


@pytest.mark.parametrize("T,V,k,dtype", [(9, 40, 256, "f32"), (7, 300, 256, "bf16"),
                                         (5, 3000, 130, "f32"), (310, 3000, 97, "bf16"),
                                         (6, 20000, 256, "bf16")])
def test_many_repeated_ids(T, V, k, dtype):
    """Lists in which most ids occur several times, in one group of 32 entries and across groups,
    one list of a single id, one of a single id but for unused entries."""
    z, _, t, w = inputs(T, V, k, dtype, T + V + k)
    g = gen(T * k)
    ids = torch.randint(0, min(V, k // 3), (T, k), generator=g).int()
    ids[1] = V - 1
    ids[2] = torch.where(torch.arange(k) % 3 == 1, 5, -1).int()
    assert verify(z, ids, t, w, 1.3, dtype) == 0


def test_gradient_against_differences():
    """Central differences of the summed loss in 64 bits, step h: the third derivative of the loss
    is below w tau^2 / tau^3, its h^2 / 6 below 1e-9; and the kernel's fp32 bound."""
    T, V, tau, h = 4, 37, 1.5, 1e-4
    z, ids, t, w = inputs(T, V, 5, "f32", 33)
    dz = run(z, ids, t, w, tau, "f32")[2].double().cpu()
    edz = reference(z, ids, t, w, tau, V)[4]
    for r in range(T):
        for v in range(V):
            zz = z.double().clone()
            zz[r, v] += h
            up = reference(zz, ids, t, w, tau, V)[0].sum()
            zz[r, v] -= 2 * h
            down = reference(zz, ids, t, w, tau, V)[0].sum()
            assert abs(dz[r, v] - (up - down) / (2 * h)) <= 1e-8 + edz[r, v]


def test_other_stream_and_graph():
    z, ids, t, w = inputs(33, 3001, 20, "bf16", 4)
    want = run(z, ids, t, w, 1.0, "bf16")
    z, ids, t, w = z.cuda(), ids.cuda(), t.cuda(), w.cuda()
    loss, stats, dz, st = empty(33), empty(33, 2), torch.empty_like(z), status()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tw.twell_distill_forward(z, 3001, ids, t, w, 33, 3001, 20, tw.TWELL_BF16, 1.0, loss, stats,
                                 dz, st)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip((loss, stats, dz), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("V,dtype", [(97, "f32"), (4200, "bf16")])
def test_one_id_twice_in_any_two_places(V, dtype):
    """A row for every two of 66 places: the id at both has one sum, kept at the first."""
    k = 66
    first, second = torch.triu_indices(k, k, offset=1)
    T = len(first)
    z, _, t, w = inputs(T, V, k, dtype, V)
    ids = torch.arange(k, dtype=torch.int32).repeat(T, 1)
    ids[torch.arange(T), second] = first.int()
    assert verify(z, ids, t, w, 1.0, dtype) == 0
    a = run(z, ids, t, w, 1.0, dtype)
    for _ in range(20):
        for u, v in zip(run(z, ids, t, w, 1.0, dtype)[:3], a):
            assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("V,rows", [(300, 12), (30011, 12), (6007, 312), (90001, 312)])
@pytest.mark.parametrize("tau", [1.0, 0.5, 1e-3])
def test_logits_of_any_size(dtype, V, rows, tau):
    """Rows of one huge value of either sign (a mask and nothing else), rows of values that differ by
    their last place there, huge values beside ordinary ones, and steps across the size from which
    differences are taken first."""
    z, ids, t, _ = inputs(rows, V, 6, dtype, V)
    big = [1e6, 1.2e7, -1e9, 2.5e9, -1e10, 1e14, -1e20, 1e30]
    for r, b in enumerate(big):
        z[r] = b * tau
    near = torch.tensor(2.0 ** 24 / 1.4426950408889634 * tau)
    z[8] = near * (1 + (torch.arange(V) % 9 - 4) * 2.0 ** (-23 if dtype == "f32" else -7))
    z[9] = -near * (1 + (torch.arange(V) % 9 - 4) * 2.0 ** (-23 if dtype == "f32" else -7))
    z[10, ::3] = -1e9
    z[11, ::3] = 1e9
    for r in range(12):   # a teacher on what the student does not exclude: the row's largest
        top = torch.nonzero(z[r] == z[r].max())[:, 0]
        ids[r] = top[torch.arange(6) % len(top)].int()
    assert verify(z, ids, t, None, tau, dtype) == 0


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("T,V,ldz", [(9, 40001, 40001), (61, 20011, 20016), (300, 9001, 9001)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_rows_of_long_rows(dtype, T, V, ldz, fused):
    """Masked rows between others where a cluster has a row, in place too: zeros, whatever stood
    there, and the others have the bits that they have beside rows that count."""
    z, ids, t, w = inputs(T, V, 9, dtype, T)
    rest = torch.arange(T) % 3 != 1
    want = [a[rest] for a in run(z, ids, t, w, 1.0, dtype, ldz=ldz, fused=fused)[:3]]
    z[~rest] = float("nan")
    w[~rest] = 0
    for in_place in (False, True):
        got = run(z, ids, t, w, 1.0, dtype, ldz=ldz, fused=fused, in_place=in_place)
        for a, b in zip(got[:3], want):
            assert (a[~rest] == 0).all() and torch.equal(a[rest], b)
    w[:] = 0
    got = run(z, ids, t, w, 1.0, dtype, ldz=ldz, fused=fused)
    assert all((a == 0).all() for a in got[:3])
