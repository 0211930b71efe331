"""The recurrence where gates close behind large states: what has been forgotten leaves nothing.

Bounds for |got - exact|, with u = 2^-24: the smaller one of a and c = 1 - a, w, is within
k u of itself, k = 2 (|gate| + |bias|) + 8 (the gate's logarithm is rounded twice, its
exponential is off by 4 u, the sum and its reciprocal by 3 u).  With the decaying sum of
magnitudes S_t = a_t S_{t-1} + c_t |x_t| (S_0 = |h0|), as w is at most a and at most c, a row
adds
    w k u |h - x| <= k u (a |h| + c |x|) <= k u S_t
for its gate.  While a >= 2^-6 (to a rounding of the exponential) a row is taken by c alone, which
the sum and its reciprocal leave off by 3 u: j u a |h| more with j = min(3 / a, 195).  Every sum on the way to the state is of terms within S_t.  A row's own
difference and step are 2 of them and what it leaves of the product of the shares is 1; behind
a row where pieces meet, at most 5 more joints add 2 for the state and 2 for the shares:
    E_t = a_t E_{t-1} + (k + j + 24) u S_t.
No term holds what the sequence was before it was forgotten.  Backward in the same way,
Q_t = |dh_t| + a_{t+1} Q_{t+1}:
    F_t = W_{t+1} + 2 u Q_t,   W_t = a_t F_t + (k + j + 24) u a_t Q_t     (of G and of a G)
    dx:    c F + (k + 2) u c Q
    dgate: a c (|h_{t-1} - x| F + Q (E_{t-1} + u |h_{t-1} - x|)) + (2 k + 8) u a c Q |h_{t-1} - x|
    dbias: the sum of dgate's, and (T + 64) u sum |dgate|;  dh0: W at the first row."""
import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import DT, U, check, empty, gen, setup, status
from test_recur_gpu import Case, ragged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


class Reset(Case):
    """Small inputs and gradients with few huge ones among them, gates that close or stay open."""

    def __init__(self, T, D, starts, dtype, seed=0):
        super().__init__(T, D, starts, dtype, seed=seed)
        g, tdt = gen(seed + 7), DT[dtype][0]
        rand = lambda: torch.rand(T, D, generator=g)  # noqa: E731
        huge = lambda: torch.where(rand() < 1 / 64, 1e4, 1e-4)  # noqa: E731
        self.x, self.dh = (self.x.float() * huge()).to(tdt), (self.dh.float() * huge()).to(tdt)
        self.h0, self.dhT = 1e4 * self.h0, 1e4 * self.dhT
        end = 8 + 40 * rand()
        which = rand()
        gate = torch.where(which < 1 / 16, -end, torch.where(which < 2 / 16, end, self.gate.float()))
        self.gate = gate.to(tdt)

    def reference(self):
        T, D, B = self.T, self.D, self.B
        x, bias = self.x.double(), self.bias.double() if self.bias is not None else torch.zeros(D).double()
        f = self.gate.double() + bias
        a, c = torch.sigmoid(f), torch.sigmoid(-f)
        k = 2 * (self.gate.double().abs() + bias.abs()) + 8
        kj = k + (3 / a).clamp_max(195)
        zero = torch.zeros(D, dtype=torch.float64)
        new = lambda *s: torch.full(s, float("nan"), dtype=torch.float64)  # noqa: E731
        out = {n: (new(T, D), new(T, D)) for n in ("h", "dx", "dgate")}
        out |= {n: (new(B, D), new(B, D)) for n in ("hT", "dh0")}
        db, dbe, dbm = zero.clone(), zero.clone(), zero.clone()
        for s in range(B):
            lo, hi = self.bounds[s], self.bounds[s + 1]
            h = self.h0[s].double()
            S, E, before = h.abs(), zero, []
            for t in range(lo, hi):
                before.append((h, E))
                h, S = a[t] * h + c[t] * x[t], a[t] * S + c[t] * x[t].abs()
                E = a[t] * E + (kj[t] + 24) * U * S
                out["h"][0][t], out["h"][1][t] = h, E
            out["hT"][0][s], out["hT"][1][s] = h, E
            v = self.dhT[s].double()
            q, W = v.abs(), zero
            for t in range(hi - 1, lo - 1, -1):
                G, Q = self.dh[t].double() + v, self.dh[t].double().abs() + q
                F = W + 2 * U * Q
                hp, Ep = before[t - lo]
                off, ac = (hp - x[t]).abs(), a[t] * c[t]
                out["dx"][0][t], out["dx"][1][t] = c[t] * G, c[t] * F + (k[t] + 2) * U * c[t] * Q
                dg = G * (hp - x[t]) * ac
                e = ac * (off * F + Q * (Ep + U * off)) + (2 * k[t] + 8) * U * ac * Q * off
                out["dgate"][0][t], out["dgate"][1][t] = dg, e
                db, dbe, dbm = db + dg, dbe + e, dbm + dg.abs()
                v, q, W = a[t] * G, a[t] * Q, a[t] * F + (kj[t] + 24) * U * a[t] * Q
            out["dh0"][0][s], out["dh0"][1][s] = v, W
        out["dbias"] = (db, dbe + (T + 64) * U * dbm)
        return out


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,starts", [
    (1, 16, [0, 1]), (5, 24, [0, 2, 5]), (64, 128, [0, 1, 1, 40, 64]), (129, 520, [3, 66, 128]),
    (300, 2048, [0, 64, 128, 290]), (1031, 72, ragged(1031, 200, 2)), (2049, 256, [0, 2049]),
    (640, 40, 4), (37, 64, 37), (4309, 264, ragged(4309, 9, 4)), (4261, 1544, [1, 2000, 4260]),
    (700, 2504, ragged(700, 40, 6)), (4205, 2504, [0, 1500, 4203])])
def test_closed_gates(T, D, starts, dtype):
    c = Reset(T, D, starts, dtype)
    c.compare(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 7, 300, 5000])
def test_a_large_state_is_forgotten(T, dtype):
    """The first gate is closed but for 1e-13: a state of 1e4 leaves 1e-9, not its rounding; and
    the last gradient, of 1e4, reaches the rows before a closed gate as little."""
    D, tdt, dt = 16, *DT[dtype]
    x = torch.full((T, D), 2.0 ** -13, device="cuda", dtype=tdt)
    gate = torch.zeros(T, D, device="cuda", dtype=tdt)
    gate[0] = -30.0
    gate[-1] = -30.0
    h0 = torch.full((1, D), 1e4, device="cuda")
    h, hT, kept, st = empty(T, D, dtype=tdt), empty(1, D), empty(tw.twell_recur_states(T), D), status()
    tw.twell_recur_forward(x, gate, D, None, None, 1, h0, T, D, dt, h, hT, kept, st) if T > 1 else \
        tw.twell_recur_forward(x, gate, D, None, torch.tensor([0, 1], dtype=torch.int32, device="cuda"),
                               1, h0, T, D, dt, h, hT, kept, st)
    # every h is a mean of equal inputs beside 1e4 e^-30 of the state; a = 1/2 doubles a row's 38 u
    left = 1e4 * 9.4e-14
    check(h, torch.full((T, D), 2.0 ** -13).double(), torch.tensor(left + 76 * U * 2.0 ** -13), dtype, "h")
    dh = torch.zeros(T, D, device="cuda", dtype=tdt)
    dhT = torch.full((1, D), 1e4, device="cuda")
    dx, dg, dh0 = empty(T, D, dtype=tdt), empty(T, D, dtype=tdt), empty(1, D)
    tw.twell_recur_backward(x, gate, D, None, None if T > 1 else
                            torch.tensor([0, 1], dtype=torch.int32, device="cuda"), 1, h0, kept, dh, dhT,
                            T, D, dt, dx, dg, None, dh0, st)
    assert (dx[-1].float() == torch.tensor(1e4).to(tdt).float()).all()
    assert (dx[:-1].float().abs() <= left).all() and (dh0.abs() <= left).all()
    assert tw.twell_read_status(st) == 0


def test_long_memory_beside_closed_gates():
    """Channels that take 2^-12 to 2^-20 of each input for thousands of rows are off by the same
    few roundings: neither share is lost where the other one is near 1."""
    T, D = 6000, 64
    c = Reset(T, D, [0, T], "f32")
    c.x, c.dh = torch.randn(T, D, generator=gen(1)), torch.randn(T, D, generator=gen(2))
    c.h0, c.dhT = 1e-4 * c.h0, 1e-4 * c.dhT
    c.gate = torch.linspace(8.3, 13.9, D).expand(T, D).contiguous()
    c.gate[3000, ::2] = -25.0
    c.bias = None
    got, ref = c.run(), c.reference()
    c.compare(got)
    # and far below the bound, which counts every rounding in full: a systematic error would
    # stand at 2^-25 of the state for each of the rows that it remembers
    off = (got["h"].cpu().double() - ref["h"][0]).abs().amax(0)
    size = ref["h"][0].abs().amax(0)
    assert (off <= 256 * U * size).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,starts", [(700, 72, [0, 100, 133, 400, 700]), (3000, 2504, [0, 1003, 3000]),
                                        (5000, 1544, ragged(5000, 12, 3)), (200, 16, 4)])
def test_a_closed_gate_changes_no_other_sequence(T, D, starts, dtype):
    """The bits of a sequence, and of a channel, are the same whatever gates stand beside it."""
    c = Case(T, D, starts, dtype)
    c.gate = c.gate.clamp_min(-2.0)  # (with the bias, from -1.3 on: open)
    want = c.run()
    s = 1
    lo, hi = c.bounds[s], c.bounds[s + 1]
    c.gate[lo:hi:5, ::3] = -20.0
    got = c.run()
    rows = torch.ones(T, dtype=torch.bool)
    rows[lo:hi] = False
    channels = torch.arange(D) % 3 != 0
    other = torch.arange(c.B) != s
    for n in ("h", "dx", "dgate"):
        v, w = (torch.nan_to_num(t[n].cpu()) for t in (got, want))
        assert torch.equal(v[rows], w[rows]) and torch.equal(v[:, channels], w[:, channels]), n
        assert hi == lo or not torch.equal(v[lo:hi], w[lo:hi])
    for n in ("hT", "dh0"):
        v, w = got[n].cpu(), want[n].cpu()
        assert torch.equal(v[other], w[other]) and torch.equal(v[:, channels], w[:, channels]), n


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("T,D,starts", [(300, 72, [0, 100, 290]), (5000, 1544, [0, 777, 4100, 5000]),
                                        (700, 16, [0, 350, 700])])
def test_infinities_reach_what_depends_on_them(T, D, starts, bad, dtype):
    """x: the states from its row on, and their gates' gradients; dh: G up to its row.  The rest has
    the bits that it has without."""
    s = 1
    lo, hi = starts[s], starts[s + 1]
    at = (lo + hi) // 2
    rows = torch.arange(T)
    c = Case(T, D, starts, dtype)
    want = {n: v.cpu() for n, v in c.run().items()}

    def compare(got, reached):
        for n, r in reached.items():
            r = r[:len(got[n])]
            v, w = got[n].cpu(), want[n]
            assert not v[r].isfinite().any(), n
            assert torch.equal(torch.nan_to_num(v[~r]), torch.nan_to_num(w[~r])), n

    nothing, mine = rows < 0, torch.arange(len(starts) - 1) == s
    after, upto = (rows >= at) & (rows < hi), (rows >= lo) & (rows <= at)
    whole, none = c.x.clone(), torch.zeros_like(mine)
    c.x[at] = bad
    compare(c.run(), {"h": after, "hT": mine, "dx": nothing, "dgate": after, "dh0": none})
    c.x = whole
    c.dh[at] = bad
    compare(c.run(), {"h": nothing, "hT": none, "dx": upto, "dgate": upto, "dh0": mine})
