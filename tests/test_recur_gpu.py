"""Gated linear recurrence over packed sequences and its backward against 64 bits.

Bounds, with u = 2^-24 and f = gate + bias.  f is rounded once and its
exponential is off by (|f| + 6) u, so a and c = 1 - a are each within
k = (2 |f| + 8) u of themselves.  Every value of the state is a mean of inputs,
at most M (the sequence's largest |x| and |h0| so far): a row adds k c 2 M for its
gate and less than 16 roundings of u M, those of the joints of a scan in pieces
among them, and passes on a times what the row before was off:
    E_t = a_t E_{t-1} + 2 k c M + 16 u M.
Backward in the same way with the sum of magnitudes Q_t = |dh_t| + a_{t+1} Q_{t+1}:
    F_t = a_{t+1} F_{t+1} + (k c + 16 u) Q_t,
    dx:    c F + (k + 2 u) c Q
    dgate: a c (|h_{t-1} - x| F + Q (E_{t-1} + 2 u M)) + (2 k + 6 u) a c Q |h_{t-1} - x|
    dbias: the sum of dgate's, and T u sum |dgate|."""
import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import DT, U, check, empty, gen, setup, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


class Case:
    """Inputs of one call on the host, in their stored type."""

    def __init__(self, T, D, starts, dtype, state=True, bias=True, seed=0, fused=True):
        g = gen(seed + T * 131 + D)
        tdt = DT[dtype][0]
        self.T, self.D, self.dtype, self.starts = T, D, dtype, starts
        self.B = len(starts) - 1 if isinstance(starts, list) else starts
        self.bounds = starts if isinstance(starts, list) else [i * (T // starts) for i in range(starts + 1)]
        self.fused = fused
        self.x, self.gate = torch.randn(T, D, generator=g).to(tdt), torch.randn(T, D, generator=g).to(tdt)
        self.bias = torch.linspace(-1, 5, D) + 0.1 * torch.randn(D, generator=g) if bias else None
        self.h0 = torch.randn(self.B, D, generator=g) if state else None
        self.dh = torch.randn(T, D, generator=g).to(tdt)
        self.dhT = torch.randn(self.B, D, generator=g) if state else None
        self.state = state

    def run(self, backward=True, stream=None):
        """(h, hT, dx, dgate, dbias, dh0) as the GPU has them; outputs start as NaN."""
        T, D, B = self.T, self.D, self.B
        tdt, dt = DT[self.dtype]
        dev = lambda v: None if v is None else v.cuda()  # noqa: E731
        ld = 2 * D if self.fused else D
        if self.fused:
            xg, dxg = torch.cat([self.x, self.gate], 1).cuda(), empty(T, 2 * D, dtype=tdt)
            x, gate, dx, dgate = xg[:, :D], xg[:, D:], dxg[:, :D], dxg[:, D:]
        else:
            x, gate, dx, dgate = self.x.cuda(), self.gate.cuda(), empty(T, D, dtype=tdt), empty(T, D, dtype=tdt)
        starts = torch.tensor(self.starts, dtype=torch.int32).cuda() if isinstance(self.starts, list) else None
        h, hT, kept, st = empty(T, D, dtype=tdt), empty(B, D), empty(tw.twell_recur_states(T), D), status()
        bias, h0, dh, dhT = dev(self.bias), dev(self.h0), dev(self.dh), dev(self.dhT)
        torch.cuda.synchronize()
        tw.twell_recur_forward(x, gate, ld, bias, starts, B, h0, T, D, dt, h, hT, kept, st, stream)
        out = {"h": h, "hT": hT}
        if backward:
            dbias, dh0 = empty(D), empty(B, D)
            tw.twell_recur_backward(x, gate, ld, bias, starts, B, h0, kept, dh, dhT, T, D, dt, dx,
                                    dgate, dbias, dh0, st, stream)
            out |= {"dx": dx, "dgate": dgate, "dbias": dbias, "dh0": dh0}
        torch.cuda.synchronize()
        assert tw.twell_read_status(st) == 0
        return out

    def reference(self):
        """{name: (value, bound)} in 64 bits; rows outside the sequences are NaN."""
        T, D, B = self.T, self.D, self.B
        x, f = self.x.double(), self.gate.double()
        if self.bias is not None:
            f = f + self.bias.double()
        a, c = torch.sigmoid(f), torch.sigmoid(-f)
        k = (2 * f.abs() + 8) * U
        zero = torch.zeros(D, dtype=torch.float64)
        new = lambda *s: torch.full(s, float("nan"), dtype=torch.float64)  # noqa: E731
        out = {n: (new(T, D), new(T, D)) for n in ("h", "dx", "dgate")}
        out |= {n: (new(B, D), new(B, D)) for n in ("hT", "dh0")}
        db, dbe, dbm = zero.clone(), zero.clone(), zero.clone()
        for s in range(B):
            lo, hi = self.bounds[s], self.bounds[s + 1]
            h = self.h0[s].double() if self.state else zero
            M, E = h.abs(), zero
            before = []
            for t in range(lo, hi):
                M = torch.maximum(M, x[t].abs())
                before.append((h, E, M))
                h = a[t] * h + c[t] * x[t]
                E = a[t] * E + 2 * k[t] * c[t] * M + 16 * U * M
                out["h"][0][t], out["h"][1][t] = h, E
            out["hT"][0][s], out["hT"][1][s] = h, E
            u = self.dhT[s].double() if self.state else zero
            q, w = u.abs(), zero
            for t in range(hi - 1, lo - 1, -1):
                G, Q = self.dh[t].double() + u, self.dh[t].double().abs() + q
                F = w + (k[t] * c[t] + 16 * U) * Q
                hp, Ep, M = before[t - lo]
                off, ac = hp - x[t], a[t] * c[t]
                out["dx"][0][t], out["dx"][1][t] = c[t] * G, c[t] * F + (k[t] + 2 * U) * c[t] * Q
                dg = G * off * ac
                e = ac * (off.abs() * F + Q * (Ep + 2 * U * M)) + (2 * k[t] + 6 * U) * ac * Q * off.abs()
                out["dgate"][0][t], out["dgate"][1][t] = dg, e
                db, dbe, dbm = db + dg, dbe + e, dbm + dg.abs()
                u, q, w = a[t] * G, a[t] * Q, a[t] * F + k[t] * Q
            out["dh0"][0][s], out["dh0"][1][s] = u, w
        out["dbias"] = (db, dbe + (T + 64) * U * dbm)
        return out

    def compare(self, got):
        ref = self.reference()
        for n, v in got.items():
            value, bound = ref[n]
            kind = self.dtype if n in ("h", "dx", "dgate") else "f32"
            # (rows outside the sequences are as they were: NaN on both sides)
            check(v, value, torch.nan_to_num(bound), kind, n)


def ragged(T, B, seed):
    """Sequences of any length, some of them empty, before the end of the buffer."""
    g = gen(seed)
    cuts = sorted(int(v) for v in torch.randint(0, T + 1, (B - 1,), generator=g))
    return [0] + cuts + [T]


SHAPES = [(1, 8, [0, 1]), (2, 16, [0, 1, 2]), (3, 72, [0, 3]), (63, 16, [0, 63]),
          (64, 128, [0, 1, 1, 1, 40, 64]), (65, 24, [0, 64, 65]), (127, 64, [0, 127]),
          (129, 520, [3, 66, 128]), (200, 64, [5, 5, 190, 190]), (300, 2048, [0, 64, 128, 290]),
          (1000, 136, ragged(1000, 17, 1)), (1031, 8, ragged(1031, 500, 2)),
          (2049, 256, [0, 2049]), (4100, 72, [0, 4099, 4100])]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,starts", SHAPES)
def test_packed(T, D, starts, dtype):
    c = Case(T, D, starts, dtype)
    c.compare(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,starts", [(5, 1544, [0, 5]), (7, 2000, [0, 3, 7]), (133, 2000, [2, 61, 131]),
                                        (519, 1672, ragged(519, 9, 3)), (1285, 1536, [0, 700, 1285]),
                                        (4099, 264, ragged(4099, 30, 4)), (2309, 1280, [0, 2309]),
                                        (700, 2504, ragged(700, 40, 6)), (4261, 1544, [1, 2000, 4260]),
                                        (4261, 2504, ragged(4261, 20, 7)), (4205, 2504, [0, 1500, 4203]),
                                        (9000, 16, ragged(9000, 60, 8))])
def test_packed_over_many_rounds(T, D, starts, dtype):
    """Lengths that cut a group of rows in two, widths that cut a warp's channels, several
    tiles a CTA."""
    c = Case(T, D, starts, dtype)
    c.compare(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_more_sequences_than_16_bits(dtype):
    g = gen(11)
    cuts = sorted(int(v) for v in torch.randint(0, 301, (66000,), generator=g))
    c = Case(300, 16, [0] + cuts + [300], dtype)
    c.compare(c.run())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,B", [(5, 64, 5), (1, 8, 1), (64, 128, 4), (600, 40, 200), (640, 1024, 2),
                                   (37, 4096, 37), (515, 1000, 1), (513, 16, 513)])
def test_sequences_of_one_length(T, D, B, dtype):
    c = Case(T, D, B, dtype)
    c.compare(c.run())


@pytest.mark.parametrize("T,D,starts", [(70, 64, [0, 30, 70]), (300, 2048, 3), (9, 128, 9)])
def test_without_states_bias_or_pitch(T, D, starts):
    c = Case(T, D, starts, "bf16", state=False, bias=False, fused=False)
    got = c.run()
    c.compare(got)


def test_optional_outputs():
    """Without hT, states, dbias and dh0 the others have the same bits."""
    c = Case(200, 64, [0, 77, 77, 180], "bf16")
    want = c.run()
    D, T, B = c.D, c.T, c.B
    x, gate, starts = c.x.cuda(), c.gate.cuda(), torch.tensor(c.starts, dtype=torch.int32).cuda()
    h, kept, st = empty(T, D, dtype=torch.bfloat16), empty(tw.twell_recur_states(T), D), status()
    args = (x, gate, D, c.bias.cuda(), starts, B, c.h0.cuda())
    tw.twell_recur_forward(*args, T, D, 1, h, None, None, st)
    assert torch.equal(h[:180], want["h"][:180])
    tw.twell_recur_forward(*args, T, D, 1, h, None, kept, st)
    dx, dg = empty(T, D, dtype=torch.bfloat16), empty(T, D, dtype=torch.bfloat16)
    tw.twell_recur_backward(*args, kept, c.dh.cuda(), c.dhT.cuda(), T, D, 1, dx, dg, None, None, st)
    assert torch.equal(dx[:180], want["dx"][:180]) and torch.equal(dg[:180], want["dgate"][:180])
    assert dx[180:].isnan().all() and h[180:].isnan().all()


def test_states_of_long_decoding():
    """A prompt and then one token at a time, the states in place, is one long sequence."""
    B, D, P, S = 3, 256, 70, 20
    c = Case(B * (P + S), D, B, "f32")
    bias, ref = c.bias.cuda(), c.reference()
    x, gate = c.x.view(B, P + S, D).cuda(), c.gate.view(B, P + S, D).cuda()
    state, st = c.h0.cuda(), status()
    h = empty(B * P, D)
    xs, gs = (v[:, :P].reshape(B * P, D).contiguous() for v in (x, gate))
    tw.twell_recur_forward(xs, gs, D, bias, None, B, state, B * P, D, 0, h, state, None, st)
    rows = [h.view(B, P, D)]
    for t in range(P, P + S):
        h = empty(B, D)
        tw.twell_recur_forward(x[:, t].contiguous(), gate[:, t].contiguous(), D, bias, None, B, state,
                               B, D, 0, h, state, None, st)
        rows.append(h.view(B, 1, D))
    got = torch.cat(rows, 1).reshape(-1, D)
    check(got, ref["h"][0], ref["h"][1], "f32", "h")
    check(state, ref["hT"][0], ref["hT"][1], "f32", "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,D,starts", [(1000, 136, ragged(1000, 17, 1)), (600, 2048, 20), (4100, 72, [0, 4099, 4100]),
                                        (300, 64, 150), (2049, 256, ragged(2049, 40, 5))])
def test_states_in_place(T, D, starts, dtype):
    """hT in the place of h0: the bits of two buffers."""
    c = Case(T, D, starts, dtype, fused=False)
    want = c.run(backward=False)
    x, gate, bias = c.x.cuda(), c.gate.cuda(), c.bias.cuda()
    s = torch.tensor(c.starts, dtype=torch.int32).cuda() if isinstance(c.starts, list) else None
    h, st = empty(T, D, dtype=DT[dtype][0]), status()
    for _ in range(20):
        state = c.h0.cuda()
        tw.twell_recur_forward(x, gate, D, bias, s, c.B, state, T, D, DT[dtype][1], h, state, None, st)
        assert torch.equal(state, want["hT"]) and torch.equal(torch.nan_to_num(h), torch.nan_to_num(want["h"]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nothing_passes_from_sequence_to_sequence(dtype):
    """NaN and infinities in one sequence, in rows outside and in unused states stay there."""
    starts = [10, 50, 50, 130, 131, 400, 690]
    c = Case(700, 72, starts, dtype)
    want = c.run()
    c.x[50:130] = float("nan")
    c.dh[130] = float("inf")
    c.gate[131:400:7] = float("nan")
    for v in (c.x, c.gate, c.dh):
        v[:10] = float("nan")
        v[690:] = float("inf")
    got = c.run()
    for s in (0, 1, 5):
        r = slice(starts[s], starts[s + 1])
        for n in ("h", "dx", "dgate"):
            assert torch.equal(got[n][r], want[n][r]), (n, s)
        for n in ("hT", "dh0"):
            assert torch.equal(got[n][s], want[n][s]), (n, s)
    assert got["h"][50:130].isnan().all()
    for n in ("h", "dx", "dgate"):
        assert got[n][:10].isnan().all() and got[n][690:].isnan().all()


def test_gates_at_the_ends():
    """Gates beyond the sigmoid's range: the state stays, or becomes the input."""
    T, D = 140, 16
    c = Case(T, D, [0, T], "f32", bias=False)
    c.gate[:, 0], c.gate[:, 1], c.gate[:, 2], c.gate[:, 3] = 200., -200., float("inf"), -float("inf")
    got = c.run()
    h, h0 = got["h"].cpu(), c.h0[0]
    for d in (0, 2):
        assert (h[:, d] == h0[d]).all()
        assert (got["dx"][:, d] == 0).all() and (got["dgate"][:, d] == 0).all()
    M = torch.cummax(torch.cat([h0[None], c.x]).abs(), 0).values[1:]
    for d in (1, 3):  # (h + (x - h), where the last state is a rounding of its own)
        assert ((h[:, d] - c.x[:, d]).abs() <= 16 * U * M[:, d]).all() and torch.equal(got["dx"][:, d].cpu(), c.dh[:-1, d].new_tensor(
            torch.cat([c.dh[:-1, d], c.dh[-1:, d] + c.dhT[0, d]]).tolist()))
    check(got["h"][:, 4:], c.reference()["h"][0][:, 4:], c.reference()["h"][1][:, 4:], "f32", "h")


@pytest.mark.parametrize("which", ["x", "gate", "bias", "h0"])
def test_gradient_against_differences(which):
    """A step of 2^-6 along a direction: the difference is within its third-order term (the
    values are of order one: 2^-12 of the sum of magnitudes) and 2^-17 for the roundings."""
    c = Case(150, 16, [0, 80, 80, 150], "f32", fused=False)
    got = c.run()
    direction = torch.randn(getattr(c, which).shape, generator=gen(5))
    name = {"x": "dx", "gate": "dgate", "bias": "dbias", "h0": "dh0"}[which]
    terms = got[name].cpu().double() * direction.double()
    value, base = [], getattr(c, which)
    for sign in (1, -1):
        setattr(c, which, base + sign * 2.0 ** -6 * direction)
        r = c.run(backward=False)
        value.append((r["h"].cpu().double() * c.dh.double()).sum() + (r["hT"].cpu().double() * c.dhT.double()).sum())
    slope = (value[0] - value[1]) / 2.0 ** -5
    assert abs(slope - terms.sum()) <= 2.0 ** -11 * terms.abs().sum() + 2.0 ** -17 * c.dh.abs().sum() * 32


def test_repeats_streams_and_graph():
    """The same bits again, on another stream, and in a replayed graph with new inputs."""
    c = Case(2000, 192, ragged(2000, 9, 3), "bf16")
    want = c.run()
    s = torch.cuda.Stream()
    for stream in (None, s, s.cuda_stream):
        got = c.run(stream=stream)
        for n in want:
            assert torch.equal(torch.nan_to_num(got[n]), torch.nan_to_num(want[n])), n
    T, D, B = c.T, c.D, c.B
    x, gate, dh = (torch.zeros(T, D, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    starts = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    bias, h0, dhT = c.bias.cuda(), c.h0.cuda(), c.dhT.cuda()
    h, dx, dg = (empty(T, D, dtype=torch.bfloat16) for _ in range(3))
    hT, kept, db, d0, st = empty(B, D), empty(tw.twell_recur_states(T), D), empty(D), empty(B, D), status()
    graph = torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        args = (x, gate, D, bias, starts, B, h0)
        tw.twell_recur_forward(*args, T, D, 1, h, hT, kept, st)
        tw.twell_recur_backward(*args, kept, dh, dhT, T, D, 1, dx, dg, db, d0, st)
    x.copy_(c.x), gate.copy_(c.gate), dh.copy_(c.dh)
    starts.copy_(torch.tensor(c.starts, dtype=torch.int32))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    for n, v in zip(("h", "hT", "dx", "dgate", "dbias", "dh0"), (h, hT, dx, dg, db, d0)):
        assert torch.equal(v, want[n]), n
    assert tw.twell_read_status(st) == 0


@pytest.mark.parametrize("starts", [[0, 40, 30, 100], [-1, 50, 100], [0, 50, 101], [7, 2 ** 30, 100],
                                    [100, 0, -2 ** 31]])
def test_malformed_starts_are_recorded(starts):
    T, D, B = 100, 64, len(starts) - 1
    x = torch.zeros(T, D, device="cuda")
    h, hT, kept, st = empty(T, D), empty(B, D), empty(tw.twell_recur_states(T), D), status()
    s = torch.tensor(starts, dtype=torch.int32).cuda()
    tw.twell_recur_forward(x, x, D, None, s, B, hT, T, D, 0, h, hT, kept, st)
    assert tw.twell_read_status(st) == -5
    kept.zero_()
    dx, dg = empty(T, D), empty(T, D)
    tw.twell_recur_backward(x, x, D, None, s, B, hT, kept, x, hT, T, D, 0, dx, dg, empty(D),
                            empty(B, D), st)
    assert tw.twell_read_status(st) == -5


def test_offsets_beyond_32_bits():
    """More than 2^31 elements: the last rows against a sequence that starts there."""
    T, D = 270000, 8192
    x = torch.randn(T, D, device="cuda", dtype=torch.bfloat16)
    h, kept, st = torch.empty_like(x), torch.empty(tw.twell_recur_states(T), D, device="cuda"), status()
    cut = T - 300
    starts = torch.tensor([0, cut, T], dtype=torch.int32, device="cuda")
    hT = empty(2, D)
    tw.twell_recur_forward(x, x, D, None, starts, 2, None, T, D, 1, h, hT, kept, st)
    tail = Case(300, D, [0, 300], "bf16", state=False, bias=False)
    tail.x = tail.gate = x[cut:].cpu()
    tail.dh = x[cut:].cpu()
    ref = tail.reference()
    check(h[cut:], ref["h"][0], ref["h"][1], "bf16", "h")
    dx, dg = torch.empty_like(x), torch.empty_like(x)
    tw.twell_recur_backward(x, x, D, None, starts, 2, None, kept, x, None, T, D, 1, dx, dg, None,
                            None, st)
    for n, v in (("dx", dx), ("dgate", dg)):
        check(v[cut:], ref[n][0], ref[n][1], "bf16", n)
    head = Case(200, D, [0, 200], "bf16", state=False, bias=False)
    head.x = head.gate = x[:200].cpu()
    ref = head.reference()
    check(h[:200], ref["h"][0], ref["h"][1], "bf16", "h")
    assert tw.twell_read_status(st) == 0
