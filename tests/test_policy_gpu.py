"""Clipped policy loss with a KL term against 64 bits.

Bounds, with u = 2^-24, s = max |z / tau| over the row: an exponent is an fma, off by
u of |z c| and of the reference's rounding, which cancels; the sum of exponentials
is off by at most (2 s + 8 + 40) u (its additions are spread over lanes: under 40
deep beside the vectors of a lane, V / 8192 + 8 more), so
    logp:   e = (6 s + 64 + V / 4096) u
    r:      e + 4 u of itself, and |logp - old| u;  exp(d) - 1: the same with d
    loss:   w (|A| r er + beta (exp(d) ed + |d| u + ...)),  slope likewise
    dz:     |slope| / tau (q (e + (2 s + 12) u) + onehot (e + 4 u)) + dslope / tau (q + onehot)."""
import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import DT, U, check, empty, gen, setup, status

pytestmark = pytest.mark.gpu
LOW, HIGH, BETA = 0.2, 0.28, 0.04


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


class Case:
    def __init__(self, T, V, dtype, tau=1.0, seed=0, old=True, ref=True, masked=False, beta=BETA):
        g = gen(seed + T * 977 + V)
        self.T, self.V, self.dtype, self.tau, self.beta = T, V, dtype, tau, beta
        self.z = (2.5 * torch.randn(T, V, generator=g)).to(DT[dtype][0])
        self.tok = torch.randint(0, V, (T,), generator=g)
        logp = torch.log_softmax(self.z.double() / tau, 1).gather(1, self.tok[:, None])[:, 0].float()
        # ratios off the clip's borders by far more than the roundings
        ratio = 1.01 + 0.04 * torch.randint(-18, 18, (T,), generator=g)
        self.old = logp - torch.log(ratio) if old else None
        self.ref = logp + 0.3 * torch.randn(T, generator=g) if ref else None
        self.adv = torch.randn(T, generator=g)
        self.w = torch.rand(T, generator=g) + 0.1
        if masked:
            self.w[torch.rand(T, generator=g) < 0.3] = 0
            self.tok[torch.rand(T, generator=g) < 0.2] = -1

    def reference(self):
        """{name: (value, bound)}, the live rows."""
        z = self.z.double() / self.tau
        live = (self.tok >= 0) & (self.w != 0 if self.w is not None else True)
        w = (self.w.double() if self.w is not None else torch.ones(self.T).double()) * live
        pick = self.tok.clamp_min(0)[:, None]
        lq = torch.log_softmax(z, 1)
        q, logp = lq.exp(), lq.gather(1, pick)[:, 0]
        finite = torch.where(torch.isinf(z), torch.zeros_like(z), z)
        s = finite.abs().amax(1)
        e = (6 * s + 64 + self.V / 4096) * U
        old = self.old.double() if self.old is not None else logp
        ref = self.ref.double() if self.ref is not None else None
        A = self.adv.double()
        r = torch.exp(logp - old)
        er = r * (e + 4 * U + (logp - old).abs() * U) if self.old is not None else torch.zeros_like(r)
        clip = torch.where(A >= 0, r > 1 + HIGH, r < 1 - LOW)
        held = r.clamp(1 - LOW, 1 + HIGH)
        loss = -torch.where(clip, held, r) * A
        eloss = torch.where(clip, 4 * U * held, er + 4 * U * r) * A.abs()
        slope = -torch.where(clip, torch.zeros_like(r), r) * A
        eslope = torch.where(clip, torch.zeros_like(r), er + 2 * U * r) * A.abs()
        if ref is not None and self.beta:
            d = ref - logp
            ed = e + d.abs() * U
            loss = loss + self.beta * (torch.expm1(d) - d)
            eloss = eloss + self.beta * (torch.expm1(d).abs() * ed + 6 * U * (torch.expm1(d).abs() + d.abs())) + 2 * U * loss.abs()
            slope = slope - self.beta * torch.expm1(d)
            eslope = eslope + self.beta * (d.exp() * ed + 6 * U * torch.expm1(d).abs()) + 2 * U * slope.abs()
        loss, eloss = w * loss, w * eloss + 2 * U * (w * loss).abs()
        slope, eslope = w * slope / self.tau, w * eslope / self.tau + 3 * U * (w * slope / self.tau).abs()
        hot = torch.zeros_like(q).scatter_(1, pick, 1.0)
        dz = slope[:, None] * (hot - q)
        keep = 1 - (hot * q).sum(1)  # (the token's own element is slope (1 - q))
        edz = slope.abs()[:, None] * (q * (1 - hot) * (2 * e + (2 * s + 12) * U)[:, None]
                                      + hot * (e * (1 - keep) + 6 * U * keep)[:, None])
        edz = edz + eslope[:, None] * (q * (1 - hot) + hot * keep[:, None])
        edz = torch.where(q < 2.0 ** -120, edz + 2.0 ** -120 * (1 + slope.abs())[:, None], edz)
        m = self.z.double().amax(1)
        stats = torch.stack([m, torch.logsumexp(z, 1) - m / self.tau], 1)
        on = live.double()
        zero = torch.zeros_like
        put = lambda v, o: (torch.where(o > 0, v, zero(v)))  # noqa: E731
        o1, o2 = on, on[:, None]
        return {"logp": (put(logp, o1), e * on), "loss": (put(loss, o1), put(eloss, o1)),
                "dz": (put(dz, o2.expand_as(dz)), put(edz, o2.expand_as(dz))),
                "stats": (put(stats, o2.expand_as(stats)), torch.stack([zero(e), e], 1) * o2)}

    def device(self, pitch=None):
        T, V = self.T, self.V
        ld = pitch or V
        z = torch.full((T, ld), 7.0, dtype=DT[self.dtype][0], device="cuda")
        z[:, :V] = self.z.cuda()
        return z, ld

    def run(self, grad=True, two=False, pitch=None, in_place=False, long=True, stream=None):
        T, V = self.T, self.V
        tdt, dt = DT[self.dtype]
        z, ld = self.device(pitch)
        dz = z if in_place and not two else torch.full_like(z, float("nan"))
        dev = lambda v: None if v is None else v.cuda()  # noqa: E731
        tok = self.tok.cuda() if long else self.tok.int().cuda()
        old, ref, adv, w = dev(self.old), dev(self.ref), dev(self.adv), dev(self.w)
        loss, logp, stats, st = empty(T), empty(T), empty(T, 2), status()
        tail = (T, V, dt, self.tau, LOW, HIGH, self.beta)
        torch.cuda.synchronize()
        tw.twell_policy_forward(z[:, :V], ld, tok, old, ref, adv, w, *tail, loss, logp, stats,
                                dz[:, :V] if grad and not two else None, st, stream)
        if two:
            dz = z if in_place else dz
            g = w if w is not None else torch.ones(T, device="cuda")
            tw.twell_policy_backward(z[:, :V], ld, tok, old, ref, adv, logp, stats, g, *tail,
                                     dz[:, :V], st, stream)
        torch.cuda.synchronize()
        assert tw.twell_read_status(st) == 0
        out = {"loss": loss, "logp": logp, "stats": stats}
        if grad or two:
            assert (dz[:, V:] == 7.0).all() if in_place else dz[:, V:].isnan().all()
            out["dz"] = dz[:, :V]
        return out

    def compare(self, got):
        ref = self.reference()
        for n, v in got.items():
            check(v, *ref[n], self.dtype if n == "dz" else "f32", n)


SHAPES = [(1, 1), (1, 2), (3, 7), (5, 100), (64, 512), (9, 1025), (4, 2048), (7, 4097), (3, 50001),
          (2, 131072), (1, 262147), (310, 2500), (320, 9000), (306, 20000), (304, 70001)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,V", SHAPES)
def test_loss_and_gradient(T, V, dtype):
    c = Case(T, V, dtype, masked=T > 3)
    one = c.run()
    c.compare(one)
    two = c.run(two=True, long=False)
    c.compare(two)
    alone = c.run(grad=False)
    for n in ("loss", "logp", "stats"):
        assert torch.equal(two[n], alone[n])
    c.compare(alone)


@pytest.mark.parametrize("T,V,pitch", [(6, 500, 507), (5, 5001, 5008), (3, 50001, 50003), (310, 5001, 5005),
                                       (304, 70001, 70003)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_pitch_and_in_place(T, V, pitch, dtype):
    c = Case(T, V, dtype, tau=1.7)
    want = c.run()
    c.compare(want)
    for got in (c.run(pitch=pitch), c.run(in_place=True), c.run(pitch=pitch, in_place=True)):
        c.compare(got)
    c.compare(c.run(pitch=pitch, two=True, in_place=True))


@pytest.mark.parametrize("kind", ["on policy", "no kl", "beta 0", "no weight", "cold", "hot"])
def test_forms(kind):
    c = Case(40, 3001, "f32", old=kind != "on policy", ref=kind != "no kl",
             beta=0.0 if kind == "beta 0" else BETA,
             tau={"cold": 0.05, "hot": 50.0}.get(kind, 1.0))
    if kind == "no weight":
        c.w = None
    c.compare(c.run())
    c.compare(c.run(two=True))


@pytest.mark.parametrize("T,V", [(5, 400), (9, 50001), (400, 4001), (310, 20000)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_log_probabilities_alone(T, V, dtype):
    c = Case(T, V, dtype, masked=True)
    want = c.run()
    z, ld = c.device()
    logp, stats, st = empty(T), empty(T, 2), status()
    tw.twell_policy_forward(z, ld, c.tok.cuda(), None, None, None, c.w.cuda(), T, V, DT[dtype][1],
                            c.tau, LOW, HIGH, BETA, None, logp, stats, None, st)
    assert tw.twell_read_status(st) == 0
    c.compare({"logp": logp, "stats": stats})
    check(logp, want["logp"].double().cpu(), c.reference()["logp"][1], "f32", "logp")


def test_clip_borders_and_signs():
    """Every side of the clip, at ratios far off and at 1, with either sign and 0."""
    V = 600
    rows = [(r, a) for r in (1e-6, 0.5, 0.79, 0.81, 1.0, 1.27, 1.29, 3.0, 1e6) for a in (-2.0, 0.0, 1.5)]
    c = Case(len(rows), V, "f32", ref=False)
    z = c.z.double()
    logp = torch.log_softmax(z, 1).gather(1, c.tok[:, None])[:, 0]
    c.old = (logp - torch.log(torch.tensor([r for r, _ in rows]).double())).float()
    c.adv = torch.tensor([a for _, a in rows])
    got = c.run()
    c.compare(got)
    for i, (r, a) in enumerate(rows):
        flat = (a > 0 and r > 1 + HIGH) or (a < 0 and r < 1 - LOW) or a == 0
        assert (got["dz"][i] == 0).all() == flat, (r, a)


@pytest.mark.parametrize("V", [300, 5000, 131072])
@pytest.mark.parametrize("T", [8, 310])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_at_the_edges(T, V, dtype):
    """Logits of -inf, the type's lowest value, huge ones; rows of NaN and of nothing; no row
    disturbs another."""
    if T * V > 2 ** 24:
        pytest.skip("long on the host")
    c = Case(T, V, dtype)
    low = torch.finfo(DT[dtype][0]).min
    c.z[1, 1:V - 1:2] = -float("inf")
    c.z[2, ::3] = low
    c.z[3] *= 1e4
    c.z[4, 5] = float("nan")
    c.z[5] = -float("inf")
    c.z[6, 9] = float("inf")
    c.tok[1], c.tok[2] = 0, 1
    c.old = c.ref = None
    for two in (False, True):
        got = c.run(two=two)
        bad = torch.zeros(T, dtype=torch.bool)
        bad[4:7] = True
        assert got["loss"][4:7].isnan().all() and got["logp"][4:7].isnan().all()
        assert got["dz"][4:7].isnan().all()
        assert not got["dz"][~bad].isnan().any()
        ref = c.reference()
        for n in ("loss", "logp", "stats", "dz"):
            kind = dtype if n == "dz" else "f32"
            check(got[n][~bad], ref[n][0][~bad], ref[n][1][~bad], kind, n)
        assert (got["dz"][1, 1:V - 1:2] == 0).all() and (got["dz"][2, ::3] == 0).all()


def test_impossible_token():
    """A token of probability 0: its own definition when it was sampled on policy."""
    c = Case(4, 700, "f32", old=False, ref=False)
    c.z[0, 3] = -float("inf")
    c.tok[0] = 3
    got = c.run()
    assert got["logp"][0] == -float("inf")
    s = (-c.w[0] * c.adv[0]).double()
    q = torch.softmax(c.z[0].double(), 0)
    want = -s * q
    want[3] = s
    assert (got["dz"][0].cpu().double() - want).abs().max() <= 1e-5 * s.abs()
    c.old = torch.full((4,), -3.0)           # and with an old log-probability: ratio 0
    got = c.run()
    want = 0.0 if c.adv[0] > 0 else -c.w[0].double() * c.adv[0].double() * (1 - LOW)
    assert abs(got["loss"][0].item() - want) <= 4 * U * abs(want)   # (1 - LOW and two products)


def test_tokens_out_of_range():
    for V in (300, 5000, 131072):
        for T in (4, 330):
            if T * V > 2 ** 24:
                continue
            c = Case(T, V, "bf16")
            want = c.run()
            good, c.tok = c.tok, c.tok.clone()
            c.tok[1], c.tok[3] = V, 2 ** 40
            z, ld = c.device()
            loss, logp, stats, st = empty(T), empty(T), empty(T, 2), status()
            dz = torch.full_like(z, float("nan"))
            args = (T, V, 1, 1.0, LOW, HIGH, BETA)
            dev = [v.cuda() for v in (c.tok, c.old, c.ref, c.adv, c.w)]
            tw.twell_policy_forward(z, ld, *dev, *args, loss, logp, stats, dz, st)
            assert tw.twell_read_status(st) == -5 and tw.twell_read_status(st) == 0
            for r in (1, 3):
                assert loss[r] == 0 and logp[r] == 0 and (stats[r] == 0).all() and (dz[r] == 0).all()
            keep = torch.ones(T, dtype=torch.bool)
            keep[1] = keep[3] = False
            assert torch.equal(dz[keep], want["dz"][keep]) and torch.equal(loss[keep], want["loss"][keep])
            dz.fill_(float("nan"))
            tw.twell_policy_backward(z, ld, *dev[:4], logp, stats, dev[4], *args, dz, st)
            assert tw.twell_read_status(st) == -5
            assert (dz[1] == 0).all() and (dz[3] == 0).all() and not dz.isnan().any()
            c.tok = good


def test_masked_rows_are_not_read():
    for T, V in ((6, 400), (6, 60000), (400, 4001), (310, 30000)):
        c = Case(T, V, "bf16")
        c.w[::2] = 0
        want = c.run()
        c.z[::2] = float("nan")
        got = c.run()
        for n in want:
            assert torch.equal(got[n], want[n]), n
        assert (got["dz"][::2] == 0).all()


def test_gradient_against_differences():
    """Central differences along a direction, step 2^-5 (the logits are of order one): third-order
    term and roundings as bounded."""
    c = Case(12, 900, "f32", masked=True)
    got = c.run()
    direction = torch.randn(c.z.shape, generator=gen(3))
    base, value = c.z, []
    for sign in (1, -1):
        c.z = base + sign * 2.0 ** -8 * direction
        value.append(c.run(grad=False)["loss"].cpu().double())
    slope = (value[0] - value[1]) / 2.0 ** -7
    want = (got["dz"].cpu().double() * direction.double()).sum(1)
    # a row's loss is off by (|A| r + beta) w times 100 u each, divided by the step
    scale = c.w.double() * (c.adv.abs().double() * 2 + 1)
    assert ((slope - want).abs() <= scale * (200 * U * 2 ** 7 + 2.0 ** -14)).all()


def test_repeats_streams_and_graph():
    for T, V in ((50, 400), (7, 60000), (320, 5001)):
        c = Case(T, V, "bf16", masked=True)
        want = c.run()
        s = torch.cuda.Stream()
        for stream in (None, s):
            got = c.run(stream=stream)
            for n in want:
                assert torch.equal(got[n], want[n])
        z = torch.zeros(T, V, dtype=torch.bfloat16, device="cuda")
        dz, dz2 = torch.empty_like(z), torch.empty_like(z)
        dev = [v.cuda() for v in (c.tok, c.old, c.ref, c.adv, c.w)]
        loss, logp, stats, st = empty(T), empty(T), empty(T, 2), status()
        args = (T, V, 1, 1.0, LOW, HIGH, BETA)
        graph = torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            tw.twell_policy_forward(z, V, *dev, *args, loss, logp, stats, dz, st)
            tw.twell_policy_backward(z, V, *dev[:4], logp, stats, dev[4], *args, dz2, st)
        z.copy_(c.z)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dz, want["dz"]) and torch.equal(loss, want["loss"])
        c.compare({"dz": dz2})


def test_offsets_beyond_32_bits():
    T, V = 17000, 131073
    z = torch.randn(T, V, device="cuda", dtype=torch.bfloat16)
    c = Case(3, V, "bf16")
    tok = torch.randint(0, V, (T,), device="cuda")
    tok[-1], tok[-2] = V - 1, 0
    c.z, c.tok = z[-3:].cpu(), tok[-3:].cpu()
    logp = torch.log_softmax(c.z.double(), 1).gather(1, c.tok[:, None])[:, 0].float()
    old = torch.full((T,), -11.0, device="cuda")
    c.old = logp - 0.05
    old[-3:] = c.old.cuda()
    adv, w = torch.randn(T, device="cuda"), torch.rand(T, device="cuda") + 0.1
    c.adv, c.w, c.ref = adv[-3:].cpu(), w[-3:].cpu(), None
    loss, lp, stats, st, dz = empty(T), empty(T), empty(T, 2), status(), torch.empty_like(z)
    args = (T, V, 1, 1.0, LOW, HIGH, BETA)
    tw.twell_policy_forward(z, V, tok, old, None, adv, w, *args, loss, lp, stats, dz, st)
    ref = c.reference()
    for n, v in (("loss", loss), ("logp", lp), ("dz", dz)):
        check(v[-3:], *ref[n], "bf16" if n == "dz" else "f32", n)
    tw.twell_policy_backward(z, V, tok, old, None, adv, lp, stats, w, *args, z, st)
    check(z[-3:], *ref["dz"], "bf16", "dz in place")
    assert tw.twell_read_status(st) == 0
