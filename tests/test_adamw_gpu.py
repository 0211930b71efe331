"""AdamW over many tensors, states in 32 and in 8 bits.

The state's arithmetic is defined operation by operation, so m and v (and the codes
and scales that they are rounded to) have to have the bits of the same operations in
fp32 on the host.  The parameter: the decay and the step are an fma each, and the
step's factor, quotient and denominator are rounded together six times at most, so it
is off by 2 u |p| + 8 u |step| (u = 2^-24); the bf16 copy is its rounding, to the
bit."""
import math

import numpy as np
import pytest
import torch

import activation_sparse_transformer_gate_gb300 as tw
from lm_testlib import U, gen, setup

pytestmark = pytest.mark.gpu
LR, B1, B2, EPS = 2e-3, 0.9, 0.99, 1e-8
f32 = lambda v: float(np.float32(v))  # noqa: E731
CODES = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    setup()


def noise(n, first, seed):
    i = np.arange(n, dtype=np.uint64) + np.uint64(first)
    m = np.uint64(0xFFFFFFFF)
    u = ((i & m) * np.uint64(0x9E3779B9) + (i >> np.uint64(32)) * np.uint64(0x3C6EF373) + np.uint64(seed)) & m
    u = ((u ^ (u >> np.uint64(16))) * np.uint64(0x6A09E667)) & m
    u = ((u ^ (u >> np.uint64(15))) * np.uint64(0xBB67AE85)) & m
    u = u ^ (u >> np.uint64(16))
    return (u & np.uint64(0xFFFF)).astype(np.int64), (u >> np.uint64(16)).astype(np.int64)


def blocks_of(x):
    n = x.numel()
    return torch.nn.functional.pad(x, (0, -n % 256)).view(-1, 256)


def quantise(x, bits16, least):
    """Codes (as bytes) and scales of a vector, by the definition."""
    n, b = x.numel(), blocks_of(x)
    top = b.abs().amax(1)
    good = torch.isfinite(top)
    top = torch.where(good, top, torch.ones_like(top)).clamp_min(1e-30)
    y = (blocks_of(x.abs()) * (torch.tensor(448.0) / top)[:, None]).view(-1)[:n].contiguous()
    y = torch.where(good.repeat_interleave(256)[:n], y, torch.zeros_like(y)).numpy()
    # in e4m3 steps, exactly: a value is a whole number of steps and a rest below one
    step = np.exp2(np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3).astype(np.float64)
    down = np.floor(y.astype(np.float64) / step)
    rest = np.floor((y.astype(np.float64) / step - down) * 2 ** 16 * 16)      # in 2^-20
    up = (rest + bits16.astype(np.float64) * 16 >= 2 ** 20)
    q = np.minimum((down + up) * step, 448.0)
    q = np.where(least.numpy(), np.maximum(q, 2.0 ** -9), q)
    code = torch.from_numpy(q).float().to(CODES).view(torch.uint8)
    code = torch.where(torch.signbit(x) & (x < 0), code | 128, code)
    ok = good.repeat_interleave(256)[:n]
    scale = torch.where(good, top * torch.tensor(1.0 / 448.0), torch.full_like(top, float("nan")))
    return torch.where(ok, code, torch.zeros_like(code)), scale


class Tensor:
    """One tensor's step on the host, and its buffers on the GPU."""

    def __init__(self, n, bits, grad=torch.float32, copy=True, decay=0.0, first=0, seed=0):
        g = gen(seed + n)
        self.n, self.bits, self.decay, self.first = n, bits, decay, first
        self.p = torch.randn(n, generator=g) * 0.02
        size = torch.exp(2 * torch.randn(-(-n // 64), generator=g)).repeat_interleave(64)[:n] * 1e-3
        self.g = (torch.randn(n, generator=g) * size).to(grad)
        m, r = torch.randn(n, generator=g) * size * 0.3, size * torch.rand(n, generator=g)
        self.copy = torch.full((n,), float("nan"), dtype=torch.bfloat16) if copy else None
        self.ms = self.vs = None
        if bits == 32:
            self.m, self.v = m, r * r
        else:
            for name, x in (("m", m), ("v", r)):
                b = blocks_of(x)
                scale = b.abs().amax(1) / 448 + 1e-33
                setattr(self, name, (b / scale[:, None]).view(-1)[:n].to(CODES))
                setattr(self, name + "s", scale)
        self.dev = [None if t is None else t.cuda() for t in
                    (self.p, self.g, self.m, self.v, self.ms, self.vs, self.copy)]

    def add(self, tensors):
        p, g, m, v, ms, vs, copy = self.dev
        tensors.add(p, g, m, v, ms, vs, copy=copy, decay=self.decay, first=self.first)

    def step(self, step, seed=0, scale=None, lr=LR):
        """The same on the host; (p in 64 bits, what it may be off)."""
        b1, b2 = f32(B1), f32(B2)
        g = self.g.float() * (1.0 if scale is None else scale)
        if self.bits == 32:
            m, v = self.m, self.v
        else:
            m = self.m.float() * self.ms.repeat_interleave(256)[:self.n]
            r = self.v.float() * self.vs.repeat_interleave(256)[:self.n]
            v = r * r
        m = m * b1 + g * f32(1 - b1)
        v = v * b2 + (g * g) * f32(1 - b2)
        c1, c2 = 1 - b1 ** step, 1 - b2 ** step
        move = f32(lr) / c1 * m.double() / (v.double().sqrt() / math.sqrt(c2) + f32(EPS))
        p = self.p.double()
        want = p * (1 - f32(lr) * f32(self.decay)) - move
        bound = 2 * U * p.abs() + 8 * U * move.abs() + 2.0 ** -149
        if self.bits == 32:
            self.m, self.v = m, v
        else:
            nm, nr = noise(self.n, self.first, seed)
            self.m, self.ms = quantise(m, nm, torch.zeros(self.n, dtype=torch.bool))
            self.v, self.vs = quantise(torch.sqrt(v), nr, v > 0)
            self.m, self.v = self.m.view(CODES), self.v.view(CODES)
        return want, bound

    def compare(self, want, bound):
        p, _, m, v, ms, vs, copy = self.dev
        bits = lambda t: t.cpu().view(torch.uint8 if self.bits == 8 else torch.int32)  # noqa: E731
        assert torch.equal(bits(m), bits(self.m)), "m"
        assert torch.equal(bits(v), bits(self.v)), "v"
        if self.bits == 8:
            assert torch.equal(ms.cpu().view(torch.int32), self.ms.view(torch.int32)), "scale of m"
            assert torch.equal(vs.cpu().view(torch.int32), self.vs.view(torch.int32)), "scale of v"
        off = (p.cpu().double() - want).abs() - bound
        assert not (off > 0).any(), off.max()
        if copy is not None:
            assert torch.equal(copy.cpu().view(torch.int16), p.cpu().bfloat16().view(torch.int16))
        self.p = p.cpu()


SIZES = [1, 2, 3, 4, 5, 127, 128, 129, 255, 256, 257, 300, 511, 2047, 2048, 2049, 5000, 70001, 262144]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_steps(bits, grad):
    """Three steps of a list of many sizes, with and without copies and decay."""
    ts = [Tensor(n, bits, grad, copy=i % 3 != 0, decay=0.1 * (i % 2), first=1000 * i)
          for i, n in enumerate(SIZES)]
    lst = tw.AdamWTensors(bits)
    for t in ts:
        t.add(lst)
    for step in (1, 2, 3):
        tw.twell_adamw_step(lst, LR, B1, B2, EPS, step, seed=77 * step)
        for t in ts:
            t.compare(*t.step(step, 77 * step))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", [torch.float32, torch.bfloat16])
def test_large_tensors(bits, grad):
    """Enough blocks for warps to go over several, across tensors and their partial blocks."""
    ts = [Tensor(n, bits, grad, decay=0.1, first=7 * n) for n in (3000001, 5, 70001, 256, 2000000, 300)]
    lst = tw.AdamWTensors(bits)
    for t in ts:
        t.add(lst)
    for step in (1, 2):
        tw.twell_adamw_step(lst, LR, B1, B2, EPS, step, seed=31 * step)
        for t in ts:
            t.compare(*t.step(step, 31 * step))


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_takes(bits):
    ts = [Tensor(1 + 37 * i % 700, bits, seed=i, first=i << 20) for i in range(1000)]
    lst = tw.AdamWTensors(bits)
    for t in ts:
        t.add(lst)
    tw.twell_adamw_step(lst, LR, B1, B2, EPS, 9, seed=2 ** 32 - 1)
    for t in ts:
        t.compare(*t.step(9, 2 ** 32 - 1))


def test_empty_tensors_are_left_out():
    ts = [Tensor(300, 32, seed=1), Tensor(40, 32, seed=2)]
    lst = tw.AdamWTensors(32)
    none = torch.empty(0, device="cuda")
    lst.add(none, none, none, none)
    ts[0].add(lst)
    lst.add(none, none, none, none)
    ts[1].add(lst)
    tw.twell_adamw_step(lst, LR, B1, B2, EPS, 1)
    for t in ts:
        t.compare(*t.step(1))
    lst = tw.AdamWTensors(32)
    lst.add(none, none, none, none)
    tw.twell_adamw_step(lst, LR, B1, B2, EPS, 1)


@pytest.mark.parametrize("n", [70001, 5000001])
def test_rounding_goes_by_the_elements_number(n):
    """Tensors cut into pieces (of whole blocks) have the bits of the whole, and those around the
    number 2^32."""
    cut, first = 256 * 100, 2 ** 32 - 30000
    whole = Tensor(n, 8, first=first)
    a = Tensor(n, 8, first=first)
    p, g, m, v, ms, vs, copy = a.dev
    for lo, hi in ((0, cut), (cut, n)):
        s, b = slice(lo, hi), slice(lo // 256, -(-hi // 256))
        lst = tw.AdamWTensors(8)
        lst.add(p[s], g[s], m[s], v[s], ms[b], vs[b], copy=copy[s], first=first + lo)
        tw.twell_adamw_step(lst, LR, B1, B2, EPS, 3, seed=5)
    lst = tw.AdamWTensors(8)
    whole.add(lst)
    tw.twell_adamw_step(lst, LR, B1, B2, EPS, 3, seed=5)
    for x, y in zip(a.dev, whole.dev):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    whole.compare(*whole.step(3, 5))


def test_overlaps_are_refused():
    """What a step writes is written once, and is no gradient; gradients may be shared."""
    x = torch.zeros(4096, device="cuda")
    p, g, m, v = x[:512], x[512:1024], x[1024:1536], x[1536:2048]
    half = torch.zeros(512, dtype=torch.bfloat16, device="cuda")

    def code(*rows):
        lst = tw.AdamWTensors(32)
        for r in rows:
            lst.add(*r[:4], copy=r[4] if len(r) > 4 else None)
        try:
            tw.twell_adamw_step(lst, 0.0, B1, B2, EPS, 1)
        except tw.TwellError as e:
            return e.code
        return 0

    other = (x[2048:2560], g, x[2560:3072], x[3072:3584])
    assert code((p, g, m, v, half), other) == 0
    for bad in ((p, g, m, v, half), (x[:512], g, *other[2:]), (other[0], g, other[2], x[1020:1532]),
                (other[0], x[256:768], *other[2:]), (other[0], other[2], *other[2:]),
                (*other, half)):
        assert code((p, g, m, v, half), bad) == -1


def test_rounding_is_unbiased():
    """The mean of many roundings of one value is the value: within 5 standard deviations, a
    rounding's being at most half a step."""
    n = 1 << 20
    t = Tensor(n, 8, copy=False)
    for value in (1.0, 0.77, 0.013, 0.0031, 2e-5):
        t.dev[1].fill_(value)
        t.dev[1][::256] = 1.0                     # (the blocks' largest)
        for x in (t.dev[2], t.dev[3]):
            x.view(torch.uint8).zero_()
        lst = tw.AdamWTensors(8)
        t.add(lst)
        tw.twell_adamw_step(lst, LR, 0.0, 0.0, EPS, 1, seed=11)
        keep = torch.arange(n, device="cuda") % 256 != 0
        for q, s in ((t.dev[2], t.dev[4]), (t.dev[3], t.dev[5])):
            got = (q.float().view(-1, 256) * s[:, None]).view(-1)[keep].double()
            step = max(2.0 ** math.floor(math.log2(value * 448)) / 8, 2.0 ** -9) / 448
            if value * 448 < 2.0 ** -9 and q is t.dev[3]:
                assert (got == got[0]).all() and got[0] > 0      # (not to zero)
                continue
            assert (got - value).abs().max() <= step * (1 + 1e-6)
            assert abs(got.mean().item() - value) <= 5 * step / 2 / math.sqrt(n) + step * 2.0 ** -16


@pytest.mark.parametrize("bits", [32, 8])
def test_averages_follow_a_change(bits):
    """Gradients that fall to a hundredth: v follows, although a step moves it by less than half of
    an 8-bit code's distance (rounded to nearest it would stay where it was)."""
    n = 4096
    t = Tensor(n, bits, copy=False)
    t.dev[1].fill_(1.0)
    t.dev[1][::256] = 10.0
    lst = tw.AdamWTensors(bits)
    t.add(lst)
    value = lambda: (t.dev[3] if bits == 32 else  # noqa: E731
                     (t.dev[3].float().view(-1, 256) * t.dev[5][:, None]).square().view(-1))
    for x in t.dev[2:4]:
        x.view(torch.uint8).zero_()
    for step in range(1, 401):
        if step == 201:
            t.dev[1].fill_(0.01)
            t.dev[1][::256] = 10.0
        tw.twell_adamw_step(lst, 0.0, B1, B2, EPS, step, seed=step)
    got = value().view(-1, 256)[:, 1:].double().mean().item()
    b2 = f32(B2)
    want = (1 - b2 ** 200) * b2 ** 200 + 1e-4 * (1 - b2 ** 200)
    # (r is unbiased; r^2 is then larger by the roundings' variance, which a step adds to and B2
    # forgets: at most (2^-4)^2 / 3 of it a step, held for 1 / (2 (1 - B2)) steps' worth; in 32
    # bits a step is three roundings of v, so 400 of them 1200 u)
    if bits == 32:
        assert abs(got - want) <= 1200 * U * want, (got, want)
    else:
        assert want * 0.98 <= got <= want * 1.1, (got, want)


def test_blocks_with_infinities():
    for bad in (float("inf"), -float("inf"), float("nan")):
        t = Tensor(1000, 8)
        t.g[300], t.dev[1][300] = bad, bad
        lst = tw.AdamWTensors(8)
        t.add(lst)
        tw.twell_adamw_step(lst, LR, B1, B2, EPS, 1, seed=3)
        want, bound = t.step(1, 3)
        p, _, m, v, ms, vs, _ = t.dev
        assert torch.equal(m.cpu().view(torch.uint8), t.m.view(torch.uint8))
        assert torch.equal(v.cpu().view(torch.uint8), t.v.view(torch.uint8))
        nan = torch.tensor([False, True, False, False])
        assert torch.equal(ms.isnan().cpu(), nan) and torch.equal(vs.isnan().cpu(), nan)
        assert p[300].isnan() and p.isnan().sum() == 1
        assert ((p.cpu().double() - want).abs() <= bound)[torch.arange(1000) != 300].all()


def test_zero_and_tiny_blocks():
    t = Tensor(1024, 8, copy=False)
    for x in t.dev[2:4]:
        x.view(torch.uint8).zero_()
    for x in (t.m, t.v):
        x.view(torch.uint8).zero_()
    t.g[:256], t.g[256:512], t.g[512:768] = 0.0, 1e-38, 1e-25
    t.dev[1].copy_(t.g)
    lst = tw.AdamWTensors(8)
    t.add(lst)
    for step in (1, 2):
        tw.twell_adamw_step(lst, LR, B1, B2, EPS, step, seed=step)
        t.compare(*t.step(step, step))
    assert (t.dev[2][:256].view(torch.uint8) == 0).all() and torch.isfinite(t.dev[0]).all()


def test_grad_scale():
    t = Tensor(700, 8)
    lst = tw.AdamWTensors(8)
    t.add(lst)
    scale = torch.tensor([0.25], device="cuda")
    tw.twell_adamw_step(lst, LR, B1, B2, EPS, 4, seed=6, grad_scale=scale)
    t.compare(*t.step(4, 6, scale=0.25))
    before = [x.clone() for x in t.dev]
    for bad in (float("inf"), float("nan")):       # a step that is given up
        scale.fill_(bad)
        tw.twell_adamw_step(lst, LR, B1, B2, EPS, 5, seed=7, grad_scale=scale)
    for x, y in zip(t.dev, before):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_once_and_replayed(bits):
    """A captured step reads lr, corrections and seed from device memory: the steps that calls
    by value make, to the bits of the state."""
    ts = [Tensor(n, bits, decay=0.05) for n in (3000, 17, 256)]
    lst = tw.AdamWTensors(bits)
    for t in ts:
        t.add(lst)
    dyn = torch.zeros(4, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        tw.twell_adamw_step(lst, 0.0, B1, B2, EPS, 1, dynamic=dyn)
    for step in range(1, 5):
        dyn.copy_(tw.adamw_dynamic(LR * step, B1, B2, step, seed=100 + step))
        graph.replay()
        torch.cuda.synchronize()
        for t in ts:
            want, bound = t.step(step, 100 + step, lr=LR * step)
            t.compare(want, 2 * bound)             # (lr / correction1 is one rounding more)


def test_on_another_stream():
    t = Tensor(100000, 32)
    lst = tw.AdamWTensors(32)
    t.add(lst)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    tw.twell_adamw_step(lst, LR, B1, B2, EPS, 1, stream=s)
    s.synchronize()
    t.compare(*t.step(1))


def test_offsets_beyond_32_bits():
    """A tensor of more than 2^31 elements, looked at around its ends and around element 2^31."""
    n = 2 ** 31 + 300
    p = torch.zeros(n, device="cuda")
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(CODES) for _ in range(2))
    ms, vs = (torch.zeros(-(-n // 256), device="cuda") for _ in range(2))
    lst = tw.AdamWTensors(8)
    lst.add(p, g, m, v, ms, vs)
    tw.twell_adamw_step(lst, LR, B1, B2, EPS, 1, seed=9)
    for at in (0, 2 ** 31 - 512, 2 ** 31, n - 300):
        assert (p[at:at + 300] + LR).abs().max() <= 1e-8
        largest = 0.5 * f32(1 - f32(B1))
        assert (ms[at // 256:at // 256 + 2].double() * 448 - largest).abs().max() <= 4 * U * largest
        assert (m[at:at + 300].float() == 448).all() and (v[at:at + 300].float() == 448).all()
