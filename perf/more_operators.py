"""The operators of a training step around the sparse feed-forward layer that
mix, judge and update: a gated linear recurrence over packed sequences (with its
backward pass and its form for decoded tokens), the clipped policy loss with a KL
term (with its gradient, and the log-probabilities alone), and an AdamW step over
all tensors of a model with states in 32 or in 8 bits.

``run`` computes a case in plain torch operations (in 32 bits, rounded once at
the end) or, where ``own`` is true, with the framework's kernels.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}
CLIP_LOW, CLIP_HIGH, BETA_KL = 0.2, 0.28, 0.04
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-3, 0.9, 0.999, 1e-8, 0.1, 10
BLOCK, E4M3_MAX = 256, 448.0


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the framework's smallest configuration (64 tokens, d_model 128, fp32): latency counts
        dict(name="mix 64x128 f32", kind="mix", T=64, D=128, B=4, dtype="f32", state=False),
        # a training step's tokens at the base d_model, packed sequences of ragged lengths
        dict(name="mix 4096x2048", kind="mix", T=4096, D=2048, B=9, dtype="bf16", state=False),
        # the long batch at the large d_model, sequences that go on from a state
        dict(name="mix 16384x4096", kind="mix", T=16384, D=4096, B=3, dtype="bf16", state=True),
        # a long document read before anything is generated: one sequence, few channels
        dict(name="prompt 131072x1024", kind="prompt", T=131072, D=1024, B=1, dtype="bf16",
             state=True),
        # a ragged batch of decoded tokens
        dict(name="step 37x4096", kind="step", T=37, D=4096, B=37, dtype="bf16", state=True),
        # the smallest configuration's loss and gradient, in one call
        dict(name="policy 64xV512 f32", kind="policy", T=64, V=512, dtype="f32", fused=True,
             masked=False),
        # the loss and its gradient as two calls (autograd's order) over an odd vocabulary;
        # an eighth of the rows are prompt tokens
        dict(name="policy 2048xV50001", kind="policy", T=2048, V=50001, dtype="bf16", fused=False,
             masked=True),
        # a large vocabulary: the loss and its gradient in one call
        dict(name="policy 8192xV131072", kind="policy", T=8192, V=131072, dtype="bf16", fused=True,
             masked=False),
        # the old or the reference policy's pass: log-probabilities alone
        dict(name="logp 4001xV50001", kind="logp", T=4001, V=50001, dtype="bf16", fused=True,
             masked=True),
        # the update of the smallest configuration's model
        dict(name="adamw V512 D128 F512", kind="adamw", V=512, D=128, F=512, layers=2, bits=32,
             grad="f32"),
        # the base model's update with states in 8 bits
        dict(name="adamw V50001 D2048 F8192 8bit", kind="adamw", V=50001, D=2048, F=8192, layers=4,
             bits=8, grad="f32"),
        # the large model's update
        dict(name="adamw V131072 D4096 F14336", kind="adamw", V=131072, D=4096, F=14336, layers=2,
             bits=32, grad="f32"),
    ]


def _log_int(rng, lo, hi, mult=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(mult, min(hi, max(lo, v)) // mult * mult)


def draw(rng):
    kind = rng.choice(["mix", "mix", "prompt", "step", "policy", "policy", "logp", "adamw",
                       "adamw"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind in ("mix", "prompt"):
        D = _log_int(rng, 64, 8192, 8)
        most = 16384 * 4096 // D // (ES[dtype] // 2)
        T = _log_int(rng, 1, min(most, 16384 if kind == "mix" else 131072))
        return dict(kind=kind, T=T, D=D, B=_log_int(rng, 1, min(T, 64)), dtype=dtype,
                    state=kind == "prompt" or rng.random() < 0.5)
    if kind == "step":
        T = _log_int(rng, 1, 512)
        return dict(kind=kind, T=T, D=_log_int(rng, 64, 8192, 8), B=T, dtype=dtype, state=True)
    if kind in ("policy", "logp"):
        V = _log_int(rng, 100, 131072)
        most = min(8192, 8192 * 131072 // (V * ES[dtype] // 2))
        return dict(kind=kind, T=_log_int(rng, 1, most), V=V, dtype=dtype,
                    fused=kind == "logp" or rng.random() < 0.5, masked=rng.random() < 0.5)
    D = _log_int(rng, 64, 4096, 8)
    return dict(kind=kind, V=_log_int(rng, 100, 131072), D=D, F=_log_int(rng, D, min(4 * D, 14336)),
                layers=rng.randint(1, 2), bits=rng.choice([8, 32]),
                grad=rng.choice(["f32", "f32", "bf16"]))


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype) * scale


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _zeros(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def _inputs_mix(c, g):
    T, D, B, dt = c["T"], c["D"], c["B"], DT[c["dtype"]]
    # inputs and gates are one projection's two halves; the bias spreads the channels'
    # memories from a few tokens to a few hundred
    st = dict(xg=_randn(g, T, 2 * D, dtype=dt),
              bias=torch.linspace(1.0, 5.0, D, device="cuda") + _randn(g, D, scale=0.1),
              h0=_randn(g, B, D) if c["state"] else None,
              h=_zeros(T, D, dtype=dt), starts=None,
              status=_zeros(1, dtype=torch.int32))
    if c["kind"] == "step":
        return st
    # sequences of any length; some are empty, and the buffer is a little longer than all of them
    end = T - int(T // 17 * float(_rand(g, 1)))
    cuts = torch.sort((_rand(g, B - 1) * (end + 1)).int()).values
    edge = torch.tensor([0, end], dtype=torch.int32, device="cuda")
    st["starts"] = torch.cat([edge[:1], cuts, edge[1:]])
    if c["state"]:
        st["hT"] = _zeros(B, D)
    if c["kind"] == "mix":
        st |= dict(dh=_randn(g, T, D, dtype=dt), dxg=_zeros(T, 2 * D, dtype=dt), dbias=_zeros(D))
        if c["state"]:
            st |= dict(dhT=_randn(g, B, D), dh0=_zeros(B, D))
    return st


def _inputs_policy(c, g):
    T, V, dt = c["T"], c["V"], DT[c["dtype"]]
    z = _randn(g, T, V, dtype=dt, scale=2.5)
    # tokens that the policy may well have sampled: a row's likeliest of a few random ones
    some = (_rand(g, T, 16) * V).long().clamp_max(V - 1)
    tok = some.gather(1, z.gather(1, some).float().argmax(1, keepdim=True))
    logp = (z.gather(1, tok).float() - torch.logsumexp(z.float(), 1, keepdim=True))[:, 0]
    # how far the policy has moved since it sampled, in steps that lie off the clip's borders
    ratio = 1.0 + 0.04 * torch.round(_randn(g, T, scale=4.0)).clamp(-20, 20) + 0.01
    f = lambda *s: torch.empty(*s, dtype=torch.float32, device="cuda")  # noqa: E731
    weight = torch.full((T,), 1.0 / T, device="cuda")
    if c["masked"]:
        weight = torch.where(_rand(g, T) < 0.125, torch.zeros_like(weight), weight)
        tok = torch.where(_rand(g, T, 1) < 0.01, torch.full_like(tok, -1), tok)
    return dict(z=z, tok=tok[:, 0].contiguous(), old=logp - torch.log(ratio),
                ref=logp + _randn(g, T, scale=0.2), adv=_randn(g, T), weight=weight, tau=1.0,
                loss=f(T), logp=f(T), stats=f(T, 2),
                dz=torch.empty_like(z) if c["kind"] == "policy" else None,
                status=_zeros(1, dtype=torch.int32))


def _model(c):
    """(elements, weight decay) of a model's tensors: matrices decay, biases and norms do not."""
    V, D, F = c["V"], c["D"], c["F"]
    layer = [(F * D, DECAY)] * 3 + [(F, 0.0), (D, 0.0)]
    return [(V * D, DECAY)] + layer * c["layers"] + [(D, 0.0), (V * D, DECAY)]


def _inputs_adamw(c, g):
    # all tensors lie in flat buffers, each from a multiple of a block on
    table, at = [], 0
    for n, decay in _model(c):
        table.append((at, n, decay))
        at += -(-n // BLOCK) * BLOCK
    blocks = at // BLOCK
    live = torch.ones(at, dtype=torch.bool, device="cuda")
    for first, n, _ in table:
        live[first + n:first + -(-n // BLOCK) * BLOCK] = False
    # gradients whose sizes differ from row to row, and averages that they may have left
    size = torch.exp(_randn(g, blocks, 1)) * 1e-3
    grad = (_randn(g, blocks, BLOCK) * size).view(-1) * live
    m = (_randn(g, blocks, BLOCK) * size * 0.3).view(-1) * live
    r = (size * (0.5 + _rand(g, blocks, BLOCK))).view(-1) * live
    st = dict(table=table, p=_randn(g, at, scale=0.02) * live, g=grad.to(DT[c["grad"]]),
              copy=_zeros(at, dtype=torch.bfloat16), seed=int(torch.randint(
                  0, 2 ** 31, (1,), generator=g, device="cuda")),
              decay=torch.cat([torch.full((-(-n // BLOCK), 1), d, device="cuda")
                               for _, n, d in table]))
    if c["bits"] == 32:
        return st | dict(m=m, v=r * r)
    for name, x in (("m", m), ("v", r)):
        scale = x.view(-1, BLOCK).abs().amax(1) / E4M3_MAX
        st[name + "scale"] = scale
        code = torch.where(scale[:, None] > 0, x.view(-1, BLOCK) / scale[:, None],
                           torch.zeros_like(x.view(-1, BLOCK)))
        st[name] = code.view(-1).to(torch.float8_e4m3fn)
    return st


INPUTS = {"mix": _inputs_mix, "prompt": _inputs_mix, "step": _inputs_mix, "policy": _inputs_policy,
          "logp": _inputs_policy, "adamw": _inputs_adamw}


def prepare(case, seed):
    st = INPUTS[case["kind"]](case, _gen(seed))
    st["case"] = case
    return st


# ------------------------------------------------------------ plain forms --
def _sequences(st):
    """For the rows: whether in a sequence, whether a sequence's first, its last, and whose."""
    starts, T = st["starts"].long(), st["case"]["T"]
    row = torch.arange(T, device="cuda")
    seq = torch.searchsorted(starts, row, right=True) - 1
    live = (row >= starts[0]) & (row < starts[-1])
    seq = torch.where(live, seq, torch.zeros_like(seq))
    return live, live & (starts[seq] == row), live & (starts[seq + 1] == row + 1), seq


def _scan(c, u, fresh):
    """y_t = (1 - c_t) y_{t-1} + u_t from y = 0 (at rows marked fresh too), by doubling."""
    C, Y = torch.where(fresh[:, None], torch.ones_like(c), c), u.clone()
    k = 1
    while k < C.shape[0]:
        Y = torch.cat([Y[:k], Y[k:] + Y[:-k] - C[k:] * Y[:-k]])
        C = torch.cat([C[:k], C[k:] + C[:-k] - C[k:] * C[:-k]])
        k *= 2
    return Y


def _plain_mix(st):
    c = st["case"]
    D, dt = c["D"], DT[c["dtype"]]
    x, gate = st["xg"][:, :D].float(), st["xg"][:, D:].float() + st["bias"]
    keep, take = torch.sigmoid(gate), torch.sigmoid(-gate)
    if c["kind"] == "step":
        h = st["h0"] + take * (x - st["h0"])
        st["h0"].copy_(h)
        return {"h": h.to(dt), "hT": st["h0"]}
    live, first, last, seq = _sequences(st)
    before = torch.zeros_like(x)
    if c["state"]:
        before = torch.where(first[:, None], st["h0"][seq], before)
    h = _scan(take, take * x + keep * before, first) * live[:, None]
    out = {"h": h.to(dt)}
    if c["state"]:
        hT = st["h0"].clone()  # (an empty sequence's state stays)
        hT[seq[last]] = h[last]
        out["hT"] = hT
    if c["kind"] == "prompt":
        return out
    before = torch.where(first[:, None], before, torch.cat([before[:1], h[:-1]]))
    dh = st["dh"].float()
    if c["state"]:
        dh = dh + torch.where(last[:, None], st["dhT"][seq], torch.zeros_like(dh))
    after = _scan(take.flip(0), (keep * dh).flip(0), last.flip(0)).flip(0)  # a_t G_t
    G = dh + torch.where(last[:, None], torch.zeros_like(dh), torch.cat([after[1:], dh[:1] * 0]))
    G = G * live[:, None]
    dgate = G * (before - x) * keep * take
    out["dxg"] = torch.cat([(take * G).to(dt), dgate.to(dt)], dim=1)
    out["dbias"] = dgate.sum(dim=0)
    if c["state"]:
        dh0 = st["dhT"].clone()
        dh0[seq[first]] = after[first]
        out["dh0"] = dh0
    return out


def _plain_policy(st):
    tau, V = st["tau"], st["case"]["V"]
    on = (st["weight"] != 0) & (st["tok"] >= 0)
    zero = torch.zeros_like(st["weight"])
    z = st["z"].float()
    top = z.amax(dim=1, keepdim=True)
    z = (z - top) / tau
    lse = torch.log(torch.exp(z).sum(dim=1, keepdim=True))
    at = st["tok"].clamp_min(0)[:, None]
    logp = (z.gather(1, at) - lse)[:, 0]
    stats = torch.cat([top, lse], dim=1) * on[:, None]
    out = {"logp": torch.where(on, logp, zero), "stats": stats}
    if st["case"]["kind"] == "logp":
        return out
    ratio, away = torch.exp(logp - st["old"]), st["ref"] - logp
    bound = ratio.clamp(1.0 - CLIP_LOW, 1.0 + CLIP_HIGH)
    gain, kept = ratio * st["adv"], bound * st["adv"]
    kl = torch.exp(away) - away - 1.0
    out["loss"] = torch.where(on, st["weight"] * (BETA_KL * kl - torch.minimum(gain, kept)), zero)
    slope = BETA_KL * (1.0 - torch.exp(away)) - torch.where(gain <= kept, gain, zero)
    slope = torch.where(on, st["weight"] * slope / tau, zero)[:, None]
    dz = torch.exp(z - lse) * -slope
    dz.scatter_add_(1, at, slope)
    out["dz"] = dz.to(st["z"].dtype)
    return out


def _noise(n, seed):
    """16 random bits for each of two roundings of element i: its number, mixed with the seed."""
    low = 0xFFFFFFFF
    x = torch.arange(n, device="cuda")
    x = (x * 0x9E3779B9 + (x >> 32) * 0x3C6EF373 + seed) & low
    x = ((x ^ (x >> 16)) * 0x6A09E667) & low
    x = ((x ^ (x >> 15)) * 0xBB67AE85) & low
    x = x ^ (x >> 16)
    return x & 0xFFFF, x >> 16


def _to_code(x, noise, least):
    """x >= 0 up to 448 as e4m3, rounded up with the chance of what rounding down would leave."""
    small = x < 2.0 ** -6
    bits = torch.where(small, x + 2.0 ** -6, x).view(torch.int32) + (noise << 4).to(torch.int32)
    code = (bits >> 20) - torch.where(small, 968, 960).to(torch.int32)
    return torch.maximum(code.clamp(0, 126), least.to(torch.int32))


def _plain_adamw(st):
    c = st["case"]
    f32 = lambda v: float(np.float32(v))  # noqa: E731
    b1, b2, lr = f32(BETA1), f32(BETA2), f32(LR)
    o1, o2 = f32(1.0 - b1), f32(1.0 - b2)
    c1, c2 = 1.0 - b1 ** STEP, 1.0 - b2 ** STEP
    g = st["g"].float().view(-1, BLOCK)
    if c["bits"] == 32:
        m, v = st["m"].view(-1, BLOCK), st["v"].view(-1, BLOCK)
    else:
        m = st["m"].float().view(-1, BLOCK) * st["mscale"][:, None]
        v = st["v"].float().view(-1, BLOCK) * st["vscale"][:, None]
        v = v * v
    m = m * b1 + g * o1
    v = v * b2 + (g * g) * o2
    r = torch.sqrt(v)
    p = st["p"].view(-1, BLOCK)
    p = p * (1.0 - lr * st["decay"]) - f32(lr / c1) * (m / (r * f32(1.0 / math.sqrt(c2)) + f32(EPS)))
    st["p"].copy_(p.view(-1))
    st["copy"].copy_(st["p"])
    out = {"p": st["p"], "copy": st["copy"]}
    if c["bits"] == 32:
        st["m"].copy_(m.view(-1))
        st["v"].copy_(v.view(-1))
        return out | {"m": st["m"], "v": st["v"]}
    nm, nr = _noise(m.numel(), st["seed"])
    for name, x, noise, least in (("m", m, nm, torch.zeros_like(v)), ("v", r, nr, (v > 0))):
        top = x.abs().amax(1, keepdim=True).clamp_min(1e-30)
        st[name + "scale"].copy_((top / E4M3_MAX)[:, 0])
        y = x.abs() * torch.div(torch.full_like(top, E4M3_MAX), top)
        code = _to_code(y, noise.view(-1, BLOCK), least) + torch.where(x < 0, 128, 0)
        st[name].copy_(code.view(-1).to(torch.uint8).view(torch.float8_e4m3fn))
        out |= {name: st[name], name + "scale": st[name + "scale"]}
    return out


PLAIN = {"mix": _plain_mix, "prompt": _plain_mix, "step": _plain_mix, "policy": _plain_policy,
         "logp": _plain_policy, "adamw": _plain_adamw}


# --------------------------------------------------- the framework's calls --
def _own_mix(tw, st):
    c = st["case"]
    dt = tw.TWELL_BF16 if c["dtype"] == "bf16" else tw.TWELL_F32
    T, D, B = c["T"], c["D"], c["B"]
    if "x" not in st:  # the halves, and what a training step keeps from forward to backward
        st["x"], st["gate"], st["kept"] = st["xg"][:, :D], st["xg"][:, D:], None
        if c["kind"] == "mix":
            st["dx"], st["dgate"] = st["dxg"][:, :D], st["dxg"][:, D:]
            st["kept"] = torch.empty(tw.twell_recur_states(T), D, device="cuda")
    hT = st["h0"] if c["kind"] == "step" else st.get("hT")  # a decoded token's state: in place
    tw.twell_recur_forward(st["x"], st["gate"], 2 * D, st["bias"], st["starts"], B, st["h0"], T, D,
                           dt, st["h"], hT, st["kept"], st["status"])
    out = {"h": st["h"]}
    if hT is not None:
        out["hT"] = hT
    if c["kind"] == "mix":
        tw.twell_recur_backward(st["x"], st["gate"], 2 * D, st["bias"], st["starts"], B, st["h0"],
                                st["kept"], st["dh"], st.get("dhT"), T, D, dt, st["dx"],
                                st["dgate"], st["dbias"], st.get("dh0"), st["status"])
        out |= {"dxg": st["dxg"], "dbias": st["dbias"]}
        if c["state"]:
            out["dh0"] = st["dh0"]
    return out


def _own_policy(tw, st):
    c = st["case"]
    dt = tw.TWELL_BF16 if c["dtype"] == "bf16" else tw.TWELL_F32
    T, V = c["T"], c["V"]
    clip = (CLIP_LOW, CLIP_HIGH, BETA_KL)
    out = {"logp": st["logp"], "stats": st["stats"]}
    if c["kind"] == "logp":
        tw.twell_policy_forward(st["z"], V, st["tok"], None, None, None, st["weight"], T, V, dt,
                                st["tau"], *clip, None, st["logp"], st["stats"], None,
                                st["status"])
        return out
    tw.twell_policy_forward(st["z"], V, st["tok"], st["old"], st["ref"], st["adv"], st["weight"],
                            T, V, dt, st["tau"], *clip, st["loss"], st["logp"], st["stats"],
                            st["dz"] if c["fused"] else None, st["status"])
    if not c["fused"]:
        tw.twell_policy_backward(st["z"], V, st["tok"], st["old"], st["ref"], st["adv"],
                                 st["logp"], st["stats"], st["weight"], T, V, dt, st["tau"], *clip,
                                 st["dz"], st["status"])
    return out | {"loss": st["loss"], "dz": st["dz"]}


def _own_adamw(tw, st):
    c = st["case"]
    if "list" not in st:  # the list that a program keeps beside its tensors
        st["list"] = tw.AdamWTensors(c["bits"])
        for first, n, decay in st["table"]:
            part = slice(first, first + n)
            blocks = slice(first // BLOCK, first // BLOCK + -(-n // BLOCK))
            scales = (st["mscale"][blocks], st["vscale"][blocks]) if c["bits"] == 8 else ()
            st["list"].add(st["p"][part], st["g"][part], st["m"][part], st["v"][part], *scales,
                           copy=st["copy"][part], decay=decay, first=first)
    tw.twell_adamw_step(st["list"], LR, BETA1, BETA2, EPS, STEP, st["seed"])
    out = {"p": st["p"], "copy": st["copy"], "m": st["m"], "v": st["v"]}
    return out | {"mscale": st["mscale"], "vscale": st["vscale"]} if c["bits"] == 8 else out


OWN = {"mix": _own_mix, "prompt": _own_mix, "step": _own_mix, "policy": _own_policy,
       "logp": _own_policy, "adamw": _own_adamw}


def run(state):
    kind = state["case"]["kind"]
    if own:
        import activation_sparse_transformer_gate_gb300 as tw
        return OWN[kind](tw, state)
    return PLAIN[kind](state)


# ------------------------------------------------------------------- work --
def work(case):
    c = case
    if c["kind"] in ("mix", "prompt", "step"):
        n, es, state = c["T"] * c["D"], ES[c["dtype"]], 4 * c["B"] * c["D"] * c["state"]
        if c["kind"] == "mix":
            # forward: x, gate in, h out; backward: x, gate, dh in, dx, dgate out
            return {"bytes": 8 * n * es + 5 * state + 12 * c["D"], "flops": 50 * n}
        return {"bytes": 3 * n * es + 2 * state + 4 * c["D"], "flops": 14 * n}
    if c["kind"] in ("policy", "logp"):
        n, es = c["T"] * c["V"], ES[c["dtype"]]
        live = 0.875 if c["masked"] else 1.0  # masked rows are not read
        if c["kind"] == "logp":
            return {"bytes": n * es * live + 24 * c["T"], "flops": 4 * n}
        reads = 1 if c["fused"] else 2        # as two calls the logits are read by each
        return {"bytes": n * es * (live * reads + 1) + 40 * c["T"] * reads, "flops": 8 * n}
    n = sum(k for k, _ in _model(c))
    state = 16.0 if c["bits"] == 32 else 4.0 + 16.0 / BLOCK
    return {"bytes": n * (8 + ES[c["grad"]] + state + 2), "flops": 18 * n}


# ---------------------------------------------------------------- 64 bits --
def _exact_mix(st):
    c = st["case"]
    T, D, B = c["T"], c["D"], c["B"]
    bounds = list(range(T + 1)) if c["kind"] == "step" else st["starts"].tolist()
    x, f = st["xg"][:, :D].double(), st["xg"][:, D:].double() + st["bias"].double()
    a, w = 1.0 / (1.0 + torch.exp(-f)), 1.0 / (1.0 + torch.exp(f))
    h = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    state = torch.zeros(B, D, dtype=torch.float64, device="cuda")
    if st["h0"] is not None:
        state += st["h0"]
    if c["kind"] == "step":
        h = a * state + w * x
        return {"h": h, "hT": h}
    if c["kind"] == "prompt":
        return _exact_long(a, w * x, h, state, bounds)
    wx, h_init = w * x, state.clone()
    for s in range(B):
        now = state[s]
        for t in range(bounds[s], bounds[s + 1]):
            now = torch.addcmul(wx[t], a[t], now)
            h[t] = now
        state[s] = now
    out = {"h": h}
    if c["state"]:
        out["hT"] = state
    prev = torch.zeros_like(h)
    prev[1:] = h[:-1]
    G = torch.zeros_like(h)
    dh, d0 = st["dh"].double(), torch.zeros_like(h_init)
    for s in range(B):
        now = st["dhT"][s].double() if c["state"] else torch.zeros(D, dtype=torch.float64,
                                                                   device="cuda")
        for t in range(bounds[s + 1] - 1, bounds[s] - 1, -1):
            G[t] = dh[t] + now
            now = a[t] * G[t]
        d0[s] = now
        if bounds[s] < bounds[s + 1]:
            prev[bounds[s]] = h_init[s]
    dgate = G * (prev - x) * a * w
    out["dxg"] = torch.cat([w * G, dgate], dim=1)
    out["dbias"] = dgate.sum(0)
    if c["state"]:
        out["dh0"] = d0
    return out


def _exact_long(a, u, h, state, bounds):
    """The states of long sequences: pieces of 256 rows, all at once from zero and from one."""
    for s in range(len(bounds) - 1):
        i, j = bounds[s], bounds[s + 1]
        k = -(-(j - i) // 256)
        if k == 0:
            continue
        pad = k * 256 - (j - i)
        A = torch.nn.functional.pad(a[i:j], (0, 0, 0, pad), value=1.0).view(k, 256, -1)
        U = torch.nn.functional.pad(u[i:j], (0, 0, 0, pad)).view(k, 256, -1)
        own_, through = torch.zeros_like(A), torch.zeros_like(A)
        y, q = torch.zeros_like(A[:, 0]), torch.ones_like(A[:, 0])
        for t in range(256):
            y, q = A[:, t] * y + U[:, t], q * A[:, t]
            own_[:, t], through[:, t] = y, q
        now = state[s].clone()
        for p in range(k):
            own_[p] += through[p] * now
            now = own_[p, -1].clone()
        h[i:j] = own_.reshape(k * 256, -1)[:j - i]
        state[s] = now
    return {"h": h, "hT": state}


def _exact_policy(st):
    tau, got = st["tau"], {"logp": [], "stats": [], "loss": [], "dz": []}
    only = st["case"]["kind"] == "logp"
    for r in range(0, st["z"].shape[0], 1024):
        part = slice(r, r + 1024)
        z = st["z"][part].double()
        top = z.max(1).values
        z /= tau
        tok, w = st["tok"][part], st["weight"][part].double()
        w = torch.where(tok < 0, torch.zeros_like(w), w)
        live = (w != 0).double()
        pick = tok.clamp_min(0)[:, None]
        total = torch.logsumexp(z, dim=1)
        logp = z.gather(1, pick)[:, 0] - total
        got["logp"].append(logp * live)
        got["stats"].append(torch.stack([top, total - top / tau], 1) * live[:, None])
        if only:
            continue
        A, ratio = st["adv"][part].double(), torch.exp(logp - st["old"][part].double())
        d = st["ref"][part].double() - logp
        held = torch.minimum(torch.maximum(ratio, torch.full_like(ratio, 1 - CLIP_LOW)),
                             torch.full_like(ratio, 1 + CLIP_HIGH))
        flat = ((A > 0) & (ratio > 1 + CLIP_HIGH)) | ((A < 0) & (ratio < 1 - CLIP_LOW))
        won = torch.where(flat, held, ratio) * A
        got["loss"].append(w * (BETA_KL * (torch.expm1(d) - d) - won))
        slope = w * (-BETA_KL * torch.expm1(d) - torch.where(flat, 0.0, 1.0) * ratio * A) / tau
        dz = torch.softmax(z, dim=1).mul_(-slope[:, None])
        dz.scatter_add_(1, pick, slope[:, None])
        got["dz"].append(dz)
    return {k: torch.cat(v) for k, v in got.items() if v}


def _exact_adamw(st):
    c = st["case"]
    b1, b2, lr = (float(np.float32(v)) for v in (BETA1, BETA2, LR))
    eps = float(np.float32(EPS))
    out = {k: [] for k in ("p", "copy", "m", "v")}
    if c["bits"] == 8:
        out |= {"mscale": [], "vscale": []}
    total, piece = st["p"].numel(), 2 ** 27
    for at in range(0, total, piece):
        part, blk = slice(at, at + piece), slice(at // BLOCK, (at + piece) // BLOCK)
        g, m, v = (st[k][part].double().view(-1, BLOCK) for k in ("g", "m", "v"))
        if c["bits"] == 8:
            m, v = m * st["mscale"][blk].double()[:, None], v * st["vscale"][blk].double()[:, None]
            v = v.square()
        m = m * b1 + (1 - b1) * g
        v = v * b2 + (1 - b2) * g.square()
        size = m / (1 - b1 ** STEP) / (torch.sqrt(v / (1 - b2 ** STEP)) + eps)
        p = st["p"][part].double().view(-1, BLOCK)
        p = p - lr * st["decay"][blk].double() * p - lr * size
        out["p"].append(p.view(-1))
        out["copy"].append(out["p"][-1])
        if c["bits"] == 32:
            out["m"].append(m.view(-1))
            out["v"].append(v.view(-1))
            continue
        # stochastic rounding: to the value below, or above with the chance of the rest
        u = torch.arange(at, at + p.numel(), device="cuda")
        u = (u * 0x9E3779B9 + (u >> 32) * 0x3C6EF373 + st["seed"]) % 2 ** 32
        u = ((u ^ (u >> 16)) * 0x6A09E667) & 0xFFFFFFFF
        u = ((u ^ (u >> 15)) * 0xBB67AE85) & 0xFFFFFFFF
        u = (u ^ (u >> 16)).view(-1, BLOCK)
        for name, x, n16 in (("m", m, u % 65536), ("v", v.sqrt(), u // 65536)):
            top = x.abs().max(1, keepdim=True).values.clamp_min(1e-30)
            y = x.abs() * (E4M3_MAX / top)
            ulp = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
            q = torch.floor(y / ulp + n16.double() / 65536) * ulp
            if name == "v":
                q = torch.where(x > 0, q.clamp_min(2.0 ** -9), q)
            out[name].append((q.clamp_max(E4M3_MAX) * x.sign()).view(-1))
            out[name + "scale"].append((top / E4M3_MAX)[:, 0])
    return {k: torch.cat(v) for k, v in out.items()}


EXACT = {"mix": _exact_mix, "prompt": _exact_mix, "step": _exact_mix, "policy": _exact_policy,
         "logp": _exact_policy, "adamw": _exact_adamw}


def exact(case, seed):
    return EXACT[case["kind"]](prepare(case, seed))
