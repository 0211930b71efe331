"""The operators that stand around the sparse feed-forward layer in a language
model, as a user's program calls them: the token embedding and its gradient,
the residual addition with the root-mean-square norm (forward and backward, or
with an 8-bit output), the 8-bit product that reads that output, and the
distillation loss against a teacher's top logits with its gradient.

``run`` computes a case in plain torch operations (in 32 bits, rounded once at
the end) or, where ``own`` is true, with the framework's kernels.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}
EPS = 1e-6


# ------------------------------------------------------------------ cases --
def listed():
    return [
        # the framework's smallest configuration (64 tokens, d_model 128, fp32) with a
        # vocabulary of characters: latency counts
        dict(name="embed 64x128 V512 f32", kind="embed", T=64, V=512, D=128, dtype="f32", pad=False),
        # one training step's tokens at the base d_model; an odd vocabulary, padded sequences
        dict(name="embed 4096x2048 V50001", kind="embed", T=4096, V=50001, D=2048, dtype="bf16",
             pad=True),
        # the large configuration: long batch, large vocabulary, the gradient table is 2.1 GB
        dict(name="embed 16384x4096 V131072", kind="embed", T=16384, V=131072, D=4096,
             dtype="bf16", pad=False),
        # residual + norm of a training step at the base d_model, forward and backward
        dict(name="norm 4096x2048", kind="norm", T=4096, D=2048, dtype="bf16"),
        # the same at the long batch and the large d_model
        dict(name="norm 16384x4096", kind="norm", T=16384, D=4096, dtype="bf16"),
        # one decoded token: residual + norm to 8 bits, then a d_model -> d_ff projection
        dict(name="project 1x2048 N8192", kind="project", T=1, D=2048, N=8192, dtype="bf16"),
        # a ragged batch of decoded tokens through the large projection
        dict(name="project 37x4096 N14336", kind="project", T=37, D=4096, N=14336, dtype="bf16"),
        # logits of an odd number of tokens over an odd vocabulary, 8-bit inputs in hand
        dict(name="q8 1001x2048 N50001", kind="q8", T=1001, D=2048, N=50001, dtype="bf16"),
        # a long prompt batch through the large projection
        dict(name="project 8192x4096 N14336", kind="project", T=8192, D=4096, N=14336,
             dtype="bf16"),
        # the smallest configuration's loss
        dict(name="distill 64xV512 k8 f32", kind="distill", T=64, V=512, k=8, dtype="f32",
             fused=True, masked=False),
        # a training step with the loss and its gradient as two calls (autograd's order);
        # odd vocabulary, ragged teacher lists, an eighth of the rows masked
        dict(name="distill 2048xV50001 k64", kind="distill", T=2048, V=50001, k=64, dtype="bf16",
             fused=False, masked=True),
        # a large vocabulary: the loss and its gradient in one call
        dict(name="distill 8192xV131072 k128", kind="distill", T=8192, V=131072, k=128,
             dtype="bf16", fused=True, masked=False),
    ]


def _log_int(rng, lo, hi, mult=1):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return max(mult, min(hi, max(lo, v)) // mult * mult)


def draw(rng):
    kind = rng.choice(["embed", "norm", "project", "q8", "distill"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "embed":
        V = _log_int(rng, 100, 131072)
        return dict(kind=kind, T=_log_int(rng, 1, 16384), V=V,
                    D=_log_int(rng, 64, 4096, 8), dtype=dtype, pad=rng.random() < 0.5)
    if kind == "norm":
        D = _log_int(rng, 64, 8192 if dtype == "bf16" else 4096, 8)
        return dict(kind=kind, T=_log_int(rng, 1, min(16384, 16384 * 4096 // D // (ES[dtype] // 2))),
                    D=D, dtype=dtype)
    if kind in ("project", "q8"):
        T, D = _log_int(rng, 1, 8192), _log_int(rng, 128, 8192, 16)
        most = 8192 * 4096 * 14336 // (T * D)
        return dict(kind=kind, T=T, D=D, N=_log_int(rng, 64, max(65, min(50001, most))),
                    dtype="bf16" if kind == "project" else dtype)
    V = _log_int(rng, 100, 131072)
    most = min(8192, 8192 * 131072 // (V * ES[dtype] // 2))
    return dict(kind=kind, T=_log_int(rng, 1, most), V=V, k=_log_int(rng, 1, min(128, V)),
                dtype=dtype, fused=rng.random() < 0.5, masked=rng.random() < 0.5)


# ----------------------------------------------------------------- inputs --
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, dtype=torch.float32, scale=1.0):
    return torch.randn(*shape, generator=g, device="cuda", dtype=dtype) * scale


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _inputs_embed(c, g):
    T, V, D, dt = c["T"], c["V"], c["D"], DT[c["dtype"]]
    # Zipf's law: the chance of a token falls as one over its rank
    tok = (torch.exp(_rand(g, T).double() * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1)
    pad_id = -1
    if c["pad"]:  # the tails of four sequences are padding
        pad_id = 0
        n = max(1, T // 4)
        at = torch.arange(T, device="cuda") % n
        tok = torch.where(at >= n - n // 8, torch.zeros_like(tok), tok)
    return dict(tok=tok, pad_id=pad_id, scale=math.sqrt(D),
                table=_randn(g, V, D, dtype=dt, scale=0.02), dy=_randn(g, T, D, dtype=dt),
                out=torch.empty(T, D, dtype=dt, device="cuda"),
                dtable=torch.empty(V, D, dtype=torch.float32, device="cuda"),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


def _hidden(g, T, D, dt):
    """Rows of a residual stream: scales differ by token, a few channels are large."""
    row = torch.exp(_randn(g, T, 1, scale=0.5))
    col = torch.where(_rand(g, D) < 0.01, 8.0, 1.0)
    return (_randn(g, T, D) * row * col).to(dt)


def _inputs_norm(c, g):
    T, D, dt = c["T"], c["D"], DT[c["dtype"]]
    e = lambda *s, d=dt: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
    return dict(x=_randn(g, T, D, dtype=dt), res=_hidden(g, T, D, dt),
                w=1.0 + _randn(g, D, scale=0.1), dy=_randn(g, T, D, dtype=dt),
                ds=_randn(g, T, D, dtype=dt),
                s=e(T, D), y=e(T, D), rstd=e(T, d=torch.float32), dx=e(T, D),
                dw=e(D, d=torch.float32))


def _inputs_project(c, g):
    T, D, N, dt = c["T"], c["D"], c["N"], DT[c["dtype"]]
    e = lambda *s, d=dt: torch.empty(*s, dtype=d, device="cuda")  # noqa: E731
    # weights in 8 bits with a scale for each output channel; the products come out near one
    wq = torch.randint(-127, 128, (N, D), generator=g, device="cuda", dtype=torch.int8)
    wscale = (0.5 + _rand(g, N)) / (127.0 * math.sqrt(D))
    st = dict(wq=wq, wscale=wscale, y=e(T, N),
              status=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if c["kind"] == "project":
        st |= dict(x=_randn(g, T, D, dtype=dt), res=_hidden(g, T, D, dt),
                   w=1.0 + _randn(g, D, scale=0.1), s=e(T, D), q=e(T, D, d=torch.int8),
                   qscale=e(T, d=torch.float32))
    else:
        a = _hidden(g, T, D, torch.float32)
        top = a.abs().amax(dim=1, keepdim=True).clamp_min(1e-20)
        st |= dict(q=torch.round(a * (127.0 / top)).to(torch.int8), qscale=top[:, 0] / 127.0,
                   bias=_randn(g, N, scale=0.1))
    return st


def _inputs_distill(c, g):
    T, V, k, dt = c["T"], c["V"], c["k"], DT[c["dtype"]]
    z = _randn(g, T, V, dtype=dt, scale=2.5)
    start = (_rand(g, T, 1) * V).long()
    step = 1 + (_rand(g, T, 1) * (V // k)).long().clamp_max(V // k - 1)
    ids = ((start + step * torch.arange(k, device="cuda")) % V).to(torch.int32)
    teacher = torch.sort(_randn(g, T, k, scale=3.0), dim=1, descending=True).values
    weight = torch.full((T,), 1.0 / T, device="cuda")
    if c["masked"]:  # lists cut by the teacher's nucleus (some to nothing); prompt rows masked
        n = (_rand(g, T, 1) * (k + 1)).long()
        ids = torch.where(torch.arange(k, device="cuda") < n, ids, torch.full_like(ids, -1))
        weight = torch.where(_rand(g, T) < 0.125, torch.zeros_like(weight), weight)
    f = lambda *s: torch.empty(*s, dtype=torch.float32, device="cuda")  # noqa: E731
    return dict(z=z, ids=ids.contiguous(), teacher=teacher, weight=weight, tau=2.0,
                loss=f(T), stats=f(T, 2), dz=torch.empty_like(z),
                status=torch.zeros(1, dtype=torch.int32, device="cuda"))


INPUTS = {"embed": _inputs_embed, "norm": _inputs_norm, "project": _inputs_project,
          "q8": _inputs_project, "distill": _inputs_distill}


def prepare(case, seed):
    st = INPUTS[case["kind"]](case, _gen(seed))
    st["case"] = case
    return st


# ------------------------------------------------------------ plain forms --
def _plain_embed(st):
    c = st["case"]
    live = st["tok"] != st["pad_id"]
    at = torch.where(live, st["tok"], torch.zeros_like(st["tok"]))
    m = live[:, None].float() * st["scale"]
    out = (st["table"][at].float() * m).to(DT[c["dtype"]])
    dtable = torch.zeros(c["V"], c["D"], dtype=torch.float32, device="cuda")
    dtable.index_add_(0, at, st["dy"].float() * m)
    return {"out": out, "dtable": dtable}


def _plain_sum(st):
    # the residual stream is stored in its type, and the norm reads what is stored
    s = (st["x"].float() + st["res"].float()).to(st["x"].dtype)
    return s, s.float()


def _plain_norm(st):
    dt = DT[st["case"]["dtype"]]
    s, sf = _plain_sum(st)
    rstd = torch.rsqrt(sf.square().mean(dim=1, keepdim=True) + EPS)
    xhat = sf * rstd
    y = (xhat * st["w"]).to(dt)
    dy = st["dy"].float()
    wdy = dy * st["w"]
    dx = st["ds"].float() + rstd * (wdy - xhat * (wdy * xhat).mean(dim=1, keepdim=True))
    return {"s": s, "y": y, "dx": dx.to(dt), "dw": (dy * xhat).sum(dim=0)}


def _plain_project(st):
    c = st["case"]
    dt = DT[c["dtype"]]
    out = {}
    if c["kind"] == "project":
        out["s"], sf = _plain_sum(st)
        h = sf * torch.rsqrt(sf.square().mean(dim=1, keepdim=True) + EPS) * st["w"]
        top = h.abs().amax(dim=1, keepdim=True)
        q, scale = torch.round(h * (127.0 / top)), top / 127.0
    else:
        q, scale = st["q"].float(), st["qscale"][:, None]
    y = torch.matmul(q, st["wq"].float().t()) * scale * st["wscale"]
    if "bias" in st:
        y = y + st["bias"]
    out["y"] = y.to(dt)
    return out


def _plain_distill(st):
    tau, ids = st["tau"], st["ids"].long()
    z = st["z"].float()
    top = z.amax(dim=1, keepdim=True)
    z = (z - top) / tau
    lse = torch.log(torch.exp(z).sum(dim=1, keepdim=True))
    live, on = ids >= 0, st["weight"] != 0
    at = torch.where(live, ids, torch.zeros_like(ids))
    t = torch.where(live, st["teacher"] / tau, torch.full_like(st["teacher"], -math.inf))
    any_ = live.any(dim=1, keepdim=True)
    big = torch.where(any_, t.amax(dim=1, keepdim=True), torch.zeros_like(lse))
    p = torch.exp(t - big)
    total = torch.where(any_, p.sum(dim=1, keepdim=True), torch.ones_like(lse))
    p = p / total
    logp = torch.where(live, t - big - torch.log(total), torch.zeros_like(p))
    kl = (p * (logp - (z.gather(1, at) - lse))).sum(dim=1)
    loss = st["weight"] * tau * tau * kl
    g = torch.where(any_, st["weight"][:, None], torch.zeros_like(lse))
    dz = torch.exp(z - lse).scatter_add_(1, at, -p) * (tau * g)
    stats = torch.cat([top, lse], dim=1) * on[:, None]
    return {"loss": loss, "stats": stats, "dz": dz.to(st["z"].dtype)}


PLAIN = {"embed": _plain_embed, "norm": _plain_norm, "project": _plain_project,
         "q8": _plain_project, "distill": _plain_distill}


# --------------------------------------------------- the framework's calls --
def _scratch(st, nbytes):
    """The workspace that a program keeps beside its buffers (allocated by the first pass)."""
    if "ws" not in st:
        st["ws"] = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
        st["nws"] = nbytes
    return st["ws"], st["nws"]


def _own_embed(tw, st):
    c = st["case"]
    dt = tw.TWELL_BF16 if c["dtype"] == "bf16" else tw.TWELL_F32
    T, V, D = c["T"], c["V"], c["D"]
    ws = st.get("ws")
    if ws is None:
        ws, _ = _scratch(st, tw.twell_embed_workspace_size(T, V, D))
    tw.twell_embed_forward(st["tok"], st["table"], T, V, D, dt, st["scale"], st["pad_id"],
                           st["out"], st["status"])
    tw.twell_embed_backward(st["tok"], st["dy"], T, V, D, dt, st["scale"], st["pad_id"],
                            st["dtable"], st["status"], ws, st["nws"])
    return {"out": st["out"], "dtable": st["dtable"]}


def _own_norm(tw, st):
    c = st["case"]
    dt = tw.TWELL_BF16 if c["dtype"] == "bf16" else tw.TWELL_F32
    T, D = c["T"], c["D"]
    ws = st.get("ws")
    if ws is None:
        ws, _ = _scratch(st, tw.twell_add_rmsnorm_workspace_size(T, D))
    tw.twell_add_rmsnorm_forward(st["x"], st["res"], st["w"], T, D, dt, EPS, st["s"], st["y"],
                                 None, None, st["rstd"])
    tw.twell_add_rmsnorm_backward(st["s"], st["w"], st["rstd"], st["dy"], st["ds"], T, D, dt,
                                  st["dx"], st["dw"], ws, st["nws"])
    return {"s": st["s"], "y": st["y"], "dx": st["dx"], "dw": st["dw"]}


def _own_project(tw, st):
    c = st["case"]
    dt = tw.TWELL_BF16 if c["dtype"] == "bf16" else tw.TWELL_F32
    T, D, N = c["T"], c["D"], c["N"]
    ws = st.get("ws")
    if ws is None:
        ws, _ = _scratch(st, tw.twell_q8_workspace_size(T, N, D))
    out = {}
    if c["kind"] == "project":
        tw.twell_add_rmsnorm_forward(st["x"], st["res"], st["w"], T, D, dt, EPS, st["s"], None,
                                     st["q"], st["qscale"], None)
        out["s"] = st["s"]
    tw.twell_q8_matmul(st["q"], st["qscale"], st["wq"], st["wscale"], st.get("bias"), T, N, D, dt,
                       st["y"], st["status"], ws, st["nws"])
    out["y"] = st["y"]
    return out


def _own_distill(tw, st):
    c = st["case"]
    dt = tw.TWELL_BF16 if c["dtype"] == "bf16" else tw.TWELL_F32
    T, V, k = c["T"], c["V"], c["k"]
    tw.twell_distill_forward(st["z"], V, st["ids"], st["teacher"], st["weight"], T, V, k, dt,
                             st["tau"], st["loss"], st["stats"], st["dz"] if c["fused"] else None,
                             st["status"])
    if not c["fused"]:
        tw.twell_distill_backward(st["z"], V, st["ids"], st["teacher"], st["stats"], st["weight"],
                                  T, V, k, dt, st["tau"], st["dz"], st["status"])
    return {"loss": st["loss"], "stats": st["stats"], "dz": st["dz"]}


OWN = {"embed": _own_embed, "norm": _own_norm, "project": _own_project, "q8": _own_project,
       "distill": _own_distill}


def run(state):
    kind = state["case"]["kind"]
    if own:
        import activation_sparse_transformer_gate_gb300 as tw
        return OWN[kind](tw, state)
    return PLAIN[kind](state)


# ------------------------------------------------------------------- work --
def work(case):
    c, es = case, ES[case["dtype"]]
    T = c["T"]
    if c["kind"] == "embed":
        V, D = c["V"], c["D"]
        p = np.diff(np.log(np.arange(1, V + 2))) / math.log(V + 1.0)
        rows = float(np.sum(-np.expm1(T * np.log1p(-p))))  # rows of the table that are looked up
        # forward: tokens, rows, out; backward: tokens, dy, the whole fp32 gradient
        return {"bytes": 16 * T + rows * D * es + 2 * T * D * es + 4 * V * D, "flops": 2 * T * D}
    if c["kind"] == "norm":
        # forward: x, residual in, s, y out; backward: s, dy, ds in, dx out; w twice, dw
        return {"bytes": 8 * T * c["D"] * es + 12 * c["D"] + 8 * T, "flops": 20 * T * c["D"]}
    if c["kind"] in ("project", "q8"):
        D, N = c["D"], c["N"]
        first = 3 * T * D * es + 4 * D if c["kind"] == "project" else T * D + 4 * T + 4 * N
        return {"bytes": first + N * D + 4 * N + T * N * es, "flops": 2.0 * T * N * D}
    V, k = c["V"], c["k"]
    live = 0.875 if c["masked"] else 1.0  # masked rows are not read
    reads = 1 if c["fused"] else 2        # as two calls the logits are read by each
    return {"bytes": T * V * es * (live * reads + 1) + T * k * 8 * reads + 16 * T,
            "flops": 8 * T * V}


# ---------------------------------------------------------------- 64 bits --
def _exact_embed(st):
    c = st["case"]
    V, D = c["V"], c["D"]
    keep = (st["tok"] != st["pad_id"]).nonzero()[:, 0]
    tok = st["tok"][keep]
    out = torch.zeros(c["T"], D, dtype=torch.float64, device="cuda")
    out[keep] = torch.index_select(st["table"], 0, tok).double() * st["scale"]
    # sums of runs of the sorted tokens
    order = torch.argsort(tok, stable=True)
    rows = torch.cumsum(st["dy"][keep][order].double(), dim=0)
    ids, count = torch.unique_consecutive(tok[order], return_counts=True)
    rows = rows[torch.cumsum(count, 0) - 1]
    rows[1:] -= rows[:-1].clone()
    dtable = torch.zeros(V, D, dtype=torch.float64, device="cuda")
    dtable[ids] = rows * st["scale"]
    return {"out": out, "dtable": dtable}


def _exact_hat(st):
    s = (st["x"].double() + st["res"].double()).to(st["x"].dtype)
    d = s.double()
    return s, d / torch.sqrt((d * d).sum(1, keepdim=True) / d.shape[1] + EPS)


def _exact_norm(st):
    s, hat = _exact_hat(st)
    d, w = s.double(), st["w"].double()
    r = 1.0 / torch.sqrt((d * d).sum(1, keepdim=True) / d.shape[1] + EPS)
    g = st["dy"].double()
    inner = torch.einsum("td,td->t", g * w, d)[:, None]
    dx = st["ds"].double() + g * w * r - d * inner * r ** 3 / d.shape[1]
    return {"s": s.double(), "y": hat * w, "dx": dx, "dw": torch.einsum("td,td->d", g, hat)}


def _exact_project(st):
    out = {}
    if st["case"]["kind"] == "project":
        s, hat = _exact_hat(st)
        h = hat * st["w"].double()
        scale = h.abs().max(1).values / 127.0
        a = torch.round(h / scale[:, None])
        out["s"] = s.double()
    else:
        a, scale = st["q"].double(), st["qscale"].double()
    w = st["wq"].double()
    y = torch.einsum("tk,nk->tn", a, w)
    y *= scale[:, None]
    y *= st["wscale"].double()
    if "bias" in st:
        y += st["bias"].double()
    out["y"] = y
    return out


def _exact_distill(st):
    tau = st["tau"]
    loss, stats, dz = [], [], []
    for r in range(0, st["z"].shape[0], 1024):
        z = st["z"][r:r + 1024].double()
        top = z.max(1).values
        z /= tau
        w = st["weight"][r:r + 1024].double()
        ids = st["ids"][r:r + 1024].long()
        t = (st["teacher"][r:r + 1024].double() / tau).masked_fill(ids < 0, -math.inf)
        p = torch.softmax(t, dim=1).nan_to_num(0.0)  # a list of nothing: no teacher
        logp = torch.log_softmax(t, dim=1)
        total = torch.logsumexp(z, dim=1)
        full = torch.zeros_like(z)
        full.scatter_add_(1, ids.clamp_min(0), p)
        has = (ids >= 0).any(1).double()
        logq = z.gather(1, ids.clamp_min(0)) - total[:, None]
        loss.append(w * tau * tau * torch.where(p > 0, p * (logp - logq), 0.0).sum(1))
        both = torch.stack([top, total - top / tau], dim=1)
        stats.append(torch.where(w[:, None] != 0, both, 0.0))
        dz.append((w * has * tau)[:, None] * (torch.softmax(z, dim=1) - full))
    return {"loss": torch.cat(loss), "stats": torch.cat(stats), "dz": torch.cat(dz)}


EXACT = {"embed": _exact_embed, "norm": _exact_norm, "project": _exact_project,
         "q8": _exact_project, "distill": _exact_distill}


def exact(case, seed):
    return EXACT[case["kind"]](prepare(case, seed))
