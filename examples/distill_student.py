"""A small language model around the activation-sparse FFN, trained by
distillation and served with an 8-bit output product.

    token ids -> embedding -> [ residual + norm -> sparse FFN ] x layers
              -> residual + norm -> logits -> distillation loss

Every step of it but the output product's matrix multiplications (torch) and
the optimizer is a call of the library.  The student sees one token at a time
(there is no attention), so what it can learn is a table of next-token
distributions: the teacher here is such a table, of which each token gives its
largest logits.

    python examples/distill_student.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import activation_sparse_transformer_gate_gb300 as tw  # noqa: E402

BF16 = tw.TWELL_BF16
EPS = 1e-6


def empty(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Teacher:
    """A fixed table of next-token logits; each token's k largest are what the student gets."""

    def __init__(self, V, k, seed=1):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.table = 2.0 * torch.randn(V, V, generator=g, device="cuda")
        top = torch.topk(self.table, k, dim=1)
        self.logits, self.ids = top.values.contiguous(), top.indices.to(torch.int32).contiguous()

    def of(self, tokens):
        return self.ids[tokens].contiguous(), self.logits[tokens].contiguous()


class Student:
    """The model's weights (fp32, with bf16 copies for the kernels) and the buffers of a step of T
    tokens; everything is allocated here, once."""

    def __init__(self, T, V, D, F, layers, k, tau=1.0, lam=1e-5, pad_id=-1, seed=0):
        self.T, self.V, self.D, self.F, self.L, self.k = T, V, D, F, layers, k
        self.tau, self.lam, self.pad_id, self.scale = tau, lam, pad_id, D ** 0.5
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)

        def w(*shape, std):
            return std * torch.randn(*shape, generator=g, device="cuda")

        self.master = {"embed": w(V, D, std=D ** -0.5), "out": w(V, D, std=D ** -0.5),
                       "norm_out": torch.ones(D, device="cuda")}
        for i in range(layers):
            self.master |= {f"norm{i}": torch.ones(D, device="cuda"),
                            f"gate{i}": w(F, D, std=D ** -0.5), f"up{i}": w(F, D, std=D ** -0.5),
                            f"down{i}": w(F, D, std=F ** -0.5),
                            f"bias{i}": torch.zeros(F, device="cuda")}
        f32 = torch.float32
        self.grad = {n: torch.zeros_like(p) for n, p in self.master.items()}
        self.adam = {n: (torch.zeros_like(p), torch.zeros_like(p)) for n, p in self.master.items()}
        self.step_no = 0
        self.cast()
        # activations kept for the backward
        self.s = [empty(T, D) for _ in range(layers + 1)]      # the residual stream
        self.n = [empty(T, D) for _ in range(layers + 1)]      # its norms
        self.rstd = [empty(T, dtype=f32) for _ in range(layers + 1)]
        self.y, self.x0 = empty(T, D), empty(T, D)
        self.act = [tw.TwellBuffers(T, F, 128, 8, BF16, train=True) for _ in range(layers)]
        self.ws_ffn, self.n_ffn = tw.workspace(T, D, F, 128, 8, BF16, True)
        n = max(tw.twell_embed_workspace_size(T, V, D), tw.twell_add_rmsnorm_workspace_size(T, D))
        self.ws, self.n_ws = empty(n, dtype=torch.uint8), n
        self.loss, self.stats = empty(T, dtype=f32), empty(T, 2, dtype=f32)
        self.ds, self.dn = empty(T, D), empty(T, D)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def cast(self):
        """bf16 copies of the matrices (norm weights and biases stay fp32)."""
        self.p = {n: p.bfloat16() if p.dim() == 2 else p for n, p in self.master.items()}

    def forward(self, tokens):
        """The final norm's rows; the residual stream and its norms stay in self.s, self.n."""
        T, D, p = self.T, self.D, self.p
        tw.twell_embed_forward(tokens, p["embed"], T, self.V, D, BF16, self.scale, self.pad_id,
                               self.x0, self.status)
        for i in range(self.L + 1):
            name = f"norm{i}" if i < self.L else "norm_out"
            # the FFN's output joins the stream; the first layer reads the embedding itself
            x, res = (self.x0, None) if i == 0 else (self.y, self.s[i - 1])
            tw.twell_add_rmsnorm_forward(x, res, p[name], T, D, BF16, EPS, self.s[i], self.n[i],
                                         None, None, self.rstd[i])
            if i < self.L:
                tw.twell_ffn_forward(self.n[i], p[f"gate{i}"], p[f"bias{i}"], None, p[f"up{i}"],
                                     p[f"down{i}"], D, 1, self.act[i].t, self.y, self.ws_ffn,
                                     self.n_ffn)
        return self.n[self.L]

    def loss_and_gradients(self, tokens, ids, teacher, row_weight):
        """The rows' losses; the gradients of every weight are left in self.grad."""
        T, V, D, p, g = self.T, self.V, self.D, self.p, self.grad
        n = self.forward(tokens)
        z = n @ p["out"].t()
        # loss and gradient in one pass, the gradient in place of the logits
        tw.twell_distill_forward(z, V, ids, teacher, row_weight, T, V, self.k, BF16, self.tau,
                                 self.loss, self.stats, z, self.status)
        g["out"] = (z.t() @ n).float()
        torch.matmul(z, p["out"], out=self.dn)
        ds = None
        for i in range(self.L, -1, -1):
            name = f"norm{i}" if i < self.L else "norm_out"
            if i < self.L:
                tw.twell_ffn_backward(self.n[i], p[f"gate{i}"], p[f"up{i}"], p[f"down{i}"],
                                      self.act[i].t, self.ds, self.lam, D, self.dn, g[f"gate{i}"],
                                      g[f"bias{i}"], g[f"up{i}"], g[f"down{i}"], self.ws_ffn,
                                      self.n_ffn)
            # what reaches the stream past the norm joins what comes through it
            tw.twell_add_rmsnorm_backward(self.s[i], p[name], self.rstd[i], self.dn, ds, T, D, BF16,
                                          self.ds, g[name], self.ws, self.n_ws)
            ds = self.ds
        tw.twell_embed_backward(tokens, self.ds, T, V, D, BF16, self.scale, self.pad_id, g["embed"],
                                self.status, self.ws, self.n_ws)
        return self.loss

    def update(self, lr):
        self.step_no += 1
        for n, p in self.master.items():
            m, v = self.adam[n]
            m.mul_(0.9).add_(self.grad[n], alpha=0.1)
            v.mul_(0.99).addcmul_(self.grad[n], self.grad[n], value=0.01)
            mh, vh = m / (1 - 0.9 ** self.step_no), v / (1 - 0.99 ** self.step_no)
            p.addcdiv_(mh, vh.sqrt().add_(1e-8), value=-lr)
        self.cast()

    def check(self):
        """Raises for what only the device could see (an id out of range, a full capacity)."""
        codes = [tw.twell_read_status(self.status)] + [tw.twell_get_status(a.t)[0] for a in self.act]
        for c in codes:
            if c != tw.TWELL_OK:
                raise tw.TwellError(c, "student")


class Server:
    """Logits with the output product in 8 bits: its weights are laid out once."""

    def __init__(self, student, T):
        self.st, self.T = student, T
        V, D = student.V, student.D
        self.wq, self.wscale = empty(V, D, dtype=torch.int8), empty(V, dtype=torch.float32)
        tw.twell_q8_quantize(student.p["out"], V, D, BF16, self.wq, self.wscale)
        self.x0, self.y = empty(T, D), empty(T, D)
        self.s, self.n = empty(T, D), empty(T, D)
        self.q, self.qscale = empty(T, D, dtype=torch.int8), empty(T, dtype=torch.float32)
        self.act = tw.TwellBuffers(T, student.F, 128, 8, BF16)
        self.ws_ffn, self.n_ffn = tw.workspace(T, D, student.F, 128, 8, BF16, False)
        self.n_ws = tw.twell_q8_workspace_size(T, V, D)
        self.ws = empty(max(self.n_ws, 1), dtype=torch.uint8)
        self.z = empty(T, V)

    def logits(self, tokens):
        st, T, D = self.st, self.T, self.st.D
        tw.twell_embed_forward(tokens, st.p["embed"], T, st.V, D, BF16, st.scale, st.pad_id, self.x0,
                               st.status)
        x, res = self.x0, None
        for i in range(st.L):
            tw.twell_add_rmsnorm_forward(x, res, st.p[f"norm{i}"], T, D, BF16, EPS, self.s, self.n,
                                         None, None, None)
            tw.twell_ffn_forward(self.n, st.p[f"gate{i}"], st.p[f"bias{i}"], None, st.p[f"up{i}"],
                                 st.p[f"down{i}"], D, 0, self.act.t, self.y, self.ws_ffn, self.n_ffn)
            x, res = self.y, self.s
        tw.twell_add_rmsnorm_forward(x, res, st.p["norm_out"], T, D, BF16, EPS, self.s, None, self.q,
                                     self.qscale, None)
        tw.twell_q8_matmul(self.q, self.qscale, self.wq, self.wscale, None, T, st.V, D, BF16, self.z,
                           st.status, self.ws, self.n_ws)
        return self.z


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    a = ap.parse_args()
    T, V, D, F, k = 4096, 1000, 256, 1024, 32
    teacher, student = Teacher(V, k), Student(T, V, D, F, layers=2, k=k)
    weight = torch.full((T,), 1.0 / T, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    for step in range(a.steps):
        tokens = torch.randint(0, V, (T,), generator=g, device="cuda")
        loss = student.loss_and_gradients(tokens, *teacher.of(tokens), weight)
        student.update(lr=2e-3)
        if step % 20 == 0 or step == a.steps - 1:
            student.check()
            print(f"step {step:4d}  loss {loss.sum().item():.4f}", flush=True)
    tokens = torch.arange(64, device="cuda")
    z = Server(student, 64).logits(tokens)
    same = (z.argmax(dim=1) == teacher.table[tokens].argmax(dim=1)).float().mean().item()
    student.check()
    print(f"served in 8 bits: the teacher's first choice for {100 * same:.0f}% of the tokens")


if __name__ == "__main__":
    main()
