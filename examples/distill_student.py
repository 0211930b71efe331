"""A small language model around the activation-sparse FFN, trained by
distillation and served with an 8-bit output product.

    token ids -> embedding -> [ residual + norm -> recurrence -> (with --mix)
                                residual + norm -> sparse FFN ] x layers
              -> residual + norm -> logits -> distillation loss, or policy loss
              -> gradients -> AdamW

Every step of it is a call of the library but the matrix multiplications of the
output product and of the recurrence's inputs, and the sampling of --tune (torch).  Without --mix the student
sees one token at a time, so what it can learn is a table of next-token
distributions: the teacher here is such a table, of which each token gives its
largest logits.  With it a gated recurrence carries a state along each sequence.
--tune goes on with the policy loss: tokens are sampled, and a reward for even ones
moves the distribution, held by the KL term to the weights that it began with.

    python examples/distill_student.py [--steps N] [--mix] [--tune N] [--bits 8]
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
    tokens; everything is allocated here, once.  With ``mix``, ``starts`` (int32, on the device)
    are the sequences' first rows and the last one's end (None: one sequence)."""

    def __init__(self, T, V, D, F, layers, k, tau=1.0, lam=1e-5, pad_id=-1, seed=0, mix=False,
                 starts=None, bits=32):
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
            if mix:  # inputs and gates in one product; the bias spreads the channels' memories
                self.master |= {f"norm_mix{i}": torch.ones(D, device="cuda"),
                                f"mix{i}": w(2 * D, D, std=D ** -0.5),
                                f"bias_mix{i}": torch.linspace(0.0, 4.0, D, device="cuda")}
        f32 = torch.float32
        # (from 16-byte boundaries, as the optimizer wants them)
        self.grad = {n: torch.zeros_like(p) for n, p in self.master.items()}
        self.cast()
        self.adam = tw.AdamWTensors(bits)
        first = 0
        for n, p in self.master.items():
            blocks = -(-p.numel() // 256)
            state = [torch.zeros_like(p, dtype=f32 if bits == 32 else torch.float8_e4m3fn)
                     for _ in range(2)]
            scales = [torch.zeros(blocks, device="cuda") for _ in range(2)] if bits == 8 else []
            self.adam.add(p, self.grad[n], *state, *scales, first=first,
                          copy=self.p[n] if p.dim() == 2 else None)
            first += 256 * blocks
        self.step_no = 0
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
        self.mix, self.starts = mix, starts
        self.B = 1 if starts is None else starts.numel() - 1
        if mix:
            z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
            # (rows of no sequence are left as they are: zeros)
            self.s_mix, self.n_mix = ([empty(T, D) for _ in range(layers)] for _ in range(2))
            self.rstd_mix = [empty(T, dtype=f32) for _ in range(layers)]
            self.xg, self.h = [empty(T, 2 * D) for _ in range(layers)], [z(T, D) for _ in range(layers)]
            self.kept = [empty(tw.twell_recur_states(T), D, dtype=f32) for _ in range(layers)]
            self.dxg = z(T, 2 * D)

    def cast(self):
        """bf16 copies of the matrices (norm weights and biases stay fp32)."""
        self.p = {n: p.bfloat16() if p.dim() == 2 else p for n, p in self.master.items()}

    def frozen(self):
        """The weights as they are, for ``forward`` once they have moved on."""
        return {n: p.clone() for n, p in self.p.items()}

    def forward(self, tokens, p=None):
        """The final norm's rows; the residual stream and its norms stay in self.s, self.n.  ``p``:
        other weights than the present ones."""
        T, D, p = self.T, self.D, p or self.p
        tw.twell_embed_forward(tokens, p["embed"], T, self.V, D, BF16, self.scale, self.pad_id,
                               self.x0, self.status)
        for i in range(self.L + 1):
            name = f"norm{i}" if i < self.L else "norm_out"
            # the FFN's output joins the stream; the first layer reads the embedding itself
            x, res = (self.x0, None) if i == 0 else (self.y, self.s[i - 1])
            if self.mix and i < self.L:
                tw.twell_add_rmsnorm_forward(x, res, p[f"norm_mix{i}"], T, D, BF16, EPS,
                                             self.s_mix[i], self.n_mix[i], None, None,
                                             self.rstd_mix[i])
                xg = torch.matmul(self.n_mix[i], p[f"mix{i}"].t(), out=self.xg[i])
                tw.twell_recur_forward(xg[:, :D], xg[:, D:], 2 * D, p[f"bias_mix{i}"], self.starts,
                                       self.B, None, T, D, BF16, self.h[i], None, self.kept[i],
                                       self.status)
                x, res = self.h[i], self.s_mix[i]
            tw.twell_add_rmsnorm_forward(x, res, p[name], T, D, BF16, EPS, self.s[i], self.n[i],
                                         None, None, self.rstd[i])
            if i < self.L:
                tw.twell_ffn_forward(self.n[i], p[f"gate{i}"], p[f"bias{i}"], None, p[f"up{i}"],
                                     p[f"down{i}"], D, 1, self.act[i].t, self.y, self.ws_ffn,
                                     self.n_ffn)
        return self.n[self.L]

    def loss_and_gradients(self, tokens, ids, teacher, row_weight):
        """The rows' losses; the gradients of every weight are left in self.grad."""
        n = self.forward(tokens)
        z = n @ self.p["out"].t()
        # loss and gradient in one pass, the gradient in place of the logits
        tw.twell_distill_forward(z, self.V, ids, teacher, row_weight, self.T, self.V, self.k, BF16,
                                 self.tau, self.loss, self.stats, z, self.status)
        self.backward(tokens, n, z)
        return self.loss

    def log_probabilities(self, tokens, sampled, row_weight, p=None):
        """Of the sampled tokens, as the old and (of frozen weights) the reference policy's are
        taken."""
        z, logp = self.forward(tokens, p) @ (p or self.p)["out"].t(), torch.empty_like(self.loss)
        tw.twell_policy_forward(z, self.V, sampled, None, None, None, row_weight, self.T, self.V,
                                BF16, self.tau, 0.2, 0.2, 0.0, None, logp, self.stats, None,
                                self.status)
        return logp

    def policy_and_gradients(self, tokens, sampled, old, ref, advantage, row_weight, clip=0.2,
                             beta=0.05):
        """The same with the policy loss."""
        n = self.forward(tokens)
        z, logp = n @ self.p["out"].t(), torch.empty_like(self.loss)
        tw.twell_policy_forward(z, self.V, sampled, old, ref, advantage, row_weight, self.T, self.V,
                                BF16, self.tau, clip, clip, beta, self.loss, logp, self.stats, z,
                                self.status)
        self.backward(tokens, n, z)
        return self.loss

    def backward(self, tokens, n, dz):
        """From the logits' gradient to every weight's."""
        T, V, D, p, g = self.T, self.V, self.D, self.p, self.grad
        g["out"].copy_(dz.t() @ n)
        torch.matmul(dz, p["out"], out=self.dn)
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
            if self.mix and i < self.L:
                xg, dxg = self.xg[i], self.dxg
                tw.twell_recur_backward(xg[:, :D], xg[:, D:], 2 * D, p[f"bias_mix{i}"], self.starts,
                                        self.B, None, self.kept[i], ds, None, T, D, BF16,
                                        dxg[:, :D], dxg[:, D:], g[f"bias_mix{i}"], None, self.status)
                g[f"mix{i}"].copy_(dxg.t() @ self.n_mix[i])
                torch.matmul(dxg, p[f"mix{i}"], out=self.dn)
                tw.twell_add_rmsnorm_backward(self.s_mix[i], p[f"norm_mix{i}"], self.rstd_mix[i],
                                              self.dn, ds, T, D, BF16, ds, g[f"norm_mix{i}"],
                                              self.ws, self.n_ws)
        tw.twell_embed_backward(tokens, self.ds, T, V, D, BF16, self.scale, self.pad_id, g["embed"],
                                self.status, self.ws, self.n_ws)

    def update(self, lr):
        """One launch: every weight, its averages, and the matrices' bf16 copies."""
        self.step_no += 1
        tw.twell_adamw_step(self.adam, lr, 0.9, 0.99, 1e-8, self.step_no, seed=self.step_no)

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
        if student.mix:
            self.xg, self.h = empty(T, 2 * D), empty(T, D)
            self.state = [torch.zeros(T, D, device="cuda") for _ in range(student.L)]

    def logits(self, tokens):
        """Of the next tokens; with the recurrence, of T sequences that go on by one token each."""
        st, T, D = self.st, self.T, self.st.D
        tw.twell_embed_forward(tokens, st.p["embed"], T, st.V, D, BF16, st.scale, st.pad_id, self.x0,
                               st.status)
        x, res = self.x0, None
        for i in range(st.L):
            if st.mix:
                tw.twell_add_rmsnorm_forward(x, res, st.p[f"norm_mix{i}"], T, D, BF16, EPS, self.s,
                                             self.n, None, None, None)
                xg = torch.matmul(self.n, st.p[f"mix{i}"].t(), out=self.xg)
                tw.twell_recur_forward(xg[:, :D], xg[:, D:], 2 * D, st.p[f"bias_mix{i}"], None, T,
                                       self.state[i], T, D, BF16, self.h, self.state[i], None,
                                       st.status)
                x, res = self.h, self.s
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


def tune(student, steps, weight, g):
    """Policy steps, two on each batch of sampled tokens; a reward for the even ones.  The policy
    that sampled is the batch's, the reference the one that tuning began with."""
    reference = student.frozen()
    for step in range(0, steps, 2):
        tokens = torch.randint(0, student.V, (student.T,), generator=g, device="cuda")
        z = student.forward(tokens) @ student.p["out"].t()
        sampled = torch.multinomial(torch.softmax(z.float() / student.tau, dim=1), 1, generator=g)[:, 0]
        reward = (sampled % 2 == 0).float()
        advantage = reward - reward.mean()
        old = student.log_probabilities(tokens, sampled, weight)
        ref = student.log_probabilities(tokens, sampled, weight, reference)
        for _ in range(min(2, steps - step)):
            student.policy_and_gradients(tokens, sampled, old, ref, advantage, weight)
            student.update(lr=5e-4)
        student.check()
        print(f"tuned {step + 2:4d}  even tokens {100 * reward.mean().item():.0f}%", flush=True)


def main():
    ap = argparse.ArgumentParser(description=__doc__,
                                 formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--mix", action="store_true", help="a gated recurrence in every layer")
    ap.add_argument("--tune", type=int, default=0, help="steps with the policy loss")
    ap.add_argument("--bits", type=int, choices=(8, 32), default=32, help="of AdamW's averages")
    a = ap.parse_args()
    T, V, D, F, k = 4096, 1000, 256, 1024, 32
    starts = torch.arange(0, T + 1, 128, dtype=torch.int32, device="cuda") if a.mix else None
    teacher = Teacher(V, k)
    student = Student(T, V, D, F, layers=2, k=k, mix=a.mix, starts=starts, bits=a.bits)
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
    tune(student, a.tune, weight, g)
    tokens = torch.arange(64, device="cuda")
    z = Server(student, 64).logits(tokens)
    same = (z.argmax(dim=1) == teacher.table[tokens].argmax(dim=1)).float().mean().item()
    student.check()
    print(f"served in 8 bits: the teacher's first choice for {100 * same:.0f}% of the tokens")


if __name__ == "__main__":
    main()
