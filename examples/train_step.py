"""A small Mixture-of-Experts language model on the library's operators.

    embedding -> [norm -> router -> experts -> norm, gate, residual] x L -> norm -> cross entropy

with its backward, the clipping of all gradients by their global norm, and a
plain SGD update.  Between two expert layers one call of ``block_norm_forward``
does the norm after the first, its channel gate, the residual update and the
norm before the second.  The residual stream is fp32; activations and matrices
are bf16; the router's product is a small library GEMM in fp32.

    python examples/train_step.py [--steps 50] [--tokens 512]

trains on a synthetic sequence whose next token depends on the present one,
and then scores single tokens.
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mixture_experts_ffn_permute_gb300 as moe  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32


class MoELM:
    """Parameters, and the workspaces of one token count (made anew when it changes)."""

    def __init__(self, vocab=1000, hidden=256, ffn=256, experts=8, top_k=2, layers=2, seed=0,
                 device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def randn(*shape, std=1.0, dtype=BF):
            return (torch.randn(*shape, generator=g) * std).to(dtype).to(device)

        V, H, F, E = vocab, hidden, ffn, experts
        self.V, self.H, self.F, self.E, self.k, self.L = V, H, F, E, top_k, layers
        self.device = device
        p = self.params = {"embed": randn(V, H, std=0.5), "head": randn(V, H, std=H ** -0.5)}
        for i in range(layers):
            p[f"router{i}"] = randn(E, H, std=H ** -0.5, dtype=F32)
            p[f"w1_{i}"] = randn(E, 2 * F, H, std=H ** -0.5)
            p[f"w2_{i}"] = randn(E, H, F, std=F ** -0.5)
            p[f"post{i}"] = torch.ones(H, device=device)
            p[f"gate{i}"] = torch.full((H,), 0.5, device=device)
        for i in range(layers + 1):  # before every layer and before the head
            p[f"pre{i}"] = torch.ones(H, device=device)
        self.grads = {k: torch.empty_like(v) for k, v in p.items()}
        self.grad_list = moe.GradList(self.grads.values())
        self.clip_ws = moe.alloc_clip_workspace(self.grad_list, device)
        self.norm = torch.zeros(2, device=device)  # the gradients' norm, the factor applied
        self.T = -1

    def _plan(self, T):
        if T == self.T:
            return
        self.T, H, dev = T, self.H, self.device

        def empty(*shape, dtype=BF):
            return torch.empty(*shape, dtype=dtype, device=dev)

        self.p_embed = moe.EmbedProblem.make(T, self.V, H, BF, F32)
        self.p_norm = moe.NormProblem.make(T, H, BF, F32, F32, gate="channel")
        self.p_first = moe.NormProblem.make(T, H, BF, F32, F32)
        self.p_ce = moe.CEProblem.make(T, H, self.V)
        self.p_moe = moe.Problem.make(T, H, self.F, self.E, self.k)
        self.ws_embed = moe.alloc_embedding_workspace(self.p_embed, dev)
        self.ws_norm = moe.alloc_block_norm_workspace(self.p_norm, dev)
        self.ws_ce = moe.alloc_linear_ce_workspace(self.p_ce, backward=True, device=dev)
        self.ws_moe = moe.alloc_workspace(self.p_moe, dev)
        self.ws_moe_bwd = moe.alloc_backward_workspace(self.p_moe, dev)
        moe.clear_device_status(self.ws_moe)
        moe.clear_device_status(self.ws_moe_bwd)
        L = self.L
        self.r = [empty(T, H, dtype=F32) for _ in range(L + 1)]   # the residual stream
        self.n = [empty(T, H) for _ in range(L + 1)]              # normed
        self.y = [empty(T, H) for _ in range(L)]                  # the experts' outputs
        self.logits = [empty(T, self.E, dtype=F32) for _ in range(L)]
        self.topk = [torch.empty(T, self.k, dtype=torch.int32, device=dev) for _ in range(L)]
        self.loss, self.lse = empty(T, dtype=F32), empty(T, dtype=F32)
        self.dr, self.dn, self.dy, self.dx = (empty(T, H, dtype=F32), empty(T, H), empty(T, H),
                                              empty(T, H))
        self.dlogits = empty(T, self.E, dtype=F32)

    def forward(self, ids, labels):
        """Losses of the tokens [T] (0 where the label is negative); ids, labels int32 [T]."""
        self._plan(ids.numel())
        p = self.params
        moe.embedding_forward(self.p_embed, ids, p["embed"], self.r[0], ws=self.ws_embed)
        moe.block_norm_forward(self.p_first, self.r[0], w_pre=p["pre0"], normed=self.n[0])
        for i in range(self.L):
            torch.matmul(self.n[i].float(), p[f"router{i}"].t(), out=self.logits[i])
            moe.forward(self.p_moe, self.n[i], self.logits[i], p[f"w1_{i}"], p[f"w2_{i}"],
                        self.y[i], self.ws_moe, topk_idx=self.topk[i])
            moe.block_norm_forward(self.p_norm, self.r[i], branch=self.y[i], w_post=p[f"post{i}"],
                                   gate=p[f"gate{i}"], w_pre=p[f"pre{i + 1}"],
                                   residual_out=self.r[i + 1], normed=self.n[i + 1])
        moe.linear_ce_forward(self.p_ce, self.n[self.L], p["head"], labels, self.loss, self.lse,
                              self.ws_ce)
        return self.loss

    def backward(self, ids, labels, d_loss, max_norm=1.0):
        """All gradients (``self.grads``) for d_loss [T] fp32 and the forward just run, clipped to
        a global norm of ``max_norm``."""
        p, g, L = self.params, self.grads, self.L
        moe.linear_ce_backward(self.p_ce, self.n[L], p["head"], labels, self.lse, d_loss, self.dn,
                               g["head"], self.ws_ce)
        later = None  # gradient of the residual stream behind the last layer
        for i in reversed(range(L)):
            moe.block_norm_backward(self.p_norm, self.r[i + 1], self.dr, self.ws_norm,
                                    branch=self.y[i], w_post=p[f"post{i}"], gate=p[f"gate{i}"],
                                    w_pre=p[f"pre{i + 1}"], d_normed=self.dn,
                                    d_residual_out=later, d_branch=self.dy,
                                    d_w_post=g[f"post{i}"], d_gate=g[f"gate{i}"],
                                    d_w_pre=g[f"pre{i + 1}"])
            moe.backward(self.p_moe, self.n[i], self.logits[i], p[f"w1_{i}"], p[f"w2_{i}"],
                         self.dy, self.dx, g[f"w1_{i}"], g[f"w2_{i}"], self.ws_moe_bwd,
                         d_logits=self.dlogits)
            torch.matmul(self.dlogits.t(), self.n[i].float(), out=g[f"router{i}"])
            self.dn.copy_(self.dx.float() + self.dlogits @ p[f"router{i}"])
            later = self.dr
        moe.block_norm_backward(self.p_first, self.r[0], self.dr, self.ws_norm, w_pre=p["pre0"],
                                d_normed=self.dn, d_residual_out=later, d_w_pre=g["pre0"])
        moe.embedding_backward(self.p_embed, ids, self.dr, g["embed"], self.ws_embed)
        moe.clip_grad_norm(self.grad_list, max_norm, self.norm, self.clip_ws)

    def step(self, ids, labels, lr, max_norm=1.0):
        """One training step on the mean loss of the valid tokens; returns that loss (on the GPU)."""
        valid = (labels >= 0).sum().clamp(min=1).float()
        loss = self.forward(ids, labels).sum() / valid
        self.backward(ids, labels, (1.0 / valid).expand(ids.numel()).contiguous(), max_norm)
        for k, v in self.params.items():
            v.sub_((lr * self.grads[k].float()).to(v.dtype))
        return loss

    def status(self):
        """The first status other than MOE_OK that a kernel recorded, else MOE_OK."""
        for ws in (self.ws_embed, self.ws_ce, self.ws_moe, self.ws_moe_bwd):
            s = moe.get_device_status(ws)
            if s != moe.MOE_OK:
                return s
        return moe.MOE_OK


def batch(T, V, g, device="cuda"):
    """A sequence in which the next token is 7 x + 3 for three tokens in four, else any."""
    seq = [int(torch.randint(V, (1,), generator=g))]
    jump = (torch.rand(T, generator=g) < 0.25).tolist()
    rand = torch.randint(V, (T,), generator=g).tolist()
    for t in range(T):
        seq.append(rand[t] if jump[t] else (7 * seq[-1] + 3) % V)
    s = torch.tensor(seq, dtype=torch.int32, device=device)
    return s[:-1].contiguous(), s[1:].contiguous()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=50)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--lr", type=float, default=1.0)
    a = ap.parse_args()
    model = MoELM(vocab=200)
    g = torch.Generator().manual_seed(1)
    for i in range(a.steps):
        ids, labels = batch(a.tokens, model.V, g)
        loss = model.step(ids, labels, a.lr)
        if i % 10 == 0 or i + 1 == a.steps:
            print(f"step {i}: loss {float(loss):.3f} (uniform {math.log(model.V):.3f}), "
                  f"gradient norm {float(model.norm[0]):.3f}")
    ids, labels = batch(8, model.V, g)
    print("single tokens:", [round(float(model.forward(ids[t:t + 1], labels[t:t + 1])), 3)
                             for t in range(8)], "status", model.status())


if __name__ == "__main__":
    main()
