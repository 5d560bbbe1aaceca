"""A tensor-parallel training step on virtual ranks, run with the library.

    python examples/tp_train_step.py [--ranks 4] [--tokens 512] [--hidden 1024] [--width 704]
                                     [--vocab 8192] [--steps 20] [--graph] [--check]

One block of a tensor-parallel model, every weight matrix split over the
ranks: row-parallel input projection, all-reduce + RMSNorm (sum saved in 8
bits), column-parallel gated feed-forward, row-parallel output projection,
all-reduce + RMSNorm, vocabulary-parallel softmax cross entropy; then the
backward pass, in which the feed-forward's input is restored from its 8-bit
checkpoint instead of being kept.  The row-parallel products are plain
torch.matmul; everything between them is the library.

It learns a fixed permutation of the vocabulary from embeddings that stay as
they are.  --graph captures the step into a CUDA graph; --check compares the
first step's gradients with autograd in float32.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import collective_all_reduce_rank_gb300 as rra  # noqa: E402

EPS = 1e-6


class Step:
    """Weights, activations and workspace of the block; buffers are made once."""

    def __init__(self, ranks=4, tokens=512, hidden=1024, width=704, vocab=8192, lr=0.5, seed=0):
        rra.rra_init(0)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        n, T, D, F, V = ranks, tokens, hidden, width, vocab
        self.n, self.T, self.D, self.F, self.V, self.lr = n, T, D, F, V, lr
        bf = dict(dtype=torch.bfloat16, device="cuda")

        def weight(*shape, scale):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)

        per = -(-V // n)
        self.shards = [max(0, min(V, (r + 1) * per) - r * per) for r in range(n)]
        self.emb = weight(V, D, scale=1.0)
        cut = [D * r // n for r in range(n + 1)]  # rank r's columns of the input projection
        self.cut = cut
        self.p = {
            "proj": [weight(D, cut[r + 1] - cut[r], scale=D ** -0.5) for r in range(n)],
            "gate": [weight(F, D, scale=D ** -0.5) for _ in range(n)],
            "up": [weight(F, D, scale=D ** -0.5) for _ in range(n)],
            "down": [weight(D, F, scale=(F * n) ** -0.5) for _ in range(n)],
            "head": [weight(v, D, scale=D ** -0.5) for v in self.shards],
            "gamma1": [torch.ones(D, **bf)], "gamma2": [torch.ones(D, **bf)],
        }
        self.g = {k: [torch.zeros_like(w, dtype=torch.float32 if k[0:5] == "gamma" else w.dtype) for w in ws]
                  for k, ws in self.p.items()}
        self.next = torch.randperm(V, generator=gen, device="cuda")  # what follows each token
        self.ids = torch.zeros(T, dtype=torch.int64, device="cuda")
        self.targets = torch.zeros(T, dtype=torch.int64, device="cuda")
        self.gen = gen

        def act(cols):
            return torch.empty(T, cols, **bf)

        def saved():  # what a norm keeps for the backward pass
            return (torch.empty(T, D, dtype=torch.float8_e4m3fn, device="cuda"),
                    torch.empty(T, -(-D // 128), dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda"))

        self.part = [act(D) for _ in range(n)]
        self.h1, self.h2 = [act(D) for _ in range(n)], [act(D) for _ in range(n)]
        self.keep1, self.keep2 = saved(), saved()
        self.acts, self.dacts = [act(F) for _ in range(n)], [act(F) for _ in range(n)]
        self.again, self.dh, self.ds = act(D), act(D), act(D)
        self.loss, self.lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
        self.grad = torch.full((T,), 1.0 / T, device="cuda")
        need = max(rra.rra_gated_ffn_workspace_bytes(n, T, D, F, True),
                   rra.rra_vocab_loss_workspace_bytes(T, D, self.shards, True),
                   rra.rra_vocab_loss_workspace_bytes(T, D, self.shards, False),
                   rra.rra_allreduce_rmsnorm_backward8_workspace_bytes(T, D))
        self.ws = torch.empty(need, dtype=torch.uint8, device="cuda")

    def batch(self):
        self.ids.copy_(torch.randint(0, self.V, (self.T,), generator=self.gen, device="cuda"))
        self.targets.copy_(self.next[self.ids])

    def forward(self):
        p, n = self.p, self.n
        x = self.emb[self.ids]
        for r in range(n):
            torch.matmul(x[:, self.cut[r]:self.cut[r + 1]], p["proj"][r].t(), out=self.part[r])
        rra.rra_allreduce_rmsnorm_save8(self.part, self.h1, p["gamma1"][0], self.D, *self.keep1, eps=EPS)
        rra.rra_gated_ffn(self.h1[0], p["gate"], p["up"], self.acts, workspace=self.ws)
        for r in range(n):
            torch.matmul(self.acts[r], p["down"][r].t(), out=self.part[r])
        rra.rra_allreduce_rmsnorm_save8(self.part, self.h2, p["gamma2"][0], self.D, *self.keep2, eps=EPS)
        rra.rra_vocab_loss(self.h2[0], p["head"], self.targets, self.loss, self.lse, workspace=self.ws)
        return x

    def backward(self, x):
        p, g, n = self.p, self.g, self.n
        rra.rra_vocab_loss_backward(self.h2[0], p["head"], self.targets, self.lse, self.grad, self.dh, g["head"],
                                    workspace=self.ws)
        rra.rra_allreduce_rmsnorm_backward8([self.dh], [self.ds], *self.keep2, p["gamma2"][0], g["gamma2"][0],
                                            workspace=self.ws)
        for r in range(n):
            torch.matmul(self.ds.t(), self.acts[r], out=g["down"][r])
            torch.matmul(self.ds, p["down"][r], out=self.dacts[r])
        rra.rra_rmsnorm_restore8(*self.keep1, p["gamma1"][0], self.again)
        rra.rra_gated_ffn_backward(self.again, p["gate"], p["up"], self.dacts, self.dh, g["gate"], g["up"],
                                   workspace=self.ws)
        rra.rra_allreduce_rmsnorm_backward8([self.dh], [self.ds], *self.keep1, p["gamma1"][0], g["gamma1"][0],
                                            workspace=self.ws)
        for r in range(n):
            torch.matmul(self.ds.t(), x[:, self.cut[r]:self.cut[r + 1]], out=g["proj"][r])

    def update(self):
        for k, ws in self.p.items():
            for w, g in zip(ws, self.g[k]):
                w.add_(g.to(w.dtype), alpha=-self.lr)

    def run(self):
        self.backward(self.forward())
        self.update()

    def capture(self):
        """The whole step as one CUDA graph (the batch is copied in before)."""
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.forward()  # warm up outside the capture: no weight changes
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.run()
        return graph


def autograd_gradients(st):
    """The same loss's gradients by autograd in float32."""
    p = {k: [w.detach().float().requires_grad_(True) for w in ws] for k, ws in st.p.items()}
    x = st.emb[st.ids].float()

    def norm(s, gamma):
        return s * torch.rsqrt((s * s).mean(1, keepdim=True) + EPS) * gamma

    s1 = sum(x[:, st.cut[r]:st.cut[r + 1]] @ p["proj"][r].t() for r in range(st.n))
    h = norm(s1, p["gamma1"][0])
    s2 = sum((torch.nn.functional.silu(h @ p["gate"][r].t()) * (h @ p["up"][r].t())) @ p["down"][r].t()
             for r in range(st.n))
    logits = norm(s2, p["gamma2"][0]) @ torch.cat(p["head"]).t()
    loss = torch.nn.functional.cross_entropy(logits, st.targets, reduction="none")
    (loss * st.grad).sum().backward()
    return loss.detach(), {k: [w.grad for w in ws] for k, ws in p.items()}


def check(st):
    """Largest relative error of the step's gradients (in the 2-norm), by weight."""
    st.batch()
    st.backward(st.forward())
    loss, want = autograd_gradients(st)
    off = {k: max(float((g.float() - w).norm() / w.norm()) for g, w in zip(st.g[k], want[k])) for k in want}
    return float((st.loss - loss).abs().max()), off


def main(argv=None):
    ap = argparse.ArgumentParser()
    for name, value in (("ranks", 4), ("tokens", 512), ("hidden", 1024), ("width", 704), ("vocab", 8192),
                        ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=value)
    ap.add_argument("--lr", type=float, default=0.5)
    ap.add_argument("--graph", action="store_true")
    ap.add_argument("--check", action="store_true")
    a = ap.parse_args(argv)
    st = Step(a.ranks, a.tokens, a.hidden, a.width, a.vocab, a.lr)
    if a.check:
        loss, off = check(st)
        print("loss off by %.2e; gradients off by %s" % (loss, {k: "%.3f" % v for k, v in off.items()}))
    graph = st.capture() if a.graph else None
    means = []
    for i in range(a.steps):
        st.batch()
        if graph is None:
            st.run()
        else:
            graph.replay()
        means.append(float(st.loss.mean()))
        print("step %3d  loss %.4f" % (i, means[-1]), flush=True)
    status, info = rra.rra_query_status()
    if status != rra.RRA_SUCCESS:
        raise RuntimeError("device status %d %s" % (status, info))
    return means


if __name__ == "__main__":
    main()
