"""Cases and plain forms of the training-step operators around the all-reduce.

Three groups, each over n virtual ranks whose shards are separate buffers:

- norm_*: the fused all-reduce + RMSNorm that saves an 8-bit checkpoint of the
  sum, the normalised activations restored from that checkpoint (the input a
  backward pass recomputes from), and the gradient taken from it;
- ffn_*: the column-parallel gated feed-forward block, forward and backward;
- loss_*: the vocabulary-parallel softmax cross entropy, forward and with its
  gradient, which never keeps the logits.

``own`` picks what ``run`` computes with: False, elementary torch operations in
32 bits; True, the library's calls.  A state holds a user's tensors; output
buffers and workspaces are made at the first pass with the library and kept,
as a training loop keeps them.
"""
import math

import torch

own = False

IGNORE = -100
EPS = 1e-6
BLOCK = 128  # columns that share a checkpoint scale
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # Eight tokens' activations after a row-parallel layer at 8 ranks: latency.
        {"name": "norm_fwd_8tok", "op": "norm_fwd", "n": 8, "tokens": 8, "hidden": 5120, "dtype": "bf16"},
        # The 512-token activations of the all-reduce benchmark: forward, then the restore that the backward makes.
        {"name": "norm_fwd_512tok", "op": "norm_fwd", "n": 8, "tokens": 512, "hidden": 5120, "dtype": "bf16"},
        # A training micro-batch: gradients of 8 ranks summed and taken through the norm.
        {"name": "norm_bwd_4096tok", "op": "norm_bwd", "n": 8, "tokens": 4096, "hidden": 5120, "dtype": "bf16"},
        # fp32 gradients of 3 ranks, ragged rows and columns.
        {"name": "norm_bwd_odd_fp32", "op": "norm_bwd", "n": 3, "tokens": 1283, "hidden": 1027, "dtype": "fp32"},
        # Serving one token through the gate and up projections of 8 ranks.
        {"name": "ffn_fwd_1tok", "op": "ffn_fwd", "n": 8, "tokens": 1, "hidden": 5120, "width": 1728, "act": "silu"},
        # A prefill chunk of 512 tokens.
        {"name": "ffn_fwd_512tok", "op": "ffn_fwd", "n": 8, "tokens": 512, "hidden": 5120, "width": 1728,
         "act": "silu"},
        # The backward pass of a training micro-batch at 4 ranks.
        {"name": "ffn_bwd_4096tok", "op": "ffn_bwd", "n": 4, "tokens": 4096, "hidden": 5120, "width": 3456,
         "act": "silu"},
        # Sizes that fill no tile and no 16-byte row.
        {"name": "ffn_bwd_odd", "op": "ffn_bwd", "n": 3, "tokens": 777, "hidden": 1027, "width": 643,
         "act": "gelu_tanh"},
        # Scoring 8 tokens against a vocabulary of 131072 held by 8 ranks.
        {"name": "loss_fwd_8tok", "op": "loss_fwd", "n": 8, "tokens": 8, "hidden": 5120, "vocab": 131072},
        # One sequence of 2048 tokens scored (evaluation: no gradient).
        {"name": "loss_fwd_2048tok", "op": "loss_fwd", "n": 8, "tokens": 2048, "hidden": 5120, "vocab": 131072},
        # A training step's loss and its gradient over a micro-batch of 8192 tokens.
        {"name": "loss_step_8192tok", "op": "loss_step", "n": 8, "tokens": 8192, "hidden": 5120, "vocab": 131072},
        # A small model with an odd vocabulary over 3 ranks (unequal shards) and odd rows.
        {"name": "loss_step_odd", "op": "loss_step", "n": 3, "tokens": 333, "hidden": 515, "vocab": 50021},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "ffn_fwd", "ffn_bwd", "loss_fwd", "loss_step"])
    n = rng.randint(1, 8)
    hidden = _log_int(rng, 128, 5120)
    if rng.random() < 0.6:
        hidden = max(64, hidden // 64 * 64)
    case = {"op": op, "n": n, "hidden": hidden}
    if op.startswith("norm"):
        case["tokens"] = _log_int(rng, 1, 4096)
        case["dtype"] = rng.choice(["bf16", "fp32"])
    elif op.startswith("ffn"):
        case["tokens"] = _log_int(rng, 1, 4096)
        case["width"] = _log_int(rng, 32, max(64, 13824 // n))
        case["act"] = rng.choice(["silu", "gelu_tanh"])
    else:
        case["tokens"] = _log_int(rng, 1, 2048)
        case["vocab"] = _log_int(rng, 1000, 131072)
    return case


def _shards(vocab, n):
    """Rows of each rank's vocabulary shard: equal but for the last ones."""
    per = -(-vocab // n)
    return [max(0, min(vocab, (r + 1) * per) - r * per) for r in range(n)]


def _randn(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    t = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
    return (t * scale).to(dtype)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, n, T, D = case["op"], case["n"], case["tokens"], case["hidden"]
    st = {"case": dict(case)}
    if op.startswith("norm"):
        dt = DT[case["dtype"]]
        # a few columns of activations are far larger than the rest
        col = torch.exp(0.5 * torch.randn(D, generator=gen, device="cuda"))
        st["gamma"] = (1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt)
        xs = [(torch.randn(T, D, generator=gen, device="cuda") * col).to(dt) for _ in range(n)]
        if op == "norm_fwd":
            st["xs"] = xs
        else:
            y, codes, scales, rstd = _plain_norm_forward(xs, st["gamma"])
            st.update(codes=codes, scales=scales, rstd=rstd)
            st["grads"] = [_randn(gen, T, D, scale=1e-2, dtype=dt) for _ in range(n)]
    elif op.startswith("ffn"):
        F = case["width"]
        st["x"] = _randn(gen, T, D)
        st["gates"] = [_randn(gen, F, D, scale=D ** -0.5) for _ in range(n)]
        st["ups"] = [_randn(gen, F, D, scale=D ** -0.5) for _ in range(n)]
        if op == "ffn_bwd":
            st["dacts"] = [_randn(gen, T, F, scale=1e-2) for _ in range(n)]
    else:
        shards = _shards(case["vocab"], n)
        st["shards"] = shards
        st["weights"] = [_randn(gen, v, D, scale=D ** -0.5) for v in shards]
        tgt = torch.randint(0, case["vocab"], (T,), generator=gen, device="cuda")
        # hidden states lean towards their target's row, as a trained model's do
        lean = torch.cat([w for w in st["weights"]])[tgt].float()
        st["x"] = (torch.randn(T, D, generator=gen, device="cuda") + 4.0 * lean).to(torch.bfloat16)
        drop = torch.rand(T, generator=gen, device="cuda") < 0.06  # padding and prompt tokens
        st["targets"] = torch.where(drop, torch.full_like(tgt, IGNORE), tgt)
        if op == "loss_step":
            valid = (st["targets"] != IGNORE).sum().clamp(min=1).float()
            st["grad"] = (1.0 / valid).expand(T).contiguous()
    return st


# ---------------------------------------------------------------------------
# the plain forms: elementary operations in 32 bits
# ---------------------------------------------------------------------------

def _e4m3(v):
    """Round float32 values of at most 448 to the nearest e4m3 value."""
    return v.to(torch.float8_e4m3fn)


def _plain_norm_forward(xs, gamma):
    s = xs[0].float()
    for x in xs[1:]:
        s = s + x.float()
    T, D = s.shape
    rstd = torch.rsqrt((s * s).mean(1) + EPS)
    y = (s * rstd[:, None] * gamma.float()).to(gamma.dtype)
    nb = -(-D // BLOCK)
    b = torch.zeros(T, nb * BLOCK, device=s.device)
    b[:, :D] = s.to(torch.bfloat16).float()
    b = b.view(T, nb, BLOCK)
    amax = b.abs().amax(2)
    # the smallest e with amax <= 448 * 2^e: frexp gives amax = m * 2^k, m in [0.5, 1); 448 = 0.875 * 2^9
    m, k = torch.frexp(amax)
    e = (k - 9 + (m > 0.875).int()).clamp(-127, 127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    codes = _e4m3(torch.ldexp(b.double(), -e[:, :, None].double()).float())
    codes = codes.view(T, nb * BLOCK)[:, :D].contiguous()
    return y, codes, (e + 127).to(torch.uint8), rstd


def _codes_value(codes, scales):
    """The values a checkpoint stands for, in 32 bits."""
    T, D = codes.shape
    e = scales.to(torch.float64) - 127.0
    mul = torch.exp2(e).repeat_interleave(BLOCK, dim=1)[:, :D]
    return (codes.to(torch.float32).double() * mul).float()


def _plain_norm_backward(grads, codes, scales, rstd, gamma):
    g = grads[0].float()
    for t in grads[1:]:
        g = g + t.float()
    h = _codes_value(codes, scales) * rstd[:, None]
    w = g * gamma.float()
    ds = rstd[:, None] * (w - h * (w * h).mean(1, keepdim=True))
    dgamma = (g * h).sum(0, dtype=torch.float64).float()
    return ds.to(gamma.dtype), dgamma


def _act_and_slope(g, act):
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * g * g)


def _plain_run(st):
    case = st["case"]
    op, n, T, D = case["op"], case["n"], case["tokens"], case["hidden"]
    if op == "norm_fwd":
        y, codes, scales, rstd = _plain_norm_forward(st["xs"], st["gamma"])
        again = (_codes_value(codes, scales) * rstd[:, None] * st["gamma"].float()).to(y.dtype)
        return {"outs": [y.clone() for _ in range(n)], "restored": again, "rstd": rstd}
    if op == "norm_bwd":
        ds, dgamma = _plain_norm_backward(st["grads"], st["codes"], st["scales"], st["rstd"], st["gamma"])
        return {"dxs": [ds.clone() for _ in range(n)], "dgamma": dgamma}
    if op.startswith("ffn"):
        x = st["x"].float()
        acts, dx, dgs, dus = [], torch.zeros(T, D, device=x.device), [], []
        for r in range(n):
            G, U = st["gates"][r].float(), st["ups"][r].float()
            g, u = x @ G.t(), x @ U.t()
            a, slope = _act_and_slope(g, case["act"])
            if op == "ffn_fwd":
                acts.append((a * u).to(torch.bfloat16))
                continue
            da = st["dacts"][r].float()
            dg, du = da * u * slope, da * a
            dx += dg @ G + du @ U
            dgs.append((dg.t() @ x).to(torch.bfloat16))
            dus.append((du.t() @ x).to(torch.bfloat16))
        if op == "ffn_fwd":
            return {"acts": acts}
        return {"dx": dx.to(torch.bfloat16), "dgates": dgs, "dups": dus}
    x = st["x"].float()
    tgt = st["targets"]
    keep = tgt != IGNORE
    logits = [x @ w.float().t() for w in st["weights"]]
    m = torch.full((T,), -math.inf, device=x.device)
    for l in logits:
        if l.shape[1]:
            m = torch.maximum(m, l.amax(1))
    z = torch.zeros(T, device=x.device)
    for l in logits:
        z += torch.exp(l - m[:, None]).sum(1)
    lse = m + torch.log(z)
    lo, hit = 0, torch.zeros(T, device=x.device)
    for l in logits:
        v = l.shape[1]
        here = keep & (tgt >= lo) & (tgt < lo + v)
        if v:
            pick = l.gather(1, (tgt - lo).clamp(0, v - 1)[:, None])[:, 0]
            hit = torch.where(here, pick, hit)
        lo += v
    loss = torch.where(keep, lse - hit, torch.zeros_like(lse))
    if op == "loss_fwd":
        return {"loss": loss, "lse": lse}
    grad = torch.where(keep, st["grad"], torch.zeros_like(st["grad"]))
    dx, dws, lo = torch.zeros(T, D, device=x.device), [], 0
    rows = torch.arange(T, device=x.device)
    for w, l in zip(st["weights"], logits):
        v = l.shape[1]
        p = torch.exp_(l.sub_(lse[:, None]))
        here = keep & (tgt >= lo) & (tgt < lo + v)
        if v:
            p[rows, (tgt - lo).clamp(0, v - 1)] -= here.float()
        p *= grad[:, None]
        dx += p @ w.float()
        dws.append((p.t() @ x).to(torch.bfloat16))
        lo += v
    return {"loss": loss, "lse": lse, "dx": dx.to(torch.bfloat16), "dweights": dws}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _workspace(nbytes):
    return torch.empty(max(16, nbytes), dtype=torch.uint8, device="cuda")


def _own_run(st):
    import collective_all_reduce_rank_gb300 as rra

    if "ready" not in st:
        rra.rra_init(0)  # once per process; later calls return at once
        st["ready"] = True
    case = st["case"]
    op, n, T, D = case["op"], case["n"], case["tokens"], case["hidden"]
    act = {"silu": 0, "gelu_tanh": 1}.get(case.get("act"), 0)
    if op == "norm_fwd":
        if "outs" not in st:
            st["outs"] = [torch.empty_like(x) for x in st["xs"]]
            st["codes"] = torch.empty(T, D, dtype=torch.float8_e4m3fn, device="cuda")
            st["scales"] = torch.empty(T, -(-D // BLOCK), dtype=torch.uint8, device="cuda")
            st["rstd"] = torch.empty(T, device="cuda")
            st["restored"] = torch.empty_like(st["xs"][0])
        rra.rra_allreduce_rmsnorm_save8(st["xs"], st["outs"], st["gamma"], D, st["codes"], st["scales"], st["rstd"],
                                        eps=EPS)
        rra.rra_rmsnorm_restore8(st["codes"], st["scales"], st["rstd"], st["gamma"], st["restored"])
        return {"outs": st["outs"], "restored": st["restored"], "rstd": st["rstd"]}
    if op == "norm_bwd":
        if "dxs" not in st:
            st["dxs"] = [torch.empty_like(g) for g in st["grads"]]
            st["dgamma"] = torch.empty(D, device="cuda")
            st["ws"] = _workspace(rra.rra_allreduce_rmsnorm_backward8_workspace_bytes(T, D))
        rra.rra_allreduce_rmsnorm_backward8(st["grads"], st["dxs"], st["codes"], st["scales"], st["rstd"],
                                            st["gamma"], st["dgamma"], workspace=st["ws"])
        return {"dxs": st["dxs"], "dgamma": st["dgamma"]}
    if op.startswith("ffn"):
        F, back = case["width"], op == "ffn_bwd"
        if "ws" not in st:
            st["ws"] = _workspace(rra.rra_gated_ffn_workspace_bytes(n, T, D, F, back))
            if back:
                st["dx"] = torch.empty_like(st["x"])
                st["dgates"] = [torch.empty_like(w) for w in st["gates"]]
                st["dups"] = [torch.empty_like(w) for w in st["ups"]]
            else:
                st["acts"] = [torch.empty(T, F, dtype=torch.bfloat16, device="cuda") for _ in range(n)]
        if not back:
            rra.rra_gated_ffn(st["x"], st["gates"], st["ups"], st["acts"], act=act, workspace=st["ws"])
            return {"acts": st["acts"]}
        rra.rra_gated_ffn_backward(st["x"], st["gates"], st["ups"], st["dacts"], st["dx"], st["dgates"], st["dups"],
                                   act=act, workspace=st["ws"])
        return {"dx": st["dx"], "dgates": st["dgates"], "dups": st["dups"]}
    back = op == "loss_step"
    if "ws" not in st:
        st["ws"] = _workspace(rra.rra_vocab_loss_workspace_bytes(T, D, st["shards"], back))
        st["loss"] = torch.empty(T, device="cuda")
        st["lse"] = torch.empty(T, device="cuda")
        if back:
            st["dx"] = torch.empty_like(st["x"])
            st["dweights"] = [torch.empty_like(w) for w in st["weights"]]
    rra.rra_vocab_loss(st["x"], st["weights"], st["targets"], st["loss"], st["lse"], ignore_index=IGNORE,
                       workspace=st["ws"])
    if not back:
        return {"loss": st["loss"], "lse": st["lse"]}
    rra.rra_vocab_loss_backward(st["x"], st["weights"], st["targets"], st["lse"], st["grad"], st["dx"],
                                st["dweights"], ignore_index=IGNORE, workspace=st["ws"])
    return {"loss": st["loss"], "lse": st["lse"], "dx": st["dx"], "dweights": st["dweights"]}


def run(state):
    return _own_run(state) if own else _plain_run(state)


# ---------------------------------------------------------------------------
# work and the definition in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op, n, T, D = case["op"], case["n"], case["tokens"], case["hidden"]
    if op.startswith("norm"):
        es = 2 if case["dtype"] == "bf16" else 4
        saved = T * D + T * (-(-D // BLOCK)) + 4 * T
        if op == "norm_fwd":  # the checkpoint is written, then read back into one restored tensor
            return {"bytes": (2 * n + 1) * T * D * es + 2 * saved + D * es, "flops": T * D * (n + 8)}
        return {"bytes": 2 * n * T * D * es + saved + D * es + 4 * D, "flops": T * D * (n + 10)}
    if op.startswith("ffn"):
        F = case["width"]
        if op == "ffn_fwd":
            return {"bytes": 2 * (T * D + 2 * n * F * D + n * T * F), "flops": 4 * n * T * D * F}
        return {"bytes": 2 * (2 * T * D + 4 * n * F * D + n * T * F), "flops": 12 * n * T * D * F}
    V = case["vocab"]
    if op == "loss_fwd":
        return {"bytes": 2 * (T * D + V * D) + 16 * T, "flops": 2 * T * D * V}
    return {"bytes": 2 * (2 * T * D + 2 * V * D) + 20 * T, "flops": 8 * T * D * V}


def exact(case, seed):
    if work(case)["flops"] > 1.5e13:
        return None
    st = prepare(case, seed)
    op, n = case["op"], case["n"]
    f64 = torch.float64
    if op == "norm_fwd":
        s = torch.stack([x.to(f64) for x in st["xs"]]).sum(0)
        inv = (s.square().mean(-1) + EPS).pow(-0.5)
        y = torch.einsum("td,t,d->td", s, inv, st["gamma"].to(f64))
        T, D = s.shape
        held = s.to(torch.float32).to(torch.bfloat16).to(f64)  # the stored activation
        saved = torch.empty_like(s)
        for lo in range(0, D, BLOCK):
            part = held[:, lo:lo + BLOCK]
            top = part.abs().amax(-1, keepdim=True)
            ex = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 448.0)).clamp(-127, 127)
            v = part / torch.exp2(ex)
            # nearest e4m3: 3 fraction bits above 2^-6, steps of 2^-9 below; ties to even
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
            saved[:, lo:lo + BLOCK] = torch.round(v / step) * step * torch.exp2(ex)
        again = torch.einsum("td,t,d->td", saved, inv, st["gamma"].to(f64))
        return {"outs": [y for _ in range(n)], "restored": again, "rstd": inv}
    if op == "norm_bwd":
        dy = torch.stack([g.to(f64) for g in st["grads"]]).sum(0)
        D = dy.shape[1]
        scale = torch.pow(2.0, st["scales"].to(f64) - 127.0)
        which = torch.arange(D, device=dy.device) // BLOCK
        xhat = st["codes"].to(torch.float32).to(f64) * scale[:, which] * st["rstd"].to(f64).unsqueeze(1)
        wy = dy * st["gamma"].to(f64)
        proj = torch.einsum("td,td->t", wy, xhat) / D
        ds = (wy - xhat * proj.unsqueeze(1)) * st["rstd"].to(f64).unsqueeze(1)
        return {"dxs": [ds for _ in range(n)], "dgamma": torch.einsum("td,td->d", dy, xhat)}
    x = st["x"].to(f64)
    if op.startswith("ffn"):
        out, dx, dgs, dus = [], torch.zeros_like(x), [], []
        for r in range(n):
            G, U = st["gates"][r].to(f64), st["ups"][r].to(f64)
            g, u = torch.einsum("td,fd->tf", x, G), torch.einsum("td,fd->tf", x, U)
            if op == "ffn_bwd":
                g.requires_grad_(True)
            if case["act"] == "silu":
                a = g * torch.sigmoid(g)
            else:
                a = g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))
            if op == "ffn_fwd":
                out.append(a * u)
                continue
            da = st["dacts"][r].to(f64)
            (dg,) = torch.autograd.grad(a, g, da * u)
            du = da * a.detach()
            dx += torch.einsum("tf,fd->td", dg, G) + torch.einsum("tf,fd->td", du, U)
            dgs.append(torch.einsum("tf,td->fd", dg, x))
            dus.append(torch.einsum("tf,td->fd", du, x))
        return {"acts": out} if op == "ffn_fwd" else {"dx": dx, "dgates": dgs, "dups": dus}
    W = torch.cat([w.to(f64) for w in st["weights"]])
    logits = torch.einsum("td,vd->tv", x, W)
    lse = torch.logsumexp(logits, 1)
    keep = st["targets"] >= 0
    safe = st["targets"].clamp(min=0)
    loss = torch.where(keep, lse - logits[torch.arange(len(safe), device=x.device), safe], 0.0)
    if op == "loss_fwd":
        return {"loss": loss, "lse": lse}
    d = torch.exp(logits - lse.unsqueeze(1))
    d.scatter_add_(1, safe.unsqueeze(1), torch.full_like(lse, -1.0).unsqueeze(1))
    d *= torch.where(keep, st["grad"].to(f64), 0.0).unsqueeze(1)
    dW = torch.einsum("tv,td->vd", d, x)
    return {"loss": loss, "lse": lse, "dx": torch.einsum("tv,vd->td", d, W),
            "dweights": list(torch.split(dW, st["shards"]))}
