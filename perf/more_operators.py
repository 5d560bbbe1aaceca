"""Cases and plain forms of the serving-step operators around the all-reduce.

Five groups over n virtual ranks whose shards are separate buffers:

- quant_*: a matrix in microscaled 4-bit floating point (MX4) and read back;
- norm_*: the fused all-reduce + residual + RMSNorm whose result is written in
  MX4, the operand of the next product;
- head_*: activations quantised and multiplied with MX4 vocabulary shards;
- ffn_*: a gated feed-forward block in MX4: column-parallel gate and up
  projections, activations requantised, row-parallel product summed over the
  ranks;
- sample_*: tokens drawn from vocabulary-parallel logits by temperature,
  top-k, top-p and min-p, from given random numbers.

MX4: 32 columns of a row share a power-of-two scale 2^e, the smallest with
max |x| <= 6 * 2^e; a code is x * 2^-e as e2m1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and
a sign), nearest, ties to even.  Codes are rows of 16 bytes a block, the even
column in the low four bits; scale bytes e + 127 lie in tiles of 128 rows x 4
blocks of 512 bytes, (row, block) at byte row % 32 * 16 + row % 128 // 32 * 4 +
block % 4 of tile (row // 128, block // 4).

``own`` picks what ``run`` computes with: False, elementary torch operations;
True, the library's calls.  A state holds a user's tensors; output buffers are
made at the first pass with the library and kept, as a server keeps them.
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 32
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # A rank's head shard quantised when weights are loaded, and read back for a check.
        {"name": "quant_weights", "op": "quant", "rows": 16384, "cols": 5120, "dtype": "bf16"},
        # fp32 rows that end inside a block, a tile of scales and a 16-byte unit.
        {"name": "quant_odd_fp32", "op": "quant", "rows": 1283, "cols": 1027, "dtype": "fp32"},
        # Eight tokens' activations between two layers at 8 ranks: latency.
        {"name": "norm_8tok", "op": "norm", "n": 8, "tokens": 8, "hidden": 5120, "dtype": "bf16", "residual": True},
        # A prefill batch of 4096 tokens.
        {"name": "norm_4096tok", "op": "norm", "n": 8, "tokens": 4096, "hidden": 5120, "dtype": "bf16",
         "residual": True},
        # One token against a vocabulary of 131072 held by 8 ranks.
        {"name": "head_1tok", "op": "head", "n": 8, "tokens": 1, "hidden": 5120, "vocab": 131072, "dtype": "fp32"},
        # A small model with an odd vocabulary over 3 ranks (unequal shards) and odd rows.
        {"name": "head_odd", "op": "head", "n": 3, "tokens": 333, "hidden": 515, "vocab": 50021, "dtype": "bf16"},
        # Serving one token through the feed-forward block of 8 ranks.
        {"name": "ffn_1tok", "op": "ffn", "n": 8, "tokens": 1, "hidden": 5120, "width": 1728, "act": "silu"},
        # A prefill chunk of 512 tokens.
        {"name": "ffn_512tok", "op": "ffn", "n": 8, "tokens": 512, "hidden": 5120, "width": 1728, "act": "silu"},
        # A prefill batch of 4096 tokens.
        {"name": "ffn_4096tok", "op": "ffn", "n": 8, "tokens": 4096, "hidden": 5120, "width": 1728,
         "act": "gelu_tanh"},
        # One request's next token.
        {"name": "sample_1row", "op": "sample", "n": 8, "rows": 1, "vocab": 131072, "dtype": "bf16"},
        # A batch of 256 requests, each with settings of its own.
        {"name": "sample_256row", "op": "sample", "n": 8, "rows": 256, "vocab": 131072, "dtype": "bf16"},
        # An odd vocabulary over 3 ranks, fp32 logits.
        {"name": "sample_odd_fp32", "op": "sample", "n": 3, "rows": 33, "vocab": 50021, "dtype": "fp32"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "norm", "head", "ffn", "sample"])
    hidden = _log_int(rng, 128, 5120)
    if rng.random() < 0.6:
        hidden = max(64, hidden // 64 * 64)
    n = rng.randint(1, 8)
    if op == "quant":
        return {"op": op, "rows": _log_int(rng, 1, 16384), "cols": hidden, "dtype": rng.choice(["bf16", "fp32"])}
    if op == "norm":
        return {"op": op, "n": n, "tokens": _log_int(rng, 1, 4096), "hidden": hidden,
                "dtype": rng.choice(["bf16", "fp32"]), "residual": rng.random() < 0.7}
    if op == "head":
        return {"op": op, "n": n, "tokens": _log_int(rng, 1, 512), "hidden": hidden,
                "vocab": _log_int(rng, 1000, 131072), "dtype": rng.choice(["bf16", "fp32"])}
    if op == "ffn":
        return {"op": op, "n": n, "tokens": _log_int(rng, 1, 4096), "hidden": hidden,
                "width": _log_int(rng, 32, max(64, 13824 // n)), "act": rng.choice(["silu", "gelu_tanh"])}
    return {"op": op, "n": n, "rows": _log_int(rng, 1, 256), "vocab": _log_int(rng, 1000, 131072),
            "dtype": rng.choice(["bf16", "fp32"])}


# ---------------------------------------------------------------------------
# MX4 in elementary operations
# ---------------------------------------------------------------------------

def _blocks(cols):
    return -(-cols // BLOCK)


def _plain_mx4(x):
    """Values [rows, blocks, 32] (zeros behind the last column) and exponents of a float32 matrix in MX4."""
    rows, cols = x.shape
    nb = _blocks(cols)
    b = torch.zeros(rows, nb * BLOCK, device=x.device)
    b[:, :cols] = x
    b = b.view(rows, nb, BLOCK)
    amax = b.abs().amax(2)
    # the smallest e with amax <= 6 * 2^e: amax = m * 2^k, m in [0.5, 1); 6 = 0.75 * 2^3
    m, k = torch.frexp(amax)
    e = (k - 3 + (m > 0.75).int()).clamp(min=-127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    v = torch.ldexp(b.double(), -e[:, :, None].double()).float()
    a = v.abs()
    # borders between neighbours; the lower code has them where it is the even one
    code = ((a > 0.25).int() + (a >= 0.75).int() + (a > 1.25).int() + (a >= 1.75).int() + (a > 2.5).int()
            + (a >= 3.5).int() + (a > 5.0).int())
    return code + 8 * (v < 0).int(), e


def _grid(device):
    half = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=device)
    return torch.cat([half, -half])


def _value(code, e):
    """What codes [rows, blocks, 32] and exponents stand for, as float32 [rows, blocks * 32]."""
    v = torch.ldexp(_grid(code.device)[code.long()], e[:, :, None].int())
    return v.reshape(v.shape[0], -1)


def _pack(code, e):
    """The library's layout of codes and scales."""
    rows, nb, _ = code.shape
    c = code.to(torch.uint8).view(rows, nb * 16, 2)
    tiles, across = -(-rows // 128), -(-nb // 4)
    s = torch.zeros(tiles * 128, across * 4, dtype=torch.uint8, device=code.device)
    s[:rows, :nb] = (e + 127).to(torch.uint8)
    s = s.view(tiles, 4, 32, across, 4).permute(0, 3, 2, 1, 4)
    return c[:, :, 0] | (c[:, :, 1] << 4), s.reshape(-1)


def _unpack(codes, scales, cols):
    """Float32 values [rows, cols] of codes and scales in the library's layout."""
    rows, nb = codes.shape[0], _blocks(cols)
    code = torch.stack([codes & 15, codes >> 4], 2).view(rows, nb, BLOCK)
    tiles, across = -(-rows // 128), -(-nb // 4)
    s = scales.view(tiles, across, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(tiles * 128, across * 4)
    return _value(code, s[:rows, :nb].int() - 127)[:, :cols]


def _quantized(gen, rows, cols, scale):
    w = (torch.randn(rows, cols, generator=gen, device="cuda") * scale).to(torch.bfloat16).float()
    return _pack(*_plain_mx4(w))


def _shards(vocab, n):
    """Rows of each rank's vocabulary shard: equal but for the last ones."""
    per = -(-vocab // n)
    return [max(0, min(vocab, (r + 1) * per) - r * per) for r in range(n)]


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op = case["op"]
    st = {"case": dict(case)}
    if op == "quant":
        x = torch.randn(case["rows"], case["cols"], generator=gen, device="cuda") * case["cols"] ** -0.5
        st["x"] = x.to(DT[case["dtype"]])
        return st
    n = case["n"]
    if op == "sample":
        rows, V = case["rows"], case["vocab"]
        logits = 2.5 * torch.randn(rows, V, generator=gen, device="cuda")
        # a few candidates stand out, as a trained model's do
        top = torch.randint(0, V, (rows, 12), generator=gen, device="cuda")
        logits.scatter_add_(1, top, 4.0 + 8.0 * torch.rand(rows, 12, generator=gen, device="cuda"))
        logits = logits.to(DT[case["dtype"]])
        st["shards"] = _shards(V, n)
        st["logits"] = [t.contiguous() for t in torch.split(logits, st["shards"], dim=1)]

        def pick(values, dtype):
            which = torch.randint(0, len(values), (rows,), generator=gen, device="cuda")
            return torch.tensor(values, dtype=dtype, device="cuda")[which]

        st["uniform"] = torch.rand(rows, generator=gen, device="cuda")
        # greedy requests among them; 0, 1 and 0 turn top-k, top-p and min-p off
        st["temperature"] = pick([0.0, 0.6, 0.7, 0.8, 1.0, 1.0, 1.3], torch.float32)
        st["top_k"] = pick([0, 0, 20, 50, 1000], torch.int32)
        st["top_p"] = pick([1.0, 0.8, 0.9, 0.95], torch.float32)
        st["min_p"] = pick([0.0, 0.0, 0.05], torch.float32)
        return st
    T, D = case["tokens"], case["hidden"]
    # a few columns of activations are far larger than the rest
    col = torch.exp(0.5 * torch.randn(D, generator=gen, device="cuda"))
    if op == "norm":
        dt = DT[case["dtype"]]
        st["gamma"] = (1.0 + 0.1 * torch.randn(D, generator=gen, device="cuda")).to(dt)
        st["xs"] = [(torch.randn(T, D, generator=gen, device="cuda") * col).to(dt) for _ in range(n)]
        # the residual stream; a pass adds to it, so each starts from this one
        st["stream"] = (2.0 * torch.randn(T, D, generator=gen, device="cuda") * col).to(dt)
        return st
    x = (torch.randn(T, D, generator=gen, device="cuda") * col).to(torch.bfloat16)
    if op == "head":
        st["shards"] = _shards(case["vocab"], n)
        st["x"] = x
        st["heads"] = [_quantized(gen, v, D, D ** -0.5) for v in st["shards"]]
        return st
    F = case["width"]
    st["x"] = _pack(*_plain_mx4(x.float()))
    st["gates"] = [_quantized(gen, F, D, D ** -0.5) for _ in range(n)]
    st["ups"] = [_quantized(gen, F, D, D ** -0.5) for _ in range(n)]
    st["downs"] = [_quantized(gen, D, F, (n * F) ** -0.5) for _ in range(n)]
    return st


# ---------------------------------------------------------------------------
# the plain forms: elementary operations in 32 bits (long sums, and the mass
# of a distribution, in 64)
# ---------------------------------------------------------------------------

def _act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    c = math.sqrt(2.0 / math.pi)
    return 0.5 * g * (1.0 + torch.tanh(c * (g + 0.044715 * g * g * g)))


def _plain_sample(st):
    logits = torch.cat(st["logits"], 1).double()
    rows, V = logits.shape
    temp = st["temperature"].double()
    greedy = temp == 0
    temp = torch.where(greedy, torch.ones_like(temp), temp)
    l, order = torch.sort(logits, dim=1, descending=True, stable=True)
    w = torch.exp((l - l[:, :1]) / temp[:, None])
    rank = torch.arange(V, device=w.device)[None, :]
    k = torch.where(greedy, torch.ones_like(st["top_k"]), st["top_k"])
    keep = (k[:, None] <= 0) | (rank < k[:, None])
    w = torch.where(keep, w, torch.zeros_like(w))
    mass = torch.cumsum(w, 1)
    p = st["top_p"].double()[:, None]
    keep &= (p >= 1.0) | (mass - w < p * mass[:, -1:])
    keep &= w >= st["min_p"].double()[:, None]
    w = torch.where(keep, w, torch.zeros_like(w))
    by_index = torch.zeros_like(w).scatter_(1, order, w)
    mass = torch.cumsum(by_index, 1)
    total = mass[:, -1:]
    token = (mass <= st["uniform"].double()[:, None] * total).sum(1)
    logprob = torch.log(by_index.gather(1, token[:, None]) / total)[:, 0]
    return {"token": token, "logprob": logprob.float()}


def _plain_run(st):
    case = st["case"]
    op = case["op"]
    if op == "sample":
        return _plain_sample(st)
    if op == "quant":
        x = st["x"]
        return {"value": _value(*_plain_mx4(x.float()))[:, :case["cols"]].to(x.dtype)}
    n, T, D = case["n"], case["tokens"], case["hidden"]
    if op == "norm":
        s = st["xs"][0].float()
        for x in st["xs"][1:]:
            s = s + x.float()
        if case["residual"]:
            s = s + st["stream"].float()
        rstd = (1.0 / torch.sqrt(s.double().square().mean(1) + EPS)).float()
        y = (s * rstd[:, None]) * st["gamma"].float()
        out = {"value": _value(*_plain_mx4(y))[:, :D].to(st["gamma"].dtype)}
        if case["residual"]:
            out["stream"] = s.to(st["gamma"].dtype)
        return out
    if op == "head":
        x = _value(*_plain_mx4(st["x"].float()))[:, :D]
        return {"logits": [(x @ _unpack(*w, D).t()).to(DT[case["dtype"]]) for w in st["heads"]]}
    F = case["width"]
    x = _unpack(*st["x"], D)
    g = x @ torch.cat([_unpack(*w, D) for w in st["gates"]]).t()
    u = x @ torch.cat([_unpack(*w, D) for w in st["ups"]]).t()
    a = (_act(g, case["act"]) * u).view(T * n, F)
    a = _value(*_plain_mx4(a))[:, :F].reshape(T, n * F)
    down = torch.cat([_unpack(*w, F) for w in st["downs"]], 1)
    return {"out": (a @ down.t()).to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# the library's calls
# ---------------------------------------------------------------------------

def _mx4(rra, rows, cols):
    """Room for an MX4 matrix: codes and scales."""
    return (torch.empty(rows, 16 * _blocks(cols), dtype=torch.uint8, device="cuda"),
            torch.empty(rra.rra_mx4_scale_bytes(rows, cols), dtype=torch.uint8, device="cuda"))


def _own_run(st):
    import collective_all_reduce_rank_gb300 as rra

    if "ready" not in st:
        rra.rra_init(0)  # once per process; later calls return at once
        st["ready"] = True
    case = st["case"]
    op = case["op"]
    if op == "sample":
        if "token" not in st:
            st["token"] = torch.empty(case["rows"], dtype=torch.int64, device="cuda")
            st["logprob"] = torch.empty(case["rows"], device="cuda")
        rra.rra_vocab_sample(st["logits"], st["uniform"], st["token"], temperature=st["temperature"],
                             top_k=st["top_k"], top_p=st["top_p"], min_p=st["min_p"], logprob=st["logprob"])
        return {"token": st["token"], "logprob": st["logprob"]}
    if op == "quant":
        x = st["x"]
        if "mx4" not in st:
            st["mx4"] = _mx4(rra, *x.shape)
            st["value"] = torch.empty_like(x)
        rra.rra_mx4_quantize(x, *st["mx4"])
        rra.rra_mx4_restore(*st["mx4"], st["value"])
        return {"value": st["value"]}
    n, T, D = case["n"], case["tokens"], case["hidden"]
    if op == "norm":
        if "mx4" not in st:
            st["mx4"] = _mx4(rra, T, D)
            st["value"] = torch.empty_like(st["stream"])
            st["next"] = torch.empty_like(st["stream"]) if case["residual"] else None
        rra.rra_allreduce_rmsnorm_mx4(st["xs"], st["gamma"], D, *st["mx4"],
                                      residual=st["stream"] if case["residual"] else None, residual_out=st["next"],
                                      eps=EPS)
        rra.rra_mx4_restore(*st["mx4"], st["value"])
        return {"value": st["value"], "stream": st["next"]} if case["residual"] else {"value": st["value"]}
    if op == "head":
        if "mx4" not in st:
            st["mx4"] = _mx4(rra, T, D)
            st["out"] = [torch.empty(T, v, dtype=DT[case["dtype"]], device="cuda") for v in st["shards"]]
        rra.rra_mx4_quantize(st["x"], *st["mx4"])
        rra.rra_mx4_product(st["mx4"], st["heads"], st["out"], D)
        return {"logits": st["out"]}
    F = case["width"]
    if "acts" not in st:
        st["acts"] = [_mx4(rra, T, F) for _ in range(n)]
        st["out"] = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
    act = {"silu": rra.RRA_ACT_SILU, "gelu_tanh": rra.RRA_ACT_GELU_TANH}[case["act"]]
    rra.rra_mx4_gated_ffn(st["x"], st["gates"], st["ups"], st["acts"], D, F, act=act)
    rra.rra_mx4_product_sum(st["acts"], st["downs"], st["out"], F)
    return {"out": st["out"]}


def run(state):
    return _own_run(state) if own else _plain_run(state)


# ---------------------------------------------------------------------------
# work and the definition in 64 bits
# ---------------------------------------------------------------------------

def _mx4_bytes(rows, cols):
    return rows * 17 * _blocks(cols)


def work(case):
    op = case["op"]
    if op == "quant":
        es, count = (2 if case["dtype"] == "bf16" else 4), case["rows"] * case["cols"]
        # the matrix in 4 bits is written, then read back
        return {"bytes": 2 * count * es + 2 * _mx4_bytes(case["rows"], case["cols"]), "flops": 6 * count}
    n = case["n"]
    if op == "sample":
        es, count = (2 if case["dtype"] == "bf16" else 4), case["rows"] * case["vocab"]
        return {"bytes": count * es + 32 * case["rows"], "flops": 8 * count}
    T, D = case["tokens"], case["hidden"]
    if op == "norm":
        es = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": (n + 1 + (2 if case["residual"] else 0)) * T * D * es + D * es + 2 * _mx4_bytes(T, D),
                "flops": T * D * (n + 10)}
    if op == "head":
        V, es = case["vocab"], (2 if case["dtype"] == "bf16" else 4)
        return {"bytes": 2 * T * D + 2 * _mx4_bytes(T, D) + _mx4_bytes(V, D) + es * T * V, "flops": 2 * T * D * V}
    F = case["width"]
    return {"bytes": _mx4_bytes(T, D) + n * (2 * _mx4_bytes(F, D) + 2 * _mx4_bytes(T, F) + _mx4_bytes(D, F)) + 2 * T * D,
            "flops": 6 * n * T * D * F}


def _exact_mx4(x):
    """A float64 matrix rounded to MX4, from the definition."""
    out = torch.empty_like(x)
    for lo in range(0, x.shape[1], BLOCK):
        part = x[:, lo:lo + BLOCK]
        top = part.abs().amax(-1, keepdim=True)
        ex = torch.ceil(torch.log2(top.clamp(min=2.0 ** -140) / 6.0)).clamp(min=-127)
        v = part / torch.exp2(ex)
        # steps of 0.5 below 2, 1 below 4, 2 from there; ties to the even multiple
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1.0))) - 1.0)
        out[:, lo:lo + BLOCK] = torch.round(v / step) * step * torch.exp2(ex)
    return out


def _exact_read(codes, scales, cols):
    """Values of codes and scales in 64 bits, each scale found by its address."""
    rows, nb = codes.shape[0], _blocks(cols)
    r = torch.arange(rows, device=codes.device)[:, None]
    b = torch.arange(nb, device=codes.device)[None, :]
    at = (r // 128 * (-(-nb // 4)) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4
    c = torch.arange(cols, device=codes.device)
    bits = (codes[:, c // 2].long() >> (4 * (c % 2))) & 15
    mag = bits & 7
    low = mag.double() / 2  # 0 and 0.5, then (1 + m / 2) 2^(e - 1)
    high = (1.0 + (mag & 1).double() / 2) * torch.exp2((mag >> 1).double() - 1)
    v = torch.where(mag < 2, low, high) * (1.0 - 2.0 * (bits >> 3).double())
    return v * torch.exp2(scales[at].double() - 127.0)[:, c // BLOCK]


def _exact_sample(st):
    tokens, logprobs = [], []
    logits = torch.cat(st["logits"], 1).double()
    for i in range(logits.shape[0]):
        l = logits[i]
        t, k = float(st["temperature"][i]), int(st["top_k"][i])
        if t == 0:
            t, k = 1.0, 1
        p, q, u = float(st["top_p"][i]), float(st["min_p"][i]), float(st["uniform"][i])
        order = torch.argsort(-l, stable=True)
        if k > 0:
            order = order[:k]
        prob = torch.softmax(l[order] / t, 0)
        if p < 1.0:
            before = torch.cumsum(prob, 0) - prob
            cut = int((before < p).sum())
            order, prob = order[:cut], prob[:cut]
        most = prob[0]
        order, prob = order[prob >= q * most], prob[prob >= q * most]
        kept, by = torch.sort(order)
        prob = prob[by] / prob.sum()
        at = int((torch.cumsum(prob, 0) <= u).sum())
        at = min(at, len(kept) - 1)
        tokens.append(kept[at])
        logprobs.append(torch.log(prob[at]))
    return {"token": torch.stack(tokens), "logprob": torch.stack(logprobs)}


def exact(case, seed):
    op = case["op"]
    if op in ("head", "ffn") and work(case)["flops"] > 8e12:
        return None
    st = prepare(case, seed)
    f64 = torch.float64
    if op == "sample":
        return _exact_sample(st)
    if op == "quant":
        return {"value": _exact_mx4(st["x"].to(f64))}
    n, T, D = case["n"], case["tokens"], case["hidden"]
    if op == "norm":
        s = torch.stack([x.to(f64) for x in st["xs"]] + ([st["stream"].to(f64)] if case["residual"] else [])).sum(0)
        inv = (s.square().mean(-1) + EPS).pow(-0.5)
        out = {"value": _exact_mx4(torch.einsum("td,t,d->td", s, inv, st["gamma"].to(f64)))}
        if case["residual"]:
            out["stream"] = s
        return out
    if op == "head":
        x = _exact_mx4(st["x"].to(f64))
        return {"logits": [torch.einsum("td,vd->tv", x, _exact_read(*w, D)) for w in st["heads"]]}
    F = case["width"]
    x = _exact_read(*st["x"], D)
    out = torch.zeros(T, D, dtype=f64, device=x.device)
    for r in range(n):
        g = torch.einsum("td,fd->tf", x, _exact_read(*st["gates"][r], D))
        u = torch.einsum("td,fd->tf", x, _exact_read(*st["ups"][r], D))
        if case["act"] == "silu":
            a = g * torch.sigmoid(g)
        else:
            a = g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))
        out += torch.einsum("tf,df->td", _exact_mx4(a * u), _exact_read(*st["downs"][r], F))
    return {"out": out}
