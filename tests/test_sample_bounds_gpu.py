"""The set of tokens that rra_vocab_sample can draw, where a bound of top-k and
one of top-p lie close to each other or to a border of the search: every row of
a call has the same logits and one of evenly spaced uniforms, so that a token
kept or dropped wrongly shows, whatever its weight.

Weights are within 2^-29 of their value: a uniform decides as the definition
does if it is further than 2^-26 from every border between two tokens, and
top-p's share from every running sum; the test asserts that of its inputs."""

import pytest
import torch

import collective_all_reduce_rank_gb300 as rra

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
DRAWS = 509
CLEAR = 2.0 ** -26


UNIFORMS = ((torch.arange(DRAWS, dtype=torch.float64) + 0.5) / DRAWS).float()


def definition(l, temperature, top_k, top_p):
    """(indices kept, ascending; the borders between them on [0, 1]; how far the
    nearest decision of top-p or a draw is from falling otherwise)."""
    l = l.double()
    order = torch.argsort(-l, stable=True)
    w = torch.exp((l - l[order[0]]) / temperature)
    if 0 < top_k < l.numel():
        order = order[:top_k]
    margin = 1.0
    if top_p < 1:
        s = w[order] / w[order].sum()
        before = torch.cumsum(s, 0) - s
        order = order[: max(1, int((before < top_p).sum()))]
        margin = float((before[1:] - top_p).abs().min()) if before.numel() > 1 else 1.0
    order, _ = torch.sort(order)
    border = torch.cumsum(w[order], 0) / w[order].sum()
    return order, border, min(margin, float((UNIFORMS.double()[:, None] - border[None, :]).abs().min()))


def check(l, shards, temperature=1.0, top_k=0, top_p=1.0):
    temperature, top_p = (float(torch.tensor(v, dtype=torch.float32)) for v in (temperature, top_p))
    order, border, margin = definition(l, temperature, top_k, top_p)
    assert margin > CLEAR
    at = (border[None, :] <= UNIFORMS.double()[:, None]).sum(1)
    want = order[at]

    def row(value, dtype=torch.float32):
        return torch.full((DRAWS,), value, dtype=dtype, device="cuda")

    token, logprob = row(-7, torch.int64), row(0.0)
    parts = [t.cuda().contiguous() for t in torch.split(l.expand(DRAWS, -1), shards, 1)]
    rra.rra_vocab_sample(parts, UNIFORMS.cuda(), token, temperature=row(temperature), top_k=row(top_k, torch.int32),
                         top_p=row(top_p), logprob=logprob)
    assert torch.equal(token.cpu(), want), (sorted(set(token.tolist())), order.tolist())
    # float32's logarithm and division: within 2^-21 of it, and of 1
    lp = torch.log(torch.diff(border, prepend=torch.zeros(1, dtype=torch.float64)))[at]
    assert ((logprob.cpu().double() - lp).abs() <= 2.0 ** -21 * (1 + lp.abs())).all()


# -- a bound of top-p in the bin that holds the one of top-k -------------------

HEADS = [[10.0, 6.9, 6.8, 6.7, -3.0], [10.0, 6.9, 6.8, 6.7, 6.6, 6.5], [3.0, 2.9, 2.8, 0.3, 0.2, 0.1],
         [10.0, 9.0, 6.9, 6.8, 6.0, 5.5, 5.1], [0.5, 0.4, -6.0, -6.1, -6.2, -6.3]]


@pytest.mark.parametrize("top_p", [0.5, 0.9, 0.99, 0.9999])
@pytest.mark.parametrize("top_k", [2, 3, 4, 5])
@pytest.mark.parametrize("head", range(len(HEADS)))
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_top_p_keeps_no_more_than_top_k(dtype, head, top_k, top_p):
    l = torch.tensor(HEADS[head]).to(DT[dtype])
    check(l, [l.numel()], 1.0, top_k, top_p)
    # the same among 300 tokens that weigh next to nothing, over two shards, the head from last to first
    far = torch.cat([torch.linspace(-40.0, -30.0, 300), torch.tensor(HEADS[head]).flip(0)]).to(DT[dtype])
    check(far, [303, far.numel() - 303], 1.0, top_k, top_p)


@pytest.mark.parametrize("top_p", [0.9, 0.99, 0.999, 0.9999])
@pytest.mark.parametrize("top_k", [2, 3, 4, 6])
def test_bounds_among_the_far_keys_of_bfloat16(top_k, top_p):
    """At a temperature of 10 the second half of the head lies beyond the 1024
    keys next to the largest, where a bin holds many keys."""
    l = torch.tensor([24.0, 0.05, 0.047, 0.044, 0.041, 0.02, -0.02, -5.0, -9.0]).to(torch.bfloat16)
    check(l, [4, 5], 10.0, top_k, top_p)


@pytest.mark.parametrize("seed", range(12))
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_random_heads(dtype, seed):
    """Clusters of near logits, all settings at random."""
    g = torch.Generator().manual_seed(1000 + seed)
    for _ in range(20):
        centre = 12.0 * torch.rand(4, generator=g) - 4.0
        spread = 10.0 ** (-3.0 * torch.rand(4, generator=g))
        n = int(torch.randint(3, 40, (1,), generator=g))
        which = torch.randint(0, 4, (n,), generator=g)
        l = (centre[which] + spread[which] * torch.randn(n, generator=g)).to(DT[dtype])
        t = float(10.0 ** (1.5 * torch.rand(1, generator=g) - 0.7))
        k = int(torch.randint(0, n + 2, (1,), generator=g))
        p = [1.0, 0.5, 0.9, 0.99, 0.999, 0.99999][int(torch.randint(0, 6, (1,), generator=g))]
        if definition(l, float(torch.tensor(t)), k, float(torch.tensor(p)))[2] > CLEAR:  # else a decision on a border
            check(l, [n], t, k, p)


# -- a bin that begins with the key of -0, which no logit has -------------------

BORDER = {
    # the largest logit's bits are 2 below a multiple of a bin of 2^22 keys
    "fp32": dict(dt=torch.float32, kind=torch.int32, top=0x3FBFFFFE, below=-0x7FFFFFFF, temperature=1.0),
    # of 2^6 keys, the 1024 next to the largest being searched one by one before
    "bf16": dict(dt=torch.bfloat16, kind=torch.int16, top=0x41BE, below=-0x7FFF, temperature=10.0),
}


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("top_k,top_p", [(2, 1.0), (0, 0.6), (0, 0.78), (2, 0.9), (3, 1.0), (5, 0.8)])
def test_zeros_above_the_smallest_negative_numbers(dtype, top_k, top_p):
    b = BORDER[dtype]
    top, below = torch.tensor([b["top"], b["below"]], dtype=b["kind"]).view(b["dt"])
    l = torch.full((300,), -1000.0, dtype=b["dt"])
    l[250], l[200], l[10:40:10] = top, 0.0, below
    assert 23 < top < 24 or 1 < top < 1.5 and below < 0
    check(l, [150, 150], b["temperature"], top_k, top_p)


# -- temperatures and logits at the ends of float32 -----------------------------

@pytest.mark.parametrize("temperature", [1e-28, 3e-31, 1e-35, 2e-38, 1e20, 1e36])
def test_temperatures_far_from_one(temperature):
    """Logits that differ by temperatures, however small or large."""
    l = (torch.tensor([1.5, 3.0, 2.75, 0.5, -1.0, 2.0], dtype=torch.float64) * temperature).float()
    check(l, [2, 4], temperature, 0, 1.0)
    check(l, [6], temperature, 4, 0.8)
