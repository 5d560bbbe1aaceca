"""The training-step operators on the GPU against their definitions in
float64: the gated feed-forward block, the vocabulary loss, and the RMSNorm
with an 8-bit checkpoint.

Elementwise bounds come from the roundings each value meets (train_ref.py).
For gradients whose terms are each rounded to bfloat16 once the bound adds
every term's half step, which is loose for long sums, so the 2-norm is held
too: independent roundings leave at most half a step of the operand and half
a step of the result, 2 x 2^-8 relative."""
import math

import pytest

torch = pytest.importorskip("torch")

import collective_all_reduce_rank_gb300 as rra  # noqa: E402
import train_ref as ref  # noqa: E402

pytestmark = pytest.mark.gpu

IGN = -100


@pytest.fixture(scope="module", autouse=True)
def _init():
    rra.rra_init(0)
    yield


def status_ok():
    st, info = rra.rra_query_status()
    assert st == rra.RRA_SUCCESS, info


def rnd(gen, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen) * scale).to(dtype)


def poison(*shape, dtype=torch.bfloat16):
    t = torch.empty(*shape, dtype=dtype, device="cuda")
    t.view(torch.uint8).fill_(0xFF)
    return t


def cuda(ts):
    return [t.cuda() for t in ts]


# -- gated feed-forward ------------------------------------------------------

FFN = [  # n, tokens, hidden, width, act
    (1, 1, 64, 128, 0), (1, 128, 64, 128, 0), (2, 24, 64, 40, 1), (1, 256, 256, 128, 1), (2, 256, 128, 256, 0), (1, 300, 200, 130, 1),
    (3, 77, 88, 33, 0), (2, 1, 512, 520, 1), (8, 16, 128, 40, 0), (2, 129, 1027, 65, 0), (3, 5, 7, 3, 1),
    (2, 513, 640, 384, 0), (1, 1, 1, 1, 0), (4, 700, 72, 1000, 0),
    # few tokens: the register path, rows on and off 16 bytes
    (1, 1, 5120, 24, 0), (8, 8, 1024, 17, 1), (3, 9, 2056, 64, 0), (2, 16, 515, 33, 0), (1, 7, 1027, 8, 1), (2, 3, 771, 100, 0),
    (1, 17, 1024, 72, 0), (2, 40, 520, 136, 1),
    (1, 2, 1027, 130, 0), (2, 8, 333, 65, 1), (1, 5, 9, 200, 0), (1, 3, 5, 64, 1), (3, 1, 4102, 12, 0),
    # a part of a tile's rows staged
    (8, 33, 512, 720, 0), (7, 128, 256, 700, 1), (8, 121, 136, 1728, 0), (1, 100, 264, 9000, 0),
]


@pytest.mark.parametrize("n,T,D,F,act", FFN)
def test_gated_ffn(n, T, D, F, act):
    gen = torch.Generator().manual_seed(T * 7 + D)
    x = rnd(gen, T, D)
    G = [rnd(gen, F, D, scale=D ** -0.5) for _ in range(n)]
    U = [rnd(gen, F, D, scale=D ** -0.5) for _ in range(n)]
    acts = [poison(T, F) for _ in range(n)]
    rra.rra_gated_ffn(x.cuda(), cuda(G), cuda(U), acts, act=act)
    status_ok()
    outs, bounds, _, _, _ = ref.ffn(x, G, U, act)
    for r in range(n):
        ref.assert_within(acts[r], outs[r], bounds[r], "acts[%d]" % r)


@pytest.mark.parametrize("n,T,D,F,act", FFN)
def test_gated_ffn_backward(n, T, D, F, act):
    gen = torch.Generator().manual_seed(T * 11 + D)
    x = rnd(gen, T, D)
    G = [rnd(gen, F, D, scale=D ** -0.5) for _ in range(n)]
    U = [rnd(gen, F, D, scale=D ** -0.5) for _ in range(n)]
    da = [rnd(gen, T, F, scale=1e-2) for _ in range(n)]
    dx = poison(T, D)
    dG, dU = [poison(F, D) for _ in range(n)], [poison(F, D) for _ in range(n)]
    rra.rra_gated_ffn_backward(x.cuda(), cuda(G), cuda(U), cuda(da), dx, dG, dU, act=act)
    status_ok()
    _, _, (rdx, bdx), rG, rU = ref.ffn(x, G, U, act, da)
    ref.assert_within(dx, rdx, bdx, "dx")
    for r in range(n):
        ref.assert_within(dG[r], *rG[r], "dgates[%d]" % r)
        ref.assert_within(dU[r], *rU[r], "dups[%d]" % r)
    ref.assert_norm_close(dx, rdx, 2 * ref.BF, "dx")


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("act", [0, 1])
def test_slope_of_large_gates(T, act):
    """Gates far out, up to where their square and cube pass float32: the slope is 0 or 1."""
    D = 64
    gen = torch.Generator().manual_seed(T)
    gates = torch.tensor([s * v for v in (90.0, 1e6, 1e12, 2e13, 1e15, 1e19, 1e25, 1e30) for s in (1.0, -1.0)])
    F = len(gates)
    x, U, da = rnd(gen, T, D), rnd(gen, F, D, scale=0.1), rnd(gen, T, F, scale=1e-2)
    x[:, 0] = 1.0
    G = torch.zeros(F, D, dtype=torch.bfloat16)
    G[:, 0] = gates  # so that every token's gate is the row's value, exactly
    dx, dG, dU = poison(T, D), poison(F, D), poison(F, D)
    rra.rra_gated_ffn_backward(x.cuda(), cuda([G]), cuda([U]), cuda([da]), dx, [dG], [dU], act=act)
    status_ok()
    X, g, W, d = x.double(), G[:, 0].double(), U.double(), da.double()
    slope = (g > 0).double()
    u, eu = X @ W.t(), ref.product_err(X.abs(), W.abs().t(), D)
    dg, du = d * u * slope, d * g.clamp(min=0)
    edg = d.abs() * eu * slope * (1 + ref.BF) + (ref.BF + 2.0 ** -20) * dg.abs()
    edu = (ref.BF + 2.0 ** -19) * du.abs()  # act by the fast exponential and division: 2^-20
    for got, v, e in ((dG, dg, edg), (dU, du, edu)):
        want = v.t() @ X
        ref.assert_within(got, want, e.t() @ X.abs() + ref.product_err(v.abs().t(), X.abs(), T)
                          + ref.BF * want.abs() + 1e-30, "weights")
    want = dg @ G.double() + du @ W
    mag = ref.product_err(dg.abs(), G.double().abs(), 2 * F) + ref.product_err(du.abs(), W.abs(), 2 * F)
    ref.assert_within(dx, want, edg @ G.double().abs() + edu @ W.abs() + mag + ref.BF * want.abs() + 1e-30, "dx")


# -- vocabulary loss ---------------------------------------------------------

LOSS = [  # tokens, hidden, shard heights
    (1, 64, (256,)), (256, 64, (256,)), (5, 64, (300, 300)), (300, 128, (512, 511)), (33, 200, (1000, 1000, 997)),
    (129, 1027, (257, 0, 64)), (7, 515, (1,)), (64, 72, (100,) * 8), (2, 8, (3, 2)), (513, 256, (2048, 2048)),
    # few tokens: the register path
    (1, 5120, (700, 700)), (8, 1024, (16, 15, 0, 33)), (16, 515, (401, 400)), (9, 1027, (3000,)), (5, 771, (17,)),
    (17, 1024, (500,)), (100, 512, (5000, 300)), (1, 1027, (1000, 129)), (8, 333, (130, 0, 300)),
    (3, 5, (260,)), (7, 4102, (140, 9)), (121, 136, (20000,)),
]


def loss_inputs(T, D, shards, seed):
    gen = torch.Generator().manual_seed(seed)
    W = [rnd(gen, v, D, scale=D ** -0.5) for v in shards]
    V = sum(shards)
    tgt = torch.randint(0, V, (T,), generator=gen)
    x = (torch.randn(T, D, generator=gen) + 3 * torch.cat(W)[tgt].float()).to(torch.bfloat16)
    tgt[torch.rand(T, generator=gen) < 0.2] = IGN
    if T > 4:
        tgt[1] = V  # outside the vocabulary
        tgt[2] = -5
        tgt[3] = V - 1
        tgt[4] = 0
    grad = torch.rand(T, generator=gen) / T
    return x, W, tgt, grad


@pytest.mark.parametrize("T,D,shards", LOSS)
def test_vocab_loss(T, D, shards):
    x, W, tgt, _ = loss_inputs(T, D, shards, T + D)
    loss, lse = poison(T, dtype=torch.float32), poison(T, dtype=torch.float32)
    rra.rra_vocab_loss(x.cuda(), cuda(W), tgt.cuda(), loss, lse, ignore_index=IGN)
    status_ok()
    want = ref.vocab_loss(x, W, tgt, IGN)
    ref.assert_within(lse, *want["lse"], "lse")
    ref.assert_within(loss, *want["loss"], "loss")


@pytest.mark.parametrize("D", [64, 515])
@pytest.mark.parametrize("size", [0.0, 97.0, 1000.0])
@pytest.mark.parametrize("T", [8, 16, 17, 300, 1300])
def test_loss_where_the_target_has_nearly_all_of_the_mass(T, size, D):
    """A target's logit of any size far above the others: the loss is next to nothing, and as exact as for small
    logits (an absolute bound, whatever the size), few tokens and many alike."""
    shards, groups = (700, 333), 5
    V = sum(shards)
    gen = torch.Generator().manual_seed(T + D)
    # every logit is exact in any order of summation: `size` for all, less 6 to 12 in eighths, and 10 more for the
    # target of the token's group
    heads = torch.randperm(V, generator=gen)[:groups]
    W, x = torch.zeros(V, D, dtype=torch.bfloat16), torch.zeros(T, D, dtype=torch.bfloat16)
    W[:, 0] = size
    W[:, 1] = -torch.randint(48, 97, (V,), generator=gen).to(torch.bfloat16) / 8
    W[heads, 1] = 0
    W[heads, 2 + torch.arange(groups)] = 10.0
    mine = torch.arange(T) % groups
    x[:, :2] = 1.0
    x[torch.arange(T), 2 + mine] = 1.0
    tgt = heads[mine]
    loss, lse = poison(T, dtype=torch.float32), poison(T, dtype=torch.float32)
    rra.rra_vocab_loss(x.cuda(), [w.contiguous().cuda() for w in torch.split(W, list(shards))], tgt.cuda(), loss, lse)
    status_ok()
    l = x.double() @ W.double().t()
    want = torch.logsumexp(l, 1)
    hit = l[torch.arange(T), tgt]
    # the largest exponential is 1, the others (3e-4 in all) are off by 2^-22 of themselves, the sum takes at most
    # 8 + 32 + 16 roundings of 2^-24 in a chain and its logarithm two more
    off = 2.0 ** -22 * 3e-4 + 60 * ref.F32
    ref.assert_within(loss, want - hit, torch.full((T,), off, dtype=torch.float64), "loss")
    assert float(loss.min()) >= 0.0
    ref.assert_within(lse, want, ref.F32 * want.abs() + off, "lse")


@pytest.mark.parametrize("room", ["default", "least", "some"])
@pytest.mark.parametrize("T,D,shards", LOSS)
def test_vocab_loss_backward(T, D, shards, room):
    x, W, tgt, grad = loss_inputs(T, D, shards, T + 3 * D)
    grad[tgt == IGN] = math.nan  # an ignored row's gradient is zero whatever stands here
    xc, Wc, tc = x.cuda(), cuda(W), tgt.cuda()
    want = ref.vocab_loss(x, W, tgt, IGN, grad)
    lse = want["lse"][0].float().cuda()
    dx, dW = poison(T, D), [poison(v, D) for v in shards]
    nb = rra.rra_vocab_loss_workspace_bytes(T, D, shards, 1 if room == "default" else 2)
    if room == "some":  # pieces of a few tiles, whose products split their K axis
        nb += 6 * T * 512 + (24 << 20)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    rra.rra_vocab_loss_backward(xc, Wc, tc, lse, grad.cuda(), dx, dW, ignore_index=IGN, workspace=ws)
    status_ok()
    ref.assert_within(dx, *want["dx"], "dx")
    for r in range(len(shards)):
        if shards[r]:
            ref.assert_within(dW[r], *want["dW"][r], "dweights[%d]" % r)
    ref.assert_norm_close(dx, want["dx"][0], 2 * ref.BF, "dx")
    ref.assert_norm_close(torch.cat(dW), torch.cat([w for w, _ in want["dW"]]), 2 * ref.BF, "dweights")


@pytest.mark.parametrize("room", ["default", "least"])
@pytest.mark.parametrize("T,D,shards", [
    (1, 64, (256,)), (1, 346, (441,) * 6), (2, 515, (129, 0, 700)), (8, 1024, (1, 300)), (17, 72, (2000,)),
    (31, 333, (129, 65)), (32, 5120, (260, 300)),
])
def test_weight_gradient_of_few_tokens(T, D, shards, room):
    """dW of up to 32 tokens has no rounding of dl in it: one half step of its own."""
    x, W, tgt, grad = loss_inputs(T, D, shards, 7 * T + D)
    want = ref.vocab_loss(x, W, tgt, IGN, grad, rest=True)
    dx, dW = poison(T, D), [poison(v, D) for v in shards]
    ws = torch.empty(rra.rra_vocab_loss_workspace_bytes(T, D, shards, 1 if room == "default" else 2),
                     dtype=torch.uint8, device="cuda")
    rra.rra_vocab_loss_backward(x.cuda(), cuda(W), tgt.cuda(), want["lse"][0].float().cuda(), grad.cuda(), dx, dW,
                                ignore_index=IGN, workspace=ws)
    status_ok()
    ref.assert_within(dx, *want["dx"], "dx")
    for r in range(len(shards)):
        if shards[r]:
            ref.assert_within(dW[r], *want["dW"][r], "dweights[%d]" % r)


@pytest.mark.parametrize("T,D,shards", [(300, 72, (40, 260)), (129, 515, (300,)), (3, 1024, (700, 90))])
def test_many_tokens_of_one_target(T, D, shards):
    """More targets in a block of rows than a warp takes at a time, and none in the others."""
    x, W, _, grad = loss_inputs(T, D, shards, T)
    tgt = torch.full((T,), sum(shards) - 9)
    tgt[::3] = 5
    tgt[1::7] = IGN
    want = ref.vocab_loss(x, W, tgt, IGN, grad)
    dx, dW = poison(T, D), [poison(v, D) for v in shards]
    rra.rra_vocab_loss_backward(x.cuda(), cuda(W), tgt.cuda(), want["lse"][0].float().cuda(), grad.cuda(), dx, dW)
    status_ok()
    ref.assert_within(dx, *want["dx"], "dx")
    for r in range(len(shards)):
        ref.assert_within(dW[r], *want["dW"][r], "dweights[%d]" % r)


# -- RMSNorm with a checkpoint -----------------------------------------------

NORM = [(1, 1, 128), (2, 3, 5120), (8, 8, 5120), (3, 5, 1027), (4, 2, 1), (5, 7, 130), (2, 64, 4096), (6, 700, 260),
        (7, 3, 51200), (1, 1300, 96)]


def depth(D, per_unit):
    """Longest chain of float32 additions in a row's reduction."""
    units = -(-D // per_unit)
    return per_unit * -(-units // 256) + 5 + 8


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n,T,D", NORM)
def test_norm_save_and_restore(n, T, D, dtype):
    dt = getattr(torch, dtype)
    gen = torch.Generator().manual_seed(n * 100 + D)
    col = torch.exp(torch.randn(D, generator=gen) * 2)
    xs = [(torch.randn(T, D, generator=gen) * col).to(dt) for _ in range(n)]
    gamma = (1 + 0.1 * torch.randn(D, generator=gen)).to(dt)
    ins = cuda(xs)
    outs, plain = [poison(T, D, dtype=dt) for _ in range(n)], [poison(T, D, dtype=dt) for _ in range(n)]
    codes = poison(T, D, dtype=torch.float8_e4m3fn)
    scales = poison(T, -(-D // 128), dtype=torch.uint8)
    rstd = poison(T, dtype=torch.float32)
    rra.rra_allreduce_rmsnorm_save8(ins, outs, gamma.cuda(), D, codes, scales, rstd, eps=1e-5)
    rra.rra_allreduce_rmsnorm(ins, plain, gamma.cuda(), D, eps=1e-5)
    for r in range(n):  # the same outputs as the operator that saves nothing, bit for bit
        assert torch.equal(outs[r], plain[r])
    s = ref.ascending_sum(xs)
    val, sc = ref.codes_of(s)
    assert torch.equal(scales.cpu(), sc)
    e = torch.exp2(sc.double() - 127).repeat_interleave(128, 1)[:, :D]
    assert torch.equal(codes.cpu().float().double() * e, val)
    q = 1 / torch.sqrt((s.double() ** 2).mean(1) + 1e-5)
    pu = 8 if dtype == "bfloat16" else 4
    ref.assert_within(rstd, q, q * (depth(D, pu) * 2.0 ** -25 + 2.0 ** -22), "rstd")
    half = ref.BF if dtype == "bfloat16" else ref.F32
    raw, norm = poison(T, D, dtype=dt), poison(T, D, dtype=dt)
    rra.rra_rmsnorm_restore8(codes, scales, None, None, raw)
    assert torch.equal(raw.cpu().double(), val)  # a code times a power of two is exact in both types
    rra.rra_rmsnorm_restore8(codes, scales, rstd, gamma.cuda(), norm)
    want = val * rstd.cpu().double()[:, None] * gamma.double()
    ref.assert_within(norm, want, want.abs() * (half + 3 * ref.F32) + 1e-40, "restored")


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("n,T,D", NORM)
def test_norm_backward(n, T, D, dtype):
    dt = getattr(torch, dtype)
    gen = torch.Generator().manual_seed(n * 31 + D)
    gamma = (1 + 0.1 * torch.randn(D, generator=gen)).to(dt)
    x = [(torch.randn(T, D, generator=gen) * 3).to(dt)]
    codes = torch.empty(T, D, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(T, -(-D // 128), dtype=torch.uint8, device="cuda")
    rstd = torch.empty(T, device="cuda")
    rra.rra_allreduce_rmsnorm_save8(cuda(x), [torch.empty_like(x[0], device="cuda")], gamma.cuda(), D, codes, scales,
                                    rstd)
    gs = [(torch.randn(T, D, generator=gen) * 1e-2).to(dt) for _ in range(n)]
    dxs, dgamma = [poison(T, D, dtype=dt) for _ in range(n)], poison(D, dtype=torch.float32)
    rra.rra_allreduce_rmsnorm_backward8(cuda(gs), dxs, codes, scales, rstd, gamma.cuda(), dgamma)
    status_ok()
    e = torch.exp2(scales.cpu().double() - 127).repeat_interleave(128, 1)[:, :D]
    q = rstd.cpu().double()[:, None]
    h = codes.cpu().float().double() * e * q
    dy = sum(g.double() for g in gs)
    mag = sum(g.double().abs() for g in gs)
    w, W = dy * gamma.double(), mag * gamma.double().abs()
    ds = q * (w - h * (w * h).mean(1, keepdim=True))
    c = (depth(D, 8 if dtype == "bfloat16" else 4) + n + 10) * ref.F32
    half = ref.BF if dtype == "bfloat16" else ref.F32
    bound = half * ds.abs() + c * q * (W + h.abs() * (W * h.abs()).mean(1, keepdim=True)) + 1e-40
    for r in range(n):
        ref.assert_within(dxs[r], ds, bound, "dxs[%d]" % r)
        assert torch.equal(dxs[r], dxs[0])
    chain = (math.ceil(T / 608) + math.ceil(608 / 8) + 8 + n + 3) * ref.F32
    ref.assert_within(dgamma, (dy * h).sum(0), chain * (mag * h.abs()).sum(0) + 1e-40, "dgamma")


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("n,T,D", [(2, 6, 256), (3, 5, 131), (1, 4, 6272)])
def test_norm_in_place_and_off_16_bytes(n, T, D, shift, dtype):
    """Buffers that start `shift` elements off 16 bytes, and outputs over
    their inputs, give the bits of aligned separate buffers."""
    dt = getattr(torch, dtype)
    gen = torch.Generator().manual_seed(D + shift)
    gamma = (1 + 0.1 * torch.randn(D, generator=gen)).to(dt).cuda()
    xs = [torch.randn(T, D, generator=gen).to(dt).cuda() for _ in range(n)]

    def off(t):
        room = torch.empty(t.numel() + shift, dtype=t.dtype, device="cuda")
        room[shift:].copy_(t.reshape(-1))
        return room[shift:].view(t.shape)

    def saved():
        return (torch.empty(T, D, dtype=torch.uint8, device="cuda"),
                torch.empty(T, -(-D // 128), dtype=torch.uint8, device="cuda"), torch.empty(T, device="cuda"))

    want = [torch.empty_like(x) for x in xs]
    keep = saved()
    rra.rra_allreduce_rmsnorm_save8(xs, want, gamma, D, *keep)
    ins, again = [off(x) for x in xs], saved()
    c = off(again[0])
    rra.rra_allreduce_rmsnorm_save8(ins, ins, off(gamma), D, c, again[1], again[2])
    assert all(torch.equal(a, b) for a, b in zip(ins, want))
    assert torch.equal(c, keep[0]) and torch.equal(again[1], keep[1]) and torch.equal(again[2], keep[2])

    y, y2 = torch.empty_like(xs[0]), off(xs[0])
    rra.rra_rmsnorm_restore8(*keep, gamma, y)
    rra.rra_rmsnorm_restore8(c, keep[1], keep[2], off(gamma), y2)
    assert torch.equal(y, y2)

    dxs, dg, dg2 = [torch.empty_like(x) for x in xs], torch.empty(D, device="cuda"), torch.empty(D, device="cuda")
    rra.rra_allreduce_rmsnorm_backward8(xs, dxs, *keep, gamma, dg)
    gs = [off(x) for x in xs]
    rra.rra_allreduce_rmsnorm_backward8(gs, gs, c, keep[1], keep[2], off(gamma), dg2)
    # the row's mean may be added in another order: one step of the type
    for a, b in zip(gs, dxs):
        half = ref.BF if dtype == "bfloat16" else 32 * ref.F32
        assert float((a.double() - b.double()).abs().max()) <= 2 * half * float(b.double().abs().max())
    assert float((dg - dg2).abs().max()) <= 64 * ref.F32 * float(sum(x.double().abs().sum(0).max() for x in xs) * 8)


def test_norm_checkpoint_of_extreme_values():
    """Zeros, subnormals, the type's largest values, infinities and NaN."""
    D = 384
    s = torch.zeros(6, D)
    s[1, :4] = torch.tensor([1e-40, -3e-39, 2.0 ** -133, 1.0e-38])
    s[2, :3] = torch.tensor([3.3895e38, -1e38, 1e30])
    s[3, 5], s[3, 6], s[3, 7] = math.inf, -math.inf, 2.5
    s[4, 130], s[4, 131] = math.nan, -7.0
    s[5] = torch.linspace(-1e-3, 1e3, D)
    x = s.cuda()
    codes = torch.empty(6, D, dtype=torch.float8_e4m3fn, device="cuda")
    scales, rstd = torch.empty(6, 3, dtype=torch.uint8, device="cuda"), torch.empty(6, device="cuda")
    rra.rra_allreduce_rmsnorm_save8([x], [torch.empty_like(x)], torch.ones(D, device="cuda"), D, codes, scales, rstd)
    val, sc = ref.codes_of(s)
    assert torch.equal(scales.cpu(), sc)
    val = val.float().double()  # restored values are rounded to float32: a code of 2^128 is infinite there
    out = torch.empty_like(x)
    rra.rra_rmsnorm_restore8(codes, scales, None, None, out)
    got = out.cpu().double()
    assert torch.equal(torch.isnan(got), torch.isnan(val))
    assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(val))


# -- how the calls behave ----------------------------------------------------

def step_inputs(T=96, D=256, F=200, V=777, n=2, seed=5):
    gen = torch.Generator().manual_seed(seed)
    d = dict(x=rnd(gen, T, D), G=[rnd(gen, F, D, scale=D ** -0.5) for _ in range(n)],
             U=[rnd(gen, F, D, scale=D ** -0.5) for _ in range(n)], da=[rnd(gen, T, F, scale=1e-2) for _ in range(n)],
             W=[rnd(gen, V, D, scale=D ** -0.5) for _ in range(n)], tgt=torch.randint(0, V * n, (T,), generator=gen),
             grad=torch.rand(T, generator=gen) / T)
    return {k: cuda(v) if isinstance(v, list) else v.cuda() for k, v in d.items()}


def step_outputs(d):
    e = lambda t: torch.empty_like(t)
    return dict(acts=[e(a) for a in d["da"]], dx=e(d["x"]), dG=[e(w) for w in d["G"]], dU=[e(w) for w in d["U"]],
                loss=torch.empty_like(d["grad"]), lse=torch.empty_like(d["grad"]), dx2=e(d["x"]),
                dW=[e(w) for w in d["W"]])


def run_step(d, o, ws, stream=None):
    rra.rra_gated_ffn(d["x"], d["G"], d["U"], o["acts"], workspace=ws, stream=stream)
    rra.rra_gated_ffn_backward(d["x"], d["G"], d["U"], d["da"], o["dx"], o["dG"], o["dU"], workspace=ws, stream=stream)
    rra.rra_vocab_loss(d["x"], d["W"], d["tgt"], o["loss"], o["lse"], workspace=ws, stream=stream)
    rra.rra_vocab_loss_backward(d["x"], d["W"], d["tgt"], o["lse"], d["grad"], o["dx2"], o["dW"], workspace=ws,
                                stream=stream)


def flat(o):
    return [t for v in o.values() for t in (v if isinstance(v, list) else [v])]


def test_repeat_stream_and_graph_give_the_same_bits():
    d = step_inputs()
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    want = step_outputs(d)
    run_step(d, want, ws)
    torch.cuda.synchronize()
    again = step_outputs(d)
    run_step(d, again, ws)
    side = step_outputs(d)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run_step(d, side, ws, stream=s)  # a stream that is not the current one
    s.synchronize()
    own = step_outputs(d)
    with torch.cuda.stream(s):
        run_step(d, own, None)  # workspaces made by the calls
    s.synchronize()
    graphed = step_outputs(d)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        run_step(d, graphed, ws)
    for t in flat(graphed):
        t.zero_()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    status_ok()
    for other in (again, side, own, graphed):
        for a, b in zip(flat(want), flat(other)):
            assert torch.equal(a, b)


def test_no_tokens_and_no_columns():
    dev = dict(device="cuda", dtype=torch.bfloat16)
    x, w = torch.empty(0, 64, **dev), [torch.ones(40, 64, **dev)]
    a, dx, dg, du = [torch.empty(0, 40, **dev)], torch.empty(0, 64, **dev), [poison(40, 64)], [poison(40, 64)]
    rra.rra_gated_ffn(x, w, w, a)
    rra.rra_gated_ffn_backward(x, w, w, a, dx, dg, du)
    assert not dg[0].any() and not du[0].any()
    none = torch.empty(0, device="cuda")
    tgt = torch.empty(0, dtype=torch.int64, device="cuda")
    dw = [poison(40, 64)]
    rra.rra_vocab_loss(x, w, tgt, none, none.clone())
    rra.rra_vocab_loss_backward(x, w, tgt, none, none.clone(), dx, dw)
    assert not dw[0].any()
    dgamma = poison(64, dtype=torch.float32)
    codes, scales = torch.empty(0, 64, device="cuda", dtype=torch.uint8), torch.empty(0, 1, device="cuda", dtype=torch.uint8)
    rra.rra_allreduce_rmsnorm_backward8([x], [torch.empty_like(x)], codes, scales, none, torch.ones(64, **dev), dgamma)
    assert not dgamma.any()
    # no columns: dx is zero
    x2, w0, dx2 = torch.ones(3, 64, **dev), [torch.empty(0, 64, **dev)], poison(3, 64)
    rra.rra_gated_ffn_backward(x2, w0, w0, [torch.empty(3, 0, **dev)], dx2, [torch.empty(0, 64, **dev)],
                               [torch.empty(0, 64, **dev)])
    assert not dx2.any()
    status_ok()


def test_every_target_ignored():
    x, W, tgt, grad = loss_inputs(40, 128, (300, 200), 3)
    tgt[:] = IGN
    xc, Wc, tc = x.cuda(), cuda(W), tgt.cuda()
    loss, lse = poison(40, dtype=torch.float32), poison(40, dtype=torch.float32)
    rra.rra_vocab_loss(xc, Wc, tc, loss, lse)
    assert not loss.any() and torch.isfinite(lse).all()
    dx, dW = poison(40, 128), [poison(300, 128), poison(200, 128)]
    rra.rra_vocab_loss_backward(xc, Wc, tc, lse, torch.full((40,), math.inf, device="cuda"), dx, dW)
    status_ok()
    assert not dx.any() and not any(w.any() for w in dW)


@pytest.mark.parametrize("T", [3, 40])
def test_what_is_not_finite_stays_in_its_row(T):
    D, shards = 640, (300, 200)
    x, W, tgt, grad = loss_inputs(T, D, shards, 11)
    tgt = torch.full((T,), 7)
    clean = [torch.empty(T, device="cuda"), torch.empty(T, device="cuda")]
    rra.rra_vocab_loss(x.cuda(), cuda(W), tgt.cuda(), *clean)
    x[1, 5] = math.nan
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    rra.rra_vocab_loss(x.cuda(), cuda(W), tgt.cuda(), loss, lse)
    assert bool(torch.isnan(loss[1])) and bool(torch.isnan(lse[1]))
    rest = [t for t in range(T) if t != 1]
    assert torch.equal(loss[rest], clean[0][rest]) and torch.equal(lse[rest], clean[1][rest])
    acts, ref_acts = [torch.empty(T, 24, dtype=torch.bfloat16, device="cuda")], [
        torch.empty(T, 24, dtype=torch.bfloat16, device="cuda")]
    w = [W[0][:24].contiguous().cuda()]
    rra.rra_gated_ffn(x.cuda(), w, w, acts)
    x[1, 5] = 0
    rra.rra_gated_ffn(x.cuda(), w, w, ref_acts)
    assert torch.isnan(acts[0][1].float()).all() and torch.equal(acts[0][rest], ref_acts[0][rest])
    status_ok()


def test_masked_logits_of_minus_infinity():
    """Vocabulary rows that are out of play: weights whose logits are -inf
    carry no probability and get no gradient beyond their own."""
    T, D = 20, 64
    gen = torch.Generator().manual_seed(2)
    x = rnd(gen, T, D).abs() + 0.25
    W = rnd(gen, 300, D, scale=0.1)
    dead = torch.zeros(300, dtype=torch.bool)
    dead[100:160] = True
    dead[299] = True
    Wd = W.clone()
    Wd[dead] = -math.inf  # every product with a positive x is -inf
    tgt = torch.randint(0, 100, (T,), generator=gen)
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    rra.rra_vocab_loss(x.cuda(), [Wd.cuda()], tgt.cuda(), loss, lse)
    want = ref.vocab_loss(x, [W[~dead]], tgt, IGN)  # the targets lie before the dead rows
    ref.assert_within(lse, *want["lse"], "lse")
    ref.assert_within(loss, *want["loss"], "loss")
    tgt[4] = 120  # a target out of play: its loss is infinite
    rra.rra_vocab_loss(x.cuda(), [Wd.cuda()], tgt.cuda(), loss, lse)
    assert float(loss[4]) == math.inf and torch.isfinite(loss[torch.arange(T) != 4]).all()
    status_ok()


def test_gradients_against_differences():
    """Central differences of the loss in float64 along random directions."""
    T, D, shards = 24, 64, (150, 83)
    x, W, tgt, grad = loss_inputs(T, D, shards, 8)
    tgt = torch.where((tgt < 0) | (tgt >= sum(shards)), torch.full_like(tgt, IGN), tgt)
    lse, loss = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    dx, dW = torch.empty(T, D, dtype=torch.bfloat16, device="cuda"), [torch.empty_like(w, device="cuda") for w in W]
    rra.rra_vocab_loss(x.cuda(), cuda(W), tgt.cuda(), loss, lse)
    rra.rra_vocab_loss_backward(x.cuda(), cuda(W), tgt.cuda(), lse, grad.cuda(), dx, dW)

    def total(xx, ww):
        return float((ref.vocab_loss(xx, ww, tgt, IGN)["loss"][0] * grad.double()).sum())

    gen = torch.Generator().manual_seed(1)
    for _ in range(4):
        vx = torch.randn(T, D, generator=gen, dtype=torch.float64)
        vw = [torch.randn(w.shape, generator=gen, dtype=torch.float64) for w in W]
        h = 1e-4
        num = (total(x.double() + h * vx, [w.double() + h * v for w, v in zip(W, vw)])
               - total(x.double() - h * vx, [w.double() - h * v for w, v in zip(W, vw)])) / (2 * h)
        parts = [(dx.cpu().double() * vx)] + [g.cpu().double() * v for g, v in zip(dW, vw)]
        # each gradient is off by at most two bfloat16 half steps of its terms' size
        slack = 4 * ref.BF * sum(float(p.norm()) for p in parts) + 1e-6 * abs(num)
        assert abs(num - sum(float(p.sum()) for p in parts)) <= slack


def test_sm_budget_and_the_recorder():
    d = step_inputs(T=300)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    want, small = step_outputs(d), step_outputs(d)
    run_step(d, want, ws)
    rra.rra_set_max_ctas(8)
    try:
        run_step(d, small, ws)
        line = [l for l in rra.rra_dump_recent().splitlines() if "gated_ffn " in l][-1]
        assert "grid=8" in line
    finally:
        rra.rra_set_max_ctas(0)
    torch.cuda.synchronize()
    status_ok()
    for a, b in zip(flat(want), flat(small)):
        assert torch.equal(a, b)


def largest_grid(call):
    """Of the launches of the last call of this name."""
    line = [l for l in rra.rra_dump_recent().splitlines() if " %s " % call in l][-1]
    return int(line.split("grid=")[1].split()[0])


def under_budget(max_ctas, call, name, least=1):
    """`call` under an SM budget: no launch of it has more CTAs."""
    rra.rra_set_max_ctas(max_ctas)
    try:
        call()
        torch.cuda.synchronize()
        assert largest_grid(name) <= max(least, max_ctas), "%s: %d CTAs" % (name, largest_grid(name))
    finally:
        rra.rra_set_max_ctas(0)


@pytest.mark.parametrize("max_ctas", [1, 7, 64])
@pytest.mark.parametrize("T,D", [(300, 5120), (130, 1027), (90, 8192), (75, 51200), (70, 51199)])
def test_norm_keeps_the_sm_budget(T, D, max_ctas):
    gen = torch.Generator().manual_seed(D)
    xs, gamma = [rnd(gen, T, D).cuda() for _ in range(2)], rnd(gen, D).cuda()

    def results():
        return dict(outs=[poison(T, D) for _ in xs], codes=poison(T, D, dtype=torch.uint8),
                    scales=poison(T, -(-D // 128), dtype=torch.uint8), rstd=poison(T, dtype=torch.float32),
                    again=poison(T, D), dxs=[poison(T, D) for _ in xs], dgamma=poison(D, dtype=torch.float32))

    def save(o):
        rra.rra_allreduce_rmsnorm_save8(xs, o["outs"], gamma, D, o["codes"], o["scales"], o["rstd"])

    def restore(o):
        rra.rra_rmsnorm_restore8(o["codes"], o["scales"], o["rstd"], gamma, o["again"])

    def back(o):
        rra.rra_allreduce_rmsnorm_backward8(xs, o["dxs"], o["codes"], o["scales"], o["rstd"], gamma, o["dgamma"])

    want, small = results(), results()
    for call in (save, restore, back):
        call(want)
    under_budget(max_ctas, lambda: save(small), "allreduce_rmsnorm_save8")
    under_budget(max_ctas, lambda: restore(small), "rmsnorm_restore8")
    under_budget(max_ctas, lambda: back(small), "allreduce_rmsnorm_backward8")
    status_ok()
    a, b = want.pop("dgamma").double(), small.pop("dgamma").double()
    for x, y in zip(flat(want), flat(small)):
        assert torch.equal(x, y)
    # rows are added in another order: chains of at most T additions
    mag = (sum(x.double().abs() for x in xs) * 4 * xs[0].double().abs().max()).sum(0)
    assert bool(((a - b).abs() <= 2 * T * ref.F32 * mag).all())


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("max_ctas", [1, 7, 64])
@pytest.mark.parametrize("T,D", [(300, 5120), (130, 1027), (66, 51200)])
def test_fused_norm_keeps_the_sm_budget(T, D, max_ctas, dtype):
    gen = torch.Generator().manual_seed(D)
    dt = getattr(torch, dtype)
    xs, gamma = [rnd(gen, T, D, dtype=dt).cuda() for _ in range(3)], rnd(gen, D, dtype=dt).cuda()
    want, small = [poison(T, D, dtype=dt) for _ in xs], [poison(T, D, dtype=dt) for _ in xs]
    rra.rra_allreduce_rmsnorm(xs, want, gamma, D)
    under_budget(max_ctas, lambda: rra.rra_allreduce_rmsnorm(xs, small, gamma, D), "allreduce_rmsnorm")
    status_ok()
    assert all(torch.equal(a, b) for a, b in zip(want, small))


@pytest.mark.parametrize("max_ctas", [1, 7, 64])
@pytest.mark.parametrize("T", [5, 20, 300, 1300])
def test_products_keep_the_sm_budget(T, max_ctas):
    d = step_inputs(T=T, D=515, F=130, V=1500)
    d["tgt"][::5] = IGN
    d["tgt"][1::7] = 40
    ws = torch.empty(256 << 20, dtype=torch.uint8, device="cuda")
    want, small = step_outputs(d), step_outputs(d)
    run_step(d, want, ws)
    calls = {
        "gated_ffn": lambda o: rra.rra_gated_ffn(d["x"], d["G"], d["U"], o["acts"], workspace=ws),
        "gated_ffn_backward": lambda o: rra.rra_gated_ffn_backward(d["x"], d["G"], d["U"], d["da"], o["dx"], o["dG"],
                                                                   o["dU"], workspace=ws),
        "vocab_loss": lambda o: rra.rra_vocab_loss(d["x"], d["W"], d["tgt"], o["loss"], o["lse"], workspace=ws),
        "vocab_loss_backward": lambda o: rra.rra_vocab_loss_backward(d["x"], d["W"], d["tgt"], want["lse"], d["grad"],
                                                                     o["dx2"], o["dW"], workspace=ws),
    }
    for name, call in calls.items():
        under_budget(max_ctas, lambda: call(small), name, least=2)  # products run as pairs of CTAs
    status_ok()
    for k in ("loss", "lse"):  # few tokens: the parts of the statistics are the CTAs'
        a, b = want.pop(k), small.pop(k)
        assert torch.allclose(a, b, rtol=0, atol=2.0 ** -19) if T <= 16 else torch.equal(a, b)
    for x, y in zip(flat(want), flat(small)):
        assert torch.equal(x, y)


def test_a_workspace_does_not_depend_on_the_sm_budget():
    """Its size is asked for under a budget, the call made without one."""
    x, W, tgt, _ = loss_inputs(8, 64, (9000,), 21)
    shards = [9000]
    rra.rra_set_max_ctas(1)
    try:
        nb = rra.rra_vocab_loss_workspace_bytes(8, 64, shards, 0)
    finally:
        rra.rra_set_max_ctas(0)
    assert nb == rra.rra_vocab_loss_workspace_bytes(8, 64, shards, 0)
    loss, lse = poison(8, dtype=torch.float32), poison(8, dtype=torch.float32)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    rra.rra_vocab_loss(x.cuda(), cuda(W), tgt.cuda(), loss, lse, ignore_index=IGN, workspace=ws)
    status_ok()
    want = ref.vocab_loss(x, W, tgt, IGN)
    ref.assert_within(lse, *want["lse"], "lse")


def test_weights_past_four_gigabytes():
    """A shard of more than 2^32 bytes: the last rows land where they belong."""
    D, V = 4096, 540_001  # 4.42 GB
    T = 20
    W = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    gen = torch.Generator().manual_seed(4)
    pick = torch.randint(V - 5000, V, (T,), generator=gen)
    W[pick, 0] = 9.0
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    rra.rra_vocab_loss(x, [W], pick.cuda(), loss, lse)
    uniq = len(set(pick.tolist()))
    want = math.log((V - uniq) + uniq * math.exp(9.0))
    assert torch.allclose(lse.cpu().double(), torch.full((T,), want, dtype=torch.float64), rtol=1e-5)
    assert torch.allclose(loss.cpu().double(), torch.full((T,), want - 9.0, dtype=torch.float64), rtol=1e-5)
    grad = torch.ones(T, device="cuda")
    dx, dW = torch.empty_like(x), torch.empty_like(W)
    rra.rra_vocab_loss_backward(x, [W], pick.cuda(), lse, grad, dx, [dW])
    status_ok()
    p9, p1 = math.exp(9.0 - want), math.exp(-want)
    col = dW[:, 0].float().cpu().double()
    assert torch.equal(dW[:, 1].float().cpu(), torch.zeros(V))
    count = torch.zeros(V, dtype=torch.float64)
    for t in pick.tolist():
        count[t] += 1
    full = torch.full((V,), T * p1, dtype=torch.float64)
    full[count > 0] = T * p9 - count[count > 0]
    assert float((col - full).abs().max()) <= 4 * ref.BF * float(full.abs().max())
    assert float((col - full)[count == 0].abs().max()) <= 4 * ref.BF * T * p1
