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
    (1, 1, 64, 128, 0), (1, 128, 64, 128, 0), (1, 256, 256, 128, 1), (2, 256, 128, 256, 0), (1, 300, 200, 130, 1),
    (3, 77, 88, 33, 0), (2, 1, 512, 520, 1), (8, 16, 128, 40, 0), (2, 129, 1027, 65, 0), (3, 5, 7, 3, 1),
    (2, 513, 640, 384, 0), (1, 1, 1, 1, 0), (4, 700, 72, 1000, 0),
    # few tokens: the register path, rows on and off 16 bytes
    (1, 1, 5120, 24, 0), (8, 8, 1024, 17, 1), (3, 9, 2056, 64, 0), (2, 16, 515, 33, 0), (1, 7, 1027, 8, 1), (2, 3, 771, 100, 0),
    (1, 17, 1024, 72, 0), (2, 40, 520, 136, 1),
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


# -- vocabulary loss ---------------------------------------------------------

LOSS = [  # tokens, hidden, shard heights
    (1, 64, (256,)), (256, 64, (256,)), (5, 64, (300, 300)), (300, 128, (512, 511)), (33, 200, (1000, 1000, 997)),
    (129, 1027, (257, 0, 64)), (7, 515, (1,)), (64, 72, (100,) * 8), (2, 8, (3, 2)), (513, 256, (2048, 2048)),
    # few tokens: the register path
    (1, 5120, (700, 700)), (8, 1024, (16, 15, 0, 33)), (16, 515, (401, 400)), (9, 1027, (3000,)), (5, 771, (17,)),
    (17, 1024, (500,)),
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


@pytest.mark.parametrize("room", ["default", "least"])
@pytest.mark.parametrize("T,D,shards", LOSS)
def test_vocab_loss_backward(T, D, shards, room):
    x, W, tgt, grad = loss_inputs(T, D, shards, T + 3 * D)
    grad[tgt == IGN] = math.nan  # an ignored row's gradient is zero whatever stands here
    xc, Wc, tc = x.cuda(), cuda(W), tgt.cuda()
    want = ref.vocab_loss(x, W, tgt, IGN, grad)
    lse = want["lse"][0].float().cuda()
    dx, dW = poison(T, D), [poison(v, D) for v in shards]
    nb = rra.rra_vocab_loss_workspace_bytes(T, D, shards, 2 if room == "least" else 1)
    ws = torch.empty(nb, dtype=torch.uint8, device="cuda")
    rra.rra_vocab_loss_backward(xc, Wc, tc, lse, grad.cuda(), dx, dW, ignore_index=IGN, workspace=ws)
    status_ok()
    ref.assert_within(dx, *want["dx"], "dx")
    for r in range(len(shards)):
        if shards[r]:
            ref.assert_within(dW[r], *want["dW"][r], "dweights[%d]" % r)
    ref.assert_norm_close(dx, want["dx"][0], 2 * ref.BF, "dx")
    ref.assert_norm_close(torch.cat(dW), torch.cat([w for w, _ in want["dW"]]), 2 * ref.BF, "dweights")


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
