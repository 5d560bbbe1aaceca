"""The serving-step operators on a GPU against their definitions in 64 bits
(serve_ref.py).

Bounds.  Quantised matrices are equal byte for byte.  A product sums exact
terms in float32: each of its ceil(K / 64) steps may lose the last bit of the
sum so far (truncation: 2^-23 of it), and so may adding up to 8 partial sums,
so a sum is off by at most (K / 64 + 10) 2^-23 times the sum of the terms'
absolute values; rounding to bfloat16 adds 2^-8 of the value (half a step,
relative), to float32 2^-24.  A gated block's activations inherit that through
the activation (|act'| <= 1.13, |act(g)| <= |g|; its own functions are within
2^-20) and are then rounded to MX4: half a step more."""
import math

import pytest
import torch

import collective_all_reduce_rank_gb300 as rra
import serve_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def ready():
    rra.rra_init(0)
    yield
    assert rra.rra_query_status()[0] == rra.RRA_SUCCESS


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def room(rows, cols, fill=0xA5):
    return (torch.full((rows, 16 * ref.blocks(cols)), fill, dtype=torch.uint8, device="cuda"),
            torch.full((ref.scale_bytes(rows, cols),), fill, dtype=torch.uint8, device="cuda"))


def matrix(g, rows, cols, scale=1.0):
    """A random matrix in MX4 on the GPU: ((codes, scales), values)."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * scale
    x *= torch.exp(torch.randn(rows, 1, generator=g, device="cuda"))
    codes, scales, v = ref.pack(x)
    return (codes.contiguous(), scales), v


def shifted(t, by):
    """A contiguous copy of t that starts `by` elements behind a 16-byte boundary."""
    buf = torch.empty(t.numel() + by + 16, dtype=t.dtype, device=t.device)
    view = buf[by:by + t.numel()].view(t.shape)
    view.copy_(t)
    return view


# -- matrices ----------------------------------------------------------------

def nasty(g, rows, cols, dt):
    x = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(4 * torch.randn(rows, cols, generator=g, device="cuda"))
    flat = x.view(-1)
    n = flat.numel()
    for i, v in enumerate([0.0, -0.0, 6.0, -6.0, 5.0, 2.5, 3.4e38, 1e-40, 2.0 ** -126, math.inf, -math.inf, math.nan]):
        if n > 300 and i < n:
            flat[(i * 977) % n] = v
    if rows > 3:
        x[1] = 0
        x[2] = torch.tensor([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25], device="cuda").repeat(cols // 8 + 1)[:cols]
    return x.to(dt)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 31), (1, 32), (1, 33), (3, 128), (5, 129), (130, 96), (257, 1027),
                                       (64, 5120), (1, 5120), (129, 2056)])
def test_quantize_and_restore(rows, cols, dtype):
    x = nasty(gen(rows + cols), rows, cols, DT[dtype])
    codes, scales = room(rows, cols)
    rra.rra_mx4_quantize(x, codes, scales)
    want, byte = ref.quantize(x)
    assert torch.equal(codes, want)
    assert torch.equal(scales, ref.tile_scales(byte, 0xA5))  # rows behind the last one are as they were
    for out_t in (torch.bfloat16, torch.float32):
        out = torch.empty(rows, cols, dtype=out_t, device="cuda")
        rra.rra_mx4_restore(codes, scales, out)
        v = ref.values(want, byte, cols)
        assert torch.equal(torch.isnan(out), torch.isnan(v))
        assert torch.equal(torch.nan_to_num(out.double()), torch.nan_to_num(v.to(out_t).double()))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("by", [1, 2, 3, 7])
def test_matrices_off_16_bytes(by, dtype):
    x = shifted(nasty(gen(by), 37, 256, DT[dtype]), by)
    codes, scales = room(37, 256)
    rra.rra_mx4_quantize(x, codes, scales)
    want, byte = ref.quantize(x)
    assert torch.equal(codes, want) and torch.equal(scales, ref.tile_scales(byte, 0xA5))
    out = shifted(torch.zeros(37, 256, dtype=DT[dtype], device="cuda"), by)
    rra.rra_mx4_restore(codes, scales, out)
    assert torch.equal(torch.nan_to_num(out.double()), torch.nan_to_num(ref.values(want, byte, 256).to(out.dtype).double()))


def test_a_byte_of_every_kind_reads_back():
    codes = torch.arange(256, dtype=torch.uint8, device="cuda").view(16, 16).repeat(16, 1)  # 256 rows, 32 columns
    byte = torch.arange(256, dtype=torch.uint8, device="cuda").view(256, 1)
    for dt in (torch.float32, torch.bfloat16):
        for by in (0, 1):
            out = shifted(torch.zeros(256, 32, dtype=dt, device="cuda"), by)
            rra.rra_mx4_restore(codes, ref.tile_scales(byte), out)
            v = ref.values(codes, byte, 32).to(dt)
            assert torch.equal(torch.isnan(out), torch.isnan(v)) and torch.equal(torch.nan_to_num(out), torch.nan_to_num(v))


# -- norm ----------------------------------------------------------------------

def norm_ref(xs, gamma, residual, eps):
    s = xs[0].float()
    for x in xs[1:]:
        s = s + x.float()
    if residual is not None:
        s = s + residual.float()
    q = (1.0 / torch.sqrt(s.double().square().mean(1) + eps)).float()
    return s, (s * q[:, None]) * gamma.float()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,rows,hidden,res,by", [
    (1, 1, 1, False, 0), (2, 3, 33, True, 0), (8, 8, 5120, True, 0), (8, 8, 5120, False, 0), (3, 400, 1027, True, 0),
    (8, 700, 2048, True, 0), (4, 5, 8192, True, 0), (2, 320, 8192, True, 0), (2, 3, 16384, False, 0),
    (2, 3, 20000, True, 0), (1, 2, 51200, True, 0), (5, 9, 512, True, 1), (3, 2, 20001, True, 3)])
def test_norm(n, rows, hidden, res, by, dtype):
    g, dt = gen(rows + hidden), DT[dtype]
    xs = [shifted(torch.randn(rows, hidden, generator=g, device="cuda").to(dt), by) for _ in range(n)]
    gamma = shifted((1 + 0.1 * torch.randn(hidden, generator=g, device="cuda")).to(dt), by)
    residual = shifted((3 * torch.randn(rows, hidden, generator=g, device="cuda")).to(dt), by) if res else None
    s, y = norm_ref(xs, gamma, residual, 1e-5)
    codes, scales = room(rows, hidden)
    out = torch.empty_like(xs[0])
    rra.rra_allreduce_rmsnorm_mx4(xs, gamma, hidden, codes, scales, residual=residual, residual_out=out, eps=1e-5)
    assert torch.equal(out, s.to(dt))
    want, byte = ref.quantize(y)
    assert torch.equal(codes, want)
    assert torch.equal(scales, ref.tile_scales(byte, 0xA5))
    again, scales2 = room(rows, hidden)
    rra.rra_allreduce_rmsnorm_mx4(xs, gamma, hidden, again, scales2, residual=residual, residual_out=residual, eps=1e-5)
    assert torch.equal(again, codes) and torch.equal(scales2, scales)
    if res:
        assert torch.equal(residual, out)  # in place


def test_norm_confines_what_is_not_finite():
    xs = [torch.randn(5, 256, generator=gen(), device="cuda") for _ in range(2)]
    xs[0][1, 7], xs[1][3, 200] = math.nan, math.inf
    codes, scales = room(5, 256)
    rra.rra_allreduce_rmsnorm_mx4(xs, torch.ones(256, device="cuda"), 256, codes, scales)
    out = torch.empty(5, 256, device="cuda")
    rra.rra_mx4_restore(codes, scales, out)
    bad = ~torch.isfinite(out)
    assert bad[1].all() and bad[3, 192:224].all() and not bad[[0, 2, 4]].any()


# -- products ------------------------------------------------------------------

def close(got, want, terms, K, dtype):
    bound = (K / 64 + 10) * 2.0 ** -23 * terms + HALF[dtype] * want.abs() * (1 + 1e-3) + 1e-30
    worst = float(((got.double() - want).abs() / bound).max())
    assert worst <= 1.0, worst


TOKENS = [1, 2, 15, 16, 17, 33, 64, 65, 100, 128, 129, 200, 256, 257, 500]


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("K,widths", [(32, [128]), (256, [5, 256, 1]), (515, [300, 130, 0, 77])])
def test_product(T, K, widths):
    g = gen(T + K)
    x, xv = matrix(g, T, K)
    ws, vs = zip(*[matrix(g, w, K, K ** -0.5) if w else (room(0, K), torch.zeros(0, K, device="cuda").double()) for w in widths])
    for dtype in ("bf16", "fp32"):
        outs = [torch.full((T, w), math.nan, dtype=DT[dtype], device="cuda") for w in widths]
        rra.rra_mx4_product(x, list(ws), outs, K)
        for o, v in zip(outs, vs):
            if o.numel():
                close(o, xv @ v.t(), xv.abs() @ v.abs().t(), K, dtype)


@pytest.mark.parametrize("T", [1, 20, 128, 129, 300])
@pytest.mark.parametrize("n,F,D", [(1, 32, 40), (3, 300, 515), (8, 129, 1024), (8, 700, 260), (2, 2048, 128)])
def test_product_sum(T, n, F, D):
    g = gen(T + F)
    xs, xv = zip(*[matrix(g, T, F) for _ in range(n)])
    ws, wv = zip(*[matrix(g, D, F, F ** -0.5) for _ in range(n)])
    want = sum(a @ b.t() for a, b in zip(xv, wv))
    terms = sum(a.abs() @ b.abs().t() for a, b in zip(xv, wv))
    for dtype in ("bf16", "fp32"):
        out = torch.full((T, D), math.nan, dtype=DT[dtype], device="cuda")
        rra.rra_mx4_product_sum(list(xs), list(ws), out, F)
        close(out, want, terms, n * F + 64 * n, dtype)
        again = torch.empty_like(out)
        rra.rra_mx4_product_sum(list(xs), list(ws), again, F)
        assert torch.equal(out, again)


@pytest.mark.parametrize("T", [33, 64, 65, 100, 128, 129])
def test_product_of_many_rows(T):
    """Weights for every SM, of several tiles a CTA: more tokens go to the kernel of few."""
    K, widths = 300, [20000, 8001]
    g = gen(T)
    x, xv = matrix(g, T, K)
    ws, vs = zip(*[matrix(g, w, K, K ** -0.5) for w in widths])
    for dtype in ("bf16", "fp32"):
        outs = [torch.full((T, w), math.nan, dtype=DT[dtype], device="cuda") for w in widths]
        rra.rra_mx4_product(x, list(ws), outs, K)
        for o, v in zip(outs, vs):
            close(o, xv @ v.t(), xv.abs() @ v.abs().t(), K, dtype)


@pytest.mark.parametrize("T", [5, 17, 64, 100])
def test_product_sum_of_long_rows(T):
    """A K axis shared by a cluster: sums of few and of many columns a CTA."""
    n, F, D = 3, 2100, 700
    g = gen(T)
    xs, xv = zip(*[matrix(g, T, F) for _ in range(n)])
    ws, wv = zip(*[matrix(g, D, F, F ** -0.5) for _ in range(n)])
    want = sum(a @ b.t() for a, b in zip(xv, wv))
    terms = sum(a.abs() @ b.abs().t() for a, b in zip(xv, wv))
    for dtype in ("bf16", "fp32"):
        out = torch.full((T, D), math.nan, dtype=DT[dtype], device="cuda")
        rra.rra_mx4_product_sum(list(xs), list(ws), out, F)
        close(out, want, terms, n * F + 64 * n, dtype)


@pytest.mark.parametrize("kind", [rra.RRA_ACT_SILU, rra.RRA_ACT_GELU_TANH])
@pytest.mark.parametrize("T", [1, 16, 40, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("n,D,F", [(1, 64, 32), (2, 515, 129), (3, 256, 300), (8, 1024, 64)])
def test_gated(T, n, D, F, kind):
    gated_case(T, n, D, F, kind)


@pytest.mark.parametrize("kind", [rra.RRA_ACT_SILU, rra.RRA_ACT_GELU_TANH])
@pytest.mark.parametrize("T", [3, 17, 20, 32, 33, 48, 49])
def test_gated_of_many_rows(T, kind):
    gated_case(T, 2, 300, 5001, kind)


@pytest.mark.parametrize("T", [2, 16])
def test_gated_of_long_rows(T):
    gated_case(T, 1, 9000, 260, rra.RRA_ACT_SILU)


def gated_case(T, n, D, F, kind):
    g = gen(T + F)
    x, xv = matrix(g, T, D)
    gates, gv = zip(*[matrix(g, F, D, D ** -0.5) for _ in range(n)])
    ups, uv = zip(*[matrix(g, F, D, D ** -0.5) for _ in range(n)])
    acts = [room(T, F, 0xFF) for _ in range(n)]
    rra.rra_mx4_gated_ffn(x, list(gates), list(ups), acts, D, F, act=kind)
    for a, gw, uw in zip(acts, gv, uv):
        G, U = xv @ gw.t(), xv @ uw.t()
        e = (D / 64 + 10) * 2.0 ** -23
        dg, du = e * (xv.abs() @ gw.abs().t()), e * (xv.abs() @ uw.abs().t())
        h = ref.act(G, kind)
        v = h * U
        dv = (1.13 * dg + 2.0 ** -20 * G.abs()) * (U.abs() + du) + h.abs() * du + 2.0 ** -22 * v.abs()
        got = ref.read(*a, F)
        worst = float(((got - v).abs() / (ref.half_step(v) + dv * 1.01 + 1e-37)).max())
        assert worst <= 1.0, worst
        # blocks behind the last one scale by 2^-127, rows behind the last one are as they were; codes end in zeros
        nb = ref.blocks(F)
        full = a[1][ref.tile_at(T, -(-nb // 4) * 4, "cuda")]
        assert int(full[:, nb:].max() if full.shape[1] > nb else 0) == 0
        mask = torch.ones_like(a[1], dtype=torch.bool)
        mask[ref.tile_at(T, -(-nb // 4) * 4, "cuda").flatten()] = False
        assert (a[1][mask] == 0xFF).all()
        if F % 32:
            tail = torch.stack([a[0] & 15, a[0] >> 4], 2).view(T, -1)[:, F:]
            assert int(tail.max()) == 0


@pytest.mark.parametrize("T", [3, 200])
def test_nan_blocks_stay_in_their_rows(T):
    g = gen(T)
    x = torch.randn(T, 128, generator=g, device="cuda")
    w = torch.randn(64, 128, generator=g, device="cuda")
    x[1, 40], w[5, 100] = math.inf, math.nan
    xc, wc = room(T, 128), room(64, 128)
    rra.rra_mx4_quantize(x, *xc)
    rra.rra_mx4_quantize(w, *wc)
    out = torch.zeros(T, 64, device="cuda")
    rra.rra_mx4_product(xc, [wc], [out], 128)
    bad = torch.isnan(out)
    assert bad[1].all() and bad[:, 5].all()
    bad[1] = False
    bad[:, 5] = False
    assert not bad.any()
    acts = room(T, 64)
    rra.rra_mx4_gated_ffn(xc, [wc], [wc], [acts], 128, 64)
    v = torch.isnan(ref.read(*acts, 64))
    assert v[1].all() and v[:, :32].all()  # the block of column 5
    v[1] = False
    assert not v[:, 32:].any()


# -- sampling ------------------------------------------------------------------

def split(l, shards):
    return [t.contiguous() for t in torch.split(l, shards, 1)]


def check_sample(l, shards, **kw):
    """Draws for a few numbers a row, against the definition; per-row settings are lists."""
    rows = l.shape[0]
    dev = {k: torch.tensor(v, dtype=torch.int32 if k == "top_k" else torch.float32, device="cuda") for k, v in kw.items()}
    token = torch.full((rows,), -7, dtype=torch.int64, device="cuda")
    logprob = torch.empty(rows, device="cuda")
    cpu = l.cpu()
    for u in torch.rand(3, rows, generator=torch.Generator().manual_seed(rows)):
        rra.rra_vocab_sample(split(l, shards), u.cuda(), token, logprob=logprob, **dev)
        for i in range(rows):
            one = {k: float(torch.tensor(v[i], dtype=torch.float32)) if k != "top_k" else v[i] for k, v in kw.items()}
            want, lp = ref.sample_row(cpu[i], float(u[i]), **one)
            assert int(token[i]) == want, (i, one, float(u[i]), int(token[i]), want)
            got = float(logprob[i])
            # float32's logarithm and division: within 2^-21 of it, and of 1
            assert got == lp or (math.isnan(got) and math.isnan(lp)) or abs(got - lp) <= 2.0 ** -21 * (1 + abs(lp))


SETTINGS = dict(temperature=[1.0, 0.7, 0.0, 1.3, 0.05, 1.0, 2.0, 1.0], top_k=[0, 50, 0, 1, 20, 3, 1000, 100000000],
                top_p=[1.0, 0.9, 0.5, 1.0, 0.99, 0.3, 0.8, 0.0], min_p=[0.0, 0.05, 0.0, 0.0, 0.0, 0.2, 0.01, 0.0])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shards", [[1], [5], [40, 0, 1], [1000, 1003], [16384] * 8, [50021], [16674, 16674, 16673]])
def test_sample(shards, dtype):
    V = sum(shards)
    l = (3.0 * torch.randn(8, V, generator=gen(V), device="cuda")).to(DT[dtype])
    check_sample(l, shards, **SETTINGS)
    check_sample(l, shards)


@pytest.mark.parametrize("rows", [1, 33, 160, 400])
def test_sample_rows(rows):
    l = (2.0 * torch.randn(rows, 4099, generator=gen(rows), device="cuda")).to(torch.bfloat16)
    k = {n: (v * (rows // 8 + 1))[:rows] for n, v in SETTINGS.items()}
    check_sample(l, [1024, 2051, 1024], **k)


@pytest.mark.parametrize("dtype,shards", [("bf16", [30001, 0, 20001, 7]), ("fp32", [20000, 20003])])
@pytest.mark.parametrize("rows,cap", [(160, 0), (24, 3), (24, 0)])
def test_sample_rows_alone_and_shared(rows, cap, dtype, shards):
    """Rows that a CTA has to itself (many of them, or few SMs) and rows that a
    cluster shares give the same tokens."""
    V = sum(shards)
    l = (3.0 * torch.randn(rows, V, generator=gen(rows + V), device="cuda")).to(DT[dtype])
    l[0] = -math.inf
    l[1, :] = 0.5
    l[2, 7] = math.inf
    l[3, V - 1] = math.nan
    l[4, 5:] = -math.inf
    k = {n: (v * (rows // 8)) for n, v in SETTINGS.items()}
    rra.rra_set_max_ctas(cap)
    try:
        check_sample(l, shards, **k)
        check_sample(l, shards)
    finally:
        rra.rra_set_max_ctas(0)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sample_equal_logits(dtype):
    """Ties at the bounds of top-k and top-p go to the lowest index."""
    V = 40000
    l = torch.full((8, V), 1.25, device="cuda").to(DT[dtype])
    l[4:] = torch.randint(0, 3, (4, V), generator=gen(), device="cuda").to(DT[dtype])
    check_sample(l, [V // 2, V // 2], temperature=[1.0] * 8, top_k=[0, 7, 0, 39999, 100, 30000, 0, 20000],
                 top_p=[1.0, 1.0, 0.5, 0.25, 1.0, 0.9, 0.6, 0.999], min_p=[0.0, 1.0, 0.5, 0.0, 0.0, 0.0, 0.4, 0.0])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sample_masks_and_extremes(dtype):
    V = 3000
    l = (2.0 * torch.randn(8, V, generator=gen(3), device="cuda"))
    inf = math.inf
    l[0] = -inf                                   # nothing to draw
    l[1, torch.arange(V, device="cuda") != 2900] = -inf
    l[2, 17] = math.nan
    l[3, [100, 2000]] = inf
    l[4] = torch.finfo(DT[dtype]).min             # a mask of the type's lowest value, everywhere
    l[5, 10:] = torch.finfo(DT[dtype]).min
    l[6] = torch.where(torch.arange(V, device="cuda") % 2 == 0, 0.0, -0.0)
    l = l.to(DT[dtype])
    for k in (dict(), dict(temperature=[0.5] * 8, top_k=[5] * 8, top_p=[0.9] * 8, min_p=[0.1] * 8),
              dict(temperature=[0.0] * 8), dict(temperature=[1e-30] * 8), dict(temperature=[1e30] * 8, top_p=[0.5] * 8),
              dict(temperature=[math.nan, -1.0] * 4)):
        check_sample(l, [1500, 1500], **k)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sample_zeros_behind_a_range(dtype):
    """The nearest logits searched first end exactly at zero: zeros count as
    theirs, not as the ones below, which end with the key of -0."""
    bits = torch.tensor([0x03FF], dtype=torch.int16).view(torch.bfloat16).float()  # 1023 keys above 0
    top = {"bf16": float(bits), "fp32": float(torch.tensor(16.0) / torch.tensor(1.44269502))}[dtype]  # 16 octaves at 1
    g = gen(77)
    l = -top * torch.rand(6, 900, generator=g, device="cuda")
    l[:, 100:250] = 0.0
    l[:, 300:360] = top * torch.rand(6, 60, generator=g, device="cuda")
    l[:, 500] = top
    l = l.to(DT[dtype])
    t = {"bf16": 1e-29, "fp32": 1.0}[dtype]
    check_sample(l, [450, 450], temperature=[t] * 6, top_k=[30, 100, 211, 212, 600, 0],
                 top_p=[1.0, 1.0, 1.0, 0.99, 1.0, 0.5], min_p=[0.0] * 6)


def test_sample_ends_of_the_range():
    l = torch.randn(4, 1000, generator=gen(9), device="cuda")
    token = torch.empty(4, dtype=torch.int64, device="cuda")
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 1.0, -1.0], device="cuda")
    rra.rra_vocab_sample([l], u, token)
    assert token.tolist() == [0, 999, 999, 0]


def test_sample_vocabulary_of_the_limit():
    V = 368640
    l = 2.0 * torch.randn(2, V, generator=gen(5), device="cuda")
    check_sample(l, [V // 8] * 8, temperature=[1.0, 0.9], top_k=[0, 5000], top_p=[0.95, 1.0], min_p=[0.0, 0.0])


def test_sample_frequencies():
    """Evenly spaced numbers draw each token as often as its weight says, to one draw."""
    l = torch.tensor([[0.3, -1.0, 2.0, 0.0, 1.1]], device="cuda").expand(4096, 5).contiguous()
    token = torch.empty(4096, dtype=torch.int64, device="cuda")
    u = (torch.arange(4096, device="cuda") + 0.5) / 4096
    rra.rra_vocab_sample([l], u, token)
    want = torch.softmax(l[0].double(), 0) * 4096
    assert ((torch.bincount(token, minlength=5) - want).abs() <= 1.0).all()


# -- together --------------------------------------------------------------------

class Step:
    """A decode step of one block on virtual ranks, buffers made once: partial
    sums -> norm -> gated feed-forward -> row-parallel product -> norm -> head
    -> token."""

    def __init__(self, T, n=4, D=512, F=320, V=1000, seed=0):
        g = gen(seed)
        self.n, self.T, self.D, self.F = n, T, D, F
        self.parts = [torch.randn(T, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(n)]
        self.stream = torch.randn(T, D, generator=g, device="cuda").to(torch.bfloat16)
        self.gamma = torch.ones(D, dtype=torch.bfloat16, device="cuda")

        def weights(rows, cols, count):
            ms = []
            for _ in range(count):
                w = torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5
                m = room(rows, cols)
                rra.rra_mx4_quantize(w, *m)
                ms.append(m)
            return ms

        self.gates, self.ups, self.downs = weights(F, D, n), weights(F, D, n), weights(D, F, n)
        self.heads = weights(V // n, D, n)
        self.mid, self.end = torch.empty_like(self.stream), torch.empty_like(self.stream)
        self.h, self.h2, self.acts = room(T, D), room(T, D), [room(T, F) for _ in range(n)]
        self.ffn = torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
        self.logits = [torch.empty(T, V // n, device="cuda") for _ in range(n)]
        self.u = torch.rand(T, generator=g, device="cuda")
        self.token = torch.empty(T, dtype=torch.int64, device="cuda")
        self.top_k = torch.full((T,), 40, dtype=torch.int32, device="cuda")

    def run(self, stream=None):
        s = dict(stream=stream)
        rra.rra_allreduce_rmsnorm_mx4(self.parts, self.gamma, self.D, *self.h, residual=self.stream, residual_out=self.mid, **s)
        rra.rra_mx4_gated_ffn(self.h, self.gates, self.ups, self.acts, self.D, self.F, **s)
        rra.rra_mx4_product_sum(self.acts, self.downs, self.ffn, self.F, **s)
        rra.rra_allreduce_rmsnorm_mx4([self.ffn], self.gamma, self.D, *self.h2, residual=self.mid, residual_out=self.end, **s)
        rra.rra_mx4_product(self.h2, self.heads, self.logits, self.D, **s)
        rra.rra_vocab_sample(self.logits, self.u, self.token, top_k=self.top_k, **s)

    def results(self):
        return [t.clone() for t in [self.token, self.end, *self.logits, *self.h2]]

    def check(self):
        """Each operator's outputs against the definition of its own inputs."""
        T, D, F = self.T, self.D, self.F
        s, y = norm_ref(self.parts, self.gamma, self.stream, 1e-6)
        assert torch.equal(self.mid, s.to(torch.bfloat16)) and torch.equal(self.h[0], ref.quantize(y)[0])
        acts = [ref.read(*a, F) for a in self.acts]
        downs = [ref.read(*w, F) for w in self.downs]
        close(self.ffn, sum(a @ w.t() for a, w in zip(acts, downs)),
              sum(a.abs() @ w.abs().t() for a, w in zip(acts, downs)), self.n * (F + 64), "bf16")
        h = ref.read(*self.h2, D)
        for o, w in zip(self.logits, self.heads):
            v = ref.read(*w, D)
            close(o, h @ v.t(), h.abs() @ v.abs().t(), D, "fp32")
        l = torch.cat(self.logits, 1).cpu()
        assert self.token.tolist() == [ref.sample_row(l[i], float(self.u[i]), top_k=40)[0] for i in range(T)]


@pytest.mark.parametrize("T", [1, 7, 130])
def test_a_step(T):
    st = Step(T)
    st.run()
    st.check()


@pytest.mark.parametrize("T", [1, 130])
def test_a_step_in_a_graph_and_on_other_streams(T):
    st = Step(T)
    st.run()
    want = st.results()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, st.results()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st.run()
    st.parts[0].mul_(0.5)  # new inputs in the captured buffers
    st.u.copy_(torch.rand(T, generator=gen(77), device="cuda"))
    graph.replay()
    st.check()
    got = st.results()
    st.run()
    assert all(torch.equal(a, b) for a, b in zip(got, st.results()))


def test_two_steps_at_once():
    a, b = Step(5, seed=1), Step(140, seed=2)
    a.run()
    b.run()
    want = a.results(), b.results()
    torch.cuda.synchronize()
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a.run(stream=s)
        b.run(stream=t)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want[0], a.results()))
    assert all(torch.equal(x, y) for x, y in zip(want[1], b.results()))


CALLS = ["allreduce_rmsnorm_mx4", "mx4_gated_ffn", "mx4_product_sum", "mx4_product", "vocab_sample"]


@pytest.mark.parametrize("cap", [1, 3, 16])
@pytest.mark.parametrize("T", [9, 200])
def test_every_launch_keeps_the_budget(T, cap):
    st = Step(T, seed=T)
    rra.rra_set_max_ctas(cap)
    try:
        st.run()
        torch.cuda.synchronize()
        st.check()
        x, m = st.stream, room(T, st.D)
        rra.rra_mx4_quantize(x, *m)
        rra.rra_mx4_restore(*m, torch.empty_like(x))
        lines = rra.rra_dump_recent().splitlines()
        for call in CALLS + ["mx4_quantize", "mx4_restore"]:
            line = [l for l in lines if " %s " % call in l][-1]
            pair = T > 128 and call in CALLS[1:4]  # products of many tokens run as pairs of CTAs, one at least
            assert int(line.split("grid=")[1].split()[0]) <= max(cap, 2 if pair else 1), line
    finally:
        rra.rra_set_max_ctas(0)
    assert rra.rra_query_status()[0] == rra.RRA_SUCCESS


@pytest.mark.parametrize("cap", [1, 2, 5, 7])
@pytest.mark.parametrize("T,K,W", [(5, 700, 650), (60, 1300, 300), (128, 515, 260), (300, 1300, 700), (513, 257, 1030)])
def test_many_tiles_for_few_ctas(T, K, W, cap):
    """A CTA's tiles one after another, over both accumulators and rings that wrap."""
    g = gen(T + W)
    x, xv = matrix(g, T, K)
    w, wv = matrix(g, W, K, K ** -0.5)
    out, acts = torch.full((T, W), math.nan, device="cuda"), room(T, W)
    two, again = torch.full((T, W), math.nan, device="cuda"), room(T, W)
    rra.rra_mx4_product(x, [w], [two], K)
    rra.rra_mx4_gated_ffn(x, [w], [w], [again], K, W)
    rra.rra_set_max_ctas(cap)
    try:
        rra.rra_mx4_product(x, [w], [out], K)
        rra.rra_mx4_gated_ffn(x, [w], [w], [acts], K, W)
        torch.cuda.synchronize()
    finally:
        rra.rra_set_max_ctas(0)
    for o in (out, two):
        close(o, xv @ wv.t(), xv.abs() @ wv.abs().t(), K, "fp32")
    v = xv @ wv.t()
    v = ref.act(v, 0) * v
    for a in (acts, again):
        off = (ref.read(*a, W) - v).abs() / (ref.half_step(v) * 1.001 + 1e-4 * v.abs().amax())
        assert float(off.max()) <= 1.0
    assert rra.rra_query_status()[0] == rra.RRA_SUCCESS


# -- more than 2^32 elements -------------------------------------------------------

def test_matrix_past_32_bits():
    rows, cols = 70000, 65536
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    some = [0, 1, 32767, 65535, 65536, 69999]
    x.zero_()
    x[some] = torch.randn(len(some), cols, generator=gen(1), device="cuda").to(torch.bfloat16)
    codes, scales = room(rows, cols)
    rra.rra_mx4_quantize(x, codes, scales)
    want, byte = ref.quantize(x[some][:, :4096])
    assert torch.equal(codes[some][:, :2048], want)
    at = ref.tile_at(rows, cols // 32, "cuda")[some]
    assert torch.equal(scales[at][:, :128], byte)
    x.fill_(1.0)
    rra.rra_mx4_restore(codes, scales, x)
    assert torch.equal(x[some][:, :4096].double(), ref.values(want, byte, 4096))
    assert not x[2:32767].any()


def test_product_past_32_bits():
    T, W, K = 130, 33_100_000, 32  # 4.3e9 outputs
    g = gen(2)
    x, xv = matrix(g, T, K)
    w, wv = matrix(g, 300, K)
    codes = torch.zeros(W, 16, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(ref.scale_bytes(W, K), dtype=torch.uint8, device="cuda")
    last = W - 300  # the last 300 rows hold the small matrix
    codes[last:] = w[0]
    row = torch.arange(300, device="cuda") + last
    scales[row // 128 * 512 + row % 32 * 16 + row % 128 // 32 * 4] = w[1][ref.tile_at(300, 1, "cuda")[:, 0]]
    out = torch.empty(T, W, dtype=torch.bfloat16, device="cuda")
    rra.rra_mx4_product(x, [(codes, scales)], [out], K)
    close(out[:, last:], xv @ wv.t(), xv.abs() @ wv.abs().t(), K, "bf16")
    assert not out[:, last - 5000:last].any() and not out[-1, :1000].any()
    few = torch.empty(1, W, dtype=torch.bfloat16, device="cuda")
    rra.rra_mx4_product((x[0][:1].contiguous(), x[1][:512]), [(codes, scales)], [few], K)
    assert torch.equal(few[:, last:], out[:1, last:]) and not few[:, :last].any()


def test_logits_past_32_bits():
    rows, V = 17000, 262144
    l = torch.zeros(rows, V, dtype=torch.bfloat16, device="cuda")
    at = torch.randint(0, V, (rows,), generator=gen(4), device="cuda")
    l[torch.arange(rows, device="cuda"), at] = 50.0  # all but sure
    token = torch.empty(rows, dtype=torch.int64, device="cuda")
    rra.rra_vocab_sample([l], torch.full((rows,), 0.5, device="cuda"), token,
                         top_k=torch.full((rows,), 5, dtype=torch.int32, device="cuda"))
    assert torch.equal(token, at)
