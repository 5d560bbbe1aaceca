"""Gated backward pass of few tokens.  Its gradients are sums over so few
entries of dg and du that what bfloat16 cuts from those does not average out (a
shard's gradient of one token was off by twice its own rounding): the entries
are kept as two bfloat16 halves, and what is left is the rounding of the result."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import collective_all_reduce_rank_gb300 as rra  # noqa: E402
import train_ref as ref  # noqa: E402
from test_train_gpu import cuda, poison, rnd, status_ok  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _ready():
    rra.rra_init(0)


def gradients(x, gates, ups, act, dacts):
    """dx, [dG], [dU] in float64 with bounds that have no rounding of dg and du in them: two halves leave
    2^-8 of 2^-8 of an entry."""
    X = x.double()
    D, n, F = X.shape[1], len(gates), len(gates[0])
    dx, bdx, out = torch.zeros_like(X), torch.zeros_like(X), []
    for G, U, da in zip(gates, ups, dacts):
        G, U, da = G.double(), U.double(), da.double()
        g, u = X @ G.t(), X @ U.t()
        eg, eu = ref.product_err(X.abs(), G.abs().t(), D), ref.product_err(X.abs(), U.abs().t(), D)
        a, sl = ref.act_slope(g, act)
        ea, es = 1.2 * eg + 2.0 ** -20 * a.abs(), 1.2 * eg + 2.0 ** -20 * (sl.abs() + 1)
        dg, du = da * u * sl, da * a
        edg = da.abs() * (u.abs() * es + (sl.abs() + es) * eu)
        edu = da.abs() * ea
        edg, edu = edg + ref.BF ** 2 * (dg.abs() + edg), edu + ref.BF ** 2 * (du.abs() + edu)
        dx += dg @ G + du @ U
        bdx += edg @ G.abs() + edu @ U.abs()
        bdx += ref.product_err(dg.abs(), G.abs(), 2 * n * F) + ref.product_err(du.abs(), U.abs(), 2 * n * F)
        for d, e in ((dg, edg), (du, edu)):
            w = d.t() @ X
            out.append((w, e.t() @ X.abs() + ref.product_err(d.abs().t(), X.abs(), 2 * len(X))
                        + ref.BF * w.abs() + 1e-30))
    return (dx, bdx + ref.BF * dx.abs() + 1e-30), out[0::2], out[1::2]


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("n,T,D,F", [
    (1, 1, 64, 8), (3, 1, 714, 48), (8, 3, 2269, 79), (2, 5, 128, 84), (5, 6, 448, 42), (4, 2, 5120, 200),
    (1, 18, 379, 71), (3, 31, 264, 300), (2, 32, 1027, 130), (8, 17, 512, 720), (1, 33, 96, 40), (2, 64, 515, 33),
    (4, 65, 128, 96), (1, 100, 1024, 640), (3, 127, 130, 35), (2, 128, 2048, 256),
])
def test_gradients_of_few_tokens_are_off_by_their_own_rounding(n, T, D, F, act):
    gen = torch.Generator().manual_seed(T * 13 + D)
    x = rnd(gen, T, D)
    G, U = ([rnd(gen, F, D, scale=D ** -0.5) for _ in range(n)] for _ in range(2))
    da = [rnd(gen, T, F, scale=1e-2) for _ in range(n)]
    dx, dG, dU = poison(T, D), [poison(F, D) for _ in range(n)], [poison(F, D) for _ in range(n)]
    ws = torch.empty(rra.rra_gated_ffn_workspace_bytes(n, T, D, F, 1), dtype=torch.uint8, device="cuda").fill_(255)
    rra.rra_gated_ffn_backward(x.cuda(), cuda(G), cuda(U), cuda(da), dx, dG, dU, act=act, workspace=ws)
    status_ok()
    (rdx, bdx), rG, rU = gradients(x, G, U, act, da)
    ref.assert_within(dx, rdx, bdx, "dx")
    for r in range(n):
        ref.assert_within(dG[r], *rG[r], "dgates[%d]" % r)
        ref.assert_within(dU[r], *rU[r], "dups[%d]" % r)


def test_entries_past_the_types_range():
    """A dg of infinity has no second half: it stays infinite, and its row alone."""
    T, D, F = 4, 64, 40
    gen = torch.Generator().manual_seed(9)
    x, G, U = rnd(gen, T, D).abs() + 0.5, rnd(gen, F, D, scale=0.1).abs(), rnd(gen, F, D, scale=0.1).abs()
    da = rnd(gen, T, F).abs()
    da[1, 7] = 3.3e38
    dx, dG, dU = poison(T, D), poison(F, D), poison(F, D)
    rra.rra_gated_ffn_backward(x.cuda(), cuda([G]), cuda([U]), cuda([da]), dx, [dG], [dU])
    status_ok()
    assert torch.isinf(dx[1].float()).all() and torch.isinf(dG[7].float()).all() and torch.isinf(dU[7].float()).all()
    rest = [t for t in range(T) if t != 1]
    rows = [f for f in range(F) if f != 7]
    assert torch.isfinite(dx[rest].float()).all() and torch.isfinite(dG[rows].float()).all()
    assert torch.isfinite(dU[rows].float()).all()
