"""The training-step operators from their definitions, in float64 on the
CPU, and bounds on what the kernels' roundings may change.  Shares no code
with the library."""
import math

import torch

BF = 2.0 ** -8   # half a bfloat16 step, relative
F32 = 2.0 ** -24


def codes_of(s32):
    """e4m3 codes' values (already times 2^e) and scale bytes of float32 sums,
    by arithmetic on the definition."""
    T, D = s32.shape
    nb = -(-D // 128)
    b = s32.to(torch.bfloat16).to(torch.float64)
    val = torch.empty_like(b)
    sc = torch.empty(T, nb, dtype=torch.uint8)
    for j in range(nb):
        p = b[:, 128 * j:128 * j + 128]
        fin = torch.where(torch.isfinite(p), p.abs(), torch.zeros_like(p))
        top = fin.amax(1)
        e = torch.full((T,), -127, dtype=torch.int64)
        for t in range(T):
            a = float(top[t])
            if a > 0:
                k = max(-127, math.ceil(math.log2(a / 448.0)) - 1)
                while a > 448.0 * 2.0 ** k:
                    k += 1
                e[t] = k
        v = p * torch.exp2(-e.double())[:, None]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        q = torch.round(v / step) * step
        q = torch.where(torch.isfinite(p), q, torch.full_like(q, math.nan))
        val[:, 128 * j:128 * j + 128] = q * torch.exp2(e.double())[:, None]
        sc[:, j] = (e + 127).to(torch.uint8)
    return val, sc


def ascending_sum(xs):
    s = xs[0].float()
    for x in xs[1:]:
        s = s + x.float()
    return s


def act_slope(g, act):
    if act == 0:
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    k = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(k)
    return g * s, s + g * s * (1 - s) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g ** 2)


def product_err(absx, absw, K):
    """Bound on the float32 accumulation of a K-long product: at most one
    rounding of 2^-23 for each of K / 8 partial sums, of the magnitudes' sum."""
    return (K / 8 + 4) * 2.0 ** -23 * (absx @ absw)


def ffn(x, gates, ups, act, dacts=None):
    """Values and elementwise bounds of the forward, and with dacts of the
    backward."""
    x = x.double()
    D = x.shape[1]
    outs, bouts = [], []
    dx = torch.zeros_like(x)
    bdx = torch.zeros_like(x)
    dG, dU, bG, bU = [], [], [], []
    for r, (G, U) in enumerate(zip(gates, ups)):
        G, U = G.double(), U.double()
        g, u = x @ G.t(), x @ U.t()
        eg, eu = product_err(x.abs(), G.abs().t(), D), product_err(x.abs(), U.abs().t(), D)
        a, sl = act_slope(g, act)
        # |act'| and |act''| are below 1.2; the fast exponential and division are good to 2^-20
        ea = 1.2 * eg + 2.0 ** -20 * a.abs()
        es = 1.2 * eg + 2.0 ** -20 * (sl.abs() + 1)
        y = a * u
        outs.append(y)
        bouts.append(ea * (u.abs() + eu) + a.abs() * eu + BF * y.abs() + 2.0 ** -22 * y.abs() + 1e-30)
        if dacts is None:
            continue
        da = dacts[r].double()
        dg, du = da * u * sl, da * a
        edg = da.abs() * (u.abs() * es + (sl.abs() + es) * eu)
        edu = da.abs() * ea
        edg = edg + BF * (dg.abs() + edg)
        edu = edu + BF * (du.abs() + edu)
        dx += dg @ G + du @ U
        bdx += edg @ G.abs() + edu @ U.abs() + product_err(dg.abs(), G.abs(), len(G) * 2 * len(gates)) \
            + product_err(du.abs(), U.abs(), len(G) * 2 * len(gates))
        for d, e, o, b in ((dg, edg, dG, bG), (du, edu, dU, bU)):
            w = d.t() @ x
            o.append(w)
            b.append(e.t() @ x.abs() + product_err(d.abs().t(), x.abs(), len(x)) + BF * w.abs() + 1e-30)
    bdx += BF * dx.abs() + 1e-30
    return outs, bouts, (dx, bdx), list(zip(dG, bG)), list(zip(dU, bU))


def vocab_loss(x, weights, targets, ignore, grad=None, rest=False):
    """(loss, lse) with bounds, and with grad (dx, [dW]) with bounds; rest: dW of two halves of each entry of dl."""
    x = x.double()
    D = x.shape[1]
    W = torch.cat([w.double() for w in weights])
    V = len(W)
    l = x @ W.t()
    el = product_err(x.abs(), W.abs().t(), D)
    lse = torch.logsumexp(l, 1)
    p = torch.exp(l - lse[:, None])
    # an error of the logits moves lse by at most their p-weighted mean; the exponentials, their float32 sums
    # (columns 2 at a time, 128 a part, parts joined) and the logarithm: (|lse| + 128 + V/128/8 + 16) roundings
    elast = (p * el).sum(1) + F32 * 2 * (lse.abs() + 3 * l.abs().amax(1) + 144 + V / 1024)
    valid = (targets != ignore)
    inside = valid & (targets >= 0) & (targets < V)
    safe = torch.where(inside, targets, torch.zeros_like(targets))
    rows = torch.arange(len(x))
    hit, ehit = l[rows, safe], el[rows, safe]
    loss = torch.where(valid, lse - hit, torch.zeros_like(lse))
    loss = torch.where(valid & ~inside, torch.full_like(loss, math.nan), loss)
    out = {"loss": (loss, elast + ehit + F32 * (lse.abs() + hit.abs())), "lse": (lse, elast)}
    if grad is None:
        return out
    w = torch.where(inside, grad.double(), torch.zeros_like(lse))
    d = p.clone()
    d[rows, safe] -= 1
    ed = p * (el + elast[:, None] + F32 * 8 * (l.abs() + lse.abs()[:, None] + 1)) + F32 * 2
    d, ed = d * w[:, None], ed * w.abs()[:, None]
    # every entry is rounded to bfloat16 but the target's, whose rest is added in float32
    step = BF * (d.abs() + ed)
    step[rows[inside], targets[inside]] = (4 * F32 * (d.abs() + ed))[rows[inside], targets[inside]]
    # two halves: the second is at most half a step of the first, and rounded in turn
    ew = ed + (BF * step + 1e-38 if rest else step)
    ed = ed + step
    dx = d @ W
    bdx = ed @ W.abs() + product_err(d.abs(), W.abs(), V) + BF * dx.abs() + 1e-30
    dW = d.t() @ x
    bW = ew.t() @ x.abs() + product_err(d.abs().t(), x.abs(), len(x)) + BF * dW.abs() + 1e-30
    sizes = [len(v) for v in weights]
    out["dx"] = (dx, bdx)
    out["dW"] = list(zip(torch.split(dW, sizes), torch.split(bW, sizes)))
    return out


def assert_within(got, want, bound, what):
    got = got.detach().cpu().double()
    same = (torch.isnan(got) & torch.isnan(want)) | ((got - want).abs() <= bound)
    if not bool(same.all()):
        bad = (~same).nonzero()
        i = tuple(bad[0].tolist())
        raise AssertionError("%s: %d of %d outside the bound, first at %s: got %r want %r bound %r"
                             % (what, len(bad), same.numel(), i, float(got[i]), float(want[i]),
                                float(bound[i] if torch.is_tensor(bound) else bound)))


def assert_norm_close(got, want, rel, what):
    if not float(want.norm()):
        return  # a vocabulary of one: the gradient is exactly zero and has no relative error
    got = got.detach().cpu().double()
    off = float((got - want).norm()) / float(want.norm())
    assert off <= rel, "%s: relative error %.3g above %.3g" % (what, off, rel)
