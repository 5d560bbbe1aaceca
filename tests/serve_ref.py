"""Definitions of the serving-step operators in 64 bits (torch, any device)."""
import math

import torch

BLOCK = 32
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
F64 = torch.float64


def blocks(cols):
    return -(-cols // BLOCK)


def scale_bytes(rows, cols):
    return 512 * -(-rows // 128) * -(-cols // 128)


def exponent(amax):
    """The smallest e >= -127 with amax <= 6 * 2^e."""
    if amax == 0:
        return -127
    m, k = math.frexp(amax / 6.0)  # amax / 6 = m 2^k, m in [0.5, 1); exact at the borders 6 * 2^e
    return max(-127, k - 1 if amax <= 6.0 * 2.0 ** (k - 1) else k)


def quantize(x):
    """Codes [rows, 16 blocks] and scale bytes [rows, blocks] (uint8) of a matrix."""
    x = x.to(F64)
    rows, cols = x.shape
    nb = blocks(cols)
    b = torch.zeros(rows, nb * BLOCK, dtype=F64, device=x.device)
    b[:, :cols] = x
    b = b.view(rows, nb, BLOCK)
    bad = ~torch.isfinite(b).all(2)
    b = torch.where(bad[:, :, None], torch.zeros_like(b), b)
    amax = b.abs().amax(2)
    e = torch.tensor([exponent(float(v)) for v in amax.flatten().tolist()], dtype=F64, device=x.device).view(rows, nb)
    v = b * torch.exp2(-e)[:, :, None]
    a = v.abs()
    code = torch.zeros_like(a, dtype=torch.int64)
    for i in range(7):
        mid = (VALUES[i] + VALUES[i + 1]) / 2
        code += (a > mid) | ((a == mid) & (i % 2 == 1))  # a tie goes to the even code
    code += 8 * (torch.signbit(v) & ~bad[:, :, None])
    byte = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    code = code.view(rows, nb * 16, 2)
    return (code[:, :, 0] | (code[:, :, 1] << 4)).to(torch.uint8), byte


def tile_at(rows, nb, device="cpu"):
    """Where the scale byte of (row, block) lies."""
    r = torch.arange(rows, device=device)[:, None]
    b = torch.arange(nb, device=device)[None, :]
    across = -(-nb // 4)
    return ((r // 128) * across + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4


def tile_scales(byte, fill=0):
    """Scale bytes [rows, blocks] in their tiles; `fill` behind the last row."""
    rows, nb = byte.shape
    across = -(-nb // 4)
    out = torch.full((-(-rows // 128) * across * 512,), fill, dtype=torch.uint8, device=byte.device)
    padded = torch.zeros(rows, across * 4, dtype=torch.uint8, device=byte.device)
    padded[:, :nb] = byte
    out[tile_at(rows, across * 4, byte.device).flatten()] = padded.flatten()
    return out


def values(codes, byte, cols):
    """What codes and scale bytes [rows, blocks] stand for."""
    rows = codes.shape[0]
    code = torch.stack([codes & 15, codes >> 4], 2).view(rows, -1).long()
    grid = torch.tensor(VALUES + [-v for v in VALUES], dtype=F64, device=codes.device)
    p = torch.exp2(byte.to(F64) - 127.0)
    p[byte == 255] = math.nan
    return (grid[code] * p.repeat_interleave(BLOCK, 1))[:, :cols]


def read(codes, scales, cols):
    """Values of a matrix in the library's layout."""
    rows, nb = codes.shape[0], blocks(cols)
    return values(codes, scales[tile_at(rows, nb, codes.device)], cols)


def pack(x, fill=255):
    """(codes, scales, values) of a matrix; scale bytes behind the last row are NaN unless told otherwise."""
    codes, byte = quantize(x)
    return codes, tile_scales(byte, fill), values(codes, byte, x.shape[1])


def act(g, kind):
    if kind == 0:
        return g * torch.sigmoid(g)
    return g * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (g + 0.044715 * g ** 3))


def half_step(v):
    """Largest rounding error of each value in MX4, its block's exponent taken a hair above the border."""
    rows, cols = v.shape
    nb = blocks(cols)
    b = torch.zeros(rows, nb * BLOCK, dtype=F64, device=v.device)
    b[:, :cols] = v
    top = b.view(rows, nb, BLOCK).abs().amax(2).clamp(min=2.0 ** -140) * (1 + 1e-4)
    p = torch.exp2(torch.ceil(torch.log2(top / 6.0)).clamp(min=-127.0)).repeat_interleave(BLOCK, 1)[:, :cols]
    a = v.abs() / p
    return p * torch.where(a < 2, 0.25, torch.where(a < 4, 0.5, 1.0))


def sample_row(l, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log of its probability) of one row of logits (64 bits)."""
    l = l.to(F64)
    if torch.isnan(l).any() or not temperature >= 0:
        return -1, math.nan
    if l.numel() == 0 or float(l.max()) == -math.inf:
        return -1, -math.inf
    order = torch.argsort(-l, stable=True)
    if temperature == 0:
        return int(order[0]), 0.0
    top = l[order[0]]
    w = torch.where(l == top, torch.ones_like(l), torch.exp((l - top) / temperature))
    w = torch.where(torch.isnan(w), torch.zeros_like(w), w)
    if 0 < top_k < l.numel():
        order = order[:top_k]
    if top_p < 1:
        s = w[order]
        before = torch.cumsum(s, 0) - s
        order = order[: max(1, int((before < top_p * s.sum()).sum()))]
    order = order[w[order] >= min(min_p, 1.0)]
    kept, _ = torch.sort(order)
    s = w[kept]
    at = int((torch.cumsum(s, 0) <= u * s.sum()).sum())
    at = min(at, kept.numel() - 1)
    return int(kept[at]), float(torch.log(s[at] / s.sum()))
