"""Refusals of the serving-step operators: every bad call returns its error
before any launch, so fake device addresses are enough and no GPU is needed.
And the reference of their tests against the definition, value by value."""
import ctypes
import math
import struct

import pytest
import torch

import collective_all_reduce_rank_gb300 as rra
import serve_ref as ref

A = 1 << 40  # never dereferenced
STEP = 1 << 34
OK, INV, UNS, ALIAS, NOT_INIT = (rra.RRA_SUCCESS, rra.RRA_ERR_INVALID_ARG, rra.RRA_ERR_UNSUPPORTED, rra.RRA_ERR_ALIAS,
                                 rra.RRA_ERR_NOT_INITIALIZED)
BF16, F32, I32 = rra.RRA_BFLOAT16, rra.RRA_FLOAT32, rra.RRA_INT32


def at(i):
    return A + i * STEP


def mx(i, codes=0, scales=0):
    """An MX4 matrix at place i, its parts moved by some bytes (None: null)."""
    return (None if codes is None else at(i) + codes, None if scales is None else at(i) + STEP // 2 + scales)


def mxs(ms):
    return b"".join(struct.pack("2P", m[0] or 0, m[1] or 0) for m in ms)


def ptrs(ps):
    return (ctypes.c_void_p * max(1, len(ps)))(*ps)


def sizes(vs):
    return (ctypes.c_size_t * max(1, len(vs)))(*vs)


@pytest.fixture(scope="module")
def lib():
    lib = rra.load()
    rra.rra_finalize()
    return lib


@pytest.mark.parametrize("rows,cols", [(0, 5), (5, 0), (1, 1), (128, 128), (129, 128), (128, 129), (1283, 1027)])
def test_scale_bytes(lib, rows, cols):
    assert rra.rra_mx4_scale_bytes(rows, cols) == ref.scale_bytes(rows, cols)


@pytest.mark.parametrize("name", ["quantize", "restore"])
@pytest.mark.parametrize("change,want", [
    (dict(x=None), INV), (dict(m=None), INV), (dict(dtype=I32), INV), (dict(dtype=9), INV), (dict(x=at(0) + 1), INV),
    (dict(x=at(0) + 2, dtype=F32), INV), (dict(m=mx(1, codes=None)), INV), (dict(m=mx(1, scales=None)), INV),
    (dict(m=mx(1, codes=8)), UNS), (dict(m=mx(1, scales=4)), UNS), (dict(rows=1 << 31), UNS), (dict(cols=1 << 31), UNS),
    (dict(m=(at(0), at(1))), ALIAS), (dict(m=(at(1), at(0))), ALIAS), (dict(rows=0), OK), (dict(cols=0), OK),
    (dict(rows=0, x=None, m=(None, None)), OK),
])
def test_matrix_refusals(lib, name, change, want):
    a = dict(x=at(0), m=mx(1), rows=4, cols=256, dtype=BF16)
    a.update(change)
    m = None if a["m"] is None else mxs([a["m"]])
    if name == "quantize":
        got = lib.rra_mx4_quantize(a["x"], m, a["rows"], a["cols"], a["dtype"], None)
    else:
        got = lib.rra_mx4_restore(m, a["x"], a["rows"], a["cols"], a["dtype"], None)
    assert got == want


def test_quantize_refuses_codes_on_scales(lib):
    assert lib.rra_mx4_quantize(at(0), mxs([(at(1), at(1))]), 4, 256, BF16, None) == ALIAS


@pytest.mark.parametrize("change,want", [
    (dict(n=0), INV), (dict(n=9), UNS), (dict(dtype=I32), INV), (dict(hidden=0), INV), (dict(hidden=51201), UNS),
    (dict(rows=1 << 31), UNS), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV), (dict(gamma=None), INV),
    (dict(gamma=at(20) + 1), INV), (dict(bufs=[at(0), None]), INV), (dict(bufs=[at(0) + 1, at(1)]), INV),
    (dict(residual=at(10) + 1), INV), (dict(residual_out=at(11) + 1), INV), (dict(out=None), INV),
    (dict(out=mx(30, codes=None)), INV), (dict(out=mx(30, codes=4)), UNS), (dict(out=mx(30, scales=4)), UNS),
    (dict(residual_out=at(0)), ALIAS), (dict(residual_out=at(10) + 64), ALIAS), (dict(residual_out=at(20)), ALIAS),
    (dict(out=(at(1), at(31))), ALIAS), (dict(out=(at(31), at(10))), ALIAS), (dict(out=(at(11), at(31))), ALIAS),
    (dict(rows=0), OK), (dict(rows=0, residual_out=at(10)), OK), (dict(rows=0, bufs=[None, None], residual=None), OK),
])
def test_norm_refusals(lib, change, want):
    n = change.get("n", 2)
    a = dict(bufs=[at(i) for i in range(n)], rows=4, hidden=256, gamma=at(20), eps=1e-6, residual=at(10),
             residual_out=at(11), out=mx(30), dtype=BF16)
    a.update(change)
    assert lib.rra_allreduce_rmsnorm_mx4(ptrs(a["bufs"]), n, a["rows"], a["hidden"], a["gamma"], a["eps"],
                                         a["residual"], a["residual_out"], None if a["out"] is None else mxs([a["out"]]),
                                         a["dtype"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(n=0), INV), (dict(n=9), UNS), (dict(x=None), INV), (dict(D=0), INV), (dict(dtype=I32), INV),
    (dict(T=1 << 31), UNS), (dict(D=1 << 31), UNS), (dict(widths=[1 << 31, 5]), UNS), (dict(outs=[at(5), None]), INV),
    (dict(outs=[at(5) + 1, at(6)]), INV), (dict(x=mx(0, codes=16, scales=8)), UNS), (dict(x=mx(0, codes=None)), INV),
    (dict(ws=[mx(1), mx(2, codes=8)]), UNS), (dict(ws=[mx(1), mx(2, scales=None)]), INV), (dict(outs=[at(5), at(5)]), ALIAS),
    (dict(outs=[at(0), at(5)]), ALIAS), (dict(outs=[at(5), at(2) + STEP // 2]), ALIAS), (dict(T=0), OK),
    (dict(widths=[0, 0]), OK), (dict(widths=[0, 0], ws=[(None, None)] * 2, outs=[None, None]), OK), (dict(), NOT_INIT),
])
def test_product_refusals(lib, change, want):
    n = change.get("n", 2)
    a = dict(x=mx(0), ws=[mx(1), mx(2)], outs=[at(5), at(6)], T=8, D=256, widths=[128, 100], dtype=BF16)
    a.update(change)
    assert lib.rra_mx4_product(None if a["x"] is None else mxs([a["x"]]), mxs(a["ws"]), ptrs(a["outs"]), n, a["T"],
                               a["D"], sizes(a["widths"]), a["dtype"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(n=0), INV), (dict(n=9), UNS), (dict(dtype=I32), INV), (dict(out=None), INV), (dict(out=at(5) + 1), INV),
    (dict(T=1 << 31), UNS), (dict(F=1 << 31), UNS), (dict(D=1 << 31), UNS), (dict(xs=[mx(0), mx(1, codes=8)]), UNS),
    (dict(ws=[mx(2), mx(3, scales=None)]), INV), (dict(out=at(1)), ALIAS), (dict(out=at(3) + STEP // 2), ALIAS),
    (dict(T=0), OK), (dict(D=0), OK), (dict(F=1 << 29), UNS), (dict(), NOT_INIT),
])
def test_product_sum_refusals(lib, change, want):
    n = change.get("n", 2)
    a = dict(xs=[mx(0), mx(1)], ws=[mx(2), mx(3)], out=at(5), T=8, F=100, D=256, dtype=BF16)
    a.update(change)
    assert lib.rra_mx4_product_sum(mxs(a["xs"]), mxs(a["ws"]), a["out"], n, a["T"], a["F"], a["D"], a["dtype"],
                                   None) == want


@pytest.mark.parametrize("change,want", [
    (dict(n=0), INV), (dict(n=9), UNS), (dict(x=None), INV), (dict(D=0), INV), (dict(act=2), INV),
    (dict(T=1 << 31), UNS), (dict(F=1 << 31), UNS), (dict(gates=[mx(1), mx(2, codes=None)]), INV),
    (dict(ups=[mx(3, scales=8), mx(4)]), UNS), (dict(acts=[mx(5), mx(6, codes=4)]), UNS),
    (dict(acts=[mx(5), mx(5)]), ALIAS), (dict(acts=[mx(5), mx(0)]), ALIAS), (dict(acts=[(at(5), at(3)), mx(6)]), ALIAS),
    (dict(T=0), OK), (dict(F=0), OK), (dict(), NOT_INIT),
])
def test_gated_refusals(lib, change, want):
    n = change.get("n", 2)
    a = dict(x=mx(0), gates=[mx(1), mx(2)], ups=[mx(3), mx(4)], acts=[mx(5), mx(6)], T=8, D=256, F=100, act=0)
    a.update(change)
    assert lib.rra_mx4_gated_ffn(None if a["x"] is None else mxs([a["x"]]), mxs(a["gates"]), mxs(a["ups"]),
                                 mxs(a["acts"]), n, a["T"], a["D"], a["F"], a["act"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(n=0), INV), (dict(n=9), UNS), (dict(dtype=I32), INV), (dict(uniform=None), INV), (dict(token=None), INV),
    (dict(token=at(11) + 4), INV), (dict(logprob=at(12) + 2), INV), (dict(top_k=at(14) + 1), INV),
    (dict(logits=[at(0), None]), INV), (dict(logits=[at(0) + 1, at(1)]), INV), (dict(vocab=[368640, 1]), UNS),
    (dict(vocab=[1 << 60, 1]), UNS), (dict(rows=1 << 31), UNS), (dict(token=at(0)), ALIAS), (dict(logprob=at(11)), ALIAS),
    (dict(logprob=at(10)), ALIAS), (dict(token=at(13)), ALIAS), (dict(rows=0), OK),
    (dict(rows=0, uniform=None, token=None, logits=[None, None]), OK),
])
def test_sample_refusals(lib, change, want):
    n = change.get("n", 2)
    a = dict(logits=[at(0), at(1)], vocab=[100, 99], rows=3, uniform=at(10), temperature=at(13), top_k=at(14),
             top_p=at(15), min_p=at(16), token=at(11), logprob=at(12), dtype=BF16)
    a.update(change)
    assert lib.rra_vocab_sample(ptrs(a["logits"]), sizes(a["vocab"]), n, a["rows"], a["uniform"], a["temperature"],
                                a["top_k"], a["top_p"], a["min_p"], a["token"], a["logprob"], a["dtype"], None) == want


def test_binding_refusals():
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)
    x = torch.zeros(4, 64)
    for bad in ((codes[:, :16], scales), (codes, scales[:256]), (codes.to(torch.int16), scales), (codes.t(), scales)):
        with pytest.raises(ValueError):
            rra.rra_mx4_quantize(x, *bad)
    with pytest.raises(TypeError):
        rra.rra_mx4_quantize(x.to(torch.float16), codes, scales)
    with pytest.raises(ValueError):
        rra.rra_allreduce_rmsnorm_mx4([x], torch.zeros(63), 63, codes, scales)
    with pytest.raises(ValueError):
        rra.rra_mx4_product((codes, scales), [(codes, scales)], [torch.zeros(4, 3), torch.zeros(4, 4)], 64)
    with pytest.raises(ValueError):
        rra.rra_vocab_sample([x], torch.zeros(4), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        rra.rra_vocab_sample([x], torch.zeros(4), torch.zeros(4, dtype=torch.int64), top_k=torch.zeros(4))
    with pytest.raises(rra.RraError):
        rra.rra_mx4_product((codes, scales), [], [], 64)
    assert rra.rra_mx4_product((codes, scales), [], [], 64, check=False) == INV


# -- the reference ------------------------------------------------------------

def test_reference_rounds_to_the_nearest_code():
    x = torch.linspace(-6, 6, 32 * 61, dtype=torch.float64).view(-1, 32)
    x[:, 0] = 6.0  # every block has the scale 1
    codes, byte = ref.quantize(x)
    v = ref.values(codes, byte, 32)
    grid = torch.tensor(ref.VALUES + [-q for q in ref.VALUES], dtype=torch.float64)
    near = (x[:, :, None] - grid).abs().amin(2)
    assert torch.equal((v - x).abs(), near) and int(byte.unique()) == 127
    ties = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0] * 4, dtype=torch.float64)[None]
    codes, byte = ref.quantize(ties)
    assert ref.values(codes, byte, 32)[0, :8].tolist() == [0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0, 6.0]


@pytest.mark.parametrize("amax,e", [(6.0, 0), (6.0 + 2.0 ** -20, 1), (3.0, -1), (3.1, 0), (1.0, -2), (2.0 ** -149, -127),
                                    (6.0 * 2.0 ** -127, -127), (6.1 * 2.0 ** -127, -126), (3.4028234663852886e38, 126)])
def test_reference_exponent(amax, e):
    assert ref.exponent(amax) == e and amax <= 6.0 * 2.0 ** e and (e == -127 or amax > 6.0 * 2.0 ** (e - 1))


def test_reference_layout_round_trip():
    x = torch.randn(133, 161, dtype=torch.float64)
    codes, scales, v = ref.pack(x)
    assert torch.equal(ref.read(codes, scales, 161), v)
    assert scales.numel() == ref.scale_bytes(133, 161)
    # row 130 (tile band 1, row 2), block 5 (tile 1, byte 1)
    assert int(scales[(1 * 2 + 1) * 512 + 2 * 16 + 0 * 4 + 1]) == int(ref.quantize(x)[1][130, 5])
