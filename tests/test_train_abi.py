"""Refusals of the training-step operators: every bad call returns its error
before any launch, so fake device addresses are enough and no GPU is needed."""
import ctypes

import pytest

import collective_all_reduce_rank_gb300 as rra

A = 1 << 40  # never dereferenced
STEP = 1 << 32
HUGE = 1 << 62
OK, INV, UNS, ALIAS, WS = (rra.RRA_SUCCESS, rra.RRA_ERR_INVALID_ARG, rra.RRA_ERR_UNSUPPORTED, rra.RRA_ERR_ALIAS,
                           rra.RRA_ERR_WORKSPACE)
NOT_INIT = rra.RRA_ERR_NOT_INITIALIZED
BF16, F32, I32 = rra.RRA_BFLOAT16, rra.RRA_FLOAT32, rra.RRA_INT32


def at(i):
    return A + i * STEP


def arr(ps):
    return (ctypes.c_void_p * max(1, len(ps)))(*ps)


def sizes(vs):
    return (ctypes.c_size_t * len(vs))(*vs)


@pytest.fixture(scope="module")
def lib():
    lib = rra.load()
    rra.rra_finalize()
    return lib


# -- norm --------------------------------------------------------------------

def save8(lib, **k):
    n = k.get("n", 2)
    a = dict(bufs=[at(i) for i in range(n)], outs=[at(10 + i) for i in range(n)], rows=4, hidden=256, gamma=at(20),
             eps=1e-6, codes=at(21), scales=at(22), rstd=at(23), dtype=BF16)
    a.update(k)
    return lib.rra_allreduce_rmsnorm_save8(arr(a["bufs"]), arr(a["outs"]), n, a["rows"], a["hidden"], a["gamma"],
                                           a["eps"], a["codes"], a["scales"], a["rstd"], a["dtype"], None)


@pytest.mark.parametrize("change,want", [
    (dict(n=0), INV), (dict(n=9), UNS), (dict(dtype=I32), INV), (dict(dtype=7), INV), (dict(hidden=0), INV),
    (dict(hidden=51201), UNS), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV), (dict(gamma=None), INV),
    (dict(codes=None), INV), (dict(scales=None), INV), (dict(rstd=None), INV), (dict(rstd=at(23) + 2), INV),
    (dict(gamma=at(20) + 1), INV), (dict(bufs=[at(0), None]), INV), (dict(outs=[at(10) + 1, at(11)]), INV),
    (dict(outs=[at(10), at(10)]), ALIAS), (dict(outs=[at(1), at(11)]), ALIAS), (dict(codes=at(0)), ALIAS),
    (dict(codes=at(20)), ALIAS), (dict(scales=at(21)), ALIAS), (dict(rstd=at(10) + 4), ALIAS),
    (dict(rows=1 << 31), UNS),
    (dict(rows=0), OK), (dict(rows=0, bufs=[None, None], outs=[None, None], codes=None, scales=None, rstd=None), OK),
    (dict(rows=0, outs=[at(0), at(1)]), OK),
])
def test_save8_refusals(lib, change, want):
    assert save8(lib, **change) == want


@pytest.mark.parametrize("change,want", [
    (dict(codes=None), INV), (dict(scales=None), INV), (dict(out=None), INV), (dict(hidden=0), INV),
    (dict(dtype=I32), INV), (dict(hidden=51201), UNS), (dict(out=at(1)), ALIAS), (dict(out=at(3)), ALIAS),
    (dict(out=at(5) + 1), INV), (dict(rstd=at(3) + 1), INV), (dict(rows=0), OK),
    (dict(rows=0, rstd=None, gamma=None), OK),
])
def test_restore8_refusals(lib, change, want):
    a = dict(codes=at(1), scales=at(2), rstd=at(3), gamma=at(4), out=at(5), rows=3, hidden=300, dtype=F32)
    a.update(change)
    assert lib.rra_rmsnorm_restore8(a["codes"], a["scales"], a["rstd"], a["gamma"], a["out"], a["rows"], a["hidden"],
                                    a["dtype"], None) == want


@pytest.mark.parametrize("change,want", [
    (dict(n=9), UNS), (dict(dtype=I32), INV), (dict(dgamma=None), INV), (dict(dgamma=at(24) + 1), INV),
    (dict(ws=None), INV), (dict(ws=at(25) + 16), INV), (dict(ws_bytes=64), WS), (dict(ws=at(0)), ALIAS),
    (dict(dgamma=at(25)), ALIAS), (dict(dgamma=at(20)), ALIAS), (dict(dxs=[at(1), at(0)]), ALIAS),
    (dict(codes=None), INV), (dict(rstd=None), INV),
])
def test_backward8_refusals(lib, change, want):
    n = change.get("n", 2)
    a = dict(grads=[at(i) for i in range(n)], dxs=[at(10 + i) for i in range(n)], rows=4, hidden=256, codes=at(21),
             scales=at(22), rstd=at(23), gamma=at(20), dgamma=at(24), ws=at(25), ws_bytes=HUGE, dtype=BF16)
    a.update(change)
    assert lib.rra_allreduce_rmsnorm_backward8(arr(a["grads"]), arr(a["dxs"]), n, a["rows"], a["hidden"], a["codes"],
                                               a["scales"], a["rstd"], a["gamma"], a["dgamma"], a["ws"],
                                               a["ws_bytes"], a["dtype"], None) == want


# -- gated feed-forward ------------------------------------------------------

FFN_BAD = [
    (dict(n=0), INV), (dict(n=9), UNS), (dict(x=None), INV), (dict(x=at(0) + 2), UNS), (dict(x=at(0) + 1), INV),
    (dict(D=0), INV), (dict(act=2), INV), (dict(dtype=F32), UNS), (dict(dtype=I32), UNS), (dict(dtype=9), INV),
    (dict(T=1 << 31), UNS), (dict(F=1 << 31), UNS), (dict(gates=[at(1), None]), INV),
    (dict(gates=[at(1) + 8, at(2)]), UNS), (dict(ups=[at(3) + 1, at(4)]), INV), (dict(ws=at(30) + 8), INV),
    (dict(T=64, D=257, ws_bytes=8), WS), (dict(T=64, D=257, ws=None), INV),
]


def ffn_args(change):
    n = change.get("n", 2)
    a = dict(n=n, x=at(0), gates=[at(1), at(2)], ups=[at(3), at(4)], acts=[at(5), at(6)], dx=at(7),
             dgates=[at(8), at(9)], dups=[at(10), at(11)], T=8, D=256, F=128, act=0, dtype=BF16, ws=at(30),
             ws_bytes=HUGE)
    a.update(change)
    return a


def ffn(lib, change):
    a = ffn_args(change)
    return lib.rra_gated_ffn(a["x"], arr(a["gates"]), arr(a["ups"]), arr(a["acts"]), a["n"], a["T"], a["D"], a["F"],
                             a["act"], a["dtype"], a["ws"], a["ws_bytes"], None)


def ffn_back(lib, change):
    a = ffn_args(change)
    return lib.rra_gated_ffn_backward(a["x"], arr(a["gates"]), arr(a["ups"]), arr(a["acts"]), a["dx"],
                                      arr(a["dgates"]), arr(a["dups"]), a["n"], a["T"], a["D"], a["F"], a["act"],
                                      a["dtype"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("change,want", FFN_BAD + [
    (dict(acts=[at(5), at(5)]), ALIAS), (dict(acts=[at(0), at(6)]), ALIAS), (dict(acts=[at(5), None]), INV),
    (dict(), NOT_INIT), (dict(T=0), OK), (dict(F=0), OK), (dict(T=0, x=None, acts=[None, None]), OK),
])
def test_gated_ffn_refusals(lib, change, want):
    assert ffn(lib, change) == want


@pytest.mark.parametrize("change,want", FFN_BAD + [
    (dict(dx=None), INV), (dict(dx=at(7) + 1), INV), (dict(dgates=[None, at(9)]), INV), (dict(dups=[at(10), at(8)]), ALIAS),
    (dict(dx=at(0)), ALIAS), (dict(dgates=[at(1), at(9)]), ALIAS), (dict(dx=at(30)), ALIAS), (dict(ws_bytes=64), WS),
    (dict(), NOT_INIT), (dict(T=0, F=0), OK),
])
def test_gated_ffn_backward_refusals(lib, change, want):
    assert ffn_back(lib, change) == want


# -- vocabulary loss ---------------------------------------------------------

LOSS_BAD = [
    (dict(n=0), INV), (dict(n=9), UNS), (dict(x=None), INV), (dict(x=at(0) + 8), UNS), (dict(D=0), INV),
    (dict(dtype=F32), UNS), (dict(dtype=9), INV), (dict(weights=[at(1), None]), INV),
    (dict(weights=[at(1), at(2) + 2]), UNS), (dict(vocab=[0, 0]), INV), (dict(vocab=[1 << 31, 4]), UNS),
    (dict(targets=None), INV), (dict(targets=at(3) + 4), INV), (dict(T=1 << 31), UNS), (dict(ws=at(30) + 64), INV),
    (dict(ws=None), INV), (dict(ws_bytes=8), WS),
]


def loss_args(change):
    a = dict(n=change.get("n", 2), x=at(0), weights=[at(1), at(2)], vocab=[300, 200], targets=at(3), T=8, D=256,
             ignore=-100, loss=at(4), lse=at(5), grad=at(6), dx=at(7), dw=[at(8), at(9)], dtype=BF16, ws=at(30),
             ws_bytes=HUGE)
    a.update(change)
    return a


def loss(lib, change):
    a = loss_args(change)
    return lib.rra_vocab_loss(a["x"], arr(a["weights"]), sizes(a["vocab"]), a["targets"], a["n"], a["T"], a["D"],
                              a["ignore"], a["loss"], a["lse"], a["dtype"], a["ws"], a["ws_bytes"], None)


def loss_back(lib, change):
    a = loss_args(change)
    return lib.rra_vocab_loss_backward(a["x"], arr(a["weights"]), sizes(a["vocab"]), a["targets"], a["lse"],
                                       a["grad"], a["dx"], arr(a["dw"]), a["n"], a["T"], a["D"], a["ignore"],
                                       a["dtype"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("change,want", LOSS_BAD + [
    (dict(loss=None), INV), (dict(lse=at(5) + 2), INV), (dict(loss=at(5)), ALIAS), (dict(loss=at(0)), ALIAS),
    (dict(lse=at(30)), ALIAS), (dict(), NOT_INIT), (dict(T=0), OK), (dict(T=0, ws=None, ws_bytes=0), OK),
    (dict(T=0, x=None, targets=None, loss=None, lse=None), OK), (dict(weights=[None, at(2)], vocab=[0, 5]), NOT_INIT),
])
def test_vocab_loss_refusals(lib, change, want):
    assert loss(lib, change) == want


@pytest.mark.parametrize("change,want", LOSS_BAD + [
    (dict(grad=None), INV), (dict(dx=None), INV), (dict(dx=at(7) + 1), INV), (dict(dw=[at(8), None]), INV),
    (dict(dw=[at(8), at(8)]), ALIAS), (dict(dx=at(0)), ALIAS), (dict(dw=[at(1), at(9)]), ALIAS), (dict(), NOT_INIT),
])
def test_vocab_loss_backward_refusals(lib, change, want):
    assert loss_back(lib, change) == want


def test_workspace_sizes_grow_with_the_call(lib):
    w = rra.rra_vocab_loss_workspace_bytes
    assert w(64, 512, [1000, 1000], 2) <= w(64, 512, [1000, 1000], 1)
    assert w(8192, 512, [16384] * 8, 1) <= (512 << 20) + 64 * 8192 * 512 * 4 + (1 << 20)
    assert w(0, 512, [100], 1) == 0
    assert rra.rra_gated_ffn_workspace_bytes(2, 64, 512, 128, 0) == 0
    assert rra.rra_gated_ffn_workspace_bytes(2, 64, 513, 128, 0) > 0
    # dg and du of both ranks, rows padded to 64 columns
    assert rra.rra_gated_ffn_workspace_bytes(2, 64, 512, 100, 1) >= 4 * 64 * 128 * 2
    assert rra.rra_allreduce_rmsnorm_backward8_workspace_bytes(4, 256) == 4 * 256 * 4


def test_binding_checks_shapes_and_types():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 16, dtype=torch.bfloat16)
    w = torch.zeros(8, 16, dtype=torch.bfloat16)
    a = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="shard"):
        rra.rra_gated_ffn(x, [w], [torch.zeros(8, 15, dtype=torch.bfloat16)], [a], stream=0)
    with pytest.raises(ValueError, match="activations"):
        rra.rra_gated_ffn(x, [w], [w], [torch.zeros(4, 9, dtype=torch.bfloat16)], stream=0)
    with pytest.raises(ValueError, match="contiguous"):
        rra.rra_gated_ffn(torch.zeros(16, 4, dtype=torch.bfloat16).t(), [w], [w], [a], stream=0,
                          workspace=torch.zeros(256, dtype=torch.uint8))
    with pytest.raises(ValueError, match="targets"):
        rra.rra_vocab_loss(x, [w], torch.zeros(4, dtype=torch.int32), torch.zeros(4), torch.zeros(4), stream=0)
    with pytest.raises(ValueError, match="scales"):
        rra.rra_allreduce_rmsnorm_save8([x], [x.clone()], x[0], 16, torch.zeros(4, 16, dtype=torch.uint8),
                                        torch.zeros(4, 2, dtype=torch.uint8), torch.zeros(4), stream=0)
    with pytest.raises(rra.RraError) as err:
        rra.rra_gated_ffn(x, [w], [w], [a], act=5, stream=0, workspace=torch.zeros(0, dtype=torch.uint8))
    assert err.value.status == INV


@pytest.mark.parametrize("n,status", [(0, INV), (9, UNS)])
def test_a_number_of_ranks_that_is_refused_is_returned_without_check(n, status):
    torch = pytest.importorskip("torch")
    bf = torch.bfloat16
    x, w, a, f = (torch.zeros(4, 16, dtype=bf), [torch.zeros(8, 16, dtype=bf)] * n, [torch.zeros(4, 8, dtype=bf)] * n,
                  torch.zeros(4))
    xs, tgt, row = [x] * n, torch.zeros(4, dtype=torch.int64), torch.zeros(16, dtype=bf)
    saved = (torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8), f)
    calls = [
        lambda **k: rra.rra_allreduce_rmsnorm_save8(xs, xs, row, 16, *saved, **k),
        lambda **k: rra.rra_allreduce_rmsnorm_backward8(xs, xs, *saved, row, torch.zeros(16), **k),
        lambda **k: rra.rra_gated_ffn(x, w, w, a, **k),
        lambda **k: rra.rra_gated_ffn_backward(x, w, w, a, x, w, w, **k),
        lambda **k: rra.rra_vocab_loss(x, w, tgt, f, f, **k),
        lambda **k: rra.rra_vocab_loss_backward(x, w, tgt, f, f, x, w, **k),
    ]
    for call in calls:
        assert call(check=False) == status
        with pytest.raises(rra.RraError) as err:
            call()
        assert err.value.status == status
