"""GB300-native all-reduce, reduce-scatter and all-gather over N virtual ranks.

A thin ctypes binding over ``librra.so`` (the C ABI declared in
``include/rra.h``).  Every function here has the C function's name and only
marshals arguments: torch tensors become device pointers, torch streams
become ``cudaStream_t``.  All computation runs in the library's CUDA kernels;
there is no CPU path.  A call whose status is not ``RRA_SUCCESS`` raises
``RraError`` (pass ``check=False`` to get the status code instead).

The library is built in-tree (``collective_all_reduce_rank_gb300/librra.so``)
by ``build.build()``; loading it builds it first when the sources are newer,
and raises if that is impossible.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import threading

from . import build as _build

RRA_OK = 0
RRA_SUCCESS = RRA_OK
RRA_ERR_INVALID_ARG = 1
RRA_ERR_UNSUPPORTED = 2
RRA_ERR_ALIAS = 3
RRA_ERR_NOT_INITIALIZED = 4
RRA_ERR_CUDA = 5
RRA_ERR_TIMEOUT = 6
RRA_ERR_WORKSPACE = 7

RRA_INT32 = 0
RRA_FLOAT32 = 1
RRA_BFLOAT16 = 2

RRA_SUM = 0

RRA_ALGO_AUTO = 0
RRA_ALGO_RING = 1
RRA_ALGO_ONE_SHOT = 2
RRA_ALGO_TWO_SHOT = 3
RRA_ALGO_DIRECT = 4
RRA_ALGO_COPY_ENGINE = 5
RRA_ALGO_TREE = 6

RRA_ACT_SILU = 0
RRA_ACT_GELU_TANH = 1

RRA_MAX_RANKS = 8

RRA_CKPT_BLOCK = 128  # columns that share a scale in an 8-bit checkpoint

DTYPE_NAMES = {RRA_INT32: "int32", RRA_FLOAT32: "float32", RRA_BFLOAT16: "bfloat16"}
ALGO_NAMES = {RRA_ALGO_AUTO: "auto", RRA_ALGO_RING: "ring", RRA_ALGO_ONE_SHOT: "one_shot",
              RRA_ALGO_TWO_SHOT: "two_shot", RRA_ALGO_DIRECT: "direct"}

_lock = threading.Lock()
_lib = None


class RraError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__("%s: %s (status %d)" % (what or "rra", rra_status_string(status), status))


def library_path() -> str:
    return _build.LIB


def load():
    """Load librra.so (building it first when it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.build()
        if not os.path.exists(path):
            raise RuntimeError("librra.so is missing and could not be built")
        lib = ctypes.CDLL(path)
        _declare(lib)
        _lib = lib
    return _lib


def _declare(lib):
    vp = ctypes.c_void_p
    vpp = ctypes.POINTER(ctypes.c_void_p)
    i, sz, u32, u64 = ctypes.c_int, ctypes.c_size_t, ctypes.c_uint32, ctypes.c_uint64
    i64 = ctypes.c_int64
    sigs = {
        "rra_init": (i, [i, sz]),
        "rra_finalize": (i, []),
        "rra_allreduce": (i, [vpp, vpp, i, sz, i, i, i, vp]),
        "rra_allreduce_two_shot_static": (i, [vpp, vpp, i, sz, i, i, vp]),
        "rra_reduce_scatter": (i, [vpp, vpp, i, sz, i, i, i, vp]),
        "rra_all_gather": (i, [vpp, vpp, i, sz, i, i, vp]),
        "rra_allreduce_rmsnorm": (i, [vpp, vpp, i, sz, sz, vp, ctypes.c_float, i, vp]),
        # host arrays of these calls travel as packed bytes
        "rra_allreduce_rmsnorm_save8": (i, [vp, vp, i, sz, sz, vp, ctypes.c_float, vp, vp, vp, i, vp]),
        "rra_rmsnorm_restore8": (i, [vp, vp, vp, vp, vp, sz, sz, i, vp]),
        "rra_allreduce_rmsnorm_backward8_workspace_bytes": (sz, [sz, sz]),
        "rra_allreduce_rmsnorm_backward8": (i, [vp, vp, i, sz, sz, vp, vp, vp, vp, vp, vp, sz, i, vp]),
        "rra_gated_ffn_workspace_bytes": (sz, [i, sz, sz, sz, i]),
        "rra_gated_ffn": (i, [vp, vp, vp, vp, i, sz, sz, sz, i, i, vp, sz, vp]),
        "rra_gated_ffn_backward": (i, [vp, vp, vp, vp, vp, vp, vp, i, sz, sz, sz, i, i, vp, sz, vp]),
        "rra_vocab_loss_workspace_bytes": (sz, [i, sz, sz, vp, i]),
        "rra_vocab_loss": (i, [vp, vp, vp, vp, i, sz, sz, i64, vp, vp, i, vp, sz, vp]),
        "rra_vocab_loss_backward": (i, [vp, vp, vp, vp, vp, vp, vp, vp, i, sz, sz, i64, i, vp, sz, vp]),
        "rra_ll_wire_bytes": (sz, [sz]),
        "rra_ll128_wire_bytes": (sz, [sz]),
        "rra_ll_pack": (i, [vp, sz, vp, u32, vp]),
        "rra_ll_unpack": (i, [vpp, i, vp, sz, i, i, u32, vp]),
        "rra_ll128_pack": (i, [vp, sz, vp, u64, vp]),
        "rra_ll128_unpack": (i, [vpp, i, vp, sz, i, i, u64, vp]),
        "rra_query_status": (i, [vp, ctypes.POINTER(ctypes.c_int32)]),
        "rra_query_status_static": (i, [vp, ctypes.POINTER(ctypes.c_int32)]),
        "rra_select_algo": (i, [i, sz, i]),
        "rra_load_tuning": (i, [ctypes.c_char_p]),
        "rra_set_timeout_ns": (None, [u64]),
        "rra_debug_skip_rank": (None, [i]),
        "rra_set_max_ctas": (None, [i]),
        "rra_status_string": (ctypes.c_char_p, [i]),
        "rra_dump_recent": (i, [ctypes.c_char_p, sz]),
    }
    for name, (res, args) in sigs.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args


def header_symbols() -> list[str]:
    """Names of every function include/rra.h declares."""
    hdr = os.path.join(_build.ROOT, "include", "rra.h")
    text = open(hdr).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(rra_[a-z0-9_]+)\s*\(", text)))


# ---------------------------------------------------------------------------
# marshalling
# ---------------------------------------------------------------------------

def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if hasattr(x, "is_contiguous") and not x.is_contiguous():
            raise ValueError("tensors passed to rra must be contiguous")
        return int(x.data_ptr())
    raise TypeError("expected a tensor or a device pointer (int), got %r" % type(x))


def _ptr_array(xs):
    return (ctypes.c_void_p * len(xs))(*[_ptr(x) for x in xs])


def _stream(stream, like=None) -> int:
    if stream is None:
        if like is not None and hasattr(like, "device"):
            import torch

            return int(torch.cuda.current_stream(like.device).cuda_stream)
        return 0
    if isinstance(stream, int):
        return stream
    return int(stream.cuda_stream)


def _dtype_of(t):
    import torch

    m = {torch.int32: RRA_INT32, torch.float32: RRA_FLOAT32, torch.bfloat16: RRA_BFLOAT16}
    if t.dtype not in m:
        raise TypeError("unsupported dtype %s (int32, float32, bfloat16)" % t.dtype)
    return m[t.dtype]


def _resolve(xs, count, dtype):
    first = xs[0] if xs else None
    if dtype is None:
        if first is None or isinstance(first, int):
            raise ValueError("dtype is required with raw pointers")
        dtype = _dtype_of(first)
    if count is None:
        if first is None or isinstance(first, int):
            raise ValueError("count is required with raw pointers")
        count = int(first.numel())
    return count, dtype


def _ret(status, what, check):
    if check and status != RRA_SUCCESS:
        raise RraError(status, what)
    return status


# ---------------------------------------------------------------------------
# the C functions
# ---------------------------------------------------------------------------

def rra_status_string(status: int) -> str:
    return load().rra_status_string(status).decode()


def rra_init(device: int = 0, workspace_bytes: int = 0, check: bool = True) -> int:
    return _ret(load().rra_init(device, workspace_bytes), "rra_init", check)


def rra_finalize(check: bool = True) -> int:
    return _ret(load().rra_finalize(), "rra_finalize", check)


def rra_allreduce(bufs, outs, count=None, dtype=None, op=RRA_SUM, algo=RRA_ALGO_AUTO, stream=None,
                  check=True, nranks=None) -> int:
    count, dtype = _resolve(bufs, count, dtype)
    n = len(bufs) if nranks is None else nranks
    st = load().rra_allreduce(_ptr_array(bufs), _ptr_array(outs), n, count, dtype, op, algo,
                              _stream(stream, bufs[0] if bufs else None))
    return _ret(st, "rra_allreduce", check)


def rra_allreduce_two_shot_static(bufs, outs, count=None, dtype=None, op=RRA_SUM, stream=None,
                                  check=True, nranks=None) -> int:
    """Two-shot all-reduce whose scratch is a static device array inside the
    library: no rra_init and no device allocation, for callers that may not
    allocate.  Calls that overlap on the GPU share that array and race."""
    count, dtype = _resolve(bufs, count, dtype)
    n = len(bufs) if nranks is None else nranks
    st = load().rra_allreduce_two_shot_static(_ptr_array(bufs), _ptr_array(outs), n, count, dtype, op,
                                              _stream(stream, bufs[0] if bufs else None))
    return _ret(st, "rra_allreduce_two_shot_static", check)


def rra_reduce_scatter(bufs, outs, recvcount=None, dtype=None, op=RRA_SUM, algo=RRA_ALGO_AUTO,
                       stream=None, check=True, nranks=None) -> int:
    if recvcount is None and outs and not isinstance(outs[0], int):
        recvcount = int(outs[0].numel())
    recvcount, dtype = _resolve(bufs, recvcount, dtype)
    n = len(bufs) if nranks is None else nranks
    st = load().rra_reduce_scatter(_ptr_array(bufs), _ptr_array(outs), n, recvcount, dtype, op, algo,
                                   _stream(stream, bufs[0] if bufs else None))
    return _ret(st, "rra_reduce_scatter", check)


def rra_all_gather(bufs, outs, sendcount=None, dtype=None, algo=RRA_ALGO_AUTO, stream=None,
                   check=True, nranks=None) -> int:
    sendcount, dtype = _resolve(bufs, sendcount, dtype)
    n = len(bufs) if nranks is None else nranks
    st = load().rra_all_gather(_ptr_array(bufs), _ptr_array(outs), n, sendcount, dtype, algo,
                               _stream(stream, bufs[0] if bufs else None))
    return _ret(st, "rra_all_gather", check)


def rra_allreduce_rmsnorm(bufs, outs, gamma, hidden, eps=1e-6, rows=None, dtype=None, stream=None,
                          check=True, nranks=None) -> int:
    count, dtype = _resolve(bufs, None if rows is None else rows * hidden, dtype)
    rows = count // hidden if rows is None else rows
    n = len(bufs) if nranks is None else nranks
    st = load().rra_allreduce_rmsnorm(_ptr_array(bufs), _ptr_array(outs), n, rows, hidden, _ptr(gamma),
                                      eps, dtype, _stream(stream, bufs[0] if bufs else None))
    return _ret(st, "rra_allreduce_rmsnorm", check)


# -- the training step around a tensor-parallel all-reduce -------------------
#
# These calls check shapes, types, devices and contiguity of every tensor.
# The small ones are bound by the host, so the checks read each attribute
# once and nothing is imported or looked up twice.

_PTRS = [struct.Struct("%dP" % n).pack for n in range(RRA_MAX_RANKS + 1)]
_SIZES = [struct.Struct("%dN" % n).pack for n in range(RRA_MAX_RANKS + 1)]
_torch_mod = None
_several = True  # more than one GPU is visible


def _t():
    """torch, and its tensor methods unbound (a call of one is cheaper than of
    a bound one)."""
    global _torch_mod, _data, _numel, _device, _dense, _several
    if _torch_mod is None:
        import torch

        t = torch.Tensor
        _data, _numel, _device, _dense = t.data_ptr, t.numel, t.get_device, t.is_contiguous
        _several = torch.cuda.device_count() > 1
        _torch_mod = torch
    return _torch_mod


def _refuse(what, t, dtype, shape, device):
    if not t.is_contiguous():
        raise ValueError("tensors passed to rra must be contiguous (%s)" % what)
    if t.get_device() != device:
        raise ValueError("tensors of one call must be on one device (%s is on %s)" % (what, t.device))
    raise ValueError("%s must be %s of %s, got %s of shape %s" % (what, dtype, shape, t.dtype, tuple(t.shape)))


def _one(what, t, dtype, shape, device):
    """Pointer of a tensor of this type, shape and device, contiguous."""
    if t.dtype is not dtype or t.shape != shape or _device(t) != device or not _dense(t):
        _refuse(what, t, dtype, shape, device)
    return _data(t)


def _flat(what, t, dtype, numel, device):
    """The same for a tensor of any shape with this many elements."""
    if t.dtype is not dtype or _numel(t) != numel or _device(t) != device or not _dense(t):
        _refuse(what, t, dtype, "%d elements" % numel, device)
    return _data(t)


def _ranks(what, ts, dtype, shape, device):
    """The pointers of one tensor per rank, as the C array of them."""
    ps = [_data(t) for t in ts if t.dtype is dtype and t.shape == shape and _device(t) == device and _dense(t)]
    if len(ps) != len(ts):
        for t in ts:
            _one(what, t, dtype, shape, device)
    return _PTRS[len(ps)](*ps)


def _flat_ranks(what, ts, dtype, numel, device):
    """The same for tensors of any shape with this many elements."""
    ps = [_data(t) for t in ts if t.dtype is dtype and _numel(t) == numel and _device(t) == device and _dense(t)]
    if len(ps) != len(ts):
        for t in ts:
            _flat(what, t, dtype, numel, device)
    return _PTRS[len(ps)](*ps)


def _same_count(n, *groups):
    """The status of a call with n ranks, which have to have a buffer each in every group."""
    if not 1 <= n <= RRA_MAX_RANKS:
        return RRA_ERR_INVALID_ARG if n < 1 else RRA_ERR_UNSUPPORTED
    for g in groups:
        if len(g) != n:
            raise ValueError("one buffer per rank is needed")
    return RRA_SUCCESS


def _on(stream, device):
    """The raw stream of the call (default: PyTorch's current one).  The
    library launches on the current device, so the tensors have to be there."""
    if device < 0:  # no GPU's: refused by the call itself
        return 0 if stream is None else stream if isinstance(stream, int) else int(stream.cuda_stream)
    cuda = _t()._C
    if _several and cuda._cuda_getDevice() != device:
        raise ValueError("the tensors are on cuda:%d, the current device is cuda:%d" % (device, cuda._cuda_getDevice()))
    if stream is None:
        return cuda._cuda_getCurrentRawStream(device)
    if isinstance(stream, int):
        return stream
    home = getattr(stream, "device_index", device)
    if home != device:
        raise ValueError("the stream is of cuda:%d, the tensors are on cuda:%d" % (home, device))
    return int(stream.cuda_stream)


def _scratch(workspace, device, stream, size, *args):
    """(pointer, bytes, tensor) of the caller's workspace, or of one made here
    from the memory of the call's stream, which PyTorch's allocator hands out
    and takes back in that stream's order (a block of another stream may still
    be in use there).  The tensor is kept until the call has been issued."""
    if workspace is None:
        torch = _t()
        if device < 0:  # refused by the call itself
            workspace = torch.empty(max(256, size(*args)), dtype=torch.uint8, device="cpu")
        elif stream is None or (isinstance(stream, int) and stream == torch._C._cuda_getCurrentRawStream(device)):
            workspace = torch.empty(max(256, size(*args)), dtype=torch.uint8, device=device)
        elif isinstance(stream, int):
            raise ValueError("a raw stream handle needs an explicit workspace unless it is the current stream's")
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(max(256, size(*args)), dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous() or workspace.get_device() != device:
        raise ValueError("the workspace must be contiguous and on the tensors' device")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _code_type(t):
    if t.element_size() != 1:
        raise ValueError("codes must be uint8 or float8_e4m3fn")
    return t.dtype


def _norm_dtype(t):
    torch = _t()
    if t.dtype is torch.bfloat16:
        return RRA_BFLOAT16
    if t.dtype is torch.float32:
        return RRA_FLOAT32
    raise TypeError("unsupported dtype %s (float32, bfloat16)" % t.dtype)


def rra_allreduce_rmsnorm_save8(bufs, outs, gamma, hidden, codes, scales, rstd, eps=1e-6, stream=None,
                                check=True) -> int:
    """All-reduce + RMSNorm that saves the sum in 8 bits for the backward
    pass: codes [rows, hidden] (float8_e4m3fn or uint8), scales
    [rows, ceil(hidden / 128)] uint8, rstd [rows] float32."""
    n = len(bufs)
    st = _same_count(n, outs)
    if st != RRA_SUCCESS:
        return _ret(st, "rra_allreduce_rmsnorm_save8", check)
    torch = _t()
    x = bufs[0]
    dev, dt, count = x.get_device(), x.dtype, x.numel()
    rows = count // hidden
    if rows * hidden != count:
        raise ValueError("a rank's buffer must hold whole rows of %d" % hidden)
    ins = _flat_ranks("a rank's buffer", bufs, dt, count, dev)
    os_ = _flat_ranks("a rank's output", outs, dt, count, dev)
    st = load().rra_allreduce_rmsnorm_save8(
        ins, os_, n, rows, hidden, _one("gamma", gamma, dt, (hidden,), dev), eps,
        _flat("codes", codes, _code_type(codes), count, dev),
        _one("scales", scales, torch.uint8, (rows, (hidden + 127) // 128), dev),
        _one("rstd", rstd, torch.float32, (rows,), dev), _norm_dtype(x), _on(stream, dev))
    return _ret(st, "rra_allreduce_rmsnorm_save8", check)


def rra_rmsnorm_restore8(codes, scales, rstd, gamma, out, stream=None, check=True) -> int:
    """out = the checkpoint's values, times rstd and gamma unless None."""
    torch = _t()
    rows, hidden = out.shape
    dev = out.get_device()
    st = load().rra_rmsnorm_restore8(
        _flat("codes", codes, _code_type(codes), rows * hidden, dev),
        _one("scales", scales, torch.uint8, (rows, (hidden + 127) // 128), dev),
        None if rstd is None else _one("rstd", rstd, torch.float32, (rows,), dev),
        None if gamma is None else _one("gamma", gamma, out.dtype, (hidden,), dev),
        _one("out", out, out.dtype, (rows, hidden), dev), rows, hidden, _norm_dtype(out), _on(stream, dev))
    return _ret(st, "rra_rmsnorm_restore8", check)


def rra_allreduce_rmsnorm_backward8_workspace_bytes(rows: int, hidden: int) -> int:
    return int(load().rra_allreduce_rmsnorm_backward8_workspace_bytes(rows, hidden))


def rra_allreduce_rmsnorm_backward8(grads, dxs, codes, scales, rstd, gamma, dgamma, workspace=None, stream=None,
                                    check=True) -> int:
    """Sum of the ranks' gradients through the norm, from the checkpoint."""
    n = len(grads)
    st = _same_count(n, dxs)
    if st != RRA_SUCCESS:
        return _ret(st, "rra_allreduce_rmsnorm_backward8", check)
    torch = _t()
    x = grads[0]
    dev, dt, count, hidden = x.get_device(), x.dtype, x.numel(), gamma.numel()
    rows = count // hidden if hidden else 0
    if rows * hidden != count:
        raise ValueError("a rank's gradient must hold whole rows of %d" % hidden)
    gs = _flat_ranks("a rank's gradient", grads, dt, count, dev)
    ds = _flat_ranks("a rank's output", dxs, dt, count, dev)
    ws, nb, _keep = _scratch(workspace, dev, stream, rra_allreduce_rmsnorm_backward8_workspace_bytes, rows, hidden)
    st = load().rra_allreduce_rmsnorm_backward8(
        gs, ds, n, rows, hidden, _flat("codes", codes, _code_type(codes), count, dev),
        _one("scales", scales, torch.uint8, (rows, (hidden + 127) // 128), dev),
        _one("rstd", rstd, torch.float32, (rows,), dev), _one("gamma", gamma, dt, (hidden,), dev),
        _one("dgamma", dgamma, torch.float32, (hidden,), dev), ws, nb, _norm_dtype(x), _on(stream, dev))
    return _ret(st, "rra_allreduce_rmsnorm_backward8", check)


def rra_gated_ffn_workspace_bytes(nranks: int, tokens: int, hidden: int, width: int, backward) -> int:
    return int(load().rra_gated_ffn_workspace_bytes(nranks, tokens, hidden, width, int(backward)))


def rra_gated_ffn(x, gates, ups, acts, act=RRA_ACT_SILU, workspace=None, stream=None, check=True) -> int:
    """acts[r] = act(x gates[r]^T) * (x ups[r]^T)."""
    n = len(gates)
    st = _same_count(n, ups, acts)
    if st != RRA_SUCCESS:
        return _ret(st, "rra_gated_ffn", check)
    _t()
    T, D = x.shape
    F, dev, dt = gates[0].shape[0], x.get_device(), x.dtype
    gs = _ranks("a gate or up shard", gates, dt, (F, D), dev)
    us = _ranks("a gate or up shard", ups, dt, (F, D), dev)
    os_ = _ranks("a rank's activations", acts, dt, (T, F), dev)
    ws, nb, _keep = _scratch(workspace, dev, stream, rra_gated_ffn_workspace_bytes, n, T, D, F, 0)
    st = load().rra_gated_ffn(_one("x", x, dt, (T, D), dev), gs, us, os_, n, T, D, F, act, _dtype_of(x), ws, nb,
                              _on(stream, dev))
    return _ret(st, "rra_gated_ffn", check)


def rra_gated_ffn_backward(x, gates, ups, dacts, dx, dgates, dups, act=RRA_ACT_SILU, workspace=None, stream=None,
                           check=True) -> int:
    """Gradients of rra_gated_ffn: dx summed over the ranks, dgates, dups."""
    n = len(gates)
    st = _same_count(n, ups, dacts, dgates, dups)
    if st != RRA_SUCCESS:
        return _ret(st, "rra_gated_ffn_backward", check)
    _t()
    T, D = x.shape
    F, dev, dt = gates[0].shape[0], x.get_device(), x.dtype
    gs = _ranks("a gate or up shard", gates, dt, (F, D), dev)
    us = _ranks("a gate or up shard", ups, dt, (F, D), dev)
    das = _ranks("a rank's activations", dacts, dt, (T, F), dev)
    dgs = _ranks("a shard's gradient", dgates, dt, (F, D), dev)
    dus = _ranks("a shard's gradient", dups, dt, (F, D), dev)
    ws, nb, _keep = _scratch(workspace, dev, stream, rra_gated_ffn_workspace_bytes, n, T, D, F, 1)
    st = load().rra_gated_ffn_backward(_one("x", x, dt, (T, D), dev), gs, us, das, _one("dx", dx, dt, (T, D), dev),
                                       dgs, dus, n, T, D, F, act, _dtype_of(x), ws, nb, _on(stream, dev))
    return _ret(st, "rra_gated_ffn_backward", check)


def _sizes(xs):
    return _SIZES[len(xs)](*xs)


def rra_vocab_loss_workspace_bytes(tokens: int, hidden: int, vocab, backward) -> int:
    """vocab: the ranks' shard heights; backward 2: the least bytes the
    backward pass runs with."""
    _ret(_same_count(len(vocab)), "rra_vocab_loss_workspace_bytes", True)
    return int(load().rra_vocab_loss_workspace_bytes(len(vocab), tokens, hidden, _sizes(vocab), int(backward)))


def rra_vocab_loss(x, weights, targets, loss, lse, ignore_index=-100, workspace=None, stream=None, check=True) -> int:
    """loss[t] = lse[t] - logit of targets[t], logits x W^T never kept; the
    vocabulary is the ranks' weight shards, one after another."""
    n = len(weights)
    st = _same_count(n)
    if st != RRA_SUCCESS:
        return _ret(st, "rra_vocab_loss", check)
    torch = _t()
    T, D = x.shape
    dev, dt = x.get_device(), x.dtype
    vocab = [w.shape[0] for w in weights]
    wp = _PTRS[n](*[_one("a vocabulary shard", w, dt, (v, D), dev) for w, v in zip(weights, vocab)])
    ws, nb, _keep = _scratch(workspace, dev, stream, rra_vocab_loss_workspace_bytes, T, D, vocab, 0)
    st = load().rra_vocab_loss(_one("x", x, dt, (T, D), dev), wp, _sizes(vocab),
                               _one("targets", targets, torch.int64, (T,), dev), n, T, D, ignore_index,
                               _one("loss", loss, torch.float32, (T,), dev), _one("lse", lse, torch.float32, (T,), dev),
                               _dtype_of(x), ws, nb, _on(stream, dev))
    return _ret(st, "rra_vocab_loss", check)


def rra_vocab_loss_backward(x, weights, targets, lse, grad_loss, dx, dweights, ignore_index=-100, workspace=None,
                            stream=None, check=True) -> int:
    """Gradients of rra_vocab_loss with respect to x and every shard."""
    n = len(weights)
    st = _same_count(n, dweights)
    if st != RRA_SUCCESS:
        return _ret(st, "rra_vocab_loss_backward", check)
    torch = _t()
    T, D = x.shape
    dev, dt = x.get_device(), x.dtype
    vocab = [w.shape[0] for w in weights]
    wp = _PTRS[n](*[_one("a vocabulary shard", w, dt, (v, D), dev) for w, v in zip(weights, vocab)])
    dp = _PTRS[n](*[_one("a shard's gradient", g, dt, (v, D), dev) for g, v in zip(dweights, vocab)])
    ws, nb, _keep = _scratch(workspace, dev, stream, rra_vocab_loss_workspace_bytes, T, D, vocab, 1)
    st = load().rra_vocab_loss_backward(
        _one("x", x, dt, (T, D), dev), wp, _sizes(vocab), _one("targets", targets, torch.int64, (T,), dev),
        _one("lse", lse, torch.float32, (T,), dev), _one("grad_loss", grad_loss, torch.float32, (T,), dev),
        _one("dx", dx, dt, (T, D), dev), dp, n, T, D, ignore_index, _dtype_of(x), ws, nb, _on(stream, dev))
    return _ret(st, "rra_vocab_loss_backward", check)


def rra_ll_wire_bytes(payload_bytes: int) -> int:
    return int(load().rra_ll_wire_bytes(payload_bytes))


def rra_ll128_wire_bytes(payload_bytes: int) -> int:
    return int(load().rra_ll128_wire_bytes(payload_bytes))


def _nbytes(t):
    return int(t.numel() * t.element_size())


def rra_ll_pack(payload, wire, flag: int, payload_bytes=None, stream=None, check=True) -> int:
    B = _nbytes(payload) if payload_bytes is None else payload_bytes
    st = load().rra_ll_pack(_ptr(payload), B, _ptr(wire), flag, _stream(stream, payload))
    return _ret(st, "rra_ll_pack", check)


def rra_ll128_pack(payload, wire, flag: int, payload_bytes=None, stream=None, check=True) -> int:
    B = _nbytes(payload) if payload_bytes is None else payload_bytes
    st = load().rra_ll128_pack(_ptr(payload), B, _ptr(wire), flag, _stream(stream, payload))
    return _ret(st, "rra_ll128_pack", check)


def rra_ll_unpack(wires, out, expected_flag: int, dtype=None, payload_bytes=None, op=RRA_SUM,
                  stream=None, check=True, nsrc=None) -> int:
    dtype = _dtype_of(out) if dtype is None else dtype
    B = _nbytes(out) if payload_bytes is None else payload_bytes
    n = len(wires) if nsrc is None else nsrc
    st = load().rra_ll_unpack(_ptr_array(wires), n, _ptr(out), B, dtype, op, expected_flag,
                              _stream(stream, out))
    return _ret(st, "rra_ll_unpack", check)


def rra_ll128_unpack(wires, out, expected_flag: int, dtype=None, payload_bytes=None, op=RRA_SUM,
                     stream=None, check=True, nsrc=None) -> int:
    dtype = _dtype_of(out) if dtype is None else dtype
    B = _nbytes(out) if payload_bytes is None else payload_bytes
    n = len(wires) if nsrc is None else nsrc
    st = load().rra_ll128_unpack(_ptr_array(wires), n, _ptr(out), B, dtype, op, expected_flag,
                                 _stream(stream, out))
    return _ret(st, "rra_ll128_unpack", check)


def rra_query_status(stream=None):
    """Synchronize the stream and read/clear the device status.
    Returns (status, [code, rank, peer, index])."""
    info = (ctypes.c_int32 * 4)()
    st = load().rra_query_status(_stream(stream), info)
    return st, list(info)


def rra_query_status_static(stream=None):
    """Synchronize the stream and read/clear the status of
    rra_allreduce_two_shot_static (allocates nothing).
    Returns (status, [code, rank, peer, index])."""
    info = (ctypes.c_int32 * 4)()
    st = load().rra_query_status_static(_stream(stream), info)
    return st, list(info)


def rra_select_algo(nranks: int, bytes_per_rank: int, dtype: int) -> int:
    return int(load().rra_select_algo(nranks, bytes_per_rank, dtype))


def rra_load_tuning(path, check=True) -> int:
    p = None if path is None else os.fsencode(path)
    return _ret(load().rra_load_tuning(p), "rra_load_tuning", check)


def rra_set_timeout_ns(ns: int) -> None:
    load().rra_set_timeout_ns(ns)


def rra_debug_skip_rank(rank: int) -> None:
    load().rra_debug_skip_rank(rank)


def rra_set_max_ctas(max_ctas: int) -> None:
    load().rra_set_max_ctas(max_ctas)


def rra_dump_recent() -> str:
    buf = ctypes.create_string_buffer(64 * 256)
    load().rra_dump_recent(buf, len(buf))
    return buf.value.decode()
