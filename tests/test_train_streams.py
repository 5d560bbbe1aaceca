"""The stream of a training operator's call and the workspace the binding makes
for it.  PyTorch's allocator hands out memory in the order of one stream, so a
block has to come from the stream the kernels run on: one of another stream may
still be in use by work pending there.  The allocator is a fake that notes the
stream of each block, so no GPU is needed."""
import contextlib
from types import SimpleNamespace

import pytest

import collective_all_reduce_rank_gb300 as rra

MAIN, OTHER = 0x10, 0x20  # raw handles


class Fake:
    """torch as far as a workspace needs it: a current stream and an allocator."""

    uint8 = "uint8"

    def __init__(self, current=MAIN):
        self.current = current
        self.made = []
        self.cuda = SimpleNamespace(stream=self._use, current_device=lambda: 0)
        self._C = SimpleNamespace(_cuda_getCurrentRawStream=lambda device: self.current, _cuda_getDevice=lambda: 0)

    @contextlib.contextmanager
    def _use(self, stream):
        old, self.current = self.current, stream.cuda_stream
        yield
        self.current = old

    def empty(self, size, dtype=None, device=None):
        self.made.append(self.current)
        return SimpleNamespace(data_ptr=lambda: 1 << 20, numel=lambda: size, element_size=lambda: 1,
                               record_stream=lambda s: None, is_contiguous=lambda: True, get_device=lambda: device)


def scratch(monkeypatch, stream, current=MAIN, device=0):
    fake = Fake(current)
    monkeypatch.setattr(rra, "_t", lambda: fake)
    out = rra._scratch(None, device, stream, lambda *a: 1000)
    assert out[1] == 1000 and fake.current == current
    return fake.made


def test_the_workspace_comes_from_the_stream_of_the_call(monkeypatch):
    assert scratch(monkeypatch, None) == [MAIN]
    assert scratch(monkeypatch, None, current=OTHER) == [OTHER]
    assert scratch(monkeypatch, SimpleNamespace(cuda_stream=OTHER)) == [OTHER]
    assert scratch(monkeypatch, SimpleNamespace(cuda_stream=0), current=OTHER) == [0]


@pytest.mark.parametrize("handle", [0, OTHER, 0x30])
def test_a_raw_handle_needs_a_workspace_unless_it_is_the_current_stream(monkeypatch, handle):
    assert scratch(monkeypatch, handle, current=handle) == [handle]
    with pytest.raises(ValueError, match="raw stream handle"):
        scratch(monkeypatch, handle, current=MAIN)


def test_tensors_of_no_gpu_have_no_stream(monkeypatch):
    """The call itself refuses them, with its own error."""
    assert scratch(monkeypatch, 0, device=-1) == [MAIN]


@pytest.mark.gpu
@pytest.mark.parametrize("call", ["ffn", "loss"])
def test_a_call_on_another_stream_makes_its_workspace_there(call):
    """Work pending on the current stream in a block that is dropped before the call: both keep their bits."""
    import torch

    rra.rra_init(0)
    gen = torch.Generator(device="cuda").manual_seed(3)
    T, D, F, V = 192, 515, 260, 1500

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)

    x, G, U, da, W = rnd(T, D), [rnd(F, D)], [rnd(F, D)], [rnd(T, F)], [rnd(V, D)]
    tgt = torch.randint(0, V, (T,), generator=gen, device="cuda")
    lse, loss, grad = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.full((T,), 1.0, device="cuda")
    rra.rra_vocab_loss(x, W, tgt, loss, lse)
    if call == "ffn":
        nb = rra.rra_gated_ffn_workspace_bytes(1, T, D, F, 1)
        outs = [torch.empty_like(x), torch.empty_like(G[0]), torch.empty_like(U[0])]
        run = lambda o, **k: rra.rra_gated_ffn_backward(x, G, U, da, o[0], [o[1]], [o[2]], **k)
    else:
        nb = rra.rra_vocab_loss_workspace_bytes(T, D, [V], 1)
        outs = [torch.empty_like(x), torch.empty_like(W[0])]
        run = lambda o, **k: rra.rra_vocab_loss_backward(x, W, tgt, lse, grad, o[0], [o[1]], **k)
    want = [torch.empty_like(o) for o in outs]
    run(want, workspace=torch.empty(nb, dtype=torch.uint8, device="cuda"))
    side = torch.cuda.Stream()
    noise = torch.randint(0, 255, (nb,), generator=gen, device="cuda", dtype=torch.uint8)
    total = torch.empty((), dtype=torch.int64, device="cuda")
    expect = noise.sum(dtype=torch.int64)
    big = torch.randn(4096, 4096, generator=gen, device="cuda")
    torch.cuda.synchronize()
    for _ in range(8):
        pending = torch.empty(nb, dtype=torch.uint8, device="cuda")  # of the current stream
        for _ in range(4):
            big @ big
        pending.copy_(noise)
        total.copy_(pending.sum(dtype=torch.int64))
        del pending
        run(outs, stream=side)
        side.synchronize()
        torch.cuda.synchronize()
        assert int(total) == int(expect)
        for a, b in zip(outs, want):
            assert torch.equal(a, b)



@pytest.mark.parametrize("stream", [None, 0, SimpleNamespace(cuda_stream=OTHER, device_index=1)])
def test_tensors_of_a_device_that_is_not_current_are_refused(monkeypatch, stream):
    """The library launches on the current device."""
    monkeypatch.setattr(rra, "_several", True)
    monkeypatch.setattr(rra, "_t", lambda: Fake())  # device 0 is current
    with pytest.raises(ValueError, match="current device"):
        rra._on(stream, 1)


def test_a_stream_of_another_device_is_refused(monkeypatch):
    monkeypatch.setattr(rra, "_t", lambda: Fake())
    with pytest.raises(ValueError, match="stream"):
        rra._on(SimpleNamespace(cuda_stream=OTHER, device_index=1), 0)
    assert rra._on(SimpleNamespace(cuda_stream=OTHER, device_index=0), 0) == OTHER
    assert rra._on(SimpleNamespace(cuda_stream=OTHER), 0) == OTHER
    assert rra._on(None, 0) == MAIN and rra._on(OTHER, 0) == OTHER and rra._on(None, -1) == 0
