"""MX4 matrices with rows so long that the bytes of their scales pass 2^32."""
import pytest
import torch

import collective_all_reduce_rank_gb300 as rra
import serve_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,more", [(torch.bfloat16, 128), (torch.float32, 131)])
def test_a_row_past_two_to_the_thirty(dtype, more):
    cols = (1 << 30) + more
    nb, n = ref.blocks(cols), 4096
    g = torch.Generator(device="cuda").manual_seed(30)
    x = torch.zeros(1, cols, dtype=dtype, device="cuda")
    ends = torch.randn(2, n, generator=g, device="cuda").to(dtype)
    x[0, :n] = ends[0]
    x[0, cols - n:] = 16.0 * ends[1]
    codes = torch.empty(1, 16 * nb, dtype=torch.uint8, device="cuda")
    scales = torch.full((ref.scale_bytes(1, cols),), 0xA5, dtype=torch.uint8, device="cuda")
    rra.rra_mx4_quantize(x, codes, scales)
    first, last = n // 32, cols // 32 * 32 - n  # a block's first column, past which lie `tail` more
    tail = x[:, last:].clone()
    want, byte = ref.quantize(x[:, :n])
    assert torch.equal(codes[:, : 16 * first], want)
    block = torch.arange(nb, device="cuda")
    at = block // 4 * 512 + block % 4
    assert torch.equal(scales[at[:first]], byte[0])
    assert not scales[at[first + 1: last // 32]].any()  # zeros between
    want, byte = ref.quantize(tail)
    assert torch.equal(codes[:, last // 2:], want)
    assert torch.equal(scales[at[last // 32:]], byte[0])
    head = ref.values(codes[:, : 16 * first], scales[at[None, :first]], n)
    end = ref.values(codes[:, last // 2:], scales[at[None, last // 32:]], cols - last)
    x.fill_(1.0)
    rra.rra_mx4_restore(codes, scales, x)
    assert torch.equal(x[:, :n].double(), head) and torch.equal(x[:, last:].double(), end)
    assert not x[:, n: last].any()
