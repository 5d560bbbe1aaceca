"""What the binding of the serving-step operators takes as codes and scales:
any type of one byte an element, and none of more, whatever its bytes."""
import pytest
import torch

import collective_all_reduce_rank_gb300 as rra


def parts():
    return torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.int64, torch.int16])
@pytest.mark.parametrize("which", [0, 1])
def test_wider_types_of_as_many_bytes_are_refused(which, dtype):
    m = list(parts())
    m[which] = m[which].view(-1).view(dtype)
    x = torch.zeros(4, 64)
    with pytest.raises(ValueError):
        rra.rra_mx4_quantize(x, *m)
    with pytest.raises(ValueError):
        rra.rra_mx4_restore(*m, x)
    with pytest.raises(ValueError):
        rra.rra_allreduce_rmsnorm_mx4([x], torch.ones(64), 64, *m)
    with pytest.raises(ValueError):
        rra.rra_mx4_product(m, [parts()], [torch.zeros(4, 4)], 64)
    with pytest.raises(ValueError):
        rra.rra_mx4_product_sum([parts()], [m], torch.zeros(4, 4), 64)
    with pytest.raises(ValueError):
        rra.rra_mx4_gated_ffn(parts(), [parts()], [m], [parts()], 64, 4)


@pytest.mark.parametrize("dtype", [torch.int8, torch.bool, torch.float8_e4m3fn])
def test_types_of_one_byte_are_taken(dtype):
    codes, scales = parts()
    # refused for what the call itself sees (a hidden size of 0), behind the checks of types
    with pytest.raises(rra.RraError):
        rra.rra_mx4_product((codes.view(dtype)[:, :0].contiguous(), scales[:0].view(dtype)),
                            [(codes.view(dtype)[:, :0].contiguous(), scales[:0])], [torch.zeros(4, 4)], 0)
