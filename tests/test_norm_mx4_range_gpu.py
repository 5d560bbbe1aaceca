"""rra_allreduce_rmsnorm_mx4 where the mean square is near an end of float32's
range: values k 2^p of small integers k, whose squares and sums of squares are
exact, so that 1 / rms is the float32 nearest to its exact value."""
import pytest
import torch

import collective_all_reduce_rank_gb300 as rra
import serve_ref as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hidden,power", [(h, p) for h in (64, 4096, 32768) for p in (-72, -66, -60, -40, -20, 20, 40, 52)]
                         + [(64, 57)])
def test_mean_squares_near_the_ends(hidden, power, dtype):
    g = torch.Generator(device="cuda").manual_seed(hidden)
    k = torch.randint(-8, 9, (5, hidden), generator=g, device="cuda").double()
    x = torch.ldexp(k, torch.tensor(float(power), device="cuda")).to(DT[dtype])
    gamma = torch.randint(1, 9, (hidden,), generator=g, device="cuda").to(DT[dtype])
    rstd = (1.0 / torch.sqrt(x.double().square().mean(1))).float()
    want, byte = ref.quantize((x.float() * rstd[:, None]) * gamma.float())
    codes = torch.full((5, 16 * ref.blocks(hidden)), 0xA5, dtype=torch.uint8, device="cuda")
    scales = torch.full((ref.scale_bytes(5, hidden),), 0xA5, dtype=torch.uint8, device="cuda")
    rra.rra_allreduce_rmsnorm_mx4([x], gamma, hidden, codes, scales, eps=0.0)
    assert torch.equal(codes, want) and torch.equal(scales, ref.tile_scales(byte, 0xA5))
