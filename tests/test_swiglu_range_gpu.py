"""GPU tests of the bf16 activation where the sigmoid leaves binary32's normal
range and the result does not."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from experts_reference import swiglu64
from test_experts_gpu import U, within

pytestmark = pytest.mark.gpu


def activation(gu):
    R, inner = gu.shape[0], gu.shape[1] // 2
    h = torch.full((R, inner), 7.0, dtype=torch.bfloat16, device="cuda")
    bounds, ws = torch.tensor([0, R], dtype=torch.int32).cuda(), torch.zeros(256, dtype=torch.uint8, device="cuda")
    M.ep_swiglu(M.moedisp_rows.contiguous(1, R), inner, gu, bounds, h, ws)
    assert M.ep_check_status(ws) == 0
    return h


# the second size is that of rows that go past the caches
@pytest.mark.parametrize("rows,inner", [(40, 256), (11011, 4096)])
def test_far_below_zero(rows, inner):
    """Every bf16 g of -300 .. -80 and some beyond, with factors u of the whole
    range, a few of them among ordinary values and many together."""
    bits = torch.arange(0xC2A0, 0xC397, dtype=torch.int32)                   # -80 .. -302
    g = torch.cat([(bits - 0x10000).to(torch.int16).view(torch.bfloat16),
                   torch.tensor([-999, -1001, -1e4, -3e38, 0.5, -1.0, 3.0]).to(torch.bfloat16)])
    u = torch.tensor([1.0, -3.0, 3.3e38, -3.3e38, 1e30, 2.0 ** -100, -(2.0 ** -133), 0.0]).to(torch.bfloat16)
    pairs = torch.cartesian_prod(torch.arange(len(g)), torch.arange(len(u)))
    order = torch.randperm(len(pairs), generator=torch.Generator().manual_seed(1))
    pairs = pairs[order][torch.arange(rows * inner) % len(pairs)].view(rows, inner, 2)
    gu = torch.cat([g[pairs[..., 0]], u[pairs[..., 1]]], 1)
    gu[::3, :inner:2] = 1.25                                                  # lanes with few of them
    gu = gu.cuda()
    h = activation(gu)
    for lo in range(0, rows, 2000):
        want, got = swiglu64(gu[lo:lo + 2000]), h[lo:lo + 2000]
        past = want.abs() > torch.finfo(torch.bfloat16).max                   # 3 * 3.3e38 and its like
        assert torch.equal(got[past].double(), want[past].sign() * torch.inf)
        want, got = want[~past], got[~past]
        # the power of two to about two steps of binary32, three products; half a step of subnormal bf16 numbers
        within(got, want, (2.0 ** -8 + 8 * U) * want.abs() + 2.0 ** -134)
    assert float(h[gu[:, :inner] < -87].abs().max()) > 1.0


def test_infinite_factor_far_below_zero():
    gu = torch.ones(1, 256)
    gu[0, :4] = torch.tensor([-100.0, -1e30, -100.0, -float("inf")])
    gu[0, 128:132] = torch.tensor([float("inf"), -float("inf"), float("nan"), 1.0])
    h = activation(gu.to(torch.bfloat16).cuda())[0].float()
    assert h[0] == -float("inf") and h[1] == float("inf") and torch.isnan(h[2]) and torch.isnan(h[3])
