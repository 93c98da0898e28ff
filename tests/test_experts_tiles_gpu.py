"""GPU tests of the experts' operators and the balance loss in the forms that
large calls take: the largest tiles of both products, tiles of several passes
and workgroups of several rows.  Every test asks the plan first whether its
sizes really take that form.  Tolerances as in test_experts_gpu.py."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from experts_reference import E4M3, Problem
from test_experts_gpu import FMTS, U, check_gemm, within

pytestmark = pytest.mark.gpu

# rows round the height of a tile of 256, below it and several of it
ROWS_256 = [0, 1, 255, 256, 257, 511, 520, 64, 3, 0, 130, 16, 17, 31, 200, 300]


def assert_tile(p, out, product=None, wgrad=None):
    plan = M.ep_expert_plan_query(p.rows, p.N, p.K, p.fmt, out)
    if product:
        assert (plan["product_rows"], plan["product_cols"]) == product, plan
    if wgrad:
        assert (plan["wgrad_cols"], plan["wgrad_channels"]) == wgrad, plan


@pytest.mark.parametrize("K", [128, 256, 640, 1152, 2176])
@pytest.mark.parametrize("padded", [None, (540, 530, 7)])
@pytest.mark.parametrize("fmt", FMTS)
def test_product_256_rows(fmt, padded, K):
    """The tile of 256 x 256: K of one scale block, of as many as its stages,
    and past one and two chunks of 8; columns cut in the last tile."""
    p = Problem(ROWS_256, 1000, K, fmt, seed=K, padded=padded, expected=1000)
    assert_tile(p, M.BF16, product=(256, 256))
    check_gemm(p, M.BF16, f"K {K} padded {padded}")


TILES = [(8, (32, 128)), (24, (64, 256)), (60, (96, 256)), (100, (128, 256)), (130, (160, 256)), (200, (256, 256))]


@pytest.mark.parametrize("out", [M.BF16, M.FP32])
@pytest.mark.parametrize("expected,tile", TILES)
def test_product_rows_do_not_depend_on_others(expected, tile, out):
    """A row's result is the same bits whatever the rows beside it hold, and
    wherever in a tile the row stands (of the same sizes and the same hint)."""
    E = 131
    counts = [(7 * e) % 5 for e in range(E - 3)] + [37, 300, 70]
    p = Problem(counts, 1160, 384, M.SCALE_FP32, seed=5, expected=expected)
    assert_tile(p, out, product=(min(tile[0], 128), tile[1]) if out == M.FP32 else tile)
    a = p.gemm(out)[:sum(counts)]
    at = p.spans[E - 2][0]
    # other values in every row but those of the last expert but one
    x, xs = p.x.clone(), p.xs.clone()
    x[:at], xs[:at] = x[:at].view(torch.uint8).flip(0).view(E4M3), xs[:at].flip(0) * 2
    # and its rows in another order, 5 of the expert before it gone, so that they stand elsewhere
    perm = torch.randperm(300, generator=torch.Generator().manual_seed(1)).cuda()
    x[at - 5:at + 295], xs[at - 5:at + 295] = p.x[at:at + 300][perm], p.xs[at:at + 300][perm]
    p.x, p.xs = x, xs
    p.bounds[E - 2:] -= 5
    b = p.gemm(out)
    assert torch.equal(b[at - 5:at + 295], a[at:at + 300][perm])
    assert p.status() == 0


# more than a round of tiles of 256 x 256, cut in both directions; rows round
# the 32 of a step and the four stages
WGRAD_ROWS = [(5 * e) % 7 for e in range(112)] + [0, 1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 161, 400]


@pytest.mark.parametrize("out,accumulate", [(M.BF16, False), (M.FP32, False), (M.FP32, True)])
@pytest.mark.parametrize("fmt", FMTS)
def test_wgrad_256_tile(fmt, out, accumulate):
    p = Problem(WGRAD_ROWS, 504, 640, fmt, seed=91)
    assert_tile(p, out, wgrad=(256, 256))
    before = torch.randn(p.E, 504, 640, device="cuda") if accumulate else None
    dw = p.wgrad(out, accumulate, before.clone() if accumulate else None)
    assert p.status() == 0
    want, s = p.wgrad64()
    if accumulate:
        want, s = want + before.double(), s + before.abs().double()
    rows = torch.tensor(WGRAD_ROWS, device="cuda").view(-1, 1, 1)
    tol = (rows + 4) * U * s
    if fmt == M.SCALE_FP32:
        tol = tol + 2.0 ** -8 * s          # scale times code, rounded to bf16
    if out == M.BF16:
        tol = tol + 2.0 ** -8 * want.abs()
    within(dw, want, tol)
    if accumulate:
        assert torch.equal(dw[0], before[0])  # an expert without rows
