"""GPU tests of the weight gradient's fp32 results for rows with FP32 scales:
they are good to binary32, stored or accumulated, as those of UE8M0 scales
are.  Tolerance, with u = 2^-24 and S the sum of the products' magnitudes:
scale times code is rounded once to binary32 (u) and split exactly into three
bf16 terms, whose products with dy are exact; 3 rows sums and one more for
accumulate, each off by u of a partial sum of at most S (1 + 2^-6)."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from experts_reference import Problem, rows64
from test_experts_gpu import COUNTS, U, within

pytestmark = pytest.mark.gpu


def check(p, accumulate=False):
    before = torch.randn(p.E, p.N, p.K, device="cuda") if accumulate else None
    dw = p.wgrad(M.FP32, accumulate, before.clone() if accumulate else None)
    assert p.status() == 0
    want, s = p.wgrad64()
    if accumulate:
        want, s = want + before.double(), s + before.abs().double()
    rows = torch.tensor([c for _, c in p.spans], device="cuda").view(-1, 1, 1)
    within(dw, want, (3 * rows + 8) * U * s * (1 + 2.0 ** -6))
    for e, (_, c) in enumerate(p.spans):
        if c == 0:
            assert torch.equal(dw[e], before[e]) if accumulate else (dw[e] == 0).all()


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("counts", COUNTS)
def test_counts(counts, accumulate):
    check(Problem(COUNTS[counts], 136, 256, M.SCALE_FP32, seed=81), accumulate)


@pytest.mark.parametrize("N,K", [(8, 128), (120, 384), (256, 256), (264, 640), (1000, 128)])
def test_sizes(N, K):
    check(Problem([33, 0, 130, 7], N, K, M.SCALE_FP32, seed=N + K))


@pytest.mark.parametrize("padded", [(16, 16, 0), (24, 16, 8), (40, 33, 3), (8, 0, 0)])
def test_padded(padded):
    check(Problem([0, 3, 16, 33, 100, 1], 136, 256, M.SCALE_FP32, seed=82, padded=padded), True)


def test_many_tiles():
    """More tiles of 256 x 128 than the device takes at once, rows round the four stages."""
    rows = [(5 * e) % 7 for e in range(112)] + [0, 1, 31, 32, 33, 63, 64, 65, 95, 96, 97, 127, 128, 129, 161, 400]
    for accumulate in (False, True):
        plan = M.ep_expert_plan_query(M.moedisp_rows.contiguous(128, sum(rows)), 504, 640, M.SCALE_FP32, M.FP32)
        assert (plan["wgrad_cols"], plan["wgrad_channels"]) == (256, 128)
        check(Problem(rows, 504, 640, M.SCALE_FP32, seed=83), accumulate)


def test_micro_batches():
    """A gradient accumulated over eight calls keeps binary32's error of the
    sum over all their rows."""
    ps = [Problem([40, 0, 130], 136, 256, M.SCALE_FP32, seed=84 + i) for i in range(8)]
    dw = torch.zeros(3, 136, 256, device="cuda")
    want = s = 0
    for p in ps:
        p.wgrad(M.FP32, True, dw)
        d, m = p.wgrad64()
        want, s = want + d, s + m
    rows = torch.tensor([8 * 40, 0, 8 * 130], device="cuda").view(-1, 1, 1)
    within(dw, want, (3 * rows + 15) * U * s * (1 + 2.0 ** -6))


def test_extreme_scales():
    """Scales that take a row to the largest and smallest values of binary32,
    infinite ones and NaN: in the sums that hold them and nowhere else."""
    p = Problem([9, 40], 136, 256, M.SCALE_FP32, seed=95)
    p.dy[:49] = 2.0 ** -10
    p.x[9:49, :128] = 448.0
    p.xs[9:49, 0] = 2.0 ** -60
    p.xs[9, 0] = 3.4e38 / 448             # 3.4e38: above bf16's largest value, below binary32's
    dw = p.wgrad(M.FP32)
    want, s = p.wgrad64()
    within(dw, want, (3 * 40 + 8) * U * s * (1 + 2.0 ** -6))
    p.xs[:9, 1] = 2.0 ** -100             # terms down to 2^-133
    dw = p.wgrad(M.FP32)
    want, s = p.wgrad64()
    within(dw[0, :, 128:], want[0, :, 128:], (3 * 9 + 8) * U * s[0, :, 128:] * (1 + 2.0 ** -6) + 9 * 2.0 ** -133)
    p = Problem([9, 40], 136, 256, M.SCALE_FP32, seed=96)
    p.x[3, 130] = 0.0
    p.xs[3, 1], p.xs[20, 0], p.xs[30, 1] = float("inf"), float("nan"), -float("inf")
    dw = p.wgrad(M.FP32)
    x = rows64(p.x[:49], p.xs[:49])
    for e, (lo, c) in enumerate(p.spans):
        want = (p.dy[lo:lo + c, :, None].double() * x[lo:lo + c, None, :]).sum(0)
        assert torch.equal(torch.isnan(dw[e]), torch.isnan(want))
        assert torch.equal(torch.isinf(dw[e]), torch.isinf(want)) and torch.equal(dw[e] > 0, want > 0)
