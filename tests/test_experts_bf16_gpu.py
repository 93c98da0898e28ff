"""GPU tests of the experts' bf16 products, their weight gradient and the bf16
activation against their definitions in 64 bits (tests/bf16_reference.py).

Tolerances, from the arithmetic (u = 2^-24, half a step of binary32): products
of two bf16 numbers are exact in binary32; a sum of m of them is off by at most
2 (m + 2) u times the sum of their magnitudes S, in any order and also where an
addition cuts off instead of rounding; a result in bf16 by 2^-8 of itself more."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from combine_ep_get_dispatch_amd import binding as B
from bf16_reference import Bf16Problem, hint_for
from experts_reference import swiglu64
from test_experts_gpu import COUNTS, within

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
LAYOUTS = [M.WEIGHTS_NK, M.WEIGHTS_KN]
OUTS = [M.BF16, M.FP32]


def check_gemm(p, layout, out, what=""):
    w = p.weights(layout)
    y = p.gemm(w, layout, out)
    assert p.status() == 0
    want, s = p.product64(lambda e: w[e].double() if layout == M.WEIGHTS_NK else w[e].double().t())
    tol = 2 * (p.K + 2) * U * s
    if out == M.BF16:
        tol = tol + 2.0 ** -8 * want.abs()
    within(y[p.live], want[p.live], tol[p.live], what)
    assert (y[~p.live] == 7.0).all(), f"{what}: rows of no expert were written"
    return y


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("counts", COUNTS)
def test_product_counts(counts, layout, out):
    check_gemm(Bf16Problem(COUNTS[counts], 264, 192, seed=len(counts)), layout, out, counts)


# channels that end inside a step, inside a half of it, at its end; columns that
# end inside a tile, a pair of products, at their ends
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("N,K", [(8, 8), (16, 16), (24, 40), (120, 72), (128, 64), (136, 128), (264, 648), (1000, 104),
                                 (512, 1152), (40, 2008)])
def test_product_sizes(N, K, layout, out):
    check_gemm(Bf16Problem([5, 0, 77, 1, 33], N, K, seed=N + K), layout, out, f"{N}x{K}")


# every tile (expected_rows only steers which), with steps before, at and past
# the stages and row counts that cut it
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("K", [56, 64, 128, 200, 1096])
@pytest.mark.parametrize("tile", [32, 64, 96, 128, 160, 256])
def test_product_every_tile(tile, K, layout, out):
    counts = [300, 0, 31, 513, 1, 256] * 3
    hint = hint_for(len(counts), 1288, K, "product_rows", tile)
    check_gemm(Bf16Problem(counts, 1288, K, seed=K, expected=hint), layout, out, f"{tile} {K}")


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("padded", [(16, 16, 0), (24, 16, 8), (40, 33, 3), (8, 0, 0)])
def test_product_padded(padded, layout, out):
    check_gemm(Bf16Problem([0, 16, 3, 40, 9, 1], 136, 328, padded=padded, seed=3, expected=4), layout, out)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_product_long_k(layout):
    check_gemm(Bf16Problem([3, 18], 72, 65536, seed=5), layout, M.FP32)


@pytest.mark.parametrize("layout", LAYOUTS)
def test_product_far_weights(layout):
    """An expert whose weights lie more than 2^32 bytes into the tensor."""
    N, K, E = 8192, 8192, 34
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device="cuda")
    p = Bf16Problem([2] * E, N, K, seed=6)
    g = torch.Generator(device="cuda").manual_seed(6)
    for e in (0, 31, 32, 33):
        w[e].normal_(generator=g)
    y = p.gemm(w, layout, M.BF16)
    assert p.status() == 0
    for e in (0, 16, 31, 32, 33):
        lo = 2 * e
        x, we = p.x[lo:lo + 2].double(), w[e].double() if layout == M.WEIGHTS_NK else w[e].double().t()
        want, s = x @ we.t(), x.abs() @ we.abs().t()
        within(y[lo:lo + 2], want, 2 * (K + 2) * U * s + 2.0 ** -8 * want.abs(), str(e))


@pytest.mark.parametrize("layout", LAYOUTS)
def test_product_special_values(layout):
    """Infinities and NaN reach the sums that hold them and no others, also in
    the last channels and next to channels and rows that are not there."""
    p = Bf16Problem([4, 3], 72, 72, seed=7)
    w = p.weights(layout)
    p.x[1, 71] = float("inf")
    p.x[2, 0] = float("nan")
    at = (1, 9, 70) if layout == M.WEIGHTS_NK else (1, 70, 9)
    w[at] = float("nan")
    for out in OUTS:
        y = p.gemm(w, layout, out)
        bad = torch.zeros(p.R, 72, dtype=torch.bool, device="cuda")
        bad[1] = bad[2] = True
        bad[4:7, 9] = True
        assert (~torch.isfinite(y[p.live]) == bad[p.live]).all()
        assert torch.isinf(y[1]).all() and torch.isnan(y[2]).all() and torch.isnan(y[4:7, 9]).all()
        assert (y[~p.live] == 7.0).all()


@pytest.mark.parametrize("layout", LAYOUTS)
def test_product_same_bits(layout):
    p = Bf16Problem([40, 0, 200, 3, 128], 520, 520, seed=8, expected=100)
    w = p.weights(layout)
    first = p.gemm(w, layout, M.FP32)
    for _ in range(5):
        assert torch.equal(first[p.live], p.gemm(w, layout, M.FP32)[p.live])


def test_bad_bounds():
    for bounds in ([0, 5, 3, 8, 9], [-1, 5, 6, 8, 9], [0, 5, 6, 8, 10 ** 9], [0, 2 ** 31 - 1, 2 ** 31 - 1, 8, 9]):
        p = Bf16Problem([5, 1, 2, 1], 136, 128)
        p.bounds = torch.tensor(bounds, dtype=torch.int32).cuda()
        for layout in LAYOUTS:
            assert (p.gemm(p.weights(layout), layout, M.BF16) == 7.0).all()
            assert p.status() == B.DEV_BAD_LAYOUT
        assert (p.wgrad(M.FP32) == 7.0).all()
        assert p.status() == B.DEV_BAD_LAYOUT
        h = torch.full((p.R, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        gu = torch.ones(p.R, 256, dtype=torch.bfloat16, device="cuda")
        M.ep_swiglu(p.rows, 128, gu, p.bounds, h, p.ws)
        assert (h == 7.0).all() and p.status() == B.DEV_BAD_LAYOUT
        assert p.status() == 0


# ---------------------------------------------------------------------------
# weight gradient
# ---------------------------------------------------------------------------

def check_wgrad(p, out, what=""):
    dw = p.wgrad(out)
    assert p.status() == 0
    want, s = p.wgrad64()
    rows = torch.tensor([c for _, c in p.spans], device="cuda").view(-1, 1, 1)
    tol = 2 * (rows + 2) * U * s
    if out == M.BF16:
        tol = tol + 2.0 ** -8 * want.abs()
    within(dw, want, tol, what)
    return dw


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("counts", COUNTS)
def test_wgrad_counts(counts, out):
    check_wgrad(Bf16Problem(COUNTS[counts], 264, 192, seed=len(counts)), out, counts)


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("N,K", [(8, 8), (24, 40), (120, 384), (256, 256), (264, 648), (1000, 128), (128, 1000)])
def test_wgrad_sizes(N, K, out):
    check_wgrad(Bf16Problem([5, 0, 77, 1, 33], N, K, seed=N + K), out, f"{N}x{K}")


# tiles of 256 x 256 (512 of them), rows before, at and past the stages
@pytest.mark.parametrize("out", OUTS)
def test_wgrad_large_tile(out):
    p = Bf16Problem([31, 32, 33, 64, 96, 128, 129, 300], 2048, 2048, seed=9)
    check_wgrad(p, out)
    check_wgrad(Bf16Problem([160, 0, 127, 1, 65, 95, 97, 128], 2040, 1992, seed=10), out)


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("padded", [(16, 16, 0), (24, 16, 8), (40, 33, 3), (8, 0, 0)])
def test_wgrad_padded(padded, out):
    check_wgrad(Bf16Problem([0, 16, 3, 40, 9, 1], 136, 328, padded=padded, seed=3), out)


@pytest.mark.parametrize("N,K", [(264, 200), (2048, 2048)])
def test_wgrad_accumulates(N, K):
    p = Bf16Problem([40, 0, 7, 65, 33, 1, 0, 12], N, K, seed=11)
    before = torch.randn(p.E, N, K, device="cuda")
    dw = p.wgrad(M.FP32, True, before.clone())
    want, s = p.wgrad64()
    want = want + before.double()
    within(dw, want, 2 * 70 * U * s + U * want.abs(), "sum")
    assert torch.equal(dw[1], before[1]) and p.status() == 0


def test_wgrad_special_values():
    """A value that is not finite stays in its column or channel; the rows
    around an expert's are not its own."""
    p = Bf16Problem([4, 33, 3], 72, 72, seed=12)
    p.dy[5, 9] = float("nan")
    p.x[36, 70] = float("inf")
    dw = p.wgrad(M.FP32)
    bad = torch.zeros_like(dw, dtype=torch.bool)
    bad[1, 9], bad[1, :, 70] = True, True
    assert (~torch.isfinite(dw) == bad).all()


def test_gradients_by_differences():
    """Both gradients of f = sum(y * c) against differences of the forward
    call, at steps that bf16 holds exactly."""
    p = Bf16Problem([3, 0, 6], 24, 40, seed=13, spare=0)
    w = p.weights(M.WEIGHTS_NK)
    c = p.dy
    f = lambda: (p.gemm(w, M.WEIGHTS_NK, M.FP32).double() * c.double()).sum()  # noqa: E731
    back = M.moedisp_rows.contiguous(p.E, p.R)
    dx = torch.empty(p.R, p.K, device="cuda")
    M.ep_expert_gemm_bf16(back, p.K, p.N, M.WEIGHTS_KN, c, w, p.bounds, dx, M.FP32, p.ws)
    dw = p.wgrad(M.FP32)
    # f is linear in each value: a difference is exact but for the sums' roundings
    scale = float((p.x.double().abs() @ w[0].double().abs().t()).max() * c.double().abs().sum())
    for r, k in ((0, 0), (2, 39), (8, 17)):
        keep = p.x[r, k].clone()
        p.x[r, k] = 4.0
        hi = f()
        p.x[r, k] = -4.0
        lo = f()
        p.x[r, k] = keep
        assert abs(float((hi - lo) / 8 - dx[r, k])) < 100 * U * scale
    for e, n, k in ((0, 0, 0), (2, 23, 39), (1, 3, 4)):
        keep = w[e, n, k].clone()
        w[e, n, k] = 4.0
        hi = f()
        w[e, n, k] = -4.0
        lo = f()
        w[e, n, k] = keep
        assert abs(float((hi - lo) / 8 - dw[e, n, k])) < 100 * U * scale
    assert p.status() == 0


# ---------------------------------------------------------------------------
# activation
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("counts,inner", [("one", 128), ("few", 256), ("cut", 1024), ("many", 2048), ("none", 128),
                                          ("first_empty", 2176), ("last_empty", 4096)])
def test_swiglu(counts, inner):
    p = Bf16Problem(COUNTS[counts], 8, 8, seed=inner)
    gu = p.rows_of(2 * inner) * 4
    h = torch.full((p.R, inner), 7.0, dtype=torch.bfloat16, device="cuda")
    M.ep_swiglu(p.rows, inner, gu, p.bounds, h, p.ws)
    assert p.status() == 0
    want = swiglu64(gu)
    # the sigmoid and two products in binary32, 4 steps at most; zero for g < -87, where |h| < 2^-110
    within(h[p.live], want[p.live], (2.0 ** -8 + 8 * U) * want[p.live].abs() + 2.0 ** -110)
    assert (h[~p.live] == 7.0).all()


@pytest.mark.parametrize("padded", [(16, 16, 0), (24, 16, 8), (8, 0, 0)])
def test_swiglu_padded(padded):
    p = Bf16Problem([0, 16, 3, 40, 9, 1], 8, 8, padded=padded, seed=14)
    gu = p.rows_of(512)
    h = torch.full((p.R, 256), 7.0, dtype=torch.bfloat16, device="cuda")
    M.ep_swiglu(p.rows, 256, gu, p.bounds, h, p.ws)
    want = swiglu64(gu)
    within(h[p.live], want[p.live], (2.0 ** -8 + 8 * U) * want[p.live].abs())
    assert (h[~p.live] == 7.0).all() and p.status() == 0


def test_swiglu_past_the_caches():
    """Rows and results of more than 256 MiB."""
    R, inner = 11011, 4096
    assert R * inner * 6 > 256 << 20
    g = torch.Generator(device="cuda").manual_seed(15)
    gu = torch.randn(R, 2 * inner, generator=g, device="cuda").to(torch.bfloat16)
    h = torch.full((R, inner), 7.0, dtype=torch.bfloat16, device="cuda")
    bounds = torch.tensor([0, 4000, 4000, R - 3], dtype=torch.int32).cuda()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    M.ep_swiglu(M.moedisp_rows.contiguous(3, R), inner, gu, bounds, h, ws)
    assert M.ep_check_status(ws) == 0 and (h[R - 3:] == 7.0).all()
    for lo in range(0, R - 3, 2000):
        want = swiglu64(gu[lo:min(lo + 2000, R - 3)])
        within(h[lo:lo + want.shape[0]], want, (2.0 ** -8 + 8 * U) * want.abs() + 2.0 ** -110)


def test_swiglu_extremes():
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([inf, -inf, nan, 1.0, 200.0, -200.0, 0.0, -0.0])
    u = torch.tensor([2.0, 2.0, 2.0, inf, 3.0, 3.0, inf, 5.0])
    gu = torch.ones(1, 256)
    gu[0, :8], gu[0, 128:136] = g, u
    gu = gu.to(torch.bfloat16).cuda()
    h = torch.empty(1, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    M.ep_swiglu(M.moedisp_rows.contiguous(1, 1), 128, gu, torch.tensor([0, 1], dtype=torch.int32).cuda(), h, ws)
    h = h[0, :8].float().cpu()
    assert h[0] == inf and torch.isnan(h[1]) and torch.isnan(h[2]) and h[3] == inf
    assert h[4] == 600.0 and h[5] == 0 and torch.isnan(h[6]) and h[7] == 0
