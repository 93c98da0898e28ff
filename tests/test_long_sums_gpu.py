"""GPU tests of the bf16 and 4-bit products over long contractions.

A bound of a sum of m terms grows with m and with the sum of their magnitudes,
the sum itself with the root of m: past some thousands of terms such a bound
lets results pass that lack many of them.  So the sums here are of small
integers and powers of two, exact in binary32 in any order, and have to be
equal.  For integers of 4 bits with arbitrary scales the bound is that of the
kernel's own sums, which are 128 channels long."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from bf16_reference import Bf16Problem, hint_for, scales4, unpack4, weights4
from test_experts_gpu import within

U = 2.0 ** -24
LAYOUTS = [M.WEIGHTS_NK, M.WEIGHTS_KN]
FMTS = [M.W4_E2M1, M.W4_INT4]
OUTS = [M.BF16, M.FP32]


def integers(p, t):
    """The rows of `t` that belong to experts become integers of -2 .. 2."""
    v = torch.randint(-2, 3, t.shape, generator=p.g).to(torch.bfloat16).cuda()
    t[p.live] = v[p.live]


def equal(p, y, want, out):
    assert p.status() == 0
    want = want.to(torch.float32)                         # exact
    assert torch.equal(y[p.live], want[p.live].to(torch.bfloat16) if out == M.BF16 else want[p.live])
    assert (y[~p.live] == 7.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("K", [65536, 65528, 30008, 4104])
def test_bf16_product(K, layout, out):
    p = Bf16Problem([3, 0, 18, 40], 72, K, seed=K)
    integers(p, p.x)
    w = torch.randint(-2, 3, (p.E, p.N, K) if layout == M.WEIGHTS_NK else (p.E, K, p.N), generator=p.g)
    w = w.to(torch.bfloat16).cuda()
    want, s = p.product64(lambda e: w[e].double() if layout == M.WEIGHTS_NK else w[e].double().t())
    assert float(s.max()) < 2 ** 24
    equal(p, p.gemm(w, layout, out), want, out)


@pytest.mark.gpu
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("tile", [32, 64, 96, 128, 160, 256])
def test_bf16_product_in_every_tile(tile, layout):
    counts, K = [300, 0, 31, 1, 256], 8200
    p = Bf16Problem(counts, 1288, K, seed=tile, expected=hint_for(len(counts), 1288, K, "product_rows", tile))
    integers(p, p.x)
    w = torch.randint(-2, 3, (p.E, p.N, K) if layout == M.WEIGHTS_NK else (p.E, K, p.N), generator=p.g)
    w = w.to(torch.bfloat16).cuda()
    want, _ = p.product64(lambda e: w[e].double() if layout == M.WEIGHTS_NK else w[e].double().t())
    equal(p, p.gemm(w, layout, M.FP32), want, M.FP32)


def four_bits(p, fmt):
    """Random codes and scales that are powers of two."""
    w, sc = p.quantised(fmt)
    steps = torch.randint(-1, 2, sc.shape, generator=p.g)
    return w, torch.exp2(steps.float()).to(torch.bfloat16).cuda() if fmt == M.W4_INT4 else (127 + steps).to(torch.uint8).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [65536, 65408, 30080, 4224])
def test_w4_product(K, fmt, out):
    p = Bf16Problem([3, 0, 18, 40], 80, K, seed=K)
    integers(p, p.x)
    w, sc = four_bits(p, fmt)
    want, s = p.product64(lambda e: weights4(w[e], sc[e], fmt))
    # integers: with the detour by 23 instead of |c| <= 8; units of 1/2 or 1/4
    assert float(s.max()) * (4 if fmt == M.W4_E2M1 else 2 * 23 / 8) < 2 ** 24
    equal(p, p.gemm4(w, sc, fmt, out), want, out)


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("tile", [16, 32, 64, 96, 160])
def test_w4_product_in_every_tile(tile, fmt):
    counts, K, N = [300, 0, 31, 513, 1, 256] * 3, 4224, 4112 if tile == 32 else 1296
    field = "int4_rows" if fmt == M.W4_INT4 else "e2m1_rows"
    p = Bf16Problem(counts, N, K, seed=tile, expected=hint_for(len(counts), N, K, field, tile))
    integers(p, p.x)
    w, sc = four_bits(p, fmt)
    want, _ = p.product64(lambda e: weights4(w[e], sc[e], fmt))
    equal(p, p.gemm4(w, sc, fmt, M.FP32), want, M.FP32)


@pytest.mark.gpu
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("N,K,E", [(72, 72, 3), (2048, 2048, 8)])
def test_weight_gradient_of_many_rows(N, K, E, out):
    """Both tiles, tens of thousands of rows of one expert."""
    p = Bf16Problem([5, 40001 if E == 3 else 20011] + [3] * (E - 2), N, K, seed=E)
    integers(p, p.x)
    integers(p, p.dy)
    want, _ = p.wgrad64()
    dw = p.wgrad(out)
    assert p.status() == 0
    want = want.to(torch.float32)
    assert torch.equal(dw, want.to(torch.bfloat16) if out == M.BF16 else want)


# ---------------------------------------------------------------------------
# integers of 4 bits, any scales
# ---------------------------------------------------------------------------
# A group's 128 channels are summed as codes q = 0 .. 15 times x on top of the
# sum of -8 x: 256 terms, exact each, off by at most 2 * 258 u of the sum of
# (q + 8) |x| in any order and also where an addition cuts off.  The K/128
# scaled sums are added by that many fused multiply-adds, each off by u of what
# has been added so far, at most the sum of |s c x| and the errors before.

def detour(w, sc):
    """float64 [N][K]: s (q + 8)."""
    return (unpack4(w, M.W4_INT4) + 16) * scales4(sc, M.W4_INT4)


def int4_tolerance(K, magnitude, s):
    return 1.01 * (516 * U * magnitude + (K // 128 + 1) * U * s)


@pytest.mark.gpu
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("counts,N,K,expected", [
    ([3, 18], 80, 65536, 0), ([5, 0, 77, 1, 33], 272, 1152, 0), ([5, 0, 77, 1, 33], 48, 384, 0),
    ([300, 0, 31, 513, 1, 256] * 3, 1296, 1152, 16), ([300, 0, 31, 513, 1, 256] * 3, 1296, 2304, 64),
    ([300, 0, 31, 513, 1, 256] * 3, 1296, 1152, 128), ([300, 0, 31, 513, 1, 256] * 3, 1296, 1152, 1000)])
def test_int4_within_its_own_bound(counts, N, K, expected, out):
    p = Bf16Problem(counts, N, K, seed=N + K, expected=expected)
    w, sc = p.quantised(M.W4_INT4)
    want, s = p.product64(lambda e: weights4(w[e], sc[e], M.W4_INT4))
    _, mag = p.product64(lambda e: detour(w[e], sc[e]))
    tol = int4_tolerance(K, mag, s)
    if out == M.BF16:
        tol = tol + 2.0 ** -8 * (want.abs() + tol)
    y = p.gemm4(w, sc, M.W4_INT4, out)
    assert p.status() == 0 and (y[~p.live] == 7.0).all()
    within(y[p.live], want[p.live], tol[p.live])


def test_the_bound_shows_what_is_missing():
    """At the largest K, results of zero and results without one group of the
    512 lie outside the bound (no GPU needed)."""
    g = torch.Generator().manual_seed(1)
    K, N = 65536, 80
    x = torch.randn(3, K, generator=g).to(torch.bfloat16).double()
    w = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    sc = torch.exp(torch.randn(K // 128, N, generator=g)).to(torch.bfloat16)
    real = weights4(w, sc, M.W4_INT4)
    want = x @ real.t()
    tol = int4_tolerance(K, x.abs() @ detour(w, sc).t(), x.abs() @ real.abs().t())
    assert float(((want.abs() - tol) > 0).double().mean()) > 0.9
    for group in (0, 255, 511):
        cut = x.clone()
        cut[:, 128 * group:128 * (group + 1)] = 0
        off = (cut @ real.t() - want).abs()
        assert float((off > tol).double().mean()) > 0.2, group


@pytest.mark.gpu
@pytest.mark.parametrize("expected", [1, 64, 1000])
def test_int4_weights_of_zero(expected):
    """-8 x and 8 x need not cancel to the last bit: within the bound, not zero;
    rows of zeros give zero."""
    p = Bf16Problem([64, 0, 300], 272, 1024, seed=9, expected=expected)
    w = torch.full((3, 272, 512), 0x88, dtype=torch.uint8, device="cuda")
    _, sc = p.quantised(M.W4_INT4)
    p.x[3] = 0
    y = p.gemm4(w, sc, M.W4_INT4, M.FP32)
    _, mag = p.product64(lambda e: detour(w[e], sc[e]))
    within(y[p.live], torch.zeros_like(mag[p.live]), int4_tolerance(1024, mag, 0.0)[p.live])
    assert p.status() == 0 and (y[3] == 0).all()
