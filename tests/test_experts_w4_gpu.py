"""GPU tests of the experts' products with 4-bit weights against their
definition in 64 bits (tests/bf16_reference.py).

Tolerances, from the arithmetic (u = 2^-24): E2M1 weights times their scales
are bf16 numbers, products are exact, and a sum of m is off by at most 2 (m +
2) u of the sum of magnitudes.  Integers: a group's sum of (q + 16) x and that of
24 x are such sums, of magnitudes up to 31 |x| and 24 |x|; their difference and
the scaled sum of the groups add four roundings.  A result in bf16 is off by
2^-8 of itself more."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from combine_ep_get_dispatch_amd import binding as B
from bf16_reference import Bf16Problem, hint_for, scales4, unpack4, weights4
from test_experts_gpu import COUNTS, within

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
FMTS = [M.W4_E2M1, M.W4_INT4]
OUTS = [M.BF16, M.FP32]


def tolerance(p, w, sc, fmt, want, s, out):
    if fmt == M.W4_INT4:
        _, s = p.product64(lambda e: 56.0 * scales4(sc[e], fmt))
    tol = 2 * (p.K + 8) * U * s
    return tol + 2.0 ** -8 * want.abs() if out == M.BF16 else tol


def check(p, fmt, out, what=""):
    w, sc = p.quantised(fmt)
    y = p.gemm4(w, sc, fmt, out)
    assert p.status() == 0
    want, s = p.product64(lambda e: weights4(w[e], sc[e], fmt))
    tol = tolerance(p, w, sc, fmt, want, s, out)
    within(y[p.live], want[p.live], tol[p.live], what)
    assert (y[~p.live] == 7.0).all(), f"{what}: rows of no expert were written"


def test_every_code():
    """Each code alone, at each place of a stage, times powers of two."""
    for fmt in FMTS:
        K, N = 384, 16
        p = Bf16Problem([16], N, K, spare=0)
        w = torch.zeros(1, N, K // 2, dtype=torch.uint8)
        if fmt == M.W4_INT4:
            w[:] = 0x88
        for n in range(N):
            for k in range(K):
                c = (n + k) % 16
                b = int(w[0, n, k // 2])
                w[0, n, k // 2] = (b & 0xF0) | c if k % 2 == 0 else (b & 0x0F) | c << 4
        w = w.cuda()
        if fmt == M.W4_INT4:
            sc = torch.full((1, K // 128, N), 0.5, dtype=torch.bfloat16, device="cuda")
        else:
            sc = torch.full((1, K // 32, N), 126, dtype=torch.uint8, device="cuda")
        want = unpack4(w[0], fmt) * 0.5
        for k0 in range(0, K, 16):
            p.x.zero_()
            for r in range(16):
                p.x[r, k0 + r] = 2.0
            y = p.gemm4(w, sc, fmt, M.FP32)
            assert torch.equal(y.double(), 2 * want[:, k0:k0 + 16].t()), (fmt, k0)


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("counts", COUNTS)
def test_counts(counts, fmt, out):
    check(Bf16Problem(COUNTS[counts], 272, 384, seed=len(counts)), fmt, out, counts)


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("N,K", [(16, 128), (32, 256), (48, 384), (112, 512), (128, 640), (144, 128), (272, 1152),
                                 (1008, 896)])
def test_sizes(N, K, fmt, out):
    check(Bf16Problem([5, 0, 77, 1, 33], N, K, seed=N + K), fmt, out, f"{N}x{K}")


# every tile (expected_rows only steers which)
@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("K", [128, 256, 640, 1152])
@pytest.mark.parametrize("tile", [16, 32, 64, 96, 160])
def test_every_tile(tile, K, fmt, out):
    counts = [300, 0, 31, 513, 1, 256] * 3
    N = 4112 if tile == 32 else 1296
    hint = hint_for(len(counts), N, K, "int4_rows" if fmt == M.W4_INT4 else "e2m1_rows", tile)
    check(Bf16Problem(counts, N, K, seed=K, expected=hint), fmt, out, f"{tile} {K}")


@pytest.mark.parametrize("out", OUTS)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("padded", [(16, 16, 0), (24, 16, 8), (40, 33, 3), (8, 0, 0)])
def test_padded(padded, fmt, out):
    check(Bf16Problem([0, 16, 3, 40, 9, 1], 144, 384, padded=padded, seed=3, expected=4), fmt, out)


@pytest.mark.parametrize("fmt", FMTS)
def test_long_k(fmt):
    check(Bf16Problem([3, 18], 80, 65536, seed=5), fmt, M.FP32)


@pytest.mark.parametrize("fmt", FMTS)
def test_far_weights(fmt):
    """An expert whose weights lie more than 2^32 bytes into the tensor, for one token."""
    N, K, E = 16384, 16384, 36
    w = torch.full((E, N, K // 2), 0x88, dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(6)
    for e in (0, 33, 35):
        w[e] = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8, device="cuda")
    counts = [0] * E
    for e in (0, 33, 35):
        counts[e] = 1
    p = Bf16Problem(counts, N, K, seed=6)
    shape = (E, K // 128, N) if fmt == M.W4_INT4 else (E, K // 32, N)
    sc = torch.ones(shape, dtype=torch.bfloat16, device="cuda") if fmt == M.W4_INT4 else \
        torch.full(shape, 127, dtype=torch.uint8, device="cuda")
    y = p.gemm4(w, sc, fmt, M.FP32)
    assert p.status() == 0
    for r, e in enumerate((0, 33, 35)):
        v, x = unpack4(w[e], fmt), p.x[r].double()
        want = v @ x
        s = (56.0 * torch.ones_like(v) if fmt == M.W4_INT4 else v.abs()) @ x.abs()
        within(y[r], want, 2 * (K + 8) * U * s, str(e))


def test_extreme_scales():
    """E2M1: scales from 2^-127 on, NaN, and weights past bf16's range."""
    K, N = 128, 256
    p = Bf16Problem([2], N, K, spare=0)
    p.x.zero_()
    p.x[0, 5], p.x[1, 100] = 1.0, 2.0 ** 60
    w = torch.full((1, N, K // 2), 0x22, dtype=torch.uint8, device="cuda")    # 1.0
    sc = torch.arange(256, dtype=torch.uint8).repeat(1, K // 32, 1).cuda()
    y = p.gemm4(w, sc, M.W4_E2M1, M.FP32).double()
    want = torch.exp2(torch.arange(255, dtype=torch.float64, device="cuda") - 127)
    assert torch.isnan(y[:, 255]).all()
    # normal bf16 weights are exact; below 2^-126 a weight may be taken as zero
    assert torch.equal(y[0, 1:255], want[1:]) and y[0, 0] in (0.0, float(want[0]))
    ok = want * 2.0 ** 60 < 2.0 ** 128
    assert torch.equal(y[1, 1:255][ok[1:]], (want * 2.0 ** 60)[1:][ok[1:]])
    w[:] = 0x77                                                                # 6.0
    y = p.gemm4(w, sc, M.W4_E2M1, M.FP32)
    # 6 * 2^126 is infinite, and so is its product with 1; those with the zeros of x are NaN, and so is the sum
    assert torch.isnan(y[0, 253:255]).all() and torch.isfinite(y[0, :253]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_special_values(fmt):
    """A row that is not finite is no other row's matter, in any place."""
    p = Bf16Problem([4, 3], 80, 384, seed=7)
    w, sc = p.quantised(fmt)
    good = p.gemm4(w, sc, fmt, M.FP32)
    p.x[1, 383] = float("inf")
    p.x[5, 0] = float("nan")
    y = p.gemm4(w, sc, fmt, M.FP32)
    assert torch.isnan(y[5]).all() and not torch.isfinite(y[1]).any()
    keep = p.live.clone()
    keep[1] = keep[5] = False
    assert torch.equal(y[keep], good[keep]) and (y[~p.live] == 7.0).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_same_bits_and_bad_bounds(fmt):
    p = Bf16Problem([40, 0, 200, 3, 128], 528, 640, seed=8, expected=4)
    w, sc = p.quantised(fmt)
    first = p.gemm4(w, sc, fmt, M.FP32)
    for _ in range(5):
        assert torch.equal(first[p.live], p.gemm4(w, sc, fmt, M.FP32)[p.live])
    p.bounds = torch.tensor([0, 40, 30, 100, 200, 300], dtype=torch.int32).cuda()
    assert (p.gemm4(w, sc, fmt, M.BF16) == 7.0).all()
    assert p.status() == B.DEV_BAD_LAYOUT and p.status() == 0
