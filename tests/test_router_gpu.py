"""GPU tests of the router's choice and its gradient against their definitions
in 64 bits (tests/bf16_reference.py).

Choices have to be equal.  Weights: a score is good to about two steps of
binary32 (u = 2^-24), sums of up to 4096 exponentials to their number of steps
at worst, the quotient and the scale to one each: 64 u for the sums over lanes
of up to 64 and 64 in a row.  Gradients: the same relative to the largest
product that enters, and half a step of bf16 where they are bf16."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from combine_ep_get_dispatch_amd import binding as B
from bf16_reference import router64
from test_experts_gpu import within

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
SCORES = [M.SCORE_SOFTMAX, M.SCORE_SIGMOID]
DTYPES = [torch.float32, torch.bfloat16]


def shape_of(z, k, score, groups=1, topk_groups=1, group_best=2, normalise=True, scale=1.0):
    dt = M.FP32 if z.dtype == torch.float32 else M.BF16
    return M.moedisp_router.make(z.shape[0], z.shape[1], k, score, dt, groups, topk_groups, group_best, normalise, scale)


def choose(z, k, score, bias=None, live=None, **kw):
    T = z.shape[0]
    idx = torch.full((T + 1, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, k), -7.0, device="cuda")
    M.ep_router_topk(shape_of(z, k, score, **kw), z, bias, live, idx, w)
    assert (idx[T] == -7).all() and (w[T] == -7).all()
    return idx[:T], w[:T]


def backward(z, idx, g, k, score, **kw):
    T, E = z.shape
    d = torch.full((T + 1, E), -7.0, dtype=z.dtype, device="cuda")
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    M.ep_router_topk_backward(shape_of(z, k, score, **kw), z, idx.contiguous(), g, d, ws)
    assert (d[T] == -7).all()
    return d[:T], M.ep_check_status(ws)


def check(z, k, score, bias=None, live=None, **kw):
    idx, w = choose(z, k, score, bias, live, **kw)
    leaf = z.double().requires_grad_()
    want_idx, want = router64(leaf, k, score, bias, live, **kw)
    assert torch.equal(idx.long(), want_idx)
    scale = kw.get("scale", 1.0)
    within(w, want.detach(), 64 * U * want.detach().abs() + 2.0 ** -120)
    g = torch.randn(w.shape, device="cuda")
    d, status = backward(z, idx, g, k, score, **kw)
    assert status == 0
    (want * g.double()).sum().backward()
    dz = leaf.grad
    # entering products: shares times gradients, with the mean that is taken away
    share = (want.detach() / scale).abs()
    gs = abs(scale) * g.double().abs()
    mean = (share * gs).sum(1, keepdim=True)
    size = torch.zeros_like(dz)
    size.scatter_add_(1, want_idx.clamp(min=0), torch.where(want_idx >= 0, share * (gs + mean), 0.0))
    if score == M.SCORE_SOFTMAX and not kw.get("normalise", True):
        size += torch.nan_to_num(torch.softmax(z.double(), 1)) * mean
    tol = 128 * U * size + 2.0 ** -120
    if z.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * dz.abs()
    within(d, dz, tol)
    return idx, w


def logits(T, E, dt, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(T, E, generator=g)).to(dt).cuda()


# one lane's experts, lanes cut inside a piece, rows of each shape of the wave
SIZES = [(1, 1, 1), (5, 8, 2), (33, 16, 16), (17, 60, 6), (9, 64, 8), (100, 100, 5), (65, 128, 32), (31, 130, 7),
         (128, 256, 8), (4100, 256, 8), (4099, 250, 9), (7, 257, 3), (19, 512, 8), (6, 513, 32), (5, 1000, 32),
         (3, 1024, 1), (4, 1025, 8), (3, 4096, 32), (2, 4095, 31)]


@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("T,E,k", SIZES)
def test_choice(T, E, k, score, dt, normalise):
    check(logits(T, E, dt, T + E), k, score, normalise=normalise, scale=2.5)


@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("T,E,k", SIZES)
def test_choice_with_bias(T, E, k, score, normalise):
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda()
    check(logits(T, E, torch.float32, T + E), k, score, bias, normalise=normalise)


@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("T,E,k,G,tg", [(40, 256, 8, 8, 4), (4100, 256, 8, 8, 3), (40, 64, 4, 64, 5), (9, 60, 6, 6, 2),
                                        (50, 128, 8, 2, 1), (21, 1024, 8, 32, 4), (5, 4096, 16, 64, 64),
                                        (13, 320, 32, 5, 2), (3, 7, 2, 7, 7), (11, 39, 3, 3, 1)])
def test_groups(T, E, k, G, tg, score, best, biased):
    z = logits(T, E, torch.float32, T + E + G)
    bias = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda() if biased else None
    check(z, k, score, bias, groups=G, topk_groups=tg, group_best=best, normalise=True)


@pytest.mark.parametrize("E,k", [(16, 4), (64, 8), (256, 8), (300, 20)])
def test_ties_go_to_the_lowest_index(E, k):
    """Rows of few different values, of both signs and zeros, with bias and
    groups as well."""
    g = torch.Generator().manual_seed(E)
    z = torch.randint(-2, 3, (500, E), generator=g).float()
    z[0], z[1], z[2, ::2] = 0.0, -0.0, -0.0
    z = z.cuda()
    bias = torch.randint(-1, 2, (E,), generator=g).float().cuda()
    for score in SCORES:
        for b in (None, bias):
            check(z, k, score, b)
            check(z, k, score, b, groups=4, topk_groups=2)
    idx, _ = choose(z[:2], k, M.SCORE_SIGMOID)
    assert (idx == torch.arange(k, device="cuda")).all()


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("score", SCORES)
def test_rows_without_experts(score, dt):
    """Logits of -inf and NaN take no part; too few experts leave masked slots;
    padding tokens have none; nothing of that reaches other tokens."""
    z = logits(40, 20, dt, 3)
    z[3, :] = -torch.inf
    z[4, :] = float("nan")
    z[5, 2:] = -torch.inf
    z[6, ::2] = float("nan")
    z[7, 5] = float("nan")
    live = torch.ones(40, dtype=torch.uint8)
    live[8] = live[39] = 0
    live = live.cuda() if score == M.SCORE_SOFTMAX else live.bool().cuda()
    z[39] = float("nan")
    for bias in (None, torch.linspace(-1, 1, 20).cuda()):
        for kw in ({}, dict(groups=5, topk_groups=2), dict(normalise=False)):
            idx, w = choose(z, 6, score, bias, live, **kw)
            want_idx, want = router64(z, 6, score, bias, live, **kw)
            assert torch.equal(idx.long(), want_idx)
            within(w, want, 64 * U * want + 2.0 ** -120)
            g = torch.randn(40, 6, device="cuda")
            d, status = backward(z, idx, g, 6, score, **kw)
            assert status == 0 and torch.isfinite(d).all()
            assert (d[3] == 0).all() and (d[4] == 0).all() and (d[8] == 0).all() and (d[39] == 0).all()
            assert (d[~(z > -torch.inf)] == 0).all()
    idx, w = choose(z, 6, score)
    assert idx[5].tolist() == [int(i) for i in torch.sort(z[5, :2], descending=True, stable=True).indices] + [-1] * 4
    assert (w[5, 2:] == 0).all() and abs(float(w[5].sum()) - 1) < 4 * U * 2


@pytest.mark.parametrize("dt", DTYPES)
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("E", [64, 256, 255])
def test_every_kind_of_nan(E, score, dt):
    """Quiet and signalling NaN of both signs, the type's lowest and highest
    values and both zeros: NaN is never chosen, the rest keep their order."""
    z = logits(16, E, dt, 9)
    if dt == torch.bfloat16:
        bits, as_int = [0x7FC0, 0xFFC0, 0x7F81, 0xFF81, 0x7FBF, 0xFFFF], torch.int16
    else:
        bits, as_int = [0x7FC00000, 0xFFC00000, 0x7F800001, 0xFF800001, 0x7FBFFFFF, 0xFFFFFFFF], torch.int32
    wide = 1 << (15 if dt == torch.bfloat16 else 31)
    bits = [b - 2 * wide if b >= wide else b for b in bits]
    for i, b in enumerate(bits):
        z.view(as_int)[i, i::3] = b           # among numbers
        z.view(as_int)[6 + i, 1:] = b         # one number left, the first
    z[12, :] = torch.finfo(dt).min
    z[13, :] = -torch.inf
    z[13, E - 1] = torch.finfo(dt).min
    z[14, ::2], z[14, 1::2] = 0.0, -0.0
    z[15, 0] = -torch.inf
    idx, w = choose(z, 8, score)
    want_idx, want = router64(z, 8, score)
    assert torch.equal(idx.long(), want_idx)
    assert torch.isfinite(w).all()
    within(w, want, 64 * U * want + 2.0 ** -120)
    assert (idx[6:12, 1:] == -1).all() and (idx[6:12, 0] == 0).all()
    assert idx[12].tolist() == idx[14].tolist() == list(range(8))
    assert idx[13].tolist() == [E - 1] + [-1] * 7


def test_bias_masks_and_forces():
    z = logits(64, 32, torch.float32, 5)
    bias = torch.zeros(32)
    bias[3], bias[7], bias[9] = -torch.inf, torch.inf, float("nan")
    bias = bias.cuda()
    for score in SCORES:
        idx, w = choose(z, 4, score, bias)
        assert (idx[:, 0] == 7).all() and not ((idx == 3) | (idx == 9)).any()
        assert torch.isfinite(w).all()
        check(z, 4, score, torch.where(torch.isnan(bias), -torch.inf, bias).clamp(max=1e30))


def test_infinite_logits():
    z = torch.zeros(3, 8)
    z[0, 5] = torch.inf
    z[1, 2] = z[1, 6] = torch.inf
    z[2] = torch.tensor([3.4e38, -3.4e38, 0, 88, -88, 100, -100, 1e30])
    z = z.cuda()
    for score in SCORES:
        for kw in (dict(normalise=True), dict(normalise=False)):
            for bias in (None, torch.zeros(8).cuda()):
                idx, w = choose(z, 2, score, bias, **kw)
                assert idx[0, 0] == 5 and idx[1].tolist() == [2, 6]
                if score == M.SCORE_SOFTMAX:
                    assert w[0].tolist() == [1.0, 0.0] and w[1].tolist() == [0.5, 0.5]
                if bias is None:
                    assert idx[2].tolist() == [0, 7]
    for bias in (None, torch.zeros(8).cuda()):
        idx, w = choose(z[2:], 8, M.SCORE_SIGMOID, bias)
        assert torch.isfinite(w).all() and sorted(idx[0].tolist()) == list(range(8))


@pytest.mark.parametrize("score", SCORES)
def test_scores_that_vanish_keep_their_shares(score):
    z = logits(50, 40, torch.float32, 6) - 500.0
    check(z, 4, score)
    idx, w = choose(z, 4, score)
    assert (abs(w.sum(1) - 1) < 8 * U).all()


@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("score", SCORES)
def test_gradient_by_differences(score, normalise):
    z = logits(6, 24, torch.float32, 7)
    kw = dict(normalise=normalise, scale=1.5)
    idx, w = choose(z, 3, score, **kw)
    g = torch.randn(6, 3, device="cuda")
    d, _ = backward(z, idx, g, 3, score, **kw)
    h = 2.0 ** -8
    for t, e in ((0, int(idx[0, 0])), (1, int(idx[1, 2])), (2, 0), (3, 23), (5, int(idx[5, 1]))):
        f = []
        for step in (h, -h):
            zz = z.double()
            zz[t, e] += step
            i, ww = router64(zz, 3, score, **kw)
            assert torch.equal(i, idx.long())
            f.append(float((ww * g.double()).sum()))
        # third derivatives of a softmax or sigmoid are below 1, of three weights' sum below 6 |g|
        assert abs((f[0] - f[1]) / (2 * h) - float(d[t, e])) < h * h * 10 * float(g.abs().max()) + 1e-6


def test_bad_and_repeated_ids():
    z = logits(70, 40, torch.float32, 8)
    idx, _ = choose(z, 4, M.SCORE_SIGMOID, normalise=False)
    g = torch.randn(70, 4, device="cuda")
    bad = idx.clone()
    bad[3, 1], bad[9, 0], bad[69, 3] = 40, -2, 2 ** 31 - 1
    masked = idx.clone()
    masked[3, 1] = masked[9, 0] = masked[69, 3] = -1
    d, status = backward(z, bad, g, 4, M.SCORE_SIGMOID, normalise=False)
    want, ok = backward(z, masked, g, 4, M.SCORE_SIGMOID, normalise=False)
    assert status == B.DEV_BAD_EXPERT_ID and ok == 0 and torch.equal(d, want)
    twice = idx.clone()
    twice[5, 1] = twice[5, 0]
    one, other = g.clone(), g.clone()
    one[5, 1], other[5, 0] = 0, 0
    d, status = backward(z, twice, g, 4, M.SCORE_SIGMOID, normalise=False)
    a, _ = backward(z, twice, one, 4, M.SCORE_SIGMOID, normalise=False)
    b, _ = backward(z, twice, other, 4, M.SCORE_SIGMOID, normalise=False)
    e = int(idx[5, 0])
    assert status == 0 and d[5, e] == a[5, e] + b[5, e]


def test_no_tokens():
    z = torch.empty(0, 16, device="cuda")
    idx, w = choose(z, 2, M.SCORE_SOFTMAX)
    assert idx.numel() == 0
    d, status = backward(z, idx, torch.empty(0, 2, device="cuda"), 2, M.SCORE_SOFTMAX)
    assert d.numel() == 0 and status == 0


@pytest.mark.parametrize("score", SCORES)
def test_many_tokens(score):
    """A large batch: more workgroups than the device holds."""
    check(logits(70001, 64, torch.bfloat16, 9), 6, score, normalise=False)
