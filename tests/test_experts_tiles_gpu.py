"""GPU tests of the experts' operators and the balance loss in the forms that
large calls take: the largest tiles of both products, tiles of several passes
and workgroups of several rows.  Every test asks the plan first whether its
sizes really take that form.  Tolerances as in test_experts_gpu.py."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from experts_reference import E4M3, Problem, balance64, scales64, swiglu64, swiglu_backward64
from test_experts_gpu import (FMTS, SCORES, SWIGLU_REL, U, Balance, balance_inputs, check_codes, check_gemm, within)

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
    # fp32 results of FP32 scales take more of LDS, and a smaller tile
    assert_tile(p, out, wgrad=(256, 128) if fmt == M.SCALE_FP32 and out == M.FP32 else (256, 256))
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


# S, L, E, k: lanes that share a row from 1 to 64, rows of one to eight chunks
# of the lanes, loads by 16 bytes and by element, more slots than lanes
PASSES = [(64, 1013, 256, 8), (40, 1013, 257, 3), (60, 350, 600, 8), (50, 463, 1030, 32), (30, 703, 4096, 5),
          (300, 4000, 5, 3), (33, 5000, 40, 12), (40, 8010, 24, 8), (1, 70001, 128, 8)]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("S,L,E,k", PASSES)
def test_balance_several_passes(S, L, E, k, score, dt):
    """Tiles of three passes and more, the last tile of a sequence shorter;
    padding tokens hold NaN beside live ones."""
    h = Balance(S, L, E, k, score, dt)
    plan = M.ep_balance_plan_query(h.b)
    assert plan["passes"] >= 3 and L % plan["tile_tokens"] % plan["rows_at_once"] != 0, plan
    g = torch.Generator(device="cuda").manual_seed(S + E)
    z = (torch.randn(S * L, E, generator=g, device="cuda") * 2).to(dt)
    idx = torch.rand(S * L, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    idx[torch.rand(S * L, k, generator=g, device="cuda") < 0.1] = -1
    idx[torch.rand(S * L, generator=g, device="cuda") < 0.2] = -1
    pad = (idx < 0).all(1)
    clean = z.clone()
    z[pad], clean[pad] = float("nan"), 0.0
    h.forward(z, idx)
    dz = h.backward(z, idx)
    assert M.ep_check_status(h.ws) == 0
    loss, counts, tokens, want = balance64(clean, idx, S, k, float(h.b.coef), score, 1.5)
    assert torch.equal(h.counts.long(), counts.long()) and torch.equal(h.tokens.long(), tokens)
    within(h.loss, loss, (2 * E + L + 40) * U * loss.abs(), "loss")
    n = tokens.double().clamp(min=1)
    w = 1.5 * h.b.coef * E * counts.double() / ((tokens > 0).sum().clamp(min=1) * k * n[:, None] ** 2)
    size = w.repeat_interleave(L, 0).amax(1, keepdim=True)
    within(dz, want, (2 * E + 40) * U * size + (2.0 ** -8 * want.abs() if dt == torch.bfloat16 else 0), "d_logits")
    assert (dz[pad] == 0).all()


def swiglu_rows(inner, padded):
    """Rows of four times what the workgroups take at once and some more, with
    gaps: (problem of the rows, gate and up values, NaN in rows of no expert)."""
    once = 2048 * max(1, 16 // (inner // 128))
    if padded:
        E, stride, cap = 37, 2 * once // 15, once // 9
        p = Problem([(e * 997) % (cap + 50) for e in range(E)], 8, 128, M.SCALE_FP32, padded=(stride, cap, 5))
    else:
        p = Problem([once, 0, 3, once + 77, 2 * once], 8, 128, M.SCALE_FP32, spare=once // 3)
    g = torch.Generator(device="cuda").manual_seed(inner)
    gu = (torch.randn(p.R, 2 * inner, generator=g, device="cuda") * 2).to(torch.bfloat16)
    gu[~p.live] = float("nan")
    return p, gu


SWIGLU = [(128, False), (128, True), (640, False), (640, True), (2048, False), (2176, True)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("inner,padded", SWIGLU)
def test_swiglu_several_rows(inner, padded, fmt):
    p, gu = swiglu_rows(inner, padded)
    plan = M.ep_expert_plan_query(p.rows, 8, inner, fmt, M.BF16)
    assert p.R > 4 * plan["swiglu_rows"] * plan["swiglu_blocks"]
    h = torch.full((p.R, inner), 7, dtype=torch.uint8, device="cuda")
    hs = torch.full((p.R, inner // 128), 7, device="cuda", dtype=torch.float32 if fmt == M.SCALE_FP32 else torch.uint8)
    M.ep_swiglu_quant(p.rows, inner, fmt, gu, p.bounds, h, hs, p.ws)
    assert p.status() == 0
    check_codes(h.view(E4M3)[p.live], hs[p.live], swiglu64(gu[p.live]), SWIGLU_REL, "h")
    assert (h[~p.live] == 7).all() and (hs[~p.live] == 7).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("inner,padded", SWIGLU)
def test_swiglu_backward_several_rows(inner, padded, fmt):
    p, gu = swiglu_rows(inner, padded)
    plan = M.ep_expert_plan_query(p.rows, 8, inner, fmt, M.BF16)
    assert p.R > 4 * plan["swiglu_rows"] * plan["swiglu_backward_blocks"]
    live = p.live
    g = torch.Generator(device="cuda").manual_seed(inner + 1)
    dh = torch.randn(p.R, inner, generator=g, device="cuda").to(torch.bfloat16)
    dh[~live] = float("nan")
    dgu = torch.full((p.R, 2 * inner), 7.0, dtype=torch.bfloat16, device="cuda")
    q = torch.full((p.R, 2 * inner), 7, dtype=torch.uint8, device="cuda")
    qs = torch.full((p.R, inner // 64), 7, device="cuda", dtype=torch.float32 if fmt == M.SCALE_FP32 else torch.uint8)
    M.ep_swiglu_backward(p.rows, inner, fmt, gu, dh, p.bounds, dgu, q, qs, p.ws)
    assert p.status() == 0
    assert (dgu[~live] == 7.0).all() and (q[~live] == 7).all() and (qs[~live] == 7).all()
    want = swiglu_backward64(gu[live], dh[live])
    gg, u = gu[live].double().chunk(2, -1)
    s = torch.sigmoid(gg)
    # dg has a factor 1 + g (1 - s) that can cancel: its error is relative to 1 + |g| (1 - s)
    size = torch.cat([(dh[live].double() * u * s).abs() * (1 + gg.abs() * (1 - s)), want[:, inner:].abs()], -1)
    own = 16 * 2.0 ** -23 * size
    within(dgu[live], want, 2.0 ** -8 * want.abs() + own, "dgu")
    real = scales64(qs[live])
    b = want.view(want.shape[0], inner // 64, 128)
    ob = own.view_as(b)
    if fmt == M.SCALE_FP32:
        amax = b.abs().amax(-1)
        within(qs[live], amax / 448, ob.amax(-1) / 448 + 2.0 ** -23 * amax / 448, "scales")
    got = q.view(E4M3)[live].double().view_as(b) * real[..., None]
    tol = torch.maximum(2.0 ** -4 * b.abs(), 2.0 ** -10 * real[..., None]) * (1 + 2.0 ** -10) + 2 * ob
    within(got, b, tol + 2.0 ** -20 * b.abs(), "codes")


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("S,L,E,k", [(4097, 3, 16, 2), (5000, 40, 33, 3), (100003, 1, 8, 2), (4500, 2, 300, 4)])
def test_balance_many_sequences(S, L, E, k, score, dt):
    """More sequences than the backward pass has workgroups; some of them hold
    padding alone."""
    h = Balance(S, L, E, k, score, dt)
    assert M.ep_balance_plan_query(h.b)["backward_blocks"] < S
    g = torch.Generator(device="cuda").manual_seed(S)
    z = (torch.randn(S * L, E, generator=g, device="cuda") * 2).to(dt)
    idx = torch.rand(S * L, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    idx[torch.rand(S * L, generator=g, device="cuda") < 0.3] = -1
    idx.view(S, L, k)[torch.rand(S, generator=g, device="cuda") < 0.2] = -1
    h.forward(z, idx)
    dz = h.backward(z, idx)
    assert M.ep_check_status(h.ws) == 0
    # the definition in 64 bits (counts by one sum over all sequences)
    z64 = z.double().view(S, L, E)
    sg = torch.sigmoid(z64)
    p = torch.softmax(z64, -1) if score == M.SCORE_SOFTMAX else sg / sg.sum(-1, keepdim=True)
    live = (idx >= 0).any(1).view(S, L)
    at = torch.where(idx < 0, E, idx).long().view(S, L * k)
    counts = torch.zeros(S, E + 1, dtype=torch.int64, device="cuda").scatter_add_(1, at, torch.ones_like(at))[:, :E]
    tokens = live.sum(1)
    n, some = tokens.double().clamp(min=1)[:, None], int((tokens > 0).sum())
    assert 0 < some < S and torch.equal(h.counts.long(), counts) and torch.equal(h.tokens.long(), tokens)
    w = float(h.b.coef) * E * counts.double() / (some * k * n ** 2)
    loss = (w * (p * live[..., None]).sum(1)).sum()
    within(h.loss, loss, (2 * E + L + 40) * U * loss.abs(), "loss")
    w = 1.5 * w[:, None, :]
    want = p * (w - (p * w).sum(-1, keepdim=True)) * live[..., None]
    if score == M.SCORE_SIGMOID:
        want = want * (1 - sg)
    tol = (2 * E + 40) * U * w.amax(-1, keepdim=True).expand_as(want)
    within(dz.view(S, L, E), want, tol + (2.0 ** -8 * want.abs() if dt == torch.bfloat16 else 0), "d_logits")


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("S,L,E,k", [(2, 64, 8, 8), (1, 4096, 64, 4), (3, 1600, 100, 5), (1, 1200, 600, 4)])
def test_balance_gradient_of_equal_counts_with_masked_slots(S, L, E, k, score):
    """Every second slot masked, experts in turn in the others: the counts are
    equal, the gradient exactly zero; one more slot masked, and it is good to
    the size of what the counts differ by, not of the counts."""
    z, _ = balance_inputs(S, L, E, k, torch.float32, 35)
    at = torch.arange(L * k, device="cuda").view(L, k)
    idx = torch.where(at % 2 == 0, (at // 2) % E, -1).repeat(S, 1).to(torch.int32).contiguous()
    assert L * k // 2 % E == 0
    h = Balance(S, L, E, k, score)
    h.forward(z, idx)
    assert (h.counts == L * k // 2 // E).all() and (h.tokens == L).all()
    assert (h.backward(z, idx) == 0).all()
    idx[3][idx[3] >= 0] = torch.where(torch.arange(int((idx[3] >= 0).sum()), device="cuda") == 0, -1, idx[3][idx[3] >= 0]).int()
    h.forward(z, idx)
    dz = h.backward(z, idx)
    _, _, tokens, want = balance64(z, idx, S, k, float(h.b.coef), score, 1.5)
    # as in check_balance, with the counts' difference from their mean (at most 1) in the place of the counts
    w = 1.5 * h.b.coef * E / (S * k * float(tokens.min()) ** 2)
    within(dz, want, (2 * E + 40) * U * w * torch.ones_like(want), "d_logits")
