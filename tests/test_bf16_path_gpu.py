"""GPU tests of the bf16 and 4-bit paths as programs run them: router, dispatch,
products, activation, combine; a training step; graphs, streams, calls at once.

Where a result passes several roundings to bf16 (2^-8 of the value each), the
tolerance adds up what each can do to it."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from bf16_reference import Bf16Problem, router64, weights4
from experts_reference import swiglu64
from test_experts_gpu import within

pytestmark = pytest.mark.gpu
B = 2.0 ** -8


def expert64(x, w1, w2):
    """(y, bound of its error) of one row: gu, h and y in bf16."""
    a = w1 @ x
    g, u = a.chunk(2)
    hv = swiglu64(a)
    # sums in binary32, far below; silu grows by at most 1.1 |dg|
    dh = B * (1.2 * g.abs() * u.abs() + hv.abs()) + B * B * a.abs().max() ** 2
    dh = dh + B * (hv.abs() + dh) + 2.0 ** -18 * a.abs().max()
    y = w2 @ hv
    bound = w2.abs() @ dh
    return y, bound + B * (y.abs() + bound) + 2.0 ** -18 * (w2.abs() @ hv.abs())


def routed(T, E, k, seed, groups=1):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g).cuda()
    live = torch.ones(T, dtype=torch.uint8)
    live[T // 3], live[T - 1] = 0, 0
    r = M.moedisp_router.make(T, E, k, M.SCORE_SIGMOID, M.FP32, groups, max(1, groups // 2), 2, True, 1.5)
    bias = (0.1 * torch.randn(E, generator=g)).cuda()
    bias[5] = -torch.inf                                # an expert without rows
    return g, r, z, bias, live.cuda()


@pytest.mark.parametrize("layout", ["contiguous", "padded"])
@pytest.mark.parametrize("form", ["bf16", "e2m1", "int4"])
def test_serving_path(layout, form):
    T, H, I, E, k = 72, 256, 128, 8, 2
    g, r, z, bias, live = routed(T, E, k, 31, groups=4)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    idx, wt = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    M.ep_router_topk(r, z, bias, live, idx, wt)
    want_idx, want_wt = router64(z, k, M.SCORE_SIGMOID, bias, live, groups=4, topk_groups=2, scale=1.5)
    assert torch.equal(idx.long(), want_idx)
    bufs = M.EpBuffers(M.moedisp_shape.make(T, H, E, 2, k), "cuda")
    if layout == "contiguous":
        bufs.layout(idx)
        bufs.dispatch(x, None, idx, wt)
        rows, bounds, rx, handle = M.moedisp_rows.contiguous(E, T * k), bufs.expert_offsets, bufs.recv_x, bufs.slot_to_row
        combine = bufs.combine
    else:
        pad = M.EpPaddedBuffers(bufs, T, T + 8, 8)
        pad.dispatch(x, None, idx, wt)
        rows, bounds = M.moedisp_rows.padded(E, T, T + 8, 8, expected_rows=18), bufs.tokens_per_expert
        rx, handle, combine = pad.recv_x, pad.slot_to_row, pad.combine
    R = rows.max_rows
    gu = torch.zeros(R, 2 * I, dtype=torch.bfloat16, device="cuda")
    h, y = torch.zeros(R, I, dtype=torch.bfloat16, device="cuda"), torch.zeros(R, H, dtype=torch.bfloat16, device="cuda")
    if form == "bf16":
        w1 = (torch.randn(E, 2 * I, H, generator=g) / H ** 0.5).to(torch.bfloat16).cuda()
        w2 = (torch.randn(E, H, I, generator=g) / I ** 0.5).to(torch.bfloat16).cuda()
        M.ep_expert_gemm_bf16(rows, 2 * I, H, M.WEIGHTS_NK, rx, w1, bounds, gu, M.BF16, bufs.ws)
        M.ep_swiglu(rows, I, gu, bounds, h, bufs.ws)
        M.ep_expert_gemm_bf16(rows, H, I, M.WEIGHTS_NK, h, w2, bounds, y, M.BF16, bufs.ws)
        w1, w2 = w1.double(), w2.double()
    else:
        fmt = M.W4_INT4 if form == "int4" else M.W4_E2M1
        c1 = torch.randint(0, 256, (E, 2 * I, H // 2), generator=g, dtype=torch.uint8).cuda()
        c2 = torch.randint(0, 256, (E, H, I // 2), generator=g, dtype=torch.uint8).cuda()
        if form == "int4":
            s1, s2 = torch.full((E, H // 128, 2 * I), 0.015).bfloat16().cuda(), torch.full((E, I // 128, H), 0.02).bfloat16().cuda()
        else:
            s1 = torch.randint(120, 123, (E, H // 32, 2 * I), generator=g, dtype=torch.uint8).cuda()
            s2 = torch.randint(120, 123, (E, I // 32, H), generator=g, dtype=torch.uint8).cuda()
        M.ep_expert_gemm_w4(rows, 2 * I, H, fmt, rx, c1, s1, bounds, gu, M.BF16, bufs.ws)
        M.ep_swiglu(rows, I, gu, bounds, h, bufs.ws)
        M.ep_expert_gemm_w4(rows, H, I, fmt, h, c2, s2, bounds, y, M.BF16, bufs.ws)
        w1, w2 = weights4(c1, s1, fmt), weights4(c2, s2, fmt)
    out = torch.empty(T, H, device="cuda")
    combine(y, out, M.FP32)
    assert M.ep_check_status(bufs.ws) == 0
    want, bound = torch.zeros(T, H, dtype=torch.float64, device="cuda"), torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(idx[t, j])
            if e < 0:
                assert int(handle[t, j]) == -1
                continue
            v, b = expert64(x[t].double(), w1[e], w2[e])
            want[t] += want_wt[t, j] * v
            bound[t] += want_wt[t, j] * (b + 2.0 ** -18 * v.abs())
    within(out, want, bound)
    assert float((out.double() - want).norm() / want.norm()) < 4 * B  # and it is no loose fit
    assert (out[T - 1] == 0).all()


@pytest.mark.parametrize("score,normalise", [(M.SCORE_SIGMOID, True), (M.SCORE_SOFTMAX, True), (M.SCORE_SOFTMAX, False)])
def test_training_step(score, normalise):
    """Forward and all gradients (tokens, router, both weights) of a layer
    against 64-bit autograd with the same choice."""
    T, H, I, E, k = 60, 128, 128, 6, 2
    g = torch.Generator().manual_seed(41)
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    wr = torch.randn(E, H, generator=g).cuda() / H ** 0.5
    z = x.float() @ wr.t()
    w1 = (torch.randn(E, 2 * I, H, generator=g) / H ** 0.5).to(torch.bfloat16).cuda()
    w2 = (torch.randn(E, H, I, generator=g) / I ** 0.5).to(torch.bfloat16).cuda()
    d_out = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    r = M.moedisp_router.make(T, E, k, score, M.FP32, normalise=normalise, scale=1.25)
    idx, wt = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    M.ep_router_topk(r, z, None, None, idx, wt)
    bufs = M.EpBuffers(M.moedisp_shape.make(T, H, E, 2, k), "cuda")
    bufs.layout(idx)
    bufs.dispatch(x, None, idx, wt)
    R, rows, off, ws = T * k, M.moedisp_rows.contiguous(E, T * k), bufs.expert_offsets, bufs.ws
    bf = lambda n: torch.empty(R, n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    rx, gu, h, y = bufs.recv_x.view(torch.bfloat16), bf(2 * I), bf(I), bf(H)
    M.ep_expert_gemm_bf16(rows, 2 * I, H, M.WEIGHTS_NK, rx, w1, off, gu, M.BF16, ws)
    M.ep_swiglu(rows, I, gu, off, h, ws)
    M.ep_expert_gemm_bf16(rows, H, I, M.WEIGHTS_NK, h, w2, off, y, M.BF16, ws)
    out = torch.empty(T, H, device="cuda")
    bufs.combine(y, out, M.FP32)
    # back: combine's gradient of a row is its weight times the token's, and of the weight their product
    row = bufs.slot_to_row.long()
    token = bufs.recv_src_idx.long()
    dy = (bufs.recv_weights[:, None] * d_out.float()[token]).to(torch.bfloat16)
    dwt = (y.float()[row] * d_out.float()[:, None]).sum(-1).contiguous()
    dh, dgu, dx_rows = bf(I), bf(2 * I), bf(H)
    dw1, dw2 = torch.empty(E, 2 * I, H, device="cuda"), torch.empty(E, H, I, device="cuda")
    M.ep_expert_gemm_bf16(rows, I, H, M.WEIGHTS_KN, dy, w2, off, dh, M.BF16, ws)
    M.ep_expert_wgrad_bf16(rows, H, I, h, dy, off, dw2, M.FP32, False, ws)
    M.ep_swiglu_backward(rows, I, M.SCALE_FP32, gu, dh, off, dgu, None, None, ws)
    M.ep_expert_gemm_bf16(rows, H, 2 * I, M.WEIGHTS_KN, dgu, w1, off, dx_rows, M.BF16, ws)
    M.ep_expert_wgrad_bf16(rows, 2 * I, H, rx, dgu, off, dw1, M.FP32, False, ws)
    dz = torch.empty_like(z)
    M.ep_router_topk_backward(r, z, idx, dwt, dz, ws)
    dx = torch.zeros(T, H, device="cuda").index_add_(0, token, dx_rows.float()) + dz @ wr
    assert M.ep_check_status(ws) == 0

    x64, wr64, w164, w264 = (t.double().requires_grad_() for t in (x, wr, w1, w2))
    z64 = x64 @ wr64.t()
    i64, wt64 = router64(z64, k, score, normalise=normalise, scale=1.25)
    assert torch.equal(i64, idx.long())
    out64 = 0
    for j in range(k):
        for e in range(E):
            at = (i64[:, j] == e).nonzero()[:, 0]
            v = swiglu64(x64[at] @ w164[e].t()) @ w264[e].t()
            out64 = out64 + torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add(0, at, wt64[at, j:j + 1] * v)
    (out64 * d_out.double()).sum().backward()
    # every path passes at most six roundings to bf16 and their like in the norm
    for name, got, want in (("out", out, out64.detach()), ("dx", dx, x64.grad), ("dw1", dw1, w164.grad),
                            ("dw2", dw2, w264.grad), ("dwr", dz.t() @ x.float(), wr64.grad)):
        off_by = float((got.double() - want).norm() / want.norm())
        assert off_by < 6 * B, (name, off_by)


def everything(seed):
    """A list of calls on buffers of their own, and the outputs they leave."""
    p = Bf16Problem([40, 0, 200, 3, 128, 17], 520, 256, seed=seed, spare=0, expected=100)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    w, wk = p.weights(M.WEIGHTS_NK), p.weights(M.WEIGHTS_KN)
    q = Bf16Problem(p.counts, 528, 256, seed=seed + 1, spare=0, expected=4)
    c, sc = q.quantised(M.W4_INT4)
    c2, sc2 = q.quantised(M.W4_E2M1)
    bf = lambda n: torch.zeros(p.R, n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    y, yk, h, y4, y42 = bf(520), bf(520), bf(256), bf(528), bf(528)
    gu = p.rows_of(512)
    dw = torch.zeros(p.E, 520, 256, device="cuda")
    z = torch.randn(300, 64, generator=p.g).cuda()
    bias = (0.1 * torch.randn(64, generator=p.g)).cuda()
    r = M.moedisp_router.make(300, 64, 6, M.SCORE_SIGMOID, M.FP32, 8, 4)
    idx, wt = torch.zeros(300, 6, dtype=torch.int32, device="cuda"), torch.zeros(300, 6, device="cuda")
    dwt, dz = torch.randn(300, 6, generator=p.g).cuda(), torch.zeros(300, 64, device="cuda")

    def step(stream=None, ws=ws):
        M.ep_expert_gemm_bf16(p.rows, 520, 256, M.WEIGHTS_NK, p.x, w, p.bounds, y, M.BF16, ws, stream)
        M.ep_expert_gemm_bf16(p.rows, 520, 256, M.WEIGHTS_KN, p.x, wk, p.bounds, yk, M.BF16, ws, stream)
        M.ep_swiglu(p.rows, 256, gu, p.bounds, h, ws, stream)
        M.ep_expert_gemm_w4(q.rows, 528, 256, M.W4_INT4, h, c, sc, q.bounds, y4, M.BF16, ws, stream)
        M.ep_expert_gemm_w4(q.rows, 528, 256, M.W4_E2M1, p.x, c2, sc2, q.bounds, y42, M.BF16, ws, stream)
        M.ep_expert_wgrad_bf16(p.rows, 520, 256, p.x, y, p.bounds, dw, M.FP32, False, ws, stream)
        M.ep_router_topk(r, z, bias, None, idx, wt, stream)
        M.ep_router_topk_backward(r, z, idx, dwt, dz, ws, stream)

    def change():
        p.x.copy_(p.x.flip(0))
        gu.copy_(gu.flip(0))
        z.copy_(z.flip(0))

    return step, change, [y, yk, h, y4, y42, dw, idx, wt, dz], ws


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_replayed_graphs_that_share_a_workspace():
    one, two = everything(51), everything(61)
    ws = one[3]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one[0](ws=ws)
        two[0](ws=ws)
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for step, _, _, _ in (one, two):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(ws=ws)
    for i in range(4):
        for (step, change, outs, _), graph in zip((one, two), graphs):
            if i:
                change()
            for o in outs:
                o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            got = [o.clone() for o in outs]
            for o in outs:
                o.zero_()
            step()
            torch.cuda.synchronize()
            assert same(got, outs), i
    assert M.ep_check_status(ws) == 0


def test_calls_at_once():
    """Two streams at the same time, many times over: each gives the bits that
    it gives alone."""
    both = [everything(71), everything(81)]
    alone = []
    for step, _, outs, _ in both:
        step()
        torch.cuda.synchronize()
        alone.append([o.clone() for o in outs])
    streams = [torch.cuda.Stream() for _ in both]
    for _ in range(20):
        for (step, _, _, _), st in zip(both, streams):
            step(st)
    torch.cuda.synchronize()
    for (_, _, outs, ws), want in zip(both, alone):
        assert same(outs, want) and M.ep_check_status(ws) == 0
