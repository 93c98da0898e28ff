"""GPU tests of what the header says of infinities and NaN in the activation
and the balance loss, and of captured graphs that share a workspace."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from experts_reference import E4M3, Problem
from test_experts_gpu import FMTS, SCORES, Balance, balance_inputs

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("fmt", FMTS)
def test_infinite_gates(fmt):
    """An infinite gate: NaN codes and scale 1 in its block forward, NaN in its
    place backward, and nothing elsewhere."""
    p = Problem([4], 8, 128, fmt, spare=0)
    gu = torch.randn(4, 512, device="cuda").to(torch.bfloat16)
    gu[1, 130], gu[2, 3] = INF, -INF
    h = torch.empty(4, 256, dtype=torch.uint8, device="cuda")
    hs = torch.empty(4, 2, device="cuda", dtype=torch.float32 if fmt == M.SCALE_FP32 else torch.uint8)
    M.ep_swiglu_quant(p.rows, 256, fmt, gu, p.bounds, h, hs, p.ws)
    bad = torch.zeros(4, 2, dtype=torch.bool, device="cuda")
    bad[1, 1] = bad[2, 0] = True
    nan = (h == 0x7F).view(4, 2, 128)
    assert nan[bad].all() and not torch.isnan(h.view(E4M3).view(4, 2, 128)[~bad].float()).any()
    assert (hs[bad] == (1.0 if fmt == M.SCALE_FP32 else 127)).all()
    dgu = torch.empty_like(gu)
    M.ep_swiglu_backward(p.rows, 256, fmt, gu, torch.ones(4, 256, device="cuda", dtype=torch.bfloat16), p.bounds, dgu,
                         None, None, p.ws)
    at = torch.zeros(4, 256, dtype=torch.bool, device="cuda")
    at[1, 130] = at[2, 3] = True
    assert torch.isnan(dgu[:, :256][at]).all() and torch.isfinite(dgu[:, :256][~at]).all()
    assert torch.isfinite(dgu[:, 256:][~at]).all()


@pytest.mark.parametrize("score", SCORES)
def test_balance_infinite_logits(score):
    """A row of -inf alone scores nothing; NaN makes the loss NaN, and so does
    +inf for softmax (the sigmoid of it is 1)."""
    z, idx = balance_inputs(2, 30, 24, 3, torch.float32, 44, pad=0.0)
    idx[7] = torch.tensor([1, 2, 3], device="cuda")
    h = Balance(2, 30, 24, 3, score)
    z[7] = -INF
    h.forward(z, idx)
    assert torch.isfinite(h.loss).all() and (h.backward(z, idx)[7] == 0).all()
    z[7, 4] = INF
    h.forward(z, idx)
    dz = h.backward(z, idx)
    assert bool(torch.isnan(h.loss)) == (score == M.SCORE_SOFTMAX)
    assert bool(torch.isnan(dz[7]).any()) == (score == M.SCORE_SOFTMAX)
    rest = torch.arange(60, device="cuda") != 7
    assert torch.isfinite(dz[rest]).all()
    z[7, 4] = float("nan")
    h.forward(z, idx)
    assert torch.isnan(h.loss).all()


def test_graphs_that_share_a_workspace():
    """Two captured graphs of losses of different shapes on one workspace,
    replayed in turn with eager calls on it between them."""
    shapes = [(4, 300, 64, 4), (1, 2000, 100, 6)]
    hs, zs = [], []
    for i, (S, L, E, k) in enumerate(shapes):
        hs.append(Balance(S, L, E, k, SCORES[i]))
        zs.append(balance_inputs(S, L, E, k, torch.float32, 45 + i))
    ws = max((h.ws for h in hs), key=lambda w: w.numel())
    for h in hs:
        h.ws = ws
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for h, (z, idx) in zip(hs, zs):
            h.forward(z, idx)
    torch.cuda.current_stream().wait_stream(side)
    graphs, grads = [], []
    for h, (z, idx) in zip(hs, zs):
        dz = torch.empty_like(z)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            h.forward(z, idx)
            M.ep_balance_loss_backward(h.b, z, idx, h.counts, h.tokens, h.d_loss, dz)
        graphs.append(g)
        grads.append(dz)
    for turn in range(4):
        for i in (0, 1, 1, 0):
            h, (z, idx) = hs[i], zs[i]
            z.mul_(1.01)
            graphs[i].replay()
            torch.cuda.synchronize()
            loss, counts, dz = h.loss.clone(), h.counts.clone(), grads[i].clone()
            h.forward(z, idx)
            want = h.backward(z, idx)
            assert torch.equal(h.loss, loss) and torch.equal(h.counts, counts) and torch.equal(dz, want), (turn, i)
    assert M.ep_check_status(ws) == 0
