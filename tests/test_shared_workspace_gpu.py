"""GPU tests of the balance loss and a split dispatch on one workspace: the
loss writes where the notify phase keeps its tables, which the scatter has to
report, whatever the loss left there; before the notify phase, after the
scatter or on another workspace it changes nothing."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from combine_ep_get_dispatch_amd import binding as B

pytestmark = pytest.mark.gpu

# tokens, experts, slots: a push scatter, and a block-pull copy
SHAPES = [(200, 16, 2), (4096, 64, 4)]


class Run:
    def __init__(self, T, E, k, quant=False, padding=False):
        g = torch.Generator().manual_seed(T)
        H = 256
        self.shape = M.moedisp_shape.make(T, H, E, 2, k)
        self.b = M.EpBuffers(self.shape, "cuda")
        if quant:
            self.b.enable_quant(128, M.SCALE_FP32)
        self.quant = quant
        self.x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
        self.idx = torch.rand(T, E, generator=g).topk(k, 1).indices.to(torch.int32).cuda()
        self.wt = torch.rand(T, k, generator=g).cuda()
        self.bal = M.moedisp_balance.make(1, T, E, k)
        self.logits = torch.randn(T, E, generator=g).cuda()
        # a loss of padding alone leaves zeros: tables that look like empty ones
        self.loss_idx = torch.full_like(self.idx, -1) if padding else self.idx
        need = max(M.ep_workspace_bytes(self.shape), M.ep_balance_workspace_bytes(self.bal))
        self.ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
        self.b.ws = self.ws
        self.loss_out = torch.zeros(1, device="cuda")
        self.counts = torch.zeros(1, E, dtype=torch.int32, device="cuda")
        self.tokens = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.b.layout(self.idx)

    def notify(self, fused):
        b = self.b
        if fused:
            b.layout_notify(self.idx)
        else:
            M.ep_dispatch_notify(self.shape, self.idx, b.tokens_per_expert, b.expert_offsets, self.ws)

    def loss(self, ws=None):
        M.ep_balance_loss(self.bal, self.logits, self.loss_idx, self.loss_out, self.counts, self.tokens,
                          self.ws if ws is None else ws)

    def scatter(self):
        b = self.b
        if self.quant:
            M.ep_dispatch_scatter_quant(self.shape, 128, M.SCALE_FP32, self.x, self.idx, self.wt, b.tokens_per_expert,
                                        b.recv_q, b.recv_qscales, b.recv_src_idx, b.recv_weights, b.expert_offsets,
                                        b.slot_to_row, self.ws)
        else:
            b.dispatch_scatter(self.x, None, self.idx, self.wt)
        return b.slot_to_row.clone()

    def status(self):
        return M.ep_check_status(self.ws)


@pytest.mark.parametrize("padding", [False, True])
@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("fused", [False, True])
@pytest.mark.parametrize("T,E,k", SHAPES)
def test_loss_between_the_phases_is_reported(T, E, k, fused, quant, padding):
    r = Run(T, E, k, quant, padding)
    assert bool(M.ep_plan_query(r.shape)["pull"]) == (T == 4096)
    r.notify(fused)
    want = r.scatter()
    assert r.status() == 0
    r.notify(fused)
    r.loss()
    r.scatter()
    assert r.status() & B.DEV_BAD_LAYOUT
    # the next notify phase writes the tables anew; the scatter may be repeated
    r.notify(fused)
    for _ in range(2):
        assert torch.equal(r.scatter(), want)
    assert r.status() == 0


@pytest.mark.parametrize("T,E,k", SHAPES)
def test_loss_around_a_dispatch(T, E, k):
    """Before the notify phase, after the scatter, around the whole dispatch,
    and on a workspace of its own between the phases."""
    r = Run(T, E, k)
    own = torch.zeros_like(r.ws)
    r.notify(False)
    want = r.scatter()
    for fused in (False, True):
        r.loss()
        r.notify(fused)
        r.loss(own)
        assert torch.equal(r.scatter(), want)
        r.loss()
        assert r.status() == 0 and M.ep_check_status(own) == 0
    r.b.dispatch(r.x, None, r.idx, r.wt)
    assert torch.equal(r.b.slot_to_row, want)
    r.loss()
    r.b.dispatch(r.x, None, r.idx, r.wt)
    assert torch.equal(r.b.slot_to_row, want) and r.status() == 0
    assert float(r.loss_out) > 0
