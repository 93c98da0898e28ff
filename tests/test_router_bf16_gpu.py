"""GPU tests of the router's choice from bf16 logits, in every shape of a wave,
against its definition in 64 bits (tests/bf16_reference.py)."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from bf16_reference import router64
from test_router_gpu import SCORES, U, choose, logits, within

pytestmark = pytest.mark.gpu

# experts of each shape of lanes and experts a lane; 256 has one for few rows and one for many
EXPERTS = [(9, 40), (9, 64), (9, 100), (9, 200), (9, 256), (4100, 256), (9, 500), (9, 1000), (3, 4096)]


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("T,E", EXPERTS)
def test_infinity_is_above_the_largest_number(T, E, score):
    """A logit of +inf counts as the largest binary32 number, which is above the
    largest bf16 one: those come after it, whatever their indexes, and get
    nothing of a softmax's weights."""
    z = logits(T, E, torch.bfloat16, E)
    top = torch.finfo(torch.bfloat16).max
    z[:, 0] = z[:, 5] = z[:, E - 2] = top
    z[:, 7] = -top
    z[:, 3] = z[:, E - 1] = torch.inf
    z[1, E - 1] = top
    z[2] = top
    z[2, E - 1] = torch.inf
    idx, w = choose(z, 5, score)
    want, _ = router64(z, 5, score)
    assert torch.equal(idx.long(), want)
    assert idx[0].tolist() == [3, E - 1, 0, 5, E - 2] and idx[2].tolist() == [E - 1, 0, 1, 2, 3]
    if score == M.SCORE_SOFTMAX:
        expect = torch.zeros(T, 5, device="cuda")
        expect[:, :2] = 0.5
        expect[1] = expect[2] = torch.tensor([1.0, 0, 0, 0, 0])
    else:
        expect = torch.full((T, 5), 0.2, device="cuda")
    within(w, expect.double(), 8 * U * expect.double())
