"""GPU tests of the router's choice from bf16 logits, in every shape of a wave,
against its definition in 64 bits (tests/bf16_reference.py)."""
import pytest
import torch

import combine_ep_get_dispatch_amd as M
from bf16_reference import router64
from test_router_gpu import SCORES, U, check, choose, logits, within

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


@pytest.mark.parametrize("normalise", [True, False])
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("T,E", EXPERTS)
def test_bias(T, E, score, normalise):
    """Rounded logits, many of which are equal, with a bias."""
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda()
    check(logits(T, E, torch.bfloat16, T + E), 8, score, bias, normalise=normalise, scale=2.5)


@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("best", [1, 2])
@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("T,E", EXPERTS)
def test_groups(T, E, score, best, biased):
    """4 of 8 groups, as for a large model's router, in every shape."""
    bias = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda() if biased else None
    check(logits(T, E, torch.bfloat16, T + E), 8, score, bias, groups=8 if E % 8 == 0 else 4, topk_groups=4,
          group_best=best)


@pytest.mark.parametrize("T,E,k,G,tg", [(5, 4096, 16, 64, 64), (40, 64, 4, 64, 5), (21, 1024, 32, 32, 4), (11, 39, 3, 3, 1)])
def test_many_groups(T, E, k, G, tg):
    bias = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda()
    check(logits(T, E, torch.bfloat16, T + E), k, M.SCORE_SIGMOID, bias, groups=G, topk_groups=tg, normalise=False)


@pytest.mark.parametrize("score", SCORES)
@pytest.mark.parametrize("T,E", EXPERTS)
def test_masked_and_infinite_logits_with_bias_and_groups(T, E, score):
    """-inf and NaN take no part; +inf has the score of the largest number."""
    z = logits(T, E, torch.bfloat16, T + E)
    z[0, ::2], z[1, 1::2], z[2, E // 2:] = -torch.inf, float("nan"), -torch.inf
    z[0, 1] = torch.finfo(torch.bfloat16).max
    bias = 0.2 * torch.randn(E, generator=torch.Generator().manual_seed(E)).cuda()
    finite = torch.where(torch.isfinite(z), z, -torch.inf)
    for kw in (dict(), dict(groups=8 if E % 8 == 0 else 4, topk_groups=2)):
        for b in (None, bias):
            idx, w = choose(z, 8, score, b, **kw)
            want_idx, want = router64(finite, 8, score, b, **kw)
            assert torch.equal(idx.long(), want_idx)
            within(w, want, 64 * U * want + 2.0 ** -120)
            top = z.clone()
            top[0, 1] = torch.inf
            again, w2 = choose(top, 8, score, b, **kw)
            assert torch.equal(again, idx) and torch.equal(w2, w)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", SCORES)
def test_scores_too_small_to_tell_apart(score, dt):
    """With groups the choice goes by scores, and those below exp(-700) are
    equal; without, it goes by logits."""
    z = torch.tensor([[0, -800, -752, -792, -704, -900, -720, -880]]).to(dt).cuda()
    idx, _ = choose(z, 8, score, groups=2, topk_groups=2)
    assert idx[0].tolist() == list(range(8))
    idx, _ = choose(z, 8, score)
    assert idx[0].tolist() == [0, 4, 6, 2, 3, 1, 7, 5]
