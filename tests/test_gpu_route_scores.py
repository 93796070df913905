"""The router's weights and choice where scores are very small or very near each
other, against the definition in 64 bits."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
gd = pytest.importorskip("greedy_decode_step_gb300")
STEP = 2.0 ** -24  # half a step of float32


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(seed, *shape):
    return torch.randn(shape, generator=rng(seed), device="cuda")


def choice(y, Wr, k, **kw):
    ids = torch.full((y.shape[0], k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((y.shape[0], k), math.nan, device="cuda")
    gd.dec_moe_route(y, Wr, ids, w, **kw)
    return ids.long(), w.double()


def shares(z, sigmoid):
    """Scores over their sum, from their logarithms: log sigmoid(z) = z - softplus(z), and a softmax's sum cancels."""
    return torch.softmax(torch.nn.functional.logsigmoid(z) if sigmoid else z, -1)


# ----------------------------------------------------------------------------- weights of small scores

def logits(T, E, at, H=16):
    """y and Wr whose logits are z = at + steps of 1/8 up to 4, exact in float32 and in 64 bits."""
    y = torch.zeros(T, H, device="cuda")
    y[:, 0], y[:, 1] = at, 0.125
    Wr = torch.zeros(E, H, device="cuda")
    Wr[:, 0] = 1.0
    Wr[:, 1] = torch.randint(0, 33, (E,), generator=rng(1), device="cuda").float()
    return y, Wr.bfloat16()


@pytest.mark.parametrize("E,k", [(8, 2), (64, 8), (300, 16)])
@pytest.mark.parametrize("at", [-60.0, -88.0, -96.0, -104.0, -1000.0, -3e4])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_all_logits_far_below_zero(sigmoid, at, E, k):
    y, Wr = logits(3, E, at)
    ids, w = choice(y, Wr, k, score="sigmoid" if sigmoid else "softmax", scale=2.5)
    z = y.double() @ Wr.double().T
    want = z.sort(dim=-1, descending=True, stable=True).indices[:, :k]
    assert torch.equal(ids, want)
    # differences of these logits are exact: two exponentials of 2 steps of 2^-23 each, sums of k, quotients and products
    assert bool(((w / 2.5 - shares(z.gather(1, want), sigmoid)).abs() <= (16 + k) * STEP * (w / 2.5)).all())


@pytest.mark.parametrize("E,k", [(8, 2), (64, 8), (300, 16)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_chosen_by_their_bias_far_below_the_others(sigmoid, E, k):
    """k experts 120 below the largest logit, which a bias of 2 puts ahead of all others."""
    y, Wr = logits(2, E, 0.0)
    y[:, 2] = 120.0
    low = torch.randperm(E, generator=rng(2), device="cuda")[:k]
    Wr[low, 2] = -1.0
    bias = torch.zeros(E, device="cuda")
    bias[low] = 2.0 + torch.arange(k, device="cuda") / 64
    ids, w = choice(y, Wr, k, bias=bias, score="sigmoid" if sigmoid else "softmax")
    assert torch.equal(ids, low.flip(0).expand(2, -1))
    z = (y.double() @ Wr.double().T).gather(1, ids)
    assert bool(((w - shares(z, sigmoid)).abs() <= (16 + k) * STEP * w).all())


def test_scores_that_are_not_numbers():
    """What the definition leaves without a value stays without one."""
    y, Wr = logits(1, 9, 1.0)
    Wr[3, 0] = math.nan
    for kw in (dict(bias=torch.zeros(9, device="cuda")), dict(renormalise=False)):
        ids, w = choice(y, Wr, 4, **kw)
        assert bool(torch.isnan(w).all()) and len(set(ids[0].tolist())) == 4
    ids, w = choice(y, Wr, 8, score="sigmoid")
    assert 3 not in ids[0].tolist() and bool(torch.isfinite(w).all())
    ids, w = choice(y, Wr, 9, score="sigmoid")
    assert ids[0, 8] == 3 and bool(torch.isnan(w).all())
