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


# ----------------------------------------------------------------------------- scores next to each other

def by_id(rank, k):
    return rank.sort(dim=-1, descending=True, stable=True).indices[:, :k]


@pytest.mark.parametrize("T,H,E,k", [(1, 256, 8, 2), (3, 1000, 33, 9), (2, 2560, 64, 8), (16, 2560, 128, 16), (1, 8200, 256, 8),
                                     (2, 4096, 200, 16)])
def test_logits_next_to_each_other(T, H, E, k):
    """Rows that differ in one weight, by a product so small that float32 sums (steps of 2^-14 and more) do not see it:
    logits of 2 H are d = H 2^-28 or more apart, where 32 products of a chain may be off by 2^-29 of their largest weight
    and value: H 2^-34 2 * 2 = d / 16, and 128 products of the one lane with weights of up to 199, 128 * 2^-34 * 199 * 2 at
    most a quarter of d (4096 2^-28; 32 in place of 199 at 1024 2^-28)."""
    y = 1.0 + torch.rand(T, H, generator=rng(5), device="cuda")
    Wr = (1.0 + torch.rand(1, H, generator=rng(6), device="cuda").mul_(0.99)).bfloat16().expand(E, -1).contiguous()
    order = torch.randperm(E, generator=rng(7), device="cuda")
    d = 2.0 ** (math.ceil(math.log2(H)) - 28)
    y[:, 7] = d * E
    Wr[:, 7] = (order.float() / E).bfloat16() if E & (E - 1) == 0 else order.bfloat16()
    if E & (E - 1):
        y[:, 7] = d
    assert torch.equal(Wr[:, 7].float() * y[0, 7], order.float() * d)  # exact
    for score in ("softmax", "sigmoid"):
        ids, w = choice(y, Wr, k, score=score)
        assert torch.equal(ids, order.argsort(descending=True)[:k].expand(T, -1))
    want = by_id(y.double() @ Wr.double().T, k)
    assert torch.equal(ids, want)


@pytest.mark.parametrize("T,H,E,k", [(16, 2560, 64, 8), (16, 1536, 80, 10), (16, 4096, 1024, 16), (16, 72, 300, 16), (5, 32768, 40, 16)])
def test_every_token_chooses_as_in_64_bits(T, H, E, k):
    """Logits off by 2^-34 H W Y at most: neighbours further apart keep their order, which leaves none out here."""
    y, Wr = normal(8, T, H), (normal(9, E, H) / math.sqrt(H)).bfloat16()
    z = y.double() @ Wr.double().T
    gap = z.sort(dim=-1, descending=True).values[:, :k + 1].diff(dim=-1).abs().min()
    off = 2.0 ** -34 * H * float(Wr.float().abs().max()) * float(y.abs().max())
    assert gap > 2 * off
    ids, w = choice(y, Wr, k)
    assert torch.equal(ids, by_id(z, k))
    p = torch.softmax(z, -1).gather(1, ids)
    p = p / p.sum(-1, keepdim=True)
    # a score's argument is rounded twice, its own and the sum's largest; two exponentials of 2 half steps, the sum of k, the
    # quotient and the factor; two logits each
    span = (z.amax(-1, keepdim=True) - z.gather(1, ids)).amax(-1, keepdim=True)
    assert bool(((w - p).abs() <= ((4 * span + 10 + k) * STEP + 4 * off) * p).all())


def test_large_small_and_unlike_values():
    """Sizes at which the sums' steps could be wrong: float32's borders, one large value among small ones, zeros."""
    E, k, H = 48, 8, 640
    Wr = (normal(10, E, H) / 8).bfloat16()
    for i, (ys, ws) in enumerate(((1e30, 1.0), (1e18, 1e18), (1e-30, 1.0), (1e-20, 1e-17), (1.0, 1e30), (1e36, 1e-36))):
        y = normal(11 + i, 2, H) * ys
        y[1, ::3] *= 1e-6
        w = (Wr.float() * ws).bfloat16()
        z = y.double() @ w.double().T
        if float(z.abs().max()) > 1e35:
            continue
        ids, _ = choice(y, w, k)
        assert torch.equal(ids, by_id(z, k)), i
    y = torch.zeros(1, H, device="cuda")
    assert choice(y, Wr, k)[0].tolist() == [list(range(k))]
    y[0, 5] = 1e-44  # the smallest floats: products below them are zero, equal ones by the lower id
    ids = choice(y, Wr, k)[0][0].tolist()
    assert len(set(ids)) == k


@pytest.mark.parametrize("E,k", [(12, 4), (64, 8), (200, 16), (700, 16)])
def test_sigmoids_next_to_one(E, k):
    """Logits of 18 to 28, whose sigmoids are 1 in float32, with a bias for all: the larger logit first."""
    y, Wr = torch.zeros(1, 8, device="cuda"), torch.zeros(E, 8, device="cuda")
    y[0, 0] = 1.0
    Wr[:, 0] = 18.0 + torch.randint(0, 81, (E,), generator=rng(20), device="cuda") / 8  # equal ones among them
    Wr = Wr.bfloat16()
    bias = torch.full((E,), 0.25, device="cuda")
    ids, w = choice(y, Wr, k, score="sigmoid", bias=bias, renormalise=False)
    z = Wr[:, 0].double()[None]
    assert torch.equal(ids, by_id(torch.sigmoid(z) + bias.double(), k))
    assert bool((w == 1.0).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(12, 4), (64, 8), (200, 16), (256, 3), (700, 16)])
def test_sums_with_a_bias_next_to_each_other(E, k, score):
    """p + bias within a step of float32 of one another: the order of 64 bits."""
    y, Wr = torch.zeros(2, 8, device="cuda"), torch.zeros(E, 8, device="cuda")
    y[:, 0] = 1.0
    Wr[:, 0] = normal(21, E)
    Wr = Wr.bfloat16()
    z = Wr[:, 0].double()
    p = torch.sigmoid(z) if score == "sigmoid" else torch.softmax(z, -1)
    bias = (0.75 - p).float()  # the rounding of the bias orders them
    rank = (p + bias.double())[None].expand(2, -1)
    assert float(rank[0].max() - rank[0].min()) < 2.0 ** -23
    best = rank[0].sort(descending=True).values[:k + 1]
    assert float(best.diff().abs().min()) > 1e-15 or bool((best.diff() == 0).any())  # or equal: by the lower id
    ids, w = choice(y, Wr, k, score=score, bias=bias)
    assert torch.equal(ids, by_id(rank, k))
