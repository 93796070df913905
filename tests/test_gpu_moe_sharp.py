"""The experts' layer held to the size its rounding errors have, and to every bit
where the result is exact (what these can tell: test_moe_bounds.py)."""
import pytest
import torch

import moe_refs as M
from test_gpu_moe import SIZES, choose, dirty, gd, make_weights, no_device_error, normal, rng  # noqa: F401

pytestmark = pytest.mark.gpu


def check(y, ids, w, held, scales, plain, residual=None):
    out = torch.full_like(y, float("nan"))
    gd.dec_moe_experts(y, ids, w, *held, out, residual=residual, scales=scales, ws=dirty(*ids.shape, y.shape[1], held[0].shape[1]))
    far = M.worst(out, *M.layer(y, ids, w, *plain, residual=residual), scales is not None)
    assert far <= 1.0, f"{far:.3g} times what the errors may be"
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,I,E,k", SIZES)
def test_experts(T, H, I, E, k, fp8):
    y = normal(20, T, H) * torch.exp(0.5 * normal(21, H))
    held, scales, plain = make_weights(22, E, H, I, fp8)
    ids, w = choose(30, T, k, E)
    check(y, ids, w, held, scales, plain)
    check(y, ids, w, held, scales, plain, residual=normal(31, T, H))


@pytest.mark.parametrize("H,I", [(264, 72), (1000, 360), (8, 8), (72, 200)])
def test_sizes_that_only_bf16_takes(H, I):
    for T in (1, 5):
        y = normal(40, T, H)
        held, scales, plain = make_weights(41, 7, H, I, False)
        ids, w = choose(42, T, 3, 7)
        check(y, ids, w, held, scales, plain)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 2, 3, 8, 9, 16])
@pytest.mark.parametrize("H,I,E,k", [(272, 208, 6, 3), (128, 64, 4, 1), (1536, 896, 20, 10), (2064, 144, 16, 16), (2560, 1216, 8, 2)])
def test_every_bit(T, H, I, E, k, fp8):
    y, ids, w, held, scales, want = M.every_bit(50 + T, T, H, I, E, k, fp8, "cuda")
    out = torch.zeros_like(y)
    gd.dec_moe_experts(y, ids, w, *held, out, scales=scales, ws=dirty(T, k, H, I))
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("H,I", [(264, 72), (1000, 360)])
@pytest.mark.parametrize("T", [2, 7])
def test_every_bit_at_sizes_that_only_bf16_takes(T, H, I):
    y, ids, w, held, scales, want = M.every_bit(70 + T, T, H, I, 6, 2, False, "cuda")
    out = torch.zeros_like(y)
    gd.dec_moe_experts(y, ids, w, *held, out, ws=dirty(T, 2, H, I))
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("fp8", [False, True])
def test_values_of_unlike_size(fp8):
    T, H, I, E, k = 12, 1024, 256, 6, 2
    y = normal(70, T, H)
    y[:, 100] *= 1e3
    y[1] *= 1e12
    y[2] *= 1e-15
    y[3] = 0.0
    y[4, 512:] = 0.0
    held, scales, plain = make_weights(71, E, H, I, fp8)
    ids, w = choose(72, T, k, E)
    check(y, ids, w, held, scales, plain)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [2, 16])
def test_particular_choices(T, fp8):
    H, I, E, k = 640, 272, 12, 4
    y = normal(50, T, H)
    held, scales, plain = make_weights(52, E, H, I, fp8)
    ids, w = choose(53, T, k, E)
    check(y, torch.full_like(ids, 11), w, held, scales, plain)  # one expert, every token four times
    twice = ids.clone()
    twice[:, 3] = twice[:, 0]
    check(y, twice, w, held, scales, plain)
    some = ids.clone()
    some[T - 1], some[0, 1:] = -1, -1
    assert not check(y, some, w, held, scales, plain)[T - 1].any()
    check(y, ids, -w, held, scales, plain)


@pytest.mark.parametrize("fp8", [False, True])
def test_weights_behind_2_to_the_31(fp8):
    """The last experts' matrices begin behind 2^31 elements; another expert's in their place would show."""
    T, H, I, E, k = 3, 8192, 8192, 40, 2
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    held = [torch.empty(E, *s, device="cuda", dtype=dt) for s in ((I, H), (I, H), (H, I))]
    scales = tuple(torch.rand(E, 64, 64, generator=rng(90), device="cuda") + 0.5 for _ in range(3)) if fp8 else None
    ids = torch.tensor([[39, 37], [38, 39], [0, 39]], dtype=torch.int32, device="cuda")
    for e in (0, 37, 38, 39):
        for i in range(3):
            held[i][e] = (0.02 * normal(91 + i + 3 * e, *held[i].shape[1:])).to(dt)
    y, w = normal(95, T, H), torch.rand(T, k, generator=rng(96), device="cuda")
    check(y, ids, w, held, scales, list(zip(held, scales)) if fp8 else held)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 2, 3, 16])
@pytest.mark.parametrize("I", [16, 64, 320])
def test_no_expert_at_all(T, I, fp8):
    """Inner vectors of less than one chunk, one and several, and nothing to compute of them."""
    H, E, k = 272, 5, 3
    y, res = normal(60, T, H), normal(61, T, H)
    held, scales, plain = make_weights(62, E, H, I, fp8)
    ids, w = torch.full((T, k), -1, dtype=torch.int32, device="cuda"), torch.rand(T, k, device="cuda")
    assert torch.equal(check(y, ids, w, held, scales, plain, res), res)
    assert not check(y, ids, w, held, scales, plain).any()
    ids[T - 1, 1] = 4  # and one expert of one token
    check(y, ids, w, held, scales, plain)
