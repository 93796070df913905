"""Attention over the 4-bit cache where the V scales of one row spread widely:
between the groups of a key, between keys, and between stretches of a row.

The cache holds any half scale next to any other, and an output dim is a sum
over its own group only, so the bound of the attention tests,
  |o - exact| <= 2^-18 (1 + A) W,  W = sum_j p_j (|z_j| + 8 s_j),
holds dim by dim whatever the other groups' scales are, and whatever the scale
of a key that has next to no probability.  The smallest normal half operand
leaves 2^-25 of the largest one, so an arithmetic that holds scales as halves
under one factor fails it from a spread of about 2^14 on.
"""
import math

import pytest
import torch

from test_gpu_kv4 import check_attention, empty_cache, gd, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def shape_of(name, G):
    """Rows, KV heads and slots that (on 152 SMs) the launch gives to clusters whose warps take one unit of 32
    keys, to clusters whose warps take several, and to the balanced runs."""
    nt = 1 if G <= 4 else 2 if G <= 8 else 4
    return {"short": (2, 1, 256), "clusters": (5, 5, 7400 // nt), "runs": (7, 8, 4500)}[name]


SHAPES = ["short", "clusters", "runs"]


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda")


def attend(gd, q, k, v, group, what):  # noqa: F811
    """The call on a cache of the rows k, v [B, Hkv, S, D], checked against the definition."""
    B, Hkv, S, D = k.shape
    pos = [S - 1 - 7 * b for b in range(B)]
    cache = empty_cache(B, Hkv, S, D, group)
    gd.dec_kv4_store(k.transpose(1, 2), v.transpose(1, 2), i32([0] * B), *cache)
    o = torch.full_like(q, float("nan"))
    gd.dec_kv4_decode_attn(q, *cache, i32(pos), o)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 0
    check_attention(gd, q, cache, pos, o, what)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("D,group,G,sizes", [
    (64, 32, 1, (1.0, 1e-3)), (64, 32, 4, (10.0, 1e-4)), (64, 32, 8, (1e-5, 1000.0)),
    (128, 32, 4, (1e3, 1e-5, 1.0, 30.0)), (128, 64, 2, (1e-4, 100.0)), (128, 32, 16, (1e-5, 1e-2, 10.0, 1e4)),
    (128, 64, 7, (5e3, 1e-5)), (128, 32, 4, (0.0, 1.0, 0.0, 1e-4)), (128, 64, 16, (1.0, 0.0)), (64, 64, 2, (0.0,))])
def test_groups_of_unlike_scale(gd, D, group, G, sizes, shape):  # noqa: F811
    B, Hkv, S = shape_of(shape, G)
    k, v, q = normal(1, B, Hkv, S, D), normal(2, B, Hkv, S, D), normal(3, B, G * Hkv, D)
    attend(gd, q, k, v * torch.tensor(sizes, device="cuda").repeat_interleave(group), group, sizes)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("D,group,G", [(64, 64, 4), (128, 32, 4), (128, 128, 8), (128, 64, 16)])
@pytest.mark.parametrize("ratio", [2.0 ** 9, 2.0 ** 20])
def test_keys_that_nobody_attends_to(gd, D, group, G, ratio, shape):  # noqa: F811
    """One key in every 256 has values `ratio` times the others' and a probability below 2^-30."""
    B, Hkv, S = shape_of(shape, G)
    k, v = normal(1, B, Hkv, S, D), normal(2, B, Hkv, S, D) * 0.02
    q = normal(3, B, Hkv, 1, D) + 0.2 * normal(4, B, Hkv, G, D)
    mean = q.mean(2, keepdim=True)
    out = torch.arange(5, S, 256, device="cuda")
    # a score of about -30 from every head of the group, where the others' lie a few around zero
    k[:, :, out] = -30.0 * math.sqrt(D) * mean / (mean ** 2).sum(-1, keepdim=True)
    v[:, :, out] *= ratio
    attend(gd, q.flatten(1, 2), k, v, group, ratio)


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("D,group,G", [(64, 32, 4), (128, 32, 2), (128, 64, 8), (128, 128, 16)])
def test_scales_that_rise_and_fall_along_the_row(gd, D, group, G, shape):  # noqa: F811
    """The values' size runs up and down by 2^22 every 2048 keys, every other group's by half as much against
    them; scores fall by 11 powers of two where the values of the first group are largest."""
    B, Hkv, S = shape_of(shape, G)
    t = torch.arange(S, device="cuda")
    wave = 22.0 * (1.0 - (t % 2048 - 1024).abs() / 1024.0)  # 0 .. 22 .. 0, in powers of two
    k, v = 0.5 * normal(1, B, Hkv, S, D), normal(2, B, Hkv, S, D) * 1e-3
    q = normal(3, B, Hkv, 1, D) + 0.1 * normal(4, B, Hkv, G, D)
    mean = q.mean(2, keepdim=True)
    k += (-0.5 * math.log(2.0) * wave * math.sqrt(D))[:, None] * mean / (mean ** 2).sum(-1, keepdim=True)
    against = torch.arange(D, device="cuda") // group % 2 == 1
    v *= torch.exp2(torch.where(against[None, :], 11.0 - 0.5 * wave[:, None], wave[:, None]))
    attend(gd, q.flatten(1, 2), k, v, group, "wave")


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("D,group,G", [(64, 32, 3), (128, 32, 4), (128, 64, 8), (128, 128, 12), (128, 32, 16)])
def test_every_key_and_group_of_a_scale_of_its_own(gd, D, group, G, shape):  # noqa: F811
    """Sizes of 2^-24 to 2^12 at random, so that the 32 keys of a unit share nothing; constant groups (a scale of
    zero) among them, and scores that fall as the first group's values grow."""
    B, Hkv, S = shape_of(shape, G)
    NG = D // group
    g = torch.Generator("cuda").manual_seed(5)
    e = torch.rand(B, Hkv, S, NG, 1, generator=g, device="cuda") * 36.0 - 24.0
    v = normal(2, B, Hkv, S, D).unflatten(-1, (NG, group)) * torch.exp2(e)
    flat = torch.rand(B, Hkv, S, NG, 1, generator=g, device="cuda") < 0.1
    v = torch.where(flat, v[..., :1], v).flatten(-2)
    q = normal(3, B, Hkv, 1, D) + 0.1 * normal(4, B, Hkv, G, D)
    mean = q.mean(2, keepdim=True)
    k = 0.3 * normal(1, B, Hkv, S, D)
    k -= 0.3 * math.log(2.0) * math.sqrt(D) * e[:, :, :, 0] * mean / (mean ** 2).sum(-1, keepdim=True)
    attend(gd, q.flatten(1, 2), k, v, group, "random")
