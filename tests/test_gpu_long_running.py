"""The long-cache attention kernels' running state: scores, and the scales of
4-bit values, that rise or fall from each unit of a warp to its next one, so
that sums are taken over to a new maximum at every step, in both launch shapes
and for every width of the groups; and sums of many values of one sign.

On 152 SMs the clusters' warps walk 8 units of 32 keys (4-bit) or 16 keys
(bf16) apart, the balanced runs' 4 or 8 units; a step of 256 or 128 keys so
meets each warp at every unit or two.  The scores' steps exceed the slack of 4
powers of two, up to which a maximum is kept.
"""
import math

import pytest
import torch

from test_gpu_blocks import check_attention as check_blocks
from test_gpu_kv4 import gd, i32  # noqa: F401
from test_gpu_kv4_value_scales import attend, normal, shape_of

pytestmark = pytest.mark.gpu

WIDTHS = [1, 4, 7, 16]


def steered(B, Hkv, G, S, D, step, rise, seed):
    """Queries and keys whose scores rise (or fall) by `rise` every `step` keys, about the same for a group's heads."""
    q = normal(seed, B, Hkv, 1, D) + 0.05 * normal(seed + 1, B, Hkv, G, D)
    mean = q.mean(2, keepdim=True)
    steps = torch.arange(S, device="cuda") // step
    want = ((steps if rise > 0 else steps.flip(0)) * abs(rise))[:, None] * math.sqrt(D)
    return q.flatten(1, 2), 0.2 * normal(seed + 2, B, Hkv, S, D) + want * mean / (mean ** 2).sum(-1, keepdim=True)


@pytest.mark.parametrize("G", WIDTHS)
@pytest.mark.parametrize("shape", ["clusters", "runs"])
@pytest.mark.parametrize("D,group", [(64, 32), (128, 32), (128, 64)])
@pytest.mark.parametrize("rise,grow", [(3.2, 0.0), (3.2, 1.0), (3.2, -1.0), (-3.2, 1.0), (0.5, 1.5)])
def test_4_bit_scores_and_scales_that_change_from_unit_to_unit(gd, D, group, shape, G, rise, grow):  # noqa: F811
    B, Hkv, S = shape_of(shape, G)
    q, k = steered(B, Hkv, G, S, D, 256, rise, 11)
    size = torch.exp2(grow * (torch.arange(S, device="cuda") // 256))
    attend(gd, q, k, normal(5, B, Hkv, S, D) * 1e-3 * size[:, None] / size.max().clamp(max=1e6), group, (rise, grow))


@pytest.mark.parametrize("G", WIDTHS)
@pytest.mark.parametrize("B,Hkv,n", [(5, 5, 116), (7, 8, 60)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rise", [3.2, -3.2])
def test_listed_blocks_with_scores_that_change_from_unit_to_unit(gd, D, B, Hkv, n, G, rise):  # noqa: F811
    if (B, Hkv) == (5, 5):  # as many as leave it to clusters
        n //= 1 if G <= 4 else 2 if G <= 8 else 4
    S = 64 * n
    q, k = steered(B, Hkv, G, S, D, 128, rise, 21)
    k, v = k.bfloat16(), normal(5, B, Hkv, S, D).bfloat16()
    pos = [S - 1 - 7 * b for b in range(B)]
    ids = torch.arange(n, dtype=torch.int32, device="cuda").expand(B, Hkv, n).contiguous()
    o = torch.full_like(q, float("nan"))
    gd.dec_block_decode_attn(q, k, v, i32(pos), ids, o)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 0
    check_blocks(q, k, v, pos, ids.tolist(), o)


@pytest.mark.parametrize("G", [4, 16])
@pytest.mark.parametrize("B,Hkv,S,D,group", [(1, 1, 131072, 64, 64), (7, 8, 9000, 128, 32), (5, 5, 1800, 128, 128)])
@pytest.mark.parametrize("kind", ["middles", "codes"])
def test_4_bit_values_of_one_sign_in_long_rows(gd, B, Hkv, S, D, group, G, kind):  # noqa: F811
    """Equal scores, so that A is zero beside 1 and the sums alone count: |o - exact| <= 2^-18 W.  Sums that the
    tensor core carried along whole rows were 4e-6 off (middles) or 3e-5 (codes that are not centred)."""
    q = torch.zeros(B, Hkv * G, D, device="cuda")
    v = normal(3, B, Hkv, S, D)
    if kind == "middles":  # constant groups
        v = (1.0 + v[..., :1].abs()).expand(-1, -1, -1, D).contiguous()
    else:  # codes of one sign per dim around a middle of about zero
        sign = torch.where(torch.arange(D, device="cuda") % 2 == 0, 1.0, -1.0)
        v = sign * (1.0 + 0.3 * torch.sin(v).abs())
    attend(gd, q, normal(2, B, Hkv, S, D), v, group, kind)


def test_listed_blocks_keep_24_bits_of_the_query(gd):  # noqa: F811
    """Two kinds of keys that meet one dim each, of values +1 and -1 and nearly equal scores X of 40 to 64:
    o = tanh(half their difference).  The query's three bf16 parts are exact, each product too (8 by 8 bits); a
    score's three additions and its scaling round by 2^-24 of it each, so o is off by 2^-22 X, and by 2^-20 for
    the exponentials (2^-22), their sums and the quotient.  Two parts would leave up to 2^-18 X in each score."""
    B, Hkv, D, S, G = 40, 2, 64, 128, 8
    q = torch.zeros(B, Hkv * G, D, device="cuda")
    x = 40.0 + 24.0 * torch.sin(normal(1, B, Hkv * G)).abs()
    q[..., 3] = x
    q[..., 50] = x + 0.1 * normal(2, B, Hkv * G)
    kind = (torch.arange(S, device="cuda") % 3 == 0)
    k = torch.zeros(B, Hkv, S, D, device="cuda")
    k[..., 3] = torch.where(kind, 8.0, 0.0)
    k[..., 50] = torch.where(kind, 0.0, 8.0)
    v = torch.where(kind, 1.0, -1.0)[:, None].expand(B, Hkv, S, D).bfloat16().contiguous()
    ids = torch.arange(2, dtype=torch.int32, device="cuda").expand(B, Hkv, 2).contiguous()
    o = torch.empty_like(q)
    gd.dec_block_decode_attn(q, k.bfloat16(), v, i32([S - 1] * B), ids, o)
    n = int(kind.sum())
    e = torch.exp(q[..., 50].double() - q[..., 3].double())
    want = ((n - (S - n) * e) / (n + (S - n) * e))[..., None]
    assert ((o.double() - want).abs() <= 2.0 ** -22 * 70.0 + 2.0 ** -20).all()
    assert gd.device_error(clear=True) == 0


def test_listed_blocks_keep_24_bits_of_the_probabilities(gd):  # noqa: F811
    """Two keys, one of value zero: o = p v / (1 + p) with p = exp(-x), x in (0, 1), v = 1.  Three bf16 parts hold
    p to 2^-24; x is off by 4 * 2^-24, the exponential by 2^-22, products, sums and the quotient by 2^-23 each:
    less than 2^-20 of o in all.  Two parts would leave up to 2^-18."""
    B, Hkv, D, S, G = 200, 2, 64, 64, 8
    q = torch.zeros(B, Hkv * G, D, device="cuda")
    q[..., 7] = torch.sin(normal(1, B, Hkv * G)).abs() * 0.99
    k = torch.zeros(B, Hkv, S, D, dtype=torch.bfloat16, device="cuda")
    k[:, :, 1, 7] = -8.0
    v = torch.zeros_like(k)
    v[:, :, 1] = 1.0
    o = torch.empty_like(q)
    gd.dec_block_decode_attn(q, k, v, i32([1] * B), torch.zeros(B, Hkv, 1, dtype=torch.int32, device="cuda"), o)
    p = torch.exp(-q[..., 7].double())
    want = (p / (1.0 + p))[..., None]
    assert ((o.double() - want).abs() <= 2.0 ** -20 * want).all()
    assert gd.device_error(clear=True) == 0
