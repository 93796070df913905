"""Attention over the 4-bit cache where groups of a query are far smaller than
others and the keys' offsets are large there, so that they decide the scores.

The bound of the attention tests goes by A, the sum of the terms' magnitudes
|q| (|z| + 16 s) over sqrt(D).  The query is held as two half parts under a
power of two per head, which leave 2^-24 beside a largest element of at least
2^14: 2^-38 of it, and as much for a group's mean, which is group * 2^-38 of
it, 2^-33 at 32 dims, for the sum that meets z.  The tests' small groups have
one dim that is not zero, 2^-14 of the head's largest or more, so that A is at
least 2^-14 of that largest one times |z| / sqrt(D), and a sum's error at most
2^-33 / 2^-14 = 2^-19 of A: within the bound's 2^-18.  (A sum held to 2^-28
would be off by up to 2^-14 of A.)
"""
import pytest
import torch

from test_gpu_kv4 import gd  # noqa: F401
from test_gpu_kv4_value_scales import SHAPES, attend, normal, shape_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("G", [1, 4, 8, 11, 16])
def test_small_groups_that_meet_large_offsets(gd, G, shape):  # noqa: F811
    """Two small groups whose terms nearly cancel, against keys of +z and -z whose values are +1 and -1: an error
    of a sum moves the two kinds of keys apart, and o by half of that."""
    D, (B, Hkv, S) = 128, shape_of(shape, G)
    q = torch.zeros(B, Hkv, G, D, device="cuda")
    q[..., 64:] = normal(3, B, Hkv, G, 64).clamp(-1.0, 1.0) * 256.0
    q[..., 70] = 256.0
    q[..., 5] = (1.0 + 0.9 * torch.sin(normal(4, B, Hkv, G)).abs()) * 2.0 ** -6
    q[..., 40] = -q[..., 5] * (1.0 + 0.01 * normal(6, B, Hkv, G))
    sign = torch.where(normal(7, B, Hkv, S, 1) > 0, 1.0, -1.0)
    k = torch.zeros(B, Hkv, S, D, device="cuda")
    k[..., :64] = sign * 2.0 ** 14
    attend(gd, q.flatten(1, 2), k, sign.expand(-1, -1, -1, D).contiguous(), 32, "small groups")


def test_a_query_of_zeros_and_one_of_a_single_dim(gd):  # noqa: F811
    B, Hkv, S, D = 3, 2, 300, 128
    q = torch.zeros(B, Hkv, 4, D, device="cuda")
    q[:, :, 1, 70] = 1e-8
    q[:, :, 2, 3] = 1e8
    q[:, :, 3] = normal(3, B, Hkv, D)
    k = normal(1, B, Hkv, S, D)
    k[..., 3] *= 1e-7
    attend(gd, q.flatten(1, 2), k, normal(2, B, Hkv, S, D), 32, "zeros")
