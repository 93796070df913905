"""Plain 64-bit forms of the long-cache operators (4-bit cache, block-sparse
attention), from their definitions, for the parity tests."""
from __future__ import annotations

import math

import torch

BLOCK = 64


def quantise(x: torch.Tensor, group: int):
    """Codes [..., D] (int64) and (s, z) [..., D/group, 2] (half) of float32 rows, by the
    definition's float32 operations on the CPU: bit for bit what the cache must hold."""
    x = x.detach().float().cpu()
    g = x.unflatten(-1, (-1, group))
    lo, hi = g.amin(-1), g.amax(-1)
    s = ((hi - lo) / 15.0).clamp(max=65504.0).half()
    z = (lo + 8.0 * s.float()).clamp(-65504.0, 65504.0).half()
    sf, zf = s.float()[..., None], z.float()[..., None]
    c = torch.where(sf > 0, torch.round((g - zf) / sf) + 8.0, torch.tensor(8.0)).clamp(0, 15)
    bad = ~torch.isfinite(g).all(-1)
    s = torch.where(bad, torch.tensor(float("nan"), dtype=torch.float16), s)
    z = torch.where(bad, torch.tensor(float("nan"), dtype=torch.float16), z)
    c = torch.where(bad[..., None], torch.tensor(8.0), c)
    return c.flatten(-2).long(), torch.stack((s, z), -1)


def pack(codes: torch.Tensor) -> torch.Tensor:
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8)


def unpack(codes: torch.Tensor) -> torch.Tensor:
    c = codes.long()
    return torch.stack((c & 15, c >> 4), -1).flatten(-2)


def values(codes: torch.Tensor, params: torch.Tensor) -> torch.Tensor:
    """What packed codes [..., D/2] with (s, z) [..., NG, 2] stand for, in float64."""
    c = unpack(codes).double() - 8.0
    p = params.double()
    return (p[..., 1:] + p[..., :1] * c.unflatten(-1, (p.shape[-2], -1))).flatten(-2)


def attention(q, k, v):
    """softmax(q k^T / sqrt(D)) v in float64 for q [G, D], k and v [n, D]; zeros without keys."""
    q, k, v = q.double(), k.double(), v.double()
    if k.shape[0] == 0:
        return torch.zeros_like(q)
    return torch.softmax(q @ k.T / math.sqrt(q.shape[-1]), -1) @ v


def bounds(k, last):
    """[NB, 2, D] largest and smallest value per dim of keys [S, D] up to slot `last`, blocks of 64."""
    nb = last // BLOCK + 1
    out = torch.empty(nb, 2, k.shape[-1], dtype=k.dtype, device=k.device)
    for j in range(nb):
        part = k[j * BLOCK:min(last + 1, (j + 1) * BLOCK)]
        out[j, 0], out[j, 1] = part.amax(0), part.amin(0)
    return out


def select(q, bd, n_select, n_first, n_last):
    """Blocks for q [G, D] and bounds [nb, 2, D]: forced ones, then by exact score, ties to the lower."""
    nb = bd.shape[0]
    if nb <= n_select:
        return list(range(nb))
    q, hi, lo = q.double().cpu(), bd[:, 0].double().cpu(), bd[:, 1].double().cpu()
    terms = torch.maximum(q[:, None] * hi, q[:, None] * lo)  # [G, nb, D]
    score = [math.fsum(terms[:, j].flatten().tolist()) if torch.isfinite(terms[:, j]).all() else
             float(terms[:, j].sum()) for j in range(nb)]
    score = [-math.inf if s != s else s for s in score]
    order = sorted(range(nb), key=lambda j: (not (j < n_first or j >= nb - n_last), -score[j], j))
    return sorted(order[:n_select])
