"""Plain 64-bit forms of the 8-bit weight operators and of the mixture-of-experts
layer, from their definitions, with bounds of what fp32 arithmetic may add."""
from __future__ import annotations

import math

import torch

BLOCK = 128
TOP = 448.0


def grid(v: torch.Tensor) -> torch.Tensor:
    """Nearest e4m3 values (float64 in and out, |v| <= 448), ties to even; NaN stays."""
    a = v.abs()
    e = torch.frexp(a)[1] - 1  # a = 1.x 2^e
    step = torch.exp2(e.clamp(min=-6).double() - 3)
    return torch.round(v / step) * step  # torch.round: half to even


def blocks(x: torch.Tensor, rows: int):
    for i in range(0, x.shape[0], rows):
        for j in range(0, x.shape[1], BLOCK):
            yield slice(i, i + rows), slice(j, j + BLOCK)


def quantise(x: torch.Tensor, rows: int):
    """What codes of a matrix stand for before scaling, and scales [ceil(R / rows), ceil(K / 128)], float64."""
    x = x.detach().double().cpu()
    codes = torch.empty_like(x)
    scales = torch.empty(-(-x.shape[0] // rows), -(-x.shape[1] // BLOCK), dtype=torch.float64)
    for a, b in blocks(x, rows):
        part = x[a, b]
        fin = part[torch.isfinite(part)].abs()
        top = float(fin.max()) if fin.numel() else 0.0
        s = 1.0
        if top > 0:
            s = 2.0 ** max(-126, math.frexp(top / TOP)[1] - 1)
            while top > TOP * s:
                s *= 2
        scales[a.start // rows, b.start // BLOCK] = s
        codes[a, b] = grid(torch.where(torch.isfinite(part), part, math.nan) / s)
    return codes, scales


def spread(scales: torch.Tensor, R: int, K: int, rows: int) -> torch.Tensor:
    return scales.double().repeat_interleave(rows, -2)[..., :R, :].repeat_interleave(BLOCK, -1)[..., :K]


def held(codes: torch.Tensor, scales: torch.Tensor, rows: int) -> torch.Tensor:
    """Codes (float8_e4m3fn) times scales, float64, on their device."""
    return codes.float().double() * spread(scales, codes.shape[-2], codes.shape[-1], rows)


# What a tensor-core sum may lose: the addends of one instruction (its products
# and the running sum) are aligned to the largest of them and cut below its
# 24th bit, each by less than 2^-23 of the largest, which no running sum's
# total of magnitudes falls short of.
CUT = 2.0 ** -23
STEP = 2.0 ** -24  # half a step of float32


def gemm(xc, xs, wc, ws, residual=None):
    """x w^T in float64 and the bound of an fp32 result's error."""
    x, w = held(xc, xs, 1), held(wc, ws, BLOCK)
    out, size = x @ w.T, x.abs() @ w.abs().T
    # four instructions of 32 products a block, then one product of scales and one fma per block
    kb = -(-xc.shape[1] // BLOCK)
    bound = size * (4 * 33 * CUT + (kb + 2) * STEP)
    if residual is not None:
        out = out + residual.double()
        bound = bound + out.abs() * STEP + size * STEP
    return out, bound + 1e-40


def route(y, Wr, k, bias=None, sigmoid=False, renormalise=True, scale=1.0):
    """ids [T, k], weights (float64) and the gap between neighbours of the ranking, per token."""
    z = y.double() @ Wr.double().T
    p = torch.sigmoid(z) if sigmoid else torch.softmax(z, -1)
    rank = z if bias is None else p + bias.double()
    rank = torch.where(torch.isnan(rank), -math.inf, rank)
    order = rank.sort(dim=-1, descending=True, stable=True)
    ids = order.indices[:, :k]
    w = p.gather(1, ids)
    if renormalise:
        w = w / w.sum(-1, keepdim=True)
    gaps = order.values[:, :k + 1].diff(dim=-1).abs()
    return ids, w * scale, gaps


def experts(y, ids, gates, wg, wu, wd, residual=None):
    """The layer in float64 and the bound of an fp32 result's error; weights are tensors [E, ., .] or lists
    (fp8: pairs of codes and scales)."""
    def matrix(w, e):
        return held(w[0][e], w[1][e], BLOCK) if isinstance(w, (tuple, list)) else w[e].double()

    T, H = y.shape
    out = torch.zeros(T, H, dtype=torch.float64, device=y.device) if residual is None else residual.double().clone()
    bound = torch.zeros_like(out)
    E = (wg[0] if isinstance(wg, (tuple, list)) else wg).shape[0]
    n = 0
    for t in range(T):
        v = y[t].double()
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            g, u, d = matrix(wg, e), matrix(wu, e), matrix(wd, e)
            a, b = g @ v, u @ v
            # parts of an element: 2^-24 of it (bf16) or 2^-23 of its 128 (e4m3: taken as if of the row's largest);
            # instructions of 16 products, H / 16 of them one behind the other
            size = v.abs() + v.abs().max() * 2.0 ** -4
            da = (g.abs() @ size) * (H * 17 / 16 + 64) * CUT
            db = (u.abs() @ size) * (H * 17 / 16 + 64) * CUT
            w = float(gates[t, j])
            s = torch.sigmoid(a)
            h = a * s * b
            # |silu'| < 1.1; expf, the quotient and two products: a few steps
            dh = 1.1 * da * b.abs() + (a * s).abs() * db + 1.1 * da * db + h.abs() * 16 * STEP
            inner = h.abs() + h.abs().max() * 2.0 ** -4
            out[t] += w * (d @ h)
            bound[t] += abs(w) * (d.abs() @ dh)
            bound[t] += abs(w) * (d.abs() @ inner) * (17 / 16 * (wd[0] if isinstance(wd, (tuple, list)) else wd).shape[2] + 64) * CUT
            n += 1
    bound = bound * (1 + ids.shape[1]) + (out.abs() + 1) * 2 * STEP  # sums run over all chosen experts' columns
    return out, bound
