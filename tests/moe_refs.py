"""The experts' layer in 64 bits beside the size that its rounding errors have,
and a case whose result is exact only if every bit of the activations is kept.

The kernels add 128 bytes of K in the tensor core (four instructions of 16
bf16 or 32 e4m3 products, each addend cut below the 24th bit of the largest) and
everything else in float32.  Taken as independent, the cuts of a chunk, each
uniform up to 2^-23 of a sum that is at most twice the root of the sum of squares
of its products, add up to

    eps = sqrt(4 (n + 1) / 3) 2 2^-23        n = 16: 1.1e-6, n = 32: 1.6e-6

of that root, and so do those of all chunks of a row.  A row's error is held
against eps times its root of the sum of squares, carried through the layer
as errors are, and a token's errors are compared as a whole (root of the mean
square): one value that is wrong, a chunk, an expert or a scale left out shows.
"""
from __future__ import annotations

import math

import torch

import fp8_refs as R


def eps(fp8: bool) -> float:
    n = 32 if fp8 else 16
    return math.sqrt(4 * (n + 1) / 3) * 2 * 2.0 ** -23


def matrix(w, e):
    return R.held(w[0][e], w[1][e], R.BLOCK) if isinstance(w, (tuple, list)) else w[e].double()


def same(v):
    return v


def layer(y, ids, gates, wg, wu, wd, residual=None, outer=same, inner=same):
    """(result, size of its errors over eps), float64.  Weights: tensors [E, ., .] or pairs of codes and scales;
    `outer` and `inner` stand for what holds y and the inner vectors."""
    fp8 = isinstance(wg, (tuple, list))
    E = (wg[0] if fp8 else wg).shape[0]
    T, H = y.shape
    out = torch.zeros(T, H, dtype=torch.float64, device=y.device)
    size = torch.zeros_like(out)

    def squares(m, v):
        """Sum of squares of the products of a row; 8-bit weights: v is held to 2^-23 of the largest of 128."""
        s = (m * m) @ (v * v)
        if fp8:
            top = torch.nn.functional.pad(v.abs(), (0, -v.numel() % 128)).view(-1, 128).amax(-1).repeat_interleave(128)[:v.numel()]
            s = s + (m * m) @ (top * top) * (2.0 ** -23 / math.sqrt(3) / eps(True)) ** 2
        return s

    for t in range(T):
        v = outer(y[t].double())
        for j in range(ids.shape[1]):
            e = int(ids[t, j])
            if not 0 <= e < E:
                continue
            g, u, d = matrix(wg, e), matrix(wu, e), matrix(wd, e)
            w = float(gates[t, j])
            a, b = g @ v, u @ v
            act = a * torch.sigmoid(a)
            h = w * act * b
            # |silu'| < 1.1; an exponential, a quotient and two products: less than eps
            errors = w * w * (1.21 * b * b * squares(g, v) + act * act * squares(u, v)) + h * h
            h = inner(h)
            out[t] += d @ h
            size[t] += (d * d) @ errors + squares(d, h)
    size = size + out * out  # the sums over the launch's parts, in float32
    if residual is not None:
        out = out + residual.double()
        size = size + out * out
    return out, size.sqrt()


def worst(got, want, size, fp8: bool) -> float:
    """The largest ratio, over the tokens, of the errors' root mean square to what it may be: 1 at most."""
    err = (got.double() - want).square().mean(-1).sqrt()
    may = eps(fp8) * size.square().mean(-1).sqrt() + 1e-40
    r = err / may
    return float(torch.where(torch.isnan(r), math.inf, r).max())


# ----------------------------------------------------------------------------- activations in parts, as mistakes have them

def bf16_parts(n):
    def hold(v):
        left, sum_ = v.clone(), torch.zeros_like(v)
        for _ in range(n):
            p = left.float().bfloat16().double()
            sum_, left = sum_ + p, left - p
        return sum_
    return hold


def e4m3_parts(n):
    def hold(v):
        x = torch.nn.functional.pad(v, (0, -v.numel() % 128)).view(-1, 128)
        top = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
        s = torch.exp2(torch.ceil(torch.log2(top / 224)))
        left, sum_ = x / s, torch.zeros_like(x)
        for i in range(n):
            p = R.grid(left.clamp(-448, 448))
            sum_, left = sum_ + p * 32.0 ** -i, (left - p) * 32
        return (sum_ * s).flatten()[:v.numel()]
    return hold


# ----------------------------------------------------------------------------- a case that needs every bit

def every_bit(seed, T, H, I, E, k, fp8, device="cpu"):
    """y: +-[1, 1.75) with 23 bits behind the point.  A gate row has one weight, of a value that is 1, and is 128, where
    silu is its argument in float32; an up row and a down row have one weight each, a power of two; an expert's down
    rows are those of its own class of k, and every token takes one expert of each class.  So each result is one y times
    a power of two, all 24 bits of it.  Returns y, ids, gates, weights, scales (None: bf16) and the result."""
    g = torch.Generator().manual_seed(seed)

    def ints(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=g)

    y = (1 + ints(0, 3 * 2 ** 21 - 1, T, H).double() * 2.0 ** -23) * (1 - 2 * ints(0, 1, T, H))
    y[:, 0] = 1.0
    ids = torch.stack([k * ints(0, E // k - 1, k) + torch.arange(k) for _ in range(T)]).int()  # a class each
    gates = torch.exp2(ints(-2, 2, T, 1).double()).expand(T, k).contiguous()
    wg, wu, wd = torch.zeros(E, I, H), torch.zeros(E, I, H), torch.zeros(E, H, I)
    wg[:, :, 0] = 128.0
    from_y = ints(0, H - 1, E, I)
    sign_u, sign_d = 1.0 - 2 * ints(0, 1, E, I), 1.0 - 2 * ints(0, 1, E, H)
    wu.scatter_(2, from_y[..., None], sign_u[..., None])
    from_h = ints(0, I - 1, E, H)
    wd.scatter_(2, from_h[..., None], (sign_d * ((torch.arange(H) % k)[None] == (torch.arange(E) % k)[:, None]))[..., None])
    scales = None
    if fp8:
        scales = tuple(torch.exp2(ints(-3, 3, E, -(-w.shape[1] // 128), 1).double()).expand(-1, -1, -(-w.shape[2] // 128)).contiguous()
                       for w in (wg, wu, wd))
        scales = (torch.ones_like(scales[0]), torch.ones_like(scales[1]), scales[2])
    want = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            h = 128.0 * gates[t, j] * sign_u[e].double() * y[t][from_y[e]]
            o = sign_d[e].double() * h[from_h[e]]
            if fp8:
                o = o * scales[2][e].repeat_interleave(128, 0)[:H, 0]
            mine = torch.arange(H) % k == e % k
            want[t][mine] += o[mine]
    assert torch.equal(want.float().double(), want) and torch.equal(y.float().double(), y)
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    to = lambda x: x.to(device)
    return (to(y.float()), to(ids), to(gates.float()), [to(w.to(dt)) for w in (wg, wu, wd)],
            None if scales is None else tuple(to(s.float()) for s in scales), to(want))
