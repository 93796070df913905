"""What the experts' tests can tell: results with a mistake planted, computed in
64 bits on the CPU, against the size that the kernels' errors may have."""
import pytest
import torch

import fp8_refs as R
import moe_refs as M


def case(seed, T, H, I, E, k, fp8):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)
    y = n(T, H) * torch.exp(0.5 * n(H))
    ws = []
    for a, b in ((I, H), (I, H), (H, I)):
        w = (0.05 * n(E, a, b) * torch.exp(0.3 * n(E, a, 1))).bfloat16()
        if fp8:
            s = torch.rand(E, -(-a // 128), -(-b // 128), generator=g) * 1e-3 + 1e-3
            w = ((w.float() / torch.stack([R.spread(s[e], a, b, 128).float() for e in range(E)])).clamp(-448, 448).to(torch.float8_e4m3fn), s)
        ws.append(w)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(T)]).int()
    return y, ids, torch.rand(T, k, generator=g), ws


def without(w, cols):
    """The weights with some columns left out."""
    if isinstance(w, tuple):
        c = w[0].view(torch.uint8).clone()
        c[:, :, cols] = 0
        return c.view(torch.float8_e4m3fn), w[1]
    w = w.clone()
    w[:, :, cols] = 0
    return w


SIZES = [(16, 1536, 896, 12, 10), (2, 2560, 1216, 4, 2), (4, 1536, 896, 4, 3), (1, 4096, 64, 3, 1), (1, 16, 16, 2, 1), (3, 272, 144, 5, 2)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,I,E,k", SIZES)
def test_mistakes_show(T, H, I, E, k, fp8):
    y, ids, w, ws = case(1, T, H, I, E, k, fp8)
    want, size = M.layer(y, ids, w, *ws)
    far = lambda *a, **kw: M.worst(M.layer(*a, **kw)[0], want, size, fp8)
    assert M.worst(want.float(), want, size, fp8) < 0.1
    whole = M.e4m3_parts(5) if fp8 else M.bf16_parts(3)
    assert far(y, ids, w, *ws, outer=whole, inner=whole) < 0.5  # the activations as they are held
    assert M.worst(torch.zeros_like(want), want, size, fp8) > 100
    one = want.clone()
    one[T - 1, H // 2] += 0.1 * want[T - 1].square().mean().sqrt()
    assert M.worst(one, want, size, fp8) > 100
    last = slice(H - 64 if H > 64 else H // 2, H)
    assert far(y, ids, w, without(ws[0], last), *ws[1:]) > 100
    assert far(y, ids, w, ws[0], without(ws[1], last), ws[2]) > 100
    assert far(y, ids, w, *ws[:2], without(ws[2], slice(I // 2, I // 2 + 8))) > 100
    less = ids.clone()
    less[T - 1, k - 1] = -1
    assert far(y, less, w, *ws) > 100
    other = (ids + 1) % E
    assert far(y, other, w, *ws) > 100
    assert far(y, ids, w.roll(1, 0) * 1.001, *ws) > 100
    rough = M.e4m3_parts(1) if fp8 else M.bf16_parts(1)
    assert far(y, ids, w, *ws, outer=rough) > 20 and far(y, ids, w, *ws, inner=rough) > 20
    if fp8:
        scaled = (ws[2][0], ws[2][1] * (1 + 2.0 ** -8))
        assert far(y, ids, w, *ws[:2], scaled) > 100


@pytest.mark.parametrize("fp8", [False, True])
def test_a_part_less_shows(fp8):
    y, ids, w, ws, scales, want = M.every_bit(3, 4, 272, 208, 6, 3, fp8)
    plain = list(zip(ws, scales)) if fp8 else ws
    def got(parts_outer, parts_inner):
        hold = M.e4m3_parts if fp8 else M.bf16_parts
        return M.layer(y, ids, w, *plain, outer=hold(parts_outer), inner=hold(parts_inner))[0]
    n = 5 if fp8 else 3
    full = got(n, n)
    assert float(((full - want) / want).abs().max()) < 2.0 ** -40  # silu(128) is 128 (1 - 2.6e-56)
    for a, b in ((n - 1, n), (n, n - 1)):
        off = got(a, b).float().double() != want
        assert float(off.double().mean()) > 0.5
