"""Rows that dec_fp8_dequant writes lie apart: layouts in which two rows of
different matrices meet are refused on the host, interleaved ones are taken."""
import itertools

import pytest
import torch

P = 0x1000  # an aligned address; nothing is launched


@pytest.fixture(scope="module")
def gd():
    import greedy_decode_step_gb300 as gd
    gd.build()
    return gd


def meet(n, sm, rows, sr, K):
    at = sorted(i * sm + j * sr for i in range(n) for j in range(rows))
    return any(b - a < K for a, b in zip(at, at[1:]))


LAYOUTS = [(n, sm, rows, sr, 32) for n, rows in ((1, 3), (3, 1), (2, 2), (2, 5), (5, 2), (4, 7))
           for sm, sr in itertools.product((0, 16, 32, 48, 64, 80, 96, 128, 160, 224, 256), repeat=2)]


def test_layouts_whose_rows_meet(gd):
    """Every one that a list of all places shows to overlap; the others are not called here."""
    refused = [c for c in LAYOUTS if meet(*c)]
    assert 200 < len(refused) < len(LAYOUTS) - 200
    for n, sm, rows, sr, K in refused:
        rc = gd.lib().dec_fp8_dequant(P, P, P, 0, sm, sr, n, rows, K, 1, None)
        assert rc == gd.DEC_EINVAL and "share memory" in gd.lib().dec_last_error().decode(), (n, sm, rows, sr)


def test_many_rows_that_meet_once(gd):
    """Strides of 1,009 and 1,013 times 16: the 1,010th row of the first matrix is the 1,014th's first."""
    for n, sm, rows, sr in ((1010, 16 * 1013, 1014, 16 * 1009), (1014, 16 * 1009, 1010, 16 * 1013), (1 << 24, 1 << 28, 1 << 24, 1 << 28),
                           (1 << 24, 1 << 62, 1 << 24, 1 << 62)):
        assert gd.lib().dec_fp8_dequant(P, P, P, 1, sm, sr, n, rows, 16, 128, None) == gd.DEC_EINVAL


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layouts_whose_rows_lie_apart(gd, dtype):
    taken = [c for c in LAYOUTS if not meet(*c)]
    assert len(taken) > 200
    for n, sm, rows, sr, K in taken:
        x = torch.randn(n, rows, K, device="cuda")
        c, s = torch.zeros(n, rows, K, dtype=torch.uint8, device="cuda"), torch.zeros(n, rows, 1, device="cuda")
        gd.dec_fp8_quant(x, c, s)
        plain = torch.zeros(n, rows, K, device="cuda", dtype=dtype)
        gd.dec_fp8_dequant(c, s, plain)
        memory = torch.full(((n - 1) * sm + (rows - 1) * sr + K,), 7.0, device="cuda", dtype=dtype)
        out = memory.as_strided((n, rows, K), (sm, sr, 1))
        gd.dec_fp8_dequant(c, s, out)
        assert torch.equal(out, plain), (n, sm, rows, sr)
        out.fill_(7.0)
        assert bool((memory == 7.0).all())
