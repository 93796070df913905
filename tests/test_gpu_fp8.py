"""8-bit rows and weights (dec_fp8_quant, dec_fp8_dequant, dec_fp8_gemm)
against their definitions in 64 bits."""
import math

import pytest
import torch

import fp8_refs as R

pytestmark = pytest.mark.gpu
gd = pytest.importorskip("greedy_decode_step_gb300")


@pytest.fixture(autouse=True)
def no_device_error():
    gd.lib()
    gd.device_error(clear=True)
    yield
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 0


def rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(seed, *shape):
    return torch.randn(shape, generator=rng(seed), device="cuda")


def empty_codes(x, rows, fill=0x55):
    c = torch.full(x.shape, fill, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    s = torch.full((*x.shape[:-2], -(-x.shape[-2] // rows), -(-x.shape[-1] // 128)), -1.0, device="cuda")
    return c, s


def check_quant(x, rows):
    c, s = empty_codes(x, rows)
    gd.dec_fp8_quant(x, c, s, block_rows=rows)
    mats = [(x, c, s)] if x.dim() == 2 else [(x[i], c[i], s[i]) for i in range(x.shape[0])]
    for xm, cm, sm in mats:
        want, scale = R.quantise(xm, rows)
        assert torch.equal(sm.double().cpu(), scale)
        got = cm.float().double().cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(want, nan=0.0))
    return c, s


# ----------------------------------------------------------------------------- quantiser

@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 16), (3, 48), (128, 128), (130, 144), (257, 640), (16, 2560), (700, 2048), (3, 200, 272)])
def test_quantised_values(shape, dtype, rows):
    x = (normal(1, *shape) * torch.exp(2.0 * normal(2, *shape[:-1], 1))).to(dtype)
    check_quant(x, rows)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_values_at_borders(dtype, rows):
    """Ties between codes, magnitudes around 448 s and 2^-9 s, zeros, the smallest and largest floats, infinities, NaN."""
    x = torch.zeros(16, 128, device="cuda")
    ties = torch.tensor([17.0, 19.0, 21.0, 2.125, 2.375, 0.0009765625, 0.0029296875, 0.0048828125], device="cuda")
    for i, top in enumerate((448.0, 447.9, 448.0 * (1 + 2 ** -7), 449.0, 1.75 * 2.0 ** -40, 1.7578125 * 2.0 ** 30, 256.0, 1e-38,
                             3e38, 0.0, 2.0 ** -149, 2.0 ** -126 * 448, 1.0)):
        x[i, 0] = top
        if top > 0:
            x[i, 1:9] = ties * 2.0 ** (math.frexp(top)[1] - 9)
            x[i, 9:17] = -x[i, 1:9]
            x[i, 17] = top * 2.0 ** -19
    x[13, 3], x[13, 4], x[13, 5], x[13, 6] = math.inf, -math.inf, math.nan, 5.0
    x[14] = math.nan
    x[15, 0], x[15, 1] = -3.38e38, 1e-45
    check_quant(x.to(dtype), rows)
    for i in range(16):
        check_quant(x[i:i + 1].to(dtype), rows)


@pytest.mark.parametrize("rows", [1, 128])
def test_rows_given_as_views(rows):
    wide = normal(3, 4, 150, 3 * 272)
    check_quant(wide[:, :, 272:544], rows)
    check_quant(wide[:, ::3, :272], rows)
    check_quant(wide[2, 5:133, 544:], rows)
    check_quant(wide[0, 7].expand(130, -1)[:, :272], rows)  # one row, repeated
    check_quant(wide[1].bfloat16()[:, 16:160], rows)


@pytest.mark.parametrize("rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(1, 16), (130, 144), (3, 200, 272), (700, 2048)])
def test_read_back(shape, dtype, rows):
    x = normal(4, *shape)
    c, s = empty_codes(x, rows)
    gd.dec_fp8_quant(x, c, s, block_rows=rows)
    s *= torch.rand(s.shape, generator=rng(5), device="cuda") - 0.3  # any scales, negative ones and all
    pad = torch.full((*shape[:-2], shape[-2] + 2, shape[-1] + 16), 7.0, device="cuda", dtype=dtype)
    out = pad[..., 1:-1, :shape[-1]]
    gd.dec_fp8_dequant(c, s, out, block_rows=rows)
    want = (c.float() * R.spread(s, shape[-2], shape[-1], rows).float()).to(dtype)
    assert torch.equal(out, want)
    out.fill_(7.0)
    assert bool((pad == 7.0).all())  # nothing around it was written


def test_every_code_reads_back():
    c = torch.arange(256, dtype=torch.uint8, device="cuda").view(2, 128).view(torch.float8_e4m3fn)
    s = torch.tensor([[0.25], [2.0 ** -20]], device="cuda")
    out = torch.zeros(2, 128, device="cuda")
    gd.dec_fp8_dequant(c, s, out)
    assert torch.equal(torch.nan_to_num(out, nan=9e9), torch.nan_to_num(c.float() * s, nan=9e9))


# ----------------------------------------------------------------------------- product

def operands(seed, M, N, K, odd_scales=True):
    x, w = normal(seed, M, K) * torch.exp(normal(seed + 1, K)), 0.05 * normal(seed + 2, N, K)
    xc, xs = empty_codes(x, 1)
    wc, ws = empty_codes(w, 128)
    gd.dec_fp8_quant(x, xc, xs)
    gd.dec_fp8_quant(w, wc, ws, block_rows=128)
    if odd_scales:
        ws *= torch.rand(ws.shape, generator=rng(seed + 3), device="cuda") + 0.5
        xs *= torch.rand(xs.shape, generator=rng(seed + 4), device="cuda") - 0.4
    return xc, xs, wc, ws


def close(got, want, bound):
    err = (got.double() - want).abs()
    worst = float((err / bound).max())
    assert worst <= 1.0, f"{worst:.3g} times the bound"


ROWS = [1, 2, 15, 16, 17, 32, 33, 64, 65, 128, 129, 200, 257, 500]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("N,K", [(1, 16), (3, 144), (128, 128), (129, 272), (256, 1040), (700, 2560), (1000, 4096)])
def test_product(M, N, K):
    ops = operands(10 + M, M, N, K)
    out = torch.full((M, N), math.nan, device="cuda")
    gd.dec_fp8_gemm(*ops, out)
    close(out, *R.gemm(*ops))


@pytest.mark.parametrize("M", [1, 16, 40, 100, 300])
def test_residual_and_views(M):
    N, K = 333, 656
    ops = operands(20 + M, M, N, K)
    res = normal(25, M, N)
    want, bound = R.gemm(*ops, residual=res)
    out = torch.full((M, N), math.nan, device="cuda")
    gd.dec_fp8_gemm(*ops, out, residual=res)
    close(out, want, bound)
    same = res.clone()  # in place
    gd.dec_fp8_gemm(*ops, same, residual=same)
    assert torch.equal(same, out)
    for left, right in ((1, 2), (4, 3), (0, 0)):  # rows of a wider result, 4-byte and 16-byte aligned
        pad = torch.full((M + 2, left + N + right), 7.0, device="cuda")
        view = pad[1:M + 1, left:left + N]
        gd.dec_fp8_gemm(*ops, view, residual=res)
        assert torch.equal(view, out)
        view.fill_(7.0)
        assert bool((pad == 7.0).all())
    one = normal(26, 1, N).expand(M, -1)  # one row for all
    gd.dec_fp8_gemm(*ops, out, residual=one)
    close(out, *R.gemm(*ops, residual=one))
    codes = (ops[0].view(torch.uint8), ops[1], ops[2].view(torch.uint8), ops[3])
    gd.dec_fp8_gemm(*codes, same, residual=one)
    assert torch.equal(same, out)


# sizes that take each form of the product (16 and 32 rows, tiles of 64, 128, 192 and 256 columns, pairs of CTAs),
# ragged on both sides, with rows of the result that are whole 16 bytes and that are not
FORMS = [(9, 700, 1040), (40, 1530, 8960), (130, 4100, 656), (250, 9000, 400), (500, 6140, 1040), (385, 9700, 144),
         (1000, 9730, 528), (2050, 9729, 272), (2047, 9700, 1040), (2041, 9702, 2576), (2040, 9704, 2576), (4200, 5003, 144)]


@pytest.mark.parametrize("M,N,K", FORMS)
def test_every_form(M, N, K):
    ops = operands(80, M, N, K)
    res = normal(85, M, N)
    want, bound = R.gemm(*ops, residual=res)
    out = torch.full((M, N), math.nan, device="cuda")
    gd.dec_fp8_gemm(*ops, out, residual=res)
    close(out, want, bound)
    again = res.clone()
    gd.dec_fp8_gemm(*ops, again, residual=again)
    assert torch.equal(again, out)


# tiles of 64, 128, 192 and 256 columns, one and several of a CTA, pairs
@pytest.mark.parametrize("M,N,K", [(130, 4100, 656), (250, 9000, 400), (500, 6140, 1040), (385, 9700, 144), (1000, 9732, 528),
                                   (2047, 9700, 1040), (2050, 9728, 272), (2040, 9704, 2576)])
def test_every_form_without_a_residual(M, N, K):
    ops = operands(89, M, N, K)
    want, bound = R.gemm(*ops)
    out = torch.full((M, N), math.nan, device="cuda")
    gd.dec_fp8_gemm(*ops, out)
    close(out, want, bound)


# three and five stages, a few blocks a tile, many tiles a CTA: blocks that arrive out of order
@pytest.mark.parametrize("M,N,K", [(2050, 9729, 272), (2050, 9728, 272), (4200, 14588, 288), (250, 9000, 400), (385, 9700, 144)])
def test_short_rows_again_and_again(M, N, K):
    ops = operands(90, M, N, K)
    res = normal(91, M, N)
    for r in (None, res):
        want, bound = R.gemm(*ops, residual=r)
        first = torch.full((M, N), math.nan, device="cuda")
        gd.dec_fp8_gemm(*ops, first, residual=r)
        close(first, want, bound)
        out = torch.empty_like(first)
        for _ in range(25):
            gd.dec_fp8_gemm(*ops, out, residual=r)
            assert torch.equal(out, first)


@pytest.mark.parametrize("M,N,K", [(500, 6140, 1040), (2047, 9700, 272), (2047, 9702, 272), (1000, 9732, 528)])
def test_rows_of_unlike_alignment(M, N, K):
    """Many rows whose residual or result is not aligned as the other is: the same bits, and nothing beside them."""
    ops = operands(87, M, N, K)
    res = normal(88, M, N)
    want = torch.empty(M, N, device="cuda")
    gd.dec_fp8_gemm(*ops, want, residual=res)
    close(want, *R.gemm(*ops, residual=res))
    for left, right in ((1, 2), (4, 4), (8, 3)):
        odd = torch.zeros(M, left + N + right, device="cuda")[:, left:left + N]
        odd.copy_(res)
        out = torch.full((M, N), math.nan, device="cuda")
        gd.dec_fp8_gemm(*ops, out, residual=odd)
        assert torch.equal(out, want)
        pad = torch.full((M + 2, left + N + right), 7.0, device="cuda")
        view = pad[1:M + 1, left:left + N]
        gd.dec_fp8_gemm(*ops, view, residual=res)
        assert torch.equal(view, want)
        view.fill_(7.0)
        assert bool((pad == 7.0).all())


def test_one_row_takes_any_strides():
    ops = operands(86, 1, 333, 160)
    want, bound = R.gemm(*ops)
    out = torch.zeros(1, 333, device="cuda")
    ptr = [t.data_ptr() for t in ops]
    assert gd.lib().dec_fp8_gemm(*ptr, out.data_ptr(), 0, out.data_ptr(), 0, 1, 333, 160, None) == gd.DEC_OK
    torch.cuda.synchronize()
    close(out, want, bound)


@pytest.mark.parametrize("M", [5, 60, 200])
def test_a_nan_stays_in_its_row_and_column(M):
    N, K = 200, 400
    xc, xs, wc, ws = operands(30, M, N, K)
    clean = torch.zeros(M, N, device="cuda")
    gd.dec_fp8_gemm(xc, xs, wc, ws, clean)
    xc.view(torch.uint8)[2, 390] = 0x7F
    wc.view(torch.uint8)[131, 5] = 0xFF
    out = torch.zeros(M, N, device="cuda")
    gd.dec_fp8_gemm(xc, xs, wc, ws, out)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[2], bad[:, 131] = True, True
    assert torch.equal(torch.isnan(out), bad)
    assert torch.equal(out[~bad], clean[~bad])


@pytest.mark.parametrize("M", [1, 16, 48, 128, 400])
def test_exact_sums_of_small_integers(M):
    """Codes that are integers with sums below 2^24: every fp32 sum is exact."""
    N, K = 385, 1024
    xc = torch.randint(-8, 9, (M, K), generator=rng(40), device="cuda").float().to(torch.float8_e4m3fn)
    wc = torch.randint(-8, 9, (N, K), generator=rng(41), device="cuda").float().to(torch.float8_e4m3fn)
    xs = torch.exp2(torch.randint(0, 4, (M, 8), generator=rng(42), device="cuda").float())
    ws = torch.exp2(torch.randint(0, 4, (4, 8), generator=rng(43), device="cuda").float())
    out = torch.zeros(M, N, device="cuda")
    gd.dec_fp8_gemm(xc, xs, wc, ws, out)
    assert torch.equal(out.double(), R.gemm(xc, xs, wc, ws)[0])


@pytest.mark.parametrize("M", [3, 70, 300])
def test_reproducible_captured_and_on_another_stream(M):
    N, K = 520, 1296
    x, w = normal(50, M, K), 0.1 * normal(51, N, K)
    xc, xs = empty_codes(x, 1)
    wc, ws = empty_codes(w, 128)
    out = torch.zeros(M, N, device="cuda")

    def layer(stream=None):
        gd.dec_fp8_quant(w, wc, ws, block_rows=128, stream=stream)
        gd.dec_fp8_quant(x, xc, xs, stream=stream)
        gd.dec_fp8_gemm(xc, xs, wc, ws, out, stream=stream)

    layer()
    first = out.clone()
    close(first, *R.gemm(xc, xs, wc, ws))
    for _ in range(20):  # launches that overlap their neighbours
        layer()
    assert torch.equal(out, first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    layer(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    x.mul_(2.0)
    out.zero_()
    for _ in range(3):
        g.replay()
    assert torch.equal(out, 2.0 * first)  # a power of two changes no rounding


@pytest.mark.parametrize("M", [1, 300])
def test_weights_made_right_before_the_product(M):
    """The rows first, then the weights, then the product, without a pause: it reads no weights of the pass before."""
    N, K = 4096, 2048
    x = normal(55, M, K)
    ws = [normal(56 + i, N, K).bfloat16() for i in range(3)]
    xc, xs = empty_codes(x, 1)
    wc, wsc = empty_codes(ws[0], 128)
    outs = [torch.zeros(M, N, device="cuda") for _ in range(12)]
    for i, out in enumerate(outs):
        gd.dec_fp8_quant(x, xc, xs)
        gd.dec_fp8_quant(ws[i % 3], wc, wsc, block_rows=128)
        gd.dec_fp8_gemm(xc, xs, wc, wsc, out)
    for i in range(3):
        gd.dec_fp8_quant(ws[i], wc, wsc, block_rows=128)
        want, bound = R.gemm(xc, xs, wc, wsc)
        for out in outs[i::3]:
            close(out, want, bound)


@pytest.mark.parametrize("M", [1, 3000])
def test_one_row_of_weights_made_right_before_the_product(M):
    """One row's blocks are the same for both kinds: the quantiser of rows may have made it."""
    K = 1 << 14
    x = normal(65, M, K)
    ws = [normal(66 + i, 1, K) for i in range(3)]
    xc, xs = empty_codes(x, 1)
    wc, wsc = empty_codes(ws[0], 1)
    gd.dec_fp8_quant(x, xc, xs)
    outs = [torch.zeros(M, 1, device="cuda") for _ in range(12)]
    for i, out in enumerate(outs):
        gd.dec_fp8_quant(ws[i % 3], wc, wsc)
        gd.dec_fp8_gemm(xc, xs, wc, wsc, out)
    for i in range(3):
        gd.dec_fp8_quant(ws[i], wc, wsc)
        want, bound = R.gemm(xc, xs, wc, wsc)
        for out in outs[i::3]:
            close(out, want, bound)


def test_two_products_at_once():
    a, b = operands(60, 16, 700, 2048), operands(61, 300, 900, 1024)
    oa, ob = torch.zeros(16, 700, device="cuda"), torch.zeros(300, 900, device="cuda")
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(30):
        gd.dec_fp8_gemm(*a, oa, stream=s)
        gd.dec_fp8_gemm(*b, ob, stream=t)
    torch.cuda.synchronize()
    close(oa, *R.gemm(*a))
    close(ob, *R.gemm(*b))


def test_results_behind_2_to_the_31():
    """70,000 x 32,001 results: the last rows lie behind 2^31 elements."""
    M, N, K = 70000, 32001, 16
    ops = operands(70, M, N, K)
    out = torch.zeros(M, N, device="cuda")
    gd.dec_fp8_gemm(*ops, out)
    for r in (slice(0, 3), slice(67105, 67112), slice(M - 130, M)):
        part = (ops[0][r], ops[1][r], *ops[2:])
        close(out[r], *R.gemm(*part))


def test_quantiser_behind_2_to_the_31():
    n, rows, K = 5, 30000, 16400  # the last block row is a ragged one
    x = torch.empty(n, rows, K, device="cuda", dtype=torch.bfloat16)
    x[-1] = normal(71, rows, K)
    c, s = empty_codes(x, 128)
    gd.dec_fp8_quant(x, c, s, block_rows=128)
    r0 = rows // 128 * 128
    want, scale = R.quantise(x[-1, r0:], 128)
    assert torch.equal(s[-1, rows // 128:].double().cpu(), scale)
    assert torch.equal(c[-1, r0:].float().double().cpu(), want)
