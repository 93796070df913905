"""The 8-bit and expert calls refuse bad arguments on the host, before any GPU
work (through the C entry points with addresses that are never read, and
through the Python binding with CPU tensors)."""
import pytest
import torch

P = 0x1000  # an aligned address; nothing is launched


@pytest.fixture(scope="module")
def gd():
    import greedy_decode_step_gb300 as gd
    gd.build()
    return gd


def refused(gd, name, good, code, word, **change):
    unknown = set(change) - set(good)
    assert not unknown, unknown
    rc = getattr(gd.lib(), name)(*{**good, **change}.values())
    msg = gd.lib().dec_last_error().decode()
    assert rc == code and word in msg, (rc, msg)


QUANT = dict(x=P, bf16=0, sm=8192, sr=256, codes=P, scales=P, n=1, rows=16, K=256, block_rows=1, stream=None)
DEQUANT = dict(codes=P, scales=P, out=P, bf16=1, sm=8192, sr=256, n=2, rows=16, K=256, block_rows=128, stream=None)
GEMM = dict(xc=P, xs=P, wc=P, ws=P, residual=P, ldr=64, out=P, ldo=64, M=4, N=64, K=256, stream=None)
ROUTE = dict(y=P, Wr=P, bias=P, sigmoid=0, renorm=1, scale=1.0, ids=P, weights=P, T=4, H=256, E=8, k=2, stream=None)
EXPERTS = dict(y=P, ids=P, weights=P, Wg=P, Wu=P, Wd=P, Sg=None, Su=None, Sd=None, residual=P, out=P, ws=P, ws_bytes=1 << 40,
               T=4, k=2, E=8, H=256, I=64, stream=None)
ALL = [("dec_fp8_quant", QUANT), ("dec_fp8_dequant", DEQUANT), ("dec_fp8_gemm", GEMM), ("dec_moe_route", ROUTE),
       ("dec_moe_experts", EXPERTS)]


@pytest.mark.parametrize("name,good", ALL, ids=[n for n, _ in ALL])
def test_pointers(gd, name, good):
    for arg, x in good.items():
        if x != P:
            continue
        if arg not in ("residual", "bias"):
            refused(gd, name, good, gd.DEC_EINVAL, "null", **{arg: None})
        refused(gd, name, good, gd.DEC_EINVAL, "aligned", **{arg: P + 2})


@pytest.mark.parametrize("name,good", ALL[:3], ids=[n for n, _ in ALL[:3]])
def test_sizes_of_codes(gd, name, good):
    for K in (0, -16, 8, 100, (1 << 24) + 16):
        refused(gd, name, good, gd.DEC_EUNSUPPORTED, "codes", K=K)
    rows = "M" if "M" in good else "rows"
    refused(gd, name, good, gd.DEC_EINVAL, ">= 0", **{rows: -1})
    refused(gd, name, good, gd.DEC_EUNSUPPORTED, "2^24", **{rows: (1 << 24) + 1})
    if "n" in good:
        refused(gd, name, good, gd.DEC_EINVAL, ">= 0", n=-1)
        for R in (0, 2, 64, 256, -1):
            refused(gd, name, good, gd.DEC_EUNSUPPORTED, "blocks", block_rows=R)
        for s in ("sm", "sr"):
            refused(gd, name, good, gd.DEC_EINVAL, "strides", **{s: 130})
            refused(gd, name, good, gd.DEC_EINVAL, "strides", **{s: -8})


def test_particular_arguments(gd):
    for s in ("sm", "sr"):
        refused(gd, "dec_fp8_dequant", DEQUANT, gd.DEC_EINVAL, "share memory", **{s: 0})
    for s in ("sm", "sr"):
        refused(gd, "dec_fp8_dequant", DEQUANT, gd.DEC_EINVAL, "share memory", **{s: 248})
    refused(gd, "dec_fp8_gemm", GEMM, gd.DEC_EINVAL, "N must", N=0)
    refused(gd, "dec_fp8_gemm", GEMM, gd.DEC_EUNSUPPORTED, "2^24", N=(1 << 24) + 1, ldo=1 << 25)
    refused(gd, "dec_fp8_gemm", GEMM, gd.DEC_EUNSUPPORTED, "2^40", N=1 << 24, M=1 << 20, ldo=1 << 24)
    refused(gd, "dec_fp8_gemm", GEMM, gd.DEC_EINVAL, "apart", ldo=63)
    refused(gd, "dec_fp8_gemm", GEMM, gd.DEC_EINVAL, "apart", ldo=-64)
    refused(gd, "dec_fp8_gemm", GEMM, gd.DEC_EINVAL, "residual", ldr=-64)


@pytest.mark.parametrize("name,good", ALL[3:], ids=[n for n, _ in ALL[3:]])
def test_sizes_of_the_layer(gd, name, good):
    refused(gd, name, good, gd.DEC_EINVAL, "T must", T=-1)
    refused(gd, name, good, gd.DEC_EUNSUPPORTED, "at most 16", T=17)
    for E in (0, 1025):
        refused(gd, name, good, gd.DEC_EUNSUPPORTED, "experts outside", E=E)
    for H in (0, 4, 250, 32776):
        refused(gd, name, good, gd.DEC_EUNSUPPORTED, "H = ", H=H)
    for k in (0, 17):
        refused(gd, name, good, gd.DEC_EUNSUPPORTED, "per token", k=k)


def test_particular_arguments_of_the_layer(gd):
    refused(gd, "dec_moe_route", ROUTE, gd.DEC_EINVAL, "there are 8", k=9)
    for s in (float("nan"), float("inf")):
        refused(gd, "dec_moe_route", ROUTE, gd.DEC_EINVAL, "finite", scale=s)
    for i in (0, 12, 32776):
        refused(gd, "dec_moe_experts", EXPERTS, gd.DEC_EUNSUPPORTED, "I = ", I=i)
    held = dict(Sg=P, Su=P, Sd=P)
    refused(gd, "dec_moe_experts", EXPERTS, gd.DEC_EUNSUPPORTED, "multiples of 16", **held, H=264)
    refused(gd, "dec_moe_experts", EXPERTS, gd.DEC_EUNSUPPORTED, "multiples of 16", **held, I=72)
    for s in held:
        refused(gd, "dec_moe_experts", EXPERTS, gd.DEC_EINVAL, s, **{**held, s: None})
    refused(gd, "dec_moe_experts", EXPERTS, gd.DEC_EINVAL, "needs", ws_bytes=gd.moe_workspace_size(4, 2, 256, 64) - 1)
    refused(gd, "dec_moe_experts", EXPERTS, gd.DEC_EINVAL, "256-byte", ws=P + 128)


def test_calls_without_work_need_no_gpu(gd):
    for name, good, change in (("dec_fp8_quant", QUANT, dict(rows=0)), ("dec_fp8_quant", QUANT, dict(n=0)),
                               ("dec_fp8_dequant", DEQUANT, dict(rows=0)), ("dec_fp8_gemm", GEMM, dict(M=0)),
                               ("dec_moe_route", ROUTE, dict(T=0)), ("dec_moe_experts", EXPERTS, dict(T=0))):
        assert getattr(gd.lib(), name)(*{**good, **change}.values()) == gd.DEC_OK


@pytest.mark.parametrize("sizes,word", [((-1, 2, 64, 64), "T must"), ((17, 2, 64, 64), "at most 16"), ((4, 0, 64, 64), "per token"),
                                        ((4, 17, 64, 64), "per token"), ((4, 2, 64, 60), "I = "),
                                        ((4, 2, 60, 64), "H = ")])
def test_a_workspace_size_of_zero_leaves_its_reason(gd, sizes, word):
    assert gd.lib().dec_add_rmsnorm(None, None, None, None, 1, 64, 0.0, None) != gd.DEC_OK  # another call's message
    assert gd.moe_workspace_size(*sizes) == 0
    assert word in gd.lib().dec_last_error().decode()


# ----------------------------------------------------------------------------- through Python

def held(n, rows, K, R):
    lead = (n,) if n else ()
    return (torch.zeros(*lead, rows, K), torch.zeros(*lead, rows, K, dtype=torch.float8_e4m3fn),
            torch.zeros(*lead, -(-rows // R), -(-K // 128)))


def test_python_quantiser(gd):
    x, c, s = held(0, 130, 160, 128)
    for call in (lambda *a, **k: gd.dec_fp8_quant(*a, **k), lambda a, b, d, **k: gd.dec_fp8_dequant(b, d, a, **k)):
        with pytest.raises(gd.DecError, match="CUDA device"):  # everything else is right
            call(x, c, s, block_rows=128)
        with pytest.raises(gd.DecError, match="CUDA device"):
            call(x, c.view(torch.uint8), s, block_rows=128)
        with pytest.raises(TypeError, match="float32 or bfloat16"):
            call(x.double(), c, s, block_rows=128)
        with pytest.raises(TypeError, match="float8_e4m3fn"):
            call(x, c.float(), s, block_rows=128)
        with pytest.raises(TypeError, match="torch.Tensor"):
            call(x, c, None, block_rows=128)
        with pytest.raises(gd.DecError, match="shape"):
            call(x, c[:-1], s, block_rows=128)
        with pytest.raises(gd.DecError, match="shape"):
            call(x, c, s, block_rows=1)
        with pytest.raises(gd.DecError, match="block_rows"):
            call(x, c, s, block_rows=0)
        with pytest.raises(gd.DecError, match="contiguous rows"):
            call(torch.zeros(160, 130).T, c, s, block_rows=128)
        with pytest.raises(ValueError, match="contiguous"):
            call(x, torch.zeros(160, 130, dtype=torch.uint8).T, s, block_rows=128)
        with pytest.raises(gd.DecError, match="must be"):
            call(x[0], c[0], s[0], block_rows=128)


def test_python_product(gd):
    xc, xs = held(0, 3, 160, 1)[1:]
    wc, ws = held(0, 130, 160, 128)[1:]
    out = torch.zeros(3, 130)
    good = [xc, xs, wc, ws, out]

    def call(i=None, x=None, **kw):
        a = list(good)
        if i is not None:
            a[i] = x
        gd.dec_fp8_gemm(*a, **kw)

    with pytest.raises(gd.DecError, match="CUDA device"):
        call()
    with pytest.raises(gd.DecError, match="CUDA device"):
        call(residual=torch.zeros(3, 200)[:, 5:135])
    for i, x in ((0, xc[:2]), (1, xs[:, :1]), (2, wc[:, :144].contiguous()), (3, ws.T)):
        with pytest.raises((gd.DecError, ValueError)):
            call(i, x)
    with pytest.raises(gd.DecError, match="rows"):
        call(4, out.T)
    with pytest.raises(TypeError):
        call(4, out.double())
    with pytest.raises(gd.DecError, match="residual"):
        call(residual=out[:2])


def test_python_layer(gd):
    T, H, I, E, k = 3, 64, 48, 5, 2
    y, Wr = torch.zeros(T, H), torch.zeros(E, H, dtype=torch.bfloat16)
    ids, w = torch.zeros(T, k, dtype=torch.int32), torch.zeros(T, k)
    with pytest.raises(gd.DecError, match="CUDA device"):
        gd.dec_moe_route(y, Wr, ids, w, bias=torch.zeros(E))
    with pytest.raises(gd.DecError, match="score"):
        gd.dec_moe_route(y, Wr, ids, w, score="linear")
    with pytest.raises(TypeError):
        gd.dec_moe_route(y, Wr.float(), ids, w)
    with pytest.raises(TypeError):
        gd.dec_moe_route(y, Wr, ids.long(), w)
    with pytest.raises(gd.DecError, match="shape"):
        gd.dec_moe_route(y, Wr, ids, w, bias=torch.zeros(E + 1))
    bf = [torch.zeros(E, *s, dtype=torch.bfloat16) for s in ((I, H), (I, H), (H, I))]
    f8 = [b.to(torch.float8_e4m3fn) for b in bf]
    sc = (torch.zeros(E, 1, 1),) * 3
    with pytest.raises(gd.DecError, match="CUDA device"):
        gd.dec_moe_experts(y, ids, w, *bf, y.clone())
    with pytest.raises(gd.DecError, match="CUDA device"):
        gd.dec_moe_experts(y, ids, w, *f8, y.clone(), residual=y, scales=sc)
    with pytest.raises(TypeError):
        gd.dec_moe_experts(y, ids, w, *f8, y.clone())  # codes without scales
    with pytest.raises(TypeError):
        gd.dec_moe_experts(y, ids, w, *bf, y.clone(), scales=sc)
    with pytest.raises(gd.DecError, match="shape"):
        gd.dec_moe_experts(y, ids, w, bf[0], bf[1], bf[0], y.clone())
    with pytest.raises(TypeError):
        gd.dec_moe_experts(y, ids, w, *f8, y.clone(), scales=(sc[0], None, sc[0]))
    with pytest.raises(TypeError):
        gd.dec_moe_experts(y, ids, w, *bf, y.clone(), scales=(None, sc[0], sc[0]))
    with pytest.raises(gd.DecError, match="shape"):
        gd.dec_moe_experts(y, ids, w, *f8, y.clone(), scales=(sc[0], sc[0], torch.zeros(E, 2, 1)))
