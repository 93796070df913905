"""The mixture-of-experts layer (dec_moe_route, dec_moe_experts) against its
definition in 64 bits."""
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


# ----------------------------------------------------------------------------- router

def check_route(y, Wr, k, bias=None, sigmoid=False, renormalise=True, scale=1.0):
    T, E = y.shape[0], Wr.shape[0]
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), math.nan, device="cuda")
    gd.dec_moe_route(y, Wr, ids, w, bias=bias, score="sigmoid" if sigmoid else "softmax", renormalise=renormalise, scale=scale)
    want, gates, gaps = R.route(y, Wr, k, bias, sigmoid, renormalise, scale)
    # a logit is a sum of H products in chains of H / 128 with 7 more additions: off by at most that many half steps
    # of its sum of magnitudes, so two logits that lie further apart than twice that keep their order.  With a bias the
    # scores rank: a sigmoid moves by a quarter of its logit's error at most, a softmax by p times twice the largest
    # error (p at most the largest score), and a score's own roundings (a dozen) and the bias's sum add half steps.
    H = y.shape[1]
    size = (y.double().abs() @ Wr.double().abs().T).amax(-1)
    moves = size * (H / 128 + 8) * R.STEP
    if bias is not None:
        z = y.double() @ Wr.double().T
        top = torch.sigmoid(z).amax(-1) if sigmoid else torch.softmax(z, -1).amax(-1)
        moves = (moves / 4 if sigmoid else 2 * top * moves) + ((16 + E * (not sigmoid)) * top + bias.abs().max()) * R.STEP
    slack = 2 * moves
    clear = (gaps > slack[:, None]).all(-1)
    assert torch.equal(ids[clear].long(), want[clear])
    # a weight's relative error: the exponents' (twice the logits'), and a dozen roundings
    rel = (2 * size * (H / 128 + 8) * R.STEP + 32 * R.STEP + E * R.STEP)[:, None]
    assert bool(((w.double() - gates).abs() <= rel * gates.abs() + 1e-37)[clear].all())
    return ids, w, clear


@pytest.mark.parametrize("sigmoid,biased,renormalise,scale", [(False, False, True, 1.0), (False, False, False, 2.5),
                                                              (True, False, True, 1.0), (True, True, True, 2.5),
                                                              (True, True, False, 1.0), (False, True, True, 1.0)])
@pytest.mark.parametrize("T,H,E,k", [(1, 8, 1, 1), (1, 256, 8, 2), (2, 1000, 33, 3), (5, 2560, 64, 8), (16, 1536, 80, 10),
                                     (16, 2560, 128, 8), (3, 4096, 1024, 16), (1, 32768, 40, 16), (16, 72, 17, 16)])
def test_choice(T, H, E, k, sigmoid, biased, renormalise, scale):
    y, Wr = normal(1, T, H), (normal(2, E, H) / math.sqrt(H)).bfloat16()
    bias = 0.1 * normal(3, E) if biased else None
    clear = check_route(y, Wr, k, bias, sigmoid, renormalise, scale)[2]
    assert int(clear.sum()) * 2 >= T  # the inputs are fixed: most tokens rank clearly


def test_equal_scores_go_to_the_lower_id():
    H, E = 512, 70
    Wr = (normal(4, 1, H) / math.sqrt(H)).bfloat16().expand(E, -1).contiguous()
    y = normal(5, 2, H)
    y[1] = 0.0
    ids, w = torch.zeros(2, 9, dtype=torch.int32, device="cuda"), torch.zeros(2, 9, device="cuda")
    for score in ("softmax", "sigmoid"):
        gd.dec_moe_route(y, Wr, ids, w, score=score)
        assert ids.tolist() == [list(range(9))] * 2
        assert torch.allclose(w, torch.full_like(w, 1 / 9), rtol=1e-6)
    bias = torch.zeros(E, device="cuda")
    bias[[3, 69]] = 0.5
    bias[5] = -0.0
    gd.dec_moe_route(y, Wr, ids, w, bias=bias, score="sigmoid")
    assert ids.tolist() == [[3, 69, 0, 1, 2, 4, 5, 6, 7]] * 2
    y[0, 0], y[1, 0] = math.nan, math.inf
    gd.dec_moe_route(y, Wr, ids, w)  # NaN and equal infinities: still distinct experts
    assert all(len(set(r)) == 9 and min(r) >= 0 and max(r) < E for r in ids.tolist())


def test_nan_ranks_last():
    H, E, k = 64, 10, 3
    y = normal(6, 1, H)
    Wr = (normal(7, E, H) / 8).bfloat16()
    Wr[2] = math.nan
    ids, w = torch.zeros(1, k, dtype=torch.int32, device="cuda"), torch.zeros(1, k, device="cuda")
    gd.dec_moe_route(y, Wr, ids, w, score="sigmoid")
    z = (y.double() @ Wr.double().T)[0]
    z[2] = -math.inf
    assert ids[0].tolist() == z.topk(k).indices.tolist() and bool(torch.isfinite(w).all())


# ----------------------------------------------------------------------------- experts

def make_weights(seed, E, H, I, fp8):
    ws = [(0.05 * normal(seed + i, E, *s) * torch.exp(0.3 * normal(seed + 3 + i, E, s[0], 1))).bfloat16()
          for i, s in enumerate(((I, H), (I, H), (H, I)))]
    if not fp8:
        return ws, None, ws
    codes, scales = [], []
    for i, w in enumerate(ws):
        c = torch.zeros(w.shape, device="cuda", dtype=torch.float8_e4m3fn)
        s = torch.zeros(E, -(-w.shape[1] // 128), -(-w.shape[2] // 128), device="cuda")
        gd.dec_fp8_quant(w, c, s, block_rows=128)
        s *= torch.rand(s.shape, generator=rng(seed + 10 + i), device="cuda") + 0.5  # any scales
        codes.append(c)
        scales.append(s)
    return codes, tuple(scales), list(zip(codes, scales))


def choose(seed, T, k, E):
    ids = torch.stack([torch.randperm(E, generator=rng(seed + t), device="cuda")[:k] for t in range(T)]).int()
    return ids, torch.rand(T, k, generator=rng(seed + 99), device="cuda")


def dirty(T, k, H, I):
    n = gd.moe_workspace_size(T, k, H, I)
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # every float a NaN


def close(got, want, bound):
    err = (got.double() - want).abs()
    worst = float((err / bound).max())
    assert worst <= 1.0, f"{worst:.3g} times the bound"


def check(y, ids, w, held, scales, plain, residual=None):
    out = torch.full_like(y, math.nan)
    ws = dirty(*ids.shape, y.shape[1], held[0].shape[1])
    gd.dec_moe_experts(y, ids, w, *held, out, residual=residual, scales=scales, ws=ws)
    close(out, *R.experts(y, ids, w, *plain, residual=residual))
    again = torch.full_like(y, math.nan)
    gd.dec_moe_experts(y, ids, w, *held, again, residual=residual, scales=scales, ws=ws)
    assert torch.equal(again, out)
    return out


SIZES = [  # T, H, I, E, k
    (1, 256, 704, 8, 2), (1, 16, 16, 1, 1), (2, 128, 64, 4, 4), (1, 2560, 1216, 64, 8), (3, 272, 144, 5, 2),
    (8, 1536, 896, 20, 10), (9, 400, 208, 33, 3), (16, 512, 128, 16, 16), (16, 1536, 896, 80, 10), (13, 2064, 80, 200, 7),
    (1, 4096, 64, 6, 1), (16, 64, 2048, 3, 2), (5, 1168, 1040, 1024, 16), (16, 128, 64, 1024, 16), (2, 144, 80, 40, 16),
    (16, 32768, 48, 2, 1), (2, 64, 32768, 2, 2), (4, 32768, 32, 3, 3)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,I,E,k", SIZES)
def test_experts(T, H, I, E, k, fp8):
    y = normal(20, T, H) * torch.exp(0.5 * normal(21, H))
    held, scales, plain = make_weights(22, E, H, I, fp8)
    ids, w = choose(30, T, k, E)
    check(y, ids, w, held, scales, plain)
    check(y, ids, w, held, scales, plain, residual=normal(31, T, H))


@pytest.mark.parametrize("H,I", [(264, 72), (1000, 360), (8, 8), (72, 200)])
def test_sizes_that_only_bf16_takes(H, I):
    y = normal(40, 5, H)
    held, scales, plain = make_weights(41, 7, H, I, False)
    ids, w = choose(42, 5, 3, 7)
    check(y, ids, w, held, scales, plain, residual=normal(43, 5, H))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,H,I,E,k", [(1, 256, 704, 8, 2), (8, 400, 208, 6, 3), (16, 2064, 144, 10, 4)])
def test_exact_sums_of_integers(T, H, I, E, k, fp8):
    """Integers throughout, gates so large that silu(g) is g in float32: every sum is exact."""
    def ints(seed, lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=rng(seed), device="cuda").float()

    y = torch.zeros(T, H, device="cuda")
    y[:, ::H // 8] = ints(1, 1, 3, T, len(range(0, H, H // 8)))
    y[:, 5] = 100.0
    wg, wu, wd = ints(2, 0, 2, E, I, H), ints(3, -2, 2, E, I, H), ints(4, -2, 2, E, H, I)
    wg[..., 5] = 1.0  # the gate is 100 at least
    wu[..., 5] = 0.0
    ids, _ = choose(5, T, k, E)
    w = ints(6, 1, 3, T, k)
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    held = [x.to(dt) for x in (wg, wu, wd)]
    scales = tuple(torch.ones(E, -(-x.shape[1] // 128), -(-x.shape[2] // 128), device="cuda") for x in held) if fp8 else None
    out = torch.zeros(T, H, device="cuda")
    gd.dec_moe_experts(y, ids, w, *held, out, scales=scales, ws=dirty(T, k, H, I))
    want = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            g, u = wg[e].double() @ y[t].double(), wu[e].double() @ y[t].double()
            want[t] += w[t, j].double() * (wd[e].double() @ (g * u))
    assert float(want.abs().max()) < 2 ** 24  # and no partial sum is much larger
    assert torch.equal(out.double(), want)


@pytest.mark.parametrize("fp8", [False, True])
def test_particular_choices(fp8):
    T, H, I, E, k = 16, 640, 272, 12, 4
    y, res = normal(50, T, H), normal(51, T, H)
    held, scales, plain = make_weights(52, E, H, I, fp8)
    ids, w = choose(53, T, k, E)
    check(y, torch.full_like(ids, 11), w, held, scales, plain, res)      # one expert, every token four times
    twice = ids.clone()
    twice[:, 3] = twice[:, 0]                                            # an expert listed twice
    check(y, twice, w, held, scales, plain, res)
    some = ids.clone()
    some[3], some[7, 1:], some[15, 0] = -1, -1, -1                       # tokens with no or fewer experts
    out = check(y, some, w, held, scales, plain, res)
    assert torch.equal(out[3], res[3])
    out = check(y, torch.full_like(ids, -1), w, held, scales, plain, res)
    assert torch.equal(out, res)
    assert not check(y, torch.full_like(ids, -1), w, held, scales, plain).any()
    check(y, ids, torch.zeros_like(w), held, scales, plain, res)         # weights of zero, negative ones
    check(y, ids, -w, held, scales, plain, res)
    one = torch.full_like(ids, -1)
    one[9, 2] = 5                                                        # one token, one expert
    check(y, one, w, held, scales, plain, res)
    ordered = (torch.arange(T, device="cuda")[:, None] // 4 + torch.arange(k, device="cuda") * 3).int() % E
    check(y, ordered.contiguous(), w, held, scales, plain, res)


def test_ids_outside_the_experts_are_passed_over():
    T, H, I, E, k = 4, 256, 128, 6, 2
    y = normal(60, T, H)
    held, scales, plain = make_weights(61, E, H, I, False)
    ids, w = choose(62, T, k, E)
    bad = ids.clone()
    bad[0, 0], bad[1, 1], bad[2] = 6, -2, 2 ** 31 - 1
    out = torch.zeros_like(y)
    gd.dec_moe_experts(y, bad, w, *held, out)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 4
    close(out, *R.experts(y, bad, w, *plain))


@pytest.mark.parametrize("fp8", [False, True])
def test_values_of_unlike_size(fp8):
    """Rows with a few large elements, tokens 10^12 apart, tiny and zero rows."""
    T, H, I, E, k = 12, 1024, 256, 6, 2
    y = normal(70, T, H)
    y[:, 100] *= 1e3
    y[1] *= 1e12
    y[2] *= 1e-30
    y[3] = 0.0
    y[4, 512:] = 0.0
    held, scales, plain = make_weights(71, E, H, I, fp8)
    ids, w = choose(72, T, k, E)
    check(y, ids, w, held, scales, plain)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_nan_stays_with_its_token(fp8):
    T, H, I, E, k = 6, 512, 320, 5, 3
    y, res = normal(75, T, H), normal(76, T, H)
    held, scales, plain = make_weights(77, E, H, I, fp8)
    ids, w = choose(78, T, k, E)
    clean = check(y, ids, w, held, scales, plain, res)
    y[1, 500], y[4, 3], w[2, 1] = math.nan, math.inf, math.nan
    out = torch.zeros_like(y)
    gd.dec_moe_experts(y, ids, w, *held, out, residual=res, scales=scales)
    assert torch.isnan(out[[1, 2, 4]]).all()
    assert torch.equal(out[[0, 3, 5]], clean[[0, 3, 5]])


@pytest.mark.parametrize("T", [2, 7, 16])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_nan_in_an_expert_stays_with_its_tokens(T, fp8):
    H, I, E, k = 512, 320, 9, 2
    y, res = normal(170, T, H), normal(171, T, H)
    held, scales, plain = make_weights(172, E, H, I, fp8)
    ids, w = choose(173, T, k, E)
    ids[0] = torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    ids[1] = torch.tensor([1, 7], dtype=torch.int32, device="cuda")
    clean = check(y, ids, w, held, scales, plain, res)
    for i in range(3):
        m = held[i].view(torch.uint8 if fp8 else torch.int16)
        was = m[4, 33, 65].clone()
        m[4, 33, 65] = 0x7F if fp8 else 0x7FC0
        out = torch.zeros_like(y)
        gd.dec_moe_experts(y, ids, w, *held, out, residual=res, scales=scales)
        hit = (ids == 4).any(-1)
        assert torch.equal(torch.isnan(out).any(-1), hit) and bool(hit[0]) and not bool(hit[1])
        assert torch.equal(out[~hit], clean[~hit])
        m[4, 33, 65] = was


@pytest.mark.parametrize("fp8", [False, True])
def test_results_over_their_inputs(fp8):
    T, H, I, E, k = 7, 528, 224, 9, 3
    y, res = normal(80, T, H), normal(81, T, H)
    held, scales, plain = make_weights(82, E, H, I, fp8)
    ids, w = choose(83, T, k, E)
    want = check(y, ids, w, held, scales, plain, res)
    r = res.clone()
    gd.dec_moe_experts(y, ids, w, *held, r, residual=r, scales=scales)
    assert torch.equal(r, want)
    v = y.clone()
    gd.dec_moe_experts(v, ids, w, *held, v, residual=res, scales=scales)
    assert torch.equal(v, want)


@pytest.mark.parametrize("fp8", [False, True])
def test_weights_behind_2_to_the_31(fp8):
    """The last experts' matrices begin behind 2^31 elements."""
    T, H, I, E, k = 3, 8192, 8192, 40, 2
    dt = torch.float8_e4m3fn if fp8 else torch.bfloat16
    held = [torch.empty(E, *s, device="cuda", dtype=dt) for s in ((I, H), (I, H), (H, I))]
    scales = tuple(torch.rand(E, 64, 64, generator=rng(90), device="cuda") + 0.5 for _ in range(3)) if fp8 else None
    ids = torch.tensor([[39, 37], [38, 39], [0, 39]], dtype=torch.int32, device="cuda")
    for e in (0, 37, 38, 39):
        for i in range(3):
            held[i][e] = (0.02 * normal(91 + i + 3 * e, *held[i].shape[1:])).to(dt)
    y, w = normal(95, T, H), torch.rand(T, k, generator=rng(96), device="cuda")
    check(y, ids, w, held, scales, list(zip(held, scales)) if fp8 else held, normal(97, T, H))


# ----------------------------------------------------------------------------- the layer as it is used

@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [1, 16])
def test_layer_in_a_captured_step(T, fp8):
    """Norm, router, experts into the residual: eager, on another stream, captured and replayed with new inputs."""
    H, I, E, k, eps = 1280, 448, 24, 6, 1e-6
    gamma = (1 + 0.1 * normal(100, H)).bfloat16()
    Wr = (normal(101, E, H) / math.sqrt(H)).bfloat16()
    held, scales, plain = make_weights(102, E, H, I, fp8)
    start = normal(103, T, H)
    r, y = start.clone(), torch.zeros(T, H, device="cuda")
    ids, w = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda")
    ws = dirty(T, k, H, I)

    def layer(stream=None):
        gd.dec_add_rmsnorm(None, r, gamma, y, eps, stream=stream)
        gd.dec_moe_route(y, Wr, ids, w, stream=stream)
        gd.dec_moe_experts(y, ids, w, *held, r, residual=r, scales=scales, ws=ws, stream=stream)

    def expect(r0):
        x = r0.double()
        n = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * gamma.double()
        close(y, n, 16 * R.STEP * n.abs() + 1e-30)  # its own tests have the rest
        assert torch.equal(ids.long(), R.route(y, Wr, k)[0])
        close(r, *R.experts(y, ids, w, *plain, residual=r0))

    layer()
    expect(start)
    first = r.clone()
    for _ in range(12):  # several layers behind one another, without a pause
        r.copy_(start)
        layer()
        layer()
        layer()
    third = r.clone()
    side = torch.cuda.Stream()
    r.copy_(start)
    side.wait_stream(torch.cuda.current_stream())
    layer(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(r, first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
        layer()
        layer()
    for _ in range(3):
        r.copy_(start)
        g.replay()
        assert torch.equal(r, third)
    other = normal(104, T, H)
    r.copy_(other)
    with torch.cuda.graph(one := torch.cuda.CUDAGraph()):
        layer()
    one.replay()
    expect(other)


def test_two_layers_at_once():
    """Calls on two streams with a workspace each."""
    sets = []
    for i, (T, fp8) in enumerate(((16, False), (4, True))):
        H, I, E, k = 1024, 512, 32, 4
        held, scales, plain = make_weights(110 + 20 * i, E, H, I, fp8)
        y = normal(111 + i, T, H)
        ids, w = choose(112 + 40 * i, T, k, E)
        sets.append((y, ids, w, held, scales, plain, torch.zeros_like(y), dirty(T, k, H, I), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(40):
        for y, ids, w, held, scales, plain, out, ws, st in sets:
            gd.dec_moe_experts(y, ids, w, *held, out, scales=scales, ws=ws, stream=st)
    torch.cuda.synchronize()
    for y, ids, w, held, scales, plain, out, ws, st in sets:
        close(out, *R.experts(y, ids, w, *plain))


def test_workspace_is_returned_and_taken():
    T, H, I, E, k = 2, 256, 64, 4, 2
    y = normal(120, T, H)
    held, _, plain = make_weights(121, E, H, I, False)
    ids, w = choose(122, T, k, E)
    out = torch.zeros_like(y)
    ws = gd.dec_moe_experts(y, ids, w, *held, out)
    assert ws.numel() == gd.moe_workspace_size(T, k, H, I)
    assert gd.dec_moe_experts(y, ids, w, *held, out, ws=ws) is ws
    with pytest.raises(gd.DecError, match="needs"):
        gd.dec_moe_experts(y, ids, w, *held, out, ws=ws[:256])
    with pytest.raises(gd.DecError, match="256-byte"):
        gd.dec_moe_experts(y, ids, w, *held, out, ws=torch.zeros(ws.numel() + 64, dtype=torch.uint8, device="cuda")[16:])
    none = torch.zeros(0, H, device="cuda")
    gd.dec_moe_route(none, held[0][0, :4].contiguous(), ids[:0], w[:0])
    gd.dec_moe_experts(none, ids[:0], w[:0], *held, none)
