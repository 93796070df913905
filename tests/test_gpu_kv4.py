"""The 4-bit KV cache on the GPU: store, read-back and decode attention
against plain forms in 64 bits.

The codes, scales and middles are defined by float32 operations, so they must
agree bit for bit; so must the values read back.

Attention: a float32 score of D products is within 2^-20 of the sum of its
terms' magnitudes (query parts 2^-22, tensor-core sums of 16 terms 2^-23 and
at most 16 further float32 roundings of 2^-24); a term's magnitude is at most
|q| (|z| + 16 s), as codes are taken uncentred (0 .. 15) and moved back by 8 s.
With A the largest such sum of a head over its keys, over sqrt(D), a
probability is then within 2 * 2^-20 A of its value (its own score and the
maximum's), plus 2^-22 for the exponential, 2^-21 for the two half parts and
2^-21 for the sum.  Numerator and denominator each have that, so
  |o - exact| <= 2^-18 (1 + A) W,  W = sum_j p_j (|z_j| + 8 s_j).
"""
import math

import pytest
import torch

import long_refs as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gd():
    import greedy_decode_step_gb300 as gd
    gd.build()
    gd.lib()
    gd.device_error(clear=True)
    return gd


def gen(seed):
    return torch.Generator().manual_seed(seed)


def rows(shape, seed, scale=1.0):
    """Rows with channels of unlike size; a few constant, huge, tiny and offset groups."""
    x = torch.randn(shape, generator=gen(seed)) * scale
    x *= torch.exp(torch.randn(shape[-1], generator=gen(seed + 1)))
    flat = x.view(-1, shape[-1])
    n = flat.shape[0]
    if n > 8:
        flat[n // 7] = 1.25
        flat[n // 6] *= 1e4
        flat[n // 5] *= 1e-6
        flat[n // 4] += 300.0
        flat[n // 3] = 0.0
    return x


def empty_cache(B, Hkv, S, D, group, fill=0xAB):
    codes = [torch.full((B, Hkv, S, D // 2), fill, dtype=torch.uint8, device="cuda") for _ in range(2)]
    params = [torch.full((B, Hkv, S, D // group, 2), 7.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    return codes[0], params[0], codes[1], params[1]


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def bits(t):
    return t.contiguous().view(torch.int16).cpu()


STORE = [
    # D, group, B, Hkv, T, S_max, pos, lens
    (64, 32, 1, 1, 1, 1, [0], None),
    (64, 64, 3, 2, 1, 40, [0, 39, 7], None),
    (128, 32, 2, 3, 5, 33, [28, 0], None),
    (128, 64, 2, 8, 67, 131, [64, 3], [67, 13]),
    (128, 128, 4, 1, 130, 130, [0, 0, 0, 0], [130, 0, 1, 129]),
    (64, 32, 17, 2, 1, 9, list(range(9)) + list(range(8)), None),
    (128, 32, 1, 2, 1000, 1003, [3], None),
]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("source", ["rows", "strided", "cache"])
@pytest.mark.parametrize("D,group,B,Hkv,T,S,pos,lens", STORE)
def test_store_and_load_are_bit_exact(gd, D, group, B, Hkv, T, S, pos, lens, source, dtype):
    cache = empty_cache(B, Hkv, S, D, group)
    if source == "cache":  # slots of [B, Hkv, S_src, D]
        src_slots = S + 3
        full = [rows((B, Hkv, src_slots, D), 5 + i).to(dtype).cuda() for i in range(2)]
        k, v = (f.transpose(1, 2) for f in full)
        ref = [torch.stack([f[b, :, pos[b]:pos[b] + T] if pos[b] + T <= src_slots else
                            torch.zeros(Hkv, T, D, dtype=dtype, device="cuda") for b in range(B)]).transpose(1, 2)
               for f in full]
    elif source == "strided":  # the k and v columns of fused rows
        fused = rows((B, T, (5 + 2 * Hkv) * D), 5).to(dtype).cuda()
        k, v = (fused[..., o * D:(o + Hkv) * D].unflatten(-1, (Hkv, D)) for o in (5, 5 + Hkv))
        ref = [k, v]
    else:
        k, v = (rows((B, T, Hkv, D), 5 + i).to(dtype).cuda() for i in range(2))
        ref = [k, v]
    ln = None if lens is None else i32(lens)
    gd.dec_kv4_store(k, v, i32(pos), *cache, tokens=T, lens=ln, from_cache=source == "cache")
    outs = [torch.full((B, T, Hkv, D), -3.0, dtype=t, device="cuda") for t in (torch.float32, torch.bfloat16)
            for _ in range(2)]
    gd.dec_kv4_load(*cache, i32(pos), outs[0], outs[1], lens=ln)
    gd.dec_kv4_load(*cache, i32(pos), outs[2], outs[3], lens=ln)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 0
    for i in range(2):
        codes, params = cache[2 * i].cpu(), cache[2 * i + 1]
        want_c = torch.full_like(codes, 0xAB)
        want_p = torch.full(params.shape, 7.0, dtype=torch.float16)
        want32 = torch.full((B, T, Hkv, D), -3.0)
        for b in range(B):
            n = T if lens is None else lens[b]
            c, p = R.quantise(ref[i][b, :n], group)  # [n, Hkv, ..]
            want_c[b, :, pos[b]:pos[b] + n] = R.pack(c).transpose(0, 1)
            want_p[b, :, pos[b]:pos[b] + n] = p.transpose(0, 1)
            want32[b, :n] = R.values(R.pack(c), p).float()
        assert torch.equal(codes, want_c)
        assert torch.equal(bits(params), bits(want_p))
        assert torch.equal(outs[i].cpu(), want32)
        assert torch.equal(bits(outs[2 + i]), bits(want32.bfloat16()))


def test_store_of_values_that_are_not_finite(gd):
    """An infinity or a NaN makes its own group NaN and nothing else; magnitudes past half saturate."""
    x = torch.randn(1, 6, 1, 128, generator=gen(3))
    x[0, 0, 0, 5] = float("nan")
    x[0, 1, 0, 70] = float("inf")
    x[0, 2, 0, 127] = -float("inf")
    x[0, 3, 0, :] = 3e38
    x[0, 4, 0, ::2] = -3e38
    x[0, 4, 0, 1::2] = 3e38
    x[0, 5, 0, 0] = 1e-44
    cache = empty_cache(1, 1, 6, 128, 32)
    gd.dec_kv4_store(x.cuda(), x.cuda(), i32([0]), *cache)
    c, p = R.quantise(x, 32)
    assert torch.equal(cache[0].cpu()[0, 0], R.pack(c)[0, :, 0])
    got = cache[1].cpu()[0, 0]
    assert torch.equal(torch.isnan(got), torch.isnan(p[0, :, 0]))
    assert torch.equal(torch.nan_to_num(got, nan=1.0), torch.nan_to_num(p[0, :, 0], nan=1.0))
    assert torch.isnan(got[:, :, 0]).sum() == 3


def test_codes_at_half_steps_round_as_the_division_does(gd):
    """Values at and next to the borders between codes, where a product with 1/s could round otherwise."""
    D, n = 128, 400
    x = torch.empty(1, n, 1, D)
    s = (torch.rand(n, generator=gen(9)) * 3 + 0.01).half().float()
    steps = torch.arange(D) % 31 * 0.5  # 0 .. 15 in half steps
    x[0, :, 0] = s[:, None] * steps
    up = torch.nextafter(x, torch.tensor(math.inf))
    x = torch.where((torch.arange(D) % 3 == 1) & (steps > 0) & (steps < 15), up, x)
    cache = empty_cache(1, 1, n, D, 128)
    gd.dec_kv4_store(x.cuda(), x.cuda(), i32([0]), *cache)
    c, p = R.quantise(x, 128)
    assert torch.equal(cache[0].cpu()[0, 0], R.pack(c)[0, :, 0])


def test_rows_that_leave_the_cache_are_refused(gd):
    B, Hkv, D, S, T = 5, 2, 64, 10, 4
    k = torch.randn(B, T, Hkv, D, generator=gen(1)).cuda()
    pos, lens = i32([7, -1, 0, 6, 2]), i32([4, 4, 5, 4, -1])  # the fourth fits, the others do not
    cache = empty_cache(B, Hkv, S, D, 32)
    gd.dec_kv4_store(k, k, pos, *cache, lens=lens)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 4
    left = [b for b in range(B) if torch.all(cache[0][b] == 0xAB) and torch.all(cache[1][b] == 7.0)]
    assert left == [0, 1, 2, 4]
    out = torch.full((B, T, Hkv, D), -3.0, device="cuda")
    gd.dec_kv4_load(*cache, pos, out, out.clone(), lens=lens)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 4
    assert [b for b in range(B) if torch.all(out[b] == -3.0)] == [0, 1, 2, 4]
    # a source cache shorter than the target: its slots count too
    src = torch.randn(B, Hkv, 8, D, generator=gen(2)).cuda().transpose(1, 2)
    gd.dec_kv4_store(src, src, i32([6, 4, 5, 3, 0]), *empty_cache(B, Hkv, S, D, 32), tokens=3, from_cache=True)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 4


# ----------------------------------------------------------------------------- attention

def make_cache(B, Hkv, S, D, group, pos, seed, k_scale=1.0, v_scale=1.0, poison=True):
    """A quantised cache whose slots behind pos hold the highest codes and NaN scales."""
    out = []
    for i, scale in enumerate((k_scale, v_scale)):
        x = torch.randn((B, Hkv, S, D), generator=gen(seed + i)) * scale
        x += 0.3 * scale * torch.randn((B, Hkv, 1, D), generator=gen(seed + 10 + i))
        c, p = R.quantise(x, group)
        c = R.pack(c)
        if poison:
            for b in range(B):
                c[b, :, pos[b] + 1:] = 0xFF
                p[b, :, pos[b] + 1:] = float("nan")
        out += [c.cuda(), p.cuda()]
    return tuple(out)


def check_attention(gd, q, cache, pos, o, what=""):
    """o against the definition, within the bound of this file's docstring."""
    B, Hq, D = q.shape
    Hkv = cache[0].shape[1]
    G, NG = Hq // Hkv, cache[1].shape[3]
    for b in range(B):
        n = pos[b] + 1
        for g in range(Hkv):
            k, v = (R.values(cache[2 * i][b, g, :n], cache[2 * i + 1][b, g, :n]) for i in range(2))
            qg = q[b, g * G:(g + 1) * G].double()
            ref = R.attention(qg, k, v)
            got = o[b, g * G:(g + 1) * G].double()
            if n == 0:
                assert torch.all(got == 0.0)
                continue

            def size(p, c):  # |z| + c s per dim
                return (p[..., 1].abs() + c * p[..., 0]).double().repeat_interleave(D // NG, -1)

            A = (qg.abs() @ size(cache[1][b, g, :n], 16).T).amax(-1) / math.sqrt(D)
            W = torch.softmax(qg @ k.T / math.sqrt(D), -1) @ size(cache[3][b, g, :n], 8)
            tol = 2.0 ** -18 * (1 + A[:, None]) * W
            bad = (got - ref).abs() > tol
            assert not bad.any(), (what, b, g, float(((got - ref).abs() / tol).max()))


ATTN = [
    # D, group, Hq, Hkv, S_max, pos
    (64, 32, 1, 1, 1, [0]),
    (64, 32, 4, 2, 300, [0, -1, 299, 31, 32, 33, 255]),
    (64, 64, 6, 3, 161, [160, 128]),
    (64, 64, 16, 1, 515, [514, 3]),
    (128, 32, 32, 8, 1025, [1024]),
    (128, 32, 8, 8, 77, [76, 0, 15, 16]),
    (128, 64, 12, 3, 700, [699, 511, 512, -1, 64, 1]),
    (128, 128, 10, 2, 333, [332, 100]),
    (128, 32, 14, 2, 600, [599, 63]),
    (128, 64, 16, 1, 2050, [2049]),
    (128, 128, 24, 2, 129, [128, 127, 0]),
    (128, 32, 33, 3, 97, [96]),
]


@pytest.mark.parametrize("D,group,Hq,Hkv,S,pos", ATTN)
def test_attention_matches_the_definition(gd, D, group, Hq, Hkv, S, pos):
    B = len(pos)
    cache = make_cache(B, Hkv, S, D, group, pos, 21)
    q = torch.randn(B, Hq, D, generator=gen(4)).cuda()
    o = torch.full_like(q, float("nan"))
    gd.dec_kv4_decode_attn(q, *cache, i32(pos), o)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 0
    check_attention(gd, q, cache, pos, o)


@pytest.mark.parametrize("k_scale,v_scale,q_scale", [(1.0, 1e-4, 1.0), (1.0, 2000.0, 1.0), (0.01, 1.0, 300.0),
                                                     (30.0, 1.0, 1.0), (1.0, 1.0, 1e-30), (1e-3, 1e-5, 1e10)])
def test_attention_over_the_range_of_scales(gd, k_scale, v_scale, q_scale):
    B, Hq, Hkv, D, S = 2, 8, 2, 128, 400
    pos = [399, 170]
    cache = make_cache(B, Hkv, S, D, 32, pos, 31, k_scale, v_scale)
    q = torch.randn(B, Hq, D, generator=gen(4)).cuda() * q_scale
    o = torch.empty_like(q)
    gd.dec_kv4_decode_attn(q, *cache, i32(pos), o)
    check_attention(gd, q, cache, pos, o)


def test_attention_with_scales_that_grow_along_the_row(gd):
    """Every 32 keys the values are 1.5 times larger (the running bound on the scales rises), or
    smaller, and scores rise likewise (the running maximum changes at every step)."""
    B, Hq, Hkv, D, S = 2, 4, 1, 128, 2000
    pos = [1999, 1999]
    x = torch.randn((B, Hkv, S, D), generator=gen(41))
    grow = 1.2 ** (torch.arange(S) // 32).float()
    cache = []
    q = torch.randn(B, Hq, D, generator=gen(4))
    for i in range(2):
        y = x.clone()
        if i == 1:
            y[0] *= 1e-2 * grow[:, None] / grow[-1] * 1e3
            y[1] *= 10.0 / grow[:, None]
        else:
            y += 0.002 * torch.arange(S)[:, None] * q[0, 0]
        c, p = R.quantise(y, 32)
        cache += [R.pack(c).cuda(), p.cuda()]
    o = torch.empty(B, Hq, D, device="cuda")
    gd.dec_kv4_decode_attn(q.cuda(), *cache, i32(pos), o)
    check_attention(gd, q.cuda(), cache, pos, o)


@pytest.mark.parametrize("B", [33, 300])
def test_attention_of_many_short_rows(gd, B):
    Hq, Hkv, D, S = 4, 2, 64, 70
    pos = [(7 * b) % (S + 1) - 1 for b in range(B)]
    cache = make_cache(B, Hkv, S, D, 32, pos, 51)
    q = torch.randn(B, Hq, D, generator=gen(4)).cuda()
    o = torch.full_like(q, float("nan"))
    gd.dec_kv4_decode_attn(q, *cache, i32(pos), o)
    check_attention(gd, q, cache, pos, o)
    assert gd.device_error(clear=True) == 0


@pytest.mark.parametrize("D,group,Hq,Hkv,S,B", [(128, 32, 18, 3, 500, 25), (128, 64, 24, 2, 401, 40), (64, 32, 16, 2, 230, 40),
                                                (128, 128, 16, 1, 333, 101), (64, 64, 8, 8, 1200, 13),
                                                (128, 32, 4, 1, 3000, 110), (128, 32, 16, 1, 40, 1024)])
def test_attention_of_many_rows(gd, D, group, Hq, Hkv, S, B):
    """More (row, KV head) items than clusters fit: runs across items, cut items joined, every group width."""
    pos = [(37 * b * b + 11 * b) % (S + 1) - 1 for b in range(B)]
    cache = make_cache(B, Hkv, S, D, group, pos, 55)
    q = torch.randn(B, Hq, D, generator=gen(4)).cuda()
    o = torch.full_like(q, float("nan"))
    gd.dec_kv4_decode_attn(q, *cache, i32(pos), o)
    check_attention(gd, q, cache, pos, o)
    assert gd.device_error(clear=True) == 0


def test_attention_of_rows_without_keys_and_refused_rows(gd):
    B, Hq, Hkv, D, S = 4, 4, 2, 64, 50
    cache = make_cache(B, Hkv, S, D, 32, [49] * B, 61)
    q = torch.randn(B, Hq, D, generator=gen(4)).cuda()
    o = torch.full_like(q, -5.0)
    gd.dec_kv4_decode_attn(q, *cache, i32([-1] * B), o)
    torch.cuda.synchronize()
    assert torch.all(o == 0) and gd.device_error(clear=True) == 0
    o.fill_(-5.0)
    gd.dec_kv4_decode_attn(q, *cache, i32([49, 50, -2, 20]), o)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 4
    assert torch.all(o[1] == -5.0) and torch.all(o[2] == -5.0)
    check_attention(gd, q[[0, 3]], tuple(c[[0, 3]] for c in cache), [49, 20], o[[0, 3]])


def test_a_nan_key_reaches_only_rows_that_attend_to_it(gd):
    B, Hq, Hkv, D, S = 2, 4, 2, 64, 100
    cache = make_cache(B, Hkv, S, D, 32, [99, 99], 71, poison=False)
    cache[1][0, 1, 40] = float("nan")   # K of row 0, head 1
    cache[3][1, 0, 41, 1] = float("nan")  # V of row 1, head 0, second group
    q = torch.randn(B, Hq, D, generator=gen(4)).cuda()
    o = torch.empty_like(q)
    gd.dec_kv4_decode_attn(q, *cache, i32([99, 99]), o)
    nan = torch.isnan(o)
    assert nan[0, 2:].all() and not nan[0, :2].any()
    assert nan[1, :2, 32:].all() and not nan[1, :2, :32].any() and not nan[1, 2:].any()
    gd.dec_kv4_decode_attn(q, *cache, i32([39, 40]), o)  # the bad slots lie behind
    assert not torch.isnan(o).any()


def test_same_bits_in_every_call_on_another_stream_and_in_a_graph(gd):
    B, Hq, Hkv, D, S = 3, 32, 8, 128, 3001
    pos = [3000, 17, 1500]
    cache = make_cache(B, Hkv, S, D, 64, pos, 81)
    q = torch.randn(B, Hq, D, generator=gen(4)).cuda()
    p = i32(pos)
    ref = torch.empty_like(q)
    ws = gd.dec_kv4_decode_attn(q, *cache, p, ref)
    ws.fill_(0xFF)  # any contents will do
    o = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gd.dec_kv4_decode_attn(q, *cache, p, o, ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(o, ref)
    # two graphs that share the workspace, replayed in turn on one stream, with other positions in between
    o2 = torch.empty_like(q)
    graphs = []
    for out in (o, o2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gd.dec_kv4_decode_attn(q, *cache, p, out, ws=ws)
        graphs.append(g)
    for _ in range(2):
        o.zero_()
        o2.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(o, ref) and torch.equal(o2, ref)
        p.copy_(i32([5, -1, 700]))
        graphs[0].replay()
        p.copy_(i32(pos))
    torch.cuda.synchronize()
    check_attention(gd, q, cache, [5, -1, 700], o)
    assert gd.device_error(clear=True) == 0


def test_two_calls_at_once_with_workspaces_of_their_own(gd):
    B, Hq, Hkv, D, S = 2, 16, 4, 128, 20000
    cases = []
    for i in range(2):
        pos = [S - 1 - 500 * i, 9000 + i]
        cache = tuple(torch.randint(0, 256, (B, Hkv, S, D // 2), dtype=torch.uint8, generator=gen(i + j)).cuda() if j % 2 == 0
                      else torch.rand(B, Hkv, S, 4, 2, generator=gen(i + j)).half().cuda() for j in range(4))
        q = torch.randn(B, Hq, D, generator=gen(i)).cuda()
        ref = torch.empty_like(q)
        gd.dec_kv4_decode_attn(q, *cache, i32(pos), ref)
        cases.append((q, cache, i32(pos), ref, torch.empty_like(q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for q, cache, pos, ref, o, s in cases:
            o.zero_()
        torch.cuda.synchronize()
        for _ in range(4):
            for q, cache, pos, ref, o, s in cases:
                gd.dec_kv4_decode_attn(q, *cache, pos, o, stream=s)
        torch.cuda.synchronize()
        for q, cache, pos, ref, o, s in cases:
            assert torch.equal(o, ref)


def test_calls_wait_for_what_comes_before_them(gd):
    """Chains of writes, stores, attention and reads without a wait of the host give what they give with one."""
    B, Hq, Hkv, D, S, group = 3, 8, 2, 64, 90, 32

    def chain(wait):
        cache = empty_cache(B, Hkv, S, D, group, fill=0)
        pos = i32([0, 0, 0])
        g = torch.Generator("cuda").manual_seed(1)
        o, ws, out = torch.empty(B, Hq, D, device="cuda"), None, []
        kv = torch.empty(2, B, 1, Hkv, D, device="cuda")
        q = torch.empty(B, Hq, D, device="cuda")
        back = torch.empty(2, B, 1, Hkv, D, device="cuda")
        for step in range(80):
            kv.normal_(generator=g)
            q.normal_(generator=g)
            gd.dec_kv4_store(kv[0], kv[1], pos, *cache)
            gd.dec_kv4_load(*cache, pos, back[0], back[1])
            ws = gd.dec_kv4_decode_attn(q, *cache, pos, o, ws=ws)
            if wait:
                torch.cuda.synchronize()
            out.append(o + back.sum())
            pos += 1
            kv.zero_()
            q.zero_()
        return torch.stack(out)

    a, b = chain(True), chain(False)
    assert torch.isfinite(a).all() and torch.equal(a, b)


FIRST_CALL = """
import sys, torch
sys.path.insert(0, {root!r})
import greedy_decode_step_gb300 as gd
B, Hq, Hkv, D, S = 2, 8, 2, 128, 100
c = [torch.zeros(B, Hkv, S, D // 2, dtype=torch.uint8, device="cuda") if i % 2 == 0 else
     torch.ones(B, Hkv, S, 4, 2, dtype=torch.float16, device="cuda") for i in range(4)]
k, v, q = (torch.randn(B, n, D, device="cuda") for n in (Hkv, Hkv, Hq))
pos, o = torch.zeros(B, dtype=torch.int32, device="cuda"), torch.empty(B, Hq, D, device="cuda")
ws = torch.empty(gd.long_attn_workspace_size(Hq, Hkv, D), dtype=torch.uint8, device="cuda")
kc = torch.zeros(B, Hkv, S, D, dtype=torch.bfloat16, device="cuda")
bd = torch.zeros(B, Hkv, 2, 2, D, dtype=torch.bfloat16, device="cuda")
bl = torch.empty(B, Hkv, 2, dtype=torch.int32, device="cuda")
o2 = torch.empty_like(o)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    gd.dec_kv4_store(k[:, None], v[:, None], pos, *c)
    gd.dec_kv4_decode_attn(q, *c, pos, o, ws=ws)
    gd.dec_block_bounds(kc, pos, bd)
    gd.dec_select_blocks(q, bd, pos, bl)
    gd.dec_block_decode_attn(q, kc, kc, pos, bl, o2, ws=ws)
g.replay()
torch.cuda.synchronize()
back = torch.empty(2, B, 1, Hkv, D, device="cuda")
gd.dec_kv4_load(*c, pos, back[0], back[1])
assert torch.equal(o.view(B, Hkv, -1, D), back[1, :, 0][:, :, None].expand(-1, -1, Hq // Hkv, -1)), "one key: its value"
assert torch.all(o2 == 0) and bl.tolist() == [[[0, -1]] * Hkv] * B
assert gd.device_error() == 0
print("ok")
"""


def test_the_first_calls_of_a_process_may_be_captured(gd):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL.format(root=root)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-2000:]


def test_graphs_whose_calls_follow_copies_and_fills(gd):
    """Every call directly behind a memory copy or fill node of the same graph sees its result."""
    B, Hq, Hkv, D, S = 2, 8, 2, 64, 300
    cache = make_cache(B, Hkv, S, D, 32, [S - 1] * B, 91, poison=False)
    src = [torch.randn(B, 1, Hkv, D, generator=gen(i)).cuda() for i in (1, 2)]
    q_src, pos_src = torch.randn(B, Hq, D, generator=gen(3)).cuda(), i32([290, 17])
    k, v, q, pos = torch.zeros_like(src[0]), torch.zeros_like(src[1]), torch.zeros_like(q_src), torch.zeros_like(pos_src)
    o, back = torch.empty_like(q), torch.empty(2, B, 1, Hkv, D, device="cuda")
    ws = gd.dec_kv4_decode_attn(q, *cache, pos, o)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pos.copy_(pos_src)
        k.copy_(src[0])
        v.copy_(src[1])
        gd.dec_kv4_store(k, v, pos, *cache)
        back.zero_()
        gd.dec_kv4_load(*cache, pos, back[0], back[1])
        q.copy_(q_src)
        gd.dec_kv4_decode_attn(q, *cache, pos, o, ws=ws)
        pos.zero_()
        q.zero_()
    for _ in range(3):
        o.zero_()
        g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        c, p = R.quantise(src[i][:, 0], 32)
        assert torch.equal(back[i][:, 0].cpu(), R.values(R.pack(c), p).float())
    check_attention(gd, q_src, cache, [290, 17], o)
    assert gd.device_error(clear=True) == 0


def test_padded_and_repeated_source_rows(gd):
    """T may be longer than the cache where lens are not, and a source may repeat one row (stride 0)."""
    B, Hkv, S, D, T = 2, 2, 6, 64, 40
    one = torch.randn(1, 1, Hkv, D, generator=gen(5)).cuda()
    k = one.expand(B, T, Hkv, D)
    cache = empty_cache(B, Hkv, S, D, 64)
    gd.dec_kv4_store(k, k, i32([0, 2]), *cache, lens=i32([6, 3]))
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 0
    c, p = R.quantise(one[0, 0], 64)
    for b, rows_ in ((0, range(6)), (1, range(2, 5))):
        for t in range(S):
            want = R.pack(c) if t in rows_ else torch.full((Hkv, D // 2), 0xAB, dtype=torch.uint8)
            assert torch.equal(cache[0][b, :, t].cpu(), want) and torch.equal(cache[2][b, :, t].cpu(), want)
    out = torch.empty(B, 3, Hkv, D, device="cuda")
    with pytest.raises(gd.DecError, match="share memory"):
        gd.dec_kv4_load(*cache, i32([0, 0]), out[:, :1].expand(B, 3, Hkv, D), out[:, 1:2].expand(B, 3, Hkv, D))


def test_offsets_past_32_bits(gd):
    """The last rows of a cache of 4.3 GB of codes: store, read back and attend there."""
    B, Hq, Hkv, D, S, group = 256, 8, 8, 128, 32800, 32
    codes = [torch.zeros(B, Hkv, S, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    params = [torch.zeros(B, Hkv, S, D // group, 2, dtype=torch.float16, device="cuda") for _ in range(2)]
    assert codes[0].numel() > 1 << 32
    cache = (codes[0], params[0], codes[1], params[1])
    T = 100
    k, v = (torch.randn(B, T, Hkv, D, generator=gen(i), dtype=torch.float32).cuda() for i in (1, 2))
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    lens[-1] = T
    at = torch.full((B,), S - T, dtype=torch.int32, device="cuda")
    gd.dec_kv4_store(k, v, at, *cache, lens=lens)
    out = [torch.zeros_like(k) for _ in range(2)]
    gd.dec_kv4_load(*cache, at, *out, lens=lens)
    for x, y in zip(out, (k, v)):
        c, p = R.quantise(y[-1], group)
        assert torch.equal(x[-1].cpu(), R.values(R.pack(c), p).float())
        assert torch.all(x[:-1] == 0)
    pos = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    pos[-1] = S - 1
    q = torch.randn(B, Hq, D, generator=gen(3)).cuda()
    o = torch.empty_like(q)
    gd.dec_kv4_decode_attn(q, *cache, pos, o)
    assert torch.all(o[:-1] == 0)
    check_attention(gd, q[-1:], tuple(t[-1:] for t in cache), [S - 1], o[-1:])
    assert gd.device_error(clear=True) == 0


def test_a_decode_loop_over_the_4_bit_cache(gd):
    """As a serving loop runs them: a prompt's bf16 cache taken over, then per step the projection with RoPE
    into a one-layer bf16 cache, its new slot quantised, and attention over the codes."""
    B, H, Hq, Hkv, D, S, P, group = 2, 256, 4, 2, 64, 64, 40, 32
    staging = [torch.randn(B, Hkv, S, D, generator=gen(i)).bfloat16().cuda() for i in (1, 2)]
    cache = empty_cache(B, Hkv, S, D, group)
    W = [(torch.randn(n * D, H, generator=gen(5 + n)) * 0.06).bfloat16().cuda() for n in (Hq, Hkv, Hkv)]
    lens = [P, P - 11]
    gd.dec_kv4_store(*(s.transpose(1, 2) for s in staging), i32([0, 0]), *cache, tokens=P, lens=i32(lens),
                     from_cache=True)
    pos = i32(lens)
    q, o = torch.empty(B, Hq * D, device="cuda"), torch.empty(B, Hq, D, device="cuda")
    ws = None
    for step in range(6):
        y = torch.randn(B, H, generator=gen(50 + step)).cuda()
        gd.dec_qkv_gemv_rope(y, *W, pos, 1e6, q, *staging)
        gd.dec_kv4_store(*(s.transpose(1, 2) for s in staging), pos, *cache, tokens=1, from_cache=True)
        ws = gd.dec_kv4_decode_attn(q.view(B, Hq, D), *cache, pos, o, ws=ws)
        at = [n + step for n in lens]
        for i in range(2):
            for b in range(B):
                c, p = R.quantise(staging[i][b, :, :at[b] + 1], group)
                assert torch.equal(cache[2 * i][b, :, :at[b] + 1].cpu(), R.pack(c))
                assert torch.equal(bits(cache[2 * i + 1][b, :, :at[b] + 1]), bits(p))
        check_attention(gd, q.view(B, Hq, D), cache, at, o)
        pos += 1
    assert gd.device_error(clear=True) == 0
