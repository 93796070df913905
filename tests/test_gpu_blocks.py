"""Block-sparse decode attention on the GPU: channel bounds, selection and
attention over listed blocks, against plain forms in 64 bits.

Bounds are values of the cache and the selection goes by exact scores: both
must agree exactly.  Attention: query and probabilities are three bf16 parts (two already leave
2^-17 of each value), tensor-core sums of 16 terms, so a score is within
2^-16 A of its value, A the largest sum of |q_d k_d| / sqrt(D) over the keys,
a probability within 2^-15 A + 2^-16 relative, and with numerator and
denominator |o - exact| <= 2^-14 (1 + A) sum_j p_j |v_j|.
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


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def n_blocks(S):
    return (S + 63) // 64


def make_k(B, Hkv, S, D, seed):
    k = torch.randn(B, Hkv, S, D, generator=gen(seed))
    drift = torch.randn(B, Hkv, n_blocks(S), D, generator=gen(seed + 1)).repeat_interleave(64, 2)[:, :, :S]
    return (0.6 * k + 0.8 * drift).bfloat16().cuda()


# ----------------------------------------------------------------------------- bounds

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("S,T,pos", [(1, 1, [0]), (64, 64, [0, 0]), (65, 1, [64, 63, 0]), (200, 70, [0, 130, 57]),
                                     (513, 2, [510, 63, 127, 128, 511]), (1000, 999, [0, 1])])
def test_bounds_of_the_touched_blocks(gd, D, S, T, pos):
    B, Hkv = len(pos), 3
    k = make_k(B, Hkv, S, D, 3)
    k[:, :, -1, 0] = 50.0  # seen only where the range reaches the last slot
    bd = torch.full((B, Hkv, n_blocks(S), 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
    gd.dec_block_bounds(k, i32(pos), bd, tokens=T)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 0
    for b in range(B):
        last = pos[b] + T - 1
        first = pos[b] // 64
        for h in range(Hkv):
            ref = torch.full((n_blocks(S), 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
            ref[first:last // 64 + 1] = R.bounds(k[b, h], last)[first:]
            assert torch.equal(bd[b, h], ref)


def test_bounds_of_refused_rows_and_nan_keys(gd):
    B, Hkv, S, D = 4, 2, 130, 64
    k = make_k(B, Hkv, S, D, 5)
    k[3, 0, 70, 7] = float("nan")
    k[3, 0, 71, 8] = float("inf")
    bd = torch.full((B, Hkv, 3, 2, D), 9.0, dtype=torch.bfloat16, device="cuda")
    gd.dec_block_bounds(k, i32([-1, 127, 130, 60]), bd, tokens=20)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 4
    assert torch.all(bd[:3] == 9.0)
    part = k[3, 0, 64:80].float()
    keep = torch.cat((part[:6], part[7:]))[:, 7]
    assert bd[3, 0, 1, 0, 7] == keep.max() and bd[3, 0, 1, 1, 7] == keep.min()
    assert bd[3, 0, 1, 0, 8] == math.inf


# ----------------------------------------------------------------------------- selection

def run_select(gd, q, bd, pos, n, n_first=1, n_last=1):
    out = torch.full((q.shape[0], bd.shape[1], n), -7, dtype=torch.int32, device="cuda")
    gd.dec_select_blocks(q, bd, i32(pos), out, n_first=n_first, n_last=n_last)
    torch.cuda.synchronize()
    return out.cpu()


def check_select(got, q, bd, pos, n, n_first, n_last):
    G = q.shape[1] // bd.shape[1]
    for b in range(q.shape[0]):
        for h in range(bd.shape[1]):
            ref = R.select(q[b, h * G:(h + 1) * G], bd[b, h, :(pos[b] // 64) + 1] if pos[b] >= 0 else bd[b, h, :0], n,
                           n_first, n_last)
            assert got[b, h].tolist() == ref + [-1] * (n - len(ref)), (b, h)


@pytest.mark.parametrize("D,Hq,Hkv,S,n,first,last,pos", [
    (64, 4, 2, 700, 4, 1, 1, [699, 0, -1, 255, 256, 320]),
    (64, 1, 1, 64, 1, 0, 0, [63]),
    (128, 32, 8, 4096, 16, 1, 2, [4095, 1000, 1024]),
    (128, 6, 3, 2111, 5, 0, 0, [2110, 64 * 6 - 1]),
    (128, 16, 1, 40000, 64, 2, 2, [39999]),
    (128, 8, 2, 3000, 7, 3, 4, [2999]),           # all places forced
    (128, 2, 1, 100000, 600, 1, 1, [99999]),      # more blocks than threads
    (64, 2, 1, 524288, 64, 1, 1, [524287]),       # the longest row that is taken
    (64, 3, 1, 524288, 8000, 0, 0, [524287 - 64 * 5]),
])
def test_selection_equals_the_exact_ranking(gd, D, Hq, Hkv, S, n, first, last, pos):
    B = len(pos)
    bd = torch.empty(B, Hkv, n_blocks(S), 2, D)
    a, c = (torch.randn(bd.shape[:3] + (D,), generator=gen(i)) for i in (1, 2))
    bd[..., 0, :], bd[..., 1, :] = torch.maximum(a, c), torch.minimum(a, c)
    bd = bd.bfloat16().cuda()
    q = torch.randn(B, Hq, D, generator=gen(3)).cuda()
    got = run_select(gd, q, bd, pos, n, first, last)
    assert gd.device_error(clear=True) == 0
    check_select(got, q, bd, pos, n, first, last)


def test_scores_closer_than_float32_and_ties(gd):
    """Blocks that differ in one dim by one bf16 step of a tiny term (scores equal in float32),
    equal blocks, and a query of zeros: exact order, then the lower block."""
    D, Hkv, NB = 128, 1, 200
    base = torch.randn(D, generator=gen(1)).bfloat16().float()
    bd = torch.empty(1, Hkv, NB, 2, D)
    bd[0, 0, :, 0], bd[0, 0, :, 1] = base + 1.0, base - 1.0
    tiny = torch.randperm(NB, generator=gen(2)).float()
    bd[0, 0, :, 0, 5] = tiny // 2 * 2.0 ** -7  # pairs of equal blocks
    q = torch.randn(1, 2, D, generator=gen(3))
    q[:, :, 5] = 2.0 ** -26
    bd = bd.bfloat16().cuda()
    for n in (2, 31, 100, 199):
        got = run_select(gd, q.cuda(), bd, [NB * 64 - 1], n, 0, 1)
        check_select(got, q, bd, [NB * 64 - 1], n, 0, 1)
    zero = torch.zeros_like(q).cuda()
    assert run_select(gd, zero, bd, [NB * 64 - 1], 6, 1, 1)[0, 0].tolist() == [0, 1, 2, 3, 4, NB - 1]
    long = torch.ones(1, 1, 8192, 2, 64, dtype=torch.bfloat16, device="cuda")  # 8192 equal blocks
    got = run_select(gd, torch.ones(1, 1, 64, device="cuda"), long, [524287], 100, 2, 3)
    assert got[0, 0].tolist() == list(range(97)) + [8189, 8190, 8191]


def test_selection_with_values_that_are_not_finite(gd):
    D, NB = 64, 40
    bd = torch.randn(1, 1, NB, 2, D, generator=gen(1)).sort(3, descending=True).values
    q = torch.randn(1, 1, D, generator=gen(2)).abs()
    bd[0, 0, 7, 0, 3] = math.inf    # score +inf
    bd[0, 0, 9, :, 4] = math.nan    # score NaN: last
    bd[0, 0, 11, 0, 5] = -math.inf  # score -inf
    bd = bd.bfloat16().cuda()
    got = run_select(gd, q.cuda(), bd, [NB * 64 - 1], 10, 1, 1)
    check_select(got, q, bd, [NB * 64 - 1], 10, 1, 1)
    assert 7 in got[0, 0].tolist() and 9 not in got[0, 0].tolist()
    got = run_select(gd, q.cuda(), bd, [NB * 64 - 1], NB - 1, 0, 0)
    check_select(got, q, bd, [NB * 64 - 1], NB - 1, 0, 0)


def test_selection_leaves_refused_rows(gd):
    bd = torch.zeros(3, 2, 4, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(3, 4, 64, device="cuda")
    got = run_select(gd, q, bd, [-2, 256, 255], 2)
    assert gd.device_error(clear=True) == 4
    assert torch.all(got[:2] == -7) and got[2].tolist() == [[0, 3], [0, 3]]


# ----------------------------------------------------------------------------- attention

def listed_keys(ids, last):
    keys = []
    for i in ids:
        if i >= 0:
            keys += range(64 * i, min(64 * i + 63, last) + 1)
    return keys


def check_attention(q, k, v, pos, ids, o):
    B, Hq, D = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    for b in range(B):
        for g in range(Hkv):
            at = listed_keys(ids[b][g], pos[b])
            qg = q[b, g * G:(g + 1) * G].double()
            kk, vv = k[b, g, at].double(), v[b, g, at].double()
            got = o[b, g * G:(g + 1) * G].double()
            if not at:
                assert torch.all(got == 0.0), (b, g)
                continue
            x = qg @ kk.T / math.sqrt(D)
            p = torch.softmax(x, -1)
            A = (qg.abs() @ kk.abs().T).amax(-1) / math.sqrt(D)
            tol = 2.0 ** -14 * (1 + A[:, None]) * (p @ vv.abs())
            bad = (got - p @ vv).abs() > tol
            assert not bad.any(), (b, g, float(((got - p @ vv).abs() / tol).max()))


ATTN = [
    # D, Hq, Hkv, S_max, pos, n_select
    (64, 1, 1, 1, [0], 1),
    (64, 4, 2, 200, [199, 0, 64], 3),
    (128, 32, 8, 2000, [1999, 1023], 9),
    (128, 12, 3, 1111, [1110, 63, 5], 4),
    (128, 16, 2, 640, [639, 600], 10),
    (64, 16, 1, 900, [899, 128], 5),
    (128, 15, 1, 4100, [4099], 64),
    (128, 6, 3, 500, [499, 499, 498], 1),
]


@pytest.mark.parametrize("D,Hq,Hkv,S,pos,n", ATTN)
def test_attention_over_listed_blocks(gd, D, Hq, Hkv, S, pos, n):
    """Random lists in any order, with empty places in between; slots behind pos hold NaN."""
    B = len(pos)
    k, v = make_k(B, Hkv, S, D, 11), make_k(B, Hkv, S, D, 13)
    r = gen(17)
    ids = torch.full((B, Hkv, n), -1, dtype=torch.int32)
    for b in range(B):
        k[b, :, pos[b] + 1:] = float("nan")
        v[b, :, pos[b] + 1:] = float("nan")
        for g in range(Hkv):
            perm = torch.randperm(n_blocks(S), generator=r)[:n].to(torch.int32)
            ids[b, g, :perm.numel()] = perm
            if n > 2:
                ids[b, g, int(torch.randint(n, (1,), generator=r))] = -1
    q = torch.randn(B, Hq, D, generator=gen(4)).cuda()
    o = torch.full_like(q, float("nan"))
    gd.dec_block_decode_attn(q, k, v, i32(pos), ids.cuda(), o)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 0
    check_attention(q, k, v, pos, ids.tolist(), o)


def test_lists_that_leave_a_row_empty_repeat_or_leave_the_cache(gd):
    B, Hq, Hkv, D, S = 5, 4, 2, 128, 320
    k, v = make_k(B, Hkv, S, D, 21), make_k(B, Hkv, S, D, 23)
    pos = [319, 100, -1, 319, 64]
    ids = [[[-1, -1, -1], [4, 4, 0]],   # a head without blocks; a block twice
           [[2, 3, 4], [1, 2, 0]],      # only blocks behind the last key; one of three
           [[0, 1, 2], [0, 1, 2]],      # a row without keys
           [[5, 0, 1], [2 ** 30, -2, 3]],  # ids outside the cache
           [[1, -1, -1], [1, 0, -1]]]   # a block of one key
    q = torch.randn(B, Hq, D, generator=gen(4)).cuda()
    o = torch.full_like(q, float("nan"))
    gd.dec_block_decode_attn(q, k, v, i32(pos), i32(ids), o)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 4
    ids[3] = [[0, 1], [3]]
    check_attention(q, k, v, pos, ids, o)
    o.fill_(-5.0)
    gd.dec_block_decode_attn(q, k, v, i32([0, 320, -2, 0, 0]), i32(ids[:3] + [[[0, 1, 2]] * 2] * 2), o)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 4 and torch.all(o[1:3] == -5.0) and torch.all(o[0, :2] == 0.0)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_keys_and_values_that_are_not_finite(gd, bad, n):
    """They reach the outputs of what attends to them and no others, and none from slots behind the last."""
    B, Hq, Hkv, D, S = 4, 8, 2, 64, 2560
    g = gen(77)
    k, v = (torch.randn(B, Hkv, S, D, generator=g).bfloat16().cuda() for _ in range(2))
    q = torch.randn(B, Hq, D, generator=g).cuda()
    k[0, 1, 70, 5] = bad         # listed
    v[1, 0, 64, 9] = bad         # listed
    k[2, 0, 151:, :] = bad       # behind the last key, the same block
    v[2, 0, 151:, :] = bad
    if n == 3:
        k[3, 1, 64 * 30, 2] = bad  # not listed
    blocks = torch.arange(n, dtype=torch.int32, device="cuda").expand(B, Hkv, -1).contiguous()
    o = torch.empty(B, Hq, D, device="cuda")
    gd.dec_block_decode_attn(q, k, v, i32([200, 200, 150, 2500]), blocks, o)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 0
    want = torch.zeros(B, Hq, D, dtype=torch.bool, device="cuda")
    want[0, 4:] = True
    want[1, :4, 9] = True
    assert torch.equal(o.isnan(), want) and torch.isfinite(o[~want]).all()


def test_many_blocks_per_warp(gd):
    """Lists long enough that a warp walks more than 64 units, and every id is read once."""
    B, Hq, Hkv, D, S = 16, 4, 4, 64, 40000
    k, v = (torch.randn(B, Hkv, S, D, generator=gen(i)).bfloat16().cuda() for i in (1, 2))
    pos = [S - 1 - 997 * b for b in range(B)]
    n = n_blocks(S)
    ids = torch.stack([torch.randperm(n, generator=gen(b)) for b in range(B * Hkv)]).view(B, Hkv, n).to(torch.int32)
    q = torch.randn(B, Hq, D, generator=gen(4)).cuda()
    o = torch.empty_like(q)
    gd.dec_block_decode_attn(q, k, v, i32(pos), ids.cuda(), o)
    check_attention(q, k, v, pos, ids.tolist(), o)
    assert gd.device_error(clear=True) == 0


@pytest.mark.parametrize("D,Hq,Hkv,S,B,n", [(128, 16, 2, 700, 40, 5), (128, 16, 1, 300, 110, 3), (64, 24, 2, 900, 33, 7),
                                            (128, 4, 4, 2000, 30, 12), (128, 16, 1, 100, 1024, 2)])
def test_attention_of_many_rows(gd, D, Hq, Hkv, S, B, n):
    """More (row, KV head) items than clusters fit: runs across items, cut items joined, every group width."""
    k, v = make_k(B, Hkv, S, D, 61), make_k(B, Hkv, S, D, 63)
    pos = [(37 * b * b + 11 * b) % (S + 1) - 1 for b in range(B)]
    r = gen(19)
    ids = torch.randint(-1, n_blocks(S), (B, Hkv, n), generator=r).to(torch.int32)
    q = torch.randn(B, Hq, D, generator=gen(4)).cuda()
    o = torch.full_like(q, float("nan"))
    gd.dec_block_decode_attn(q, k, v, i32(pos), ids.cuda(), o)
    check_attention(q, k, v, pos, ids.tolist(), o)
    assert gd.device_error(clear=True) == 0


def test_selection_of_many_rows(gd):
    """One CTA per (row, KV head), where clusters of them do not fit."""
    B, Hq, Hkv, D, S, n = 60, 8, 4, 64, 5000, 9
    bd = torch.randn(B, Hkv, n_blocks(S), 2, D, generator=gen(1)).sort(3, descending=True).values.bfloat16().cuda()
    q = torch.randn(B, Hq, D, generator=gen(3)).cuda()
    pos = [(131 * b) % (S + 1) - 1 for b in range(B)]
    got = run_select(gd, q, bd, pos, n, 1, 1)
    assert gd.device_error(clear=True) == 0
    check_select(got, q, bd, pos, n, 1, 1)


def test_a_decode_step_with_selected_blocks(gd):
    """As a decode loop runs them: bounds of the prompt, then per step the new slot's bounds, the selection and
    the attention.  With every block listed it is dec_gqa_decode_attn; captured, it replays to the same bits."""
    B, H, Hq, Hkv, D, S = 2, 256, 8, 2, 64, 1024
    k, v = make_k(B, Hkv, S, D, 31), make_k(B, Hkv, S, D, 33)
    W = [(torch.randn(n * D, H, generator=gen(5 + n)) * 0.06).bfloat16().cuda() for n in (Hq, Hkv, Hkv)]
    start = [700, 510]
    bd = torch.zeros(B, Hkv, n_blocks(S), 2, D, dtype=torch.bfloat16, device="cuda")
    gd.dec_block_bounds(k, i32([0, 0]), bd, tokens=700)
    pos = i32(start)
    y = torch.empty(B, H, device="cuda")
    q, o, full = (torch.empty(B, Hq, D, device="cuda") for _ in range(3))
    blocks = torch.empty(B, Hkv, 6, dtype=torch.int32, device="cuda")
    every = torch.arange(n_blocks(S), dtype=torch.int32, device="cuda").expand(B, Hkv, -1).contiguous()
    ws = None

    def step():
        nonlocal ws
        gd.dec_qkv_gemv_rope(y, *W, pos, 1e6, q.view(B, -1), k, v)
        gd.dec_block_bounds(k, pos, bd)
        gd.dec_select_blocks(q, bd, pos, blocks)
        ws = gd.dec_block_decode_attn(q, k, v, pos, blocks, o, ws=ws)

    for i in range(4):
        y.copy_(torch.randn(B, H, generator=gen(50 + i)))
        step()
        at = [s + i for s in start]
        # the second row's bounds of the prompt reach past its keys until its blocks are written again
        for b in range(B):
            for h in range(Hkv):
                assert torch.equal(bd[b, h, at[b] // 64], R.bounds(k[b, h], at[b])[-1])
        check_select(blocks.cpu(), q, bd, at, 6, 1, 1)
        check_attention(q, k, v, at, blocks.tolist(), o)
        pos += 1
    pos -= 1
    gd.dec_block_decode_attn(q, k, v, pos, every, o, ws=ws)
    gd.dec_gqa_decode_attn(q, k, v, pos, full)
    at = [s + 3 for s in start]
    check_attention(q, k, v, at, every.tolist(), o)
    check_attention(q, k, v, at, every.tolist(), full)
    step()
    ref = [t.clone() for t in (bd, blocks, o)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    o.zero_()
    blocks.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(ref, (bd, blocks, o)))
    assert gd.device_error(clear=True) == 0


def test_offsets_past_32_bits(gd):
    """The last row of caches of 4.3 GB each."""
    B, Hq, Hkv, D, S = 64, 8, 8, 128, 32832
    k, v = (torch.zeros(B, Hkv, S, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    assert k.numel() * 2 > 1 << 32
    k[-1, :, -500:] = torch.randn(Hkv, 500, D, generator=gen(1)).bfloat16().cuda()
    v[-1, :, -500:] = torch.randn(Hkv, 500, D, generator=gen(2)).bfloat16().cuda()
    q = torch.randn(B, Hq, D, generator=gen(3)).cuda()
    bd = torch.zeros(B, Hkv, n_blocks(S), 2, D, dtype=torch.bfloat16, device="cuda")
    pos = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    pos[-1] = S - 1
    at = torch.zeros(B, dtype=torch.int32, device="cuda")
    at[-1] = S - 500
    gd.dec_block_bounds(k, at, bd, tokens=500)
    blocks = torch.empty(B, Hkv, 8, dtype=torch.int32, device="cuda")
    gd.dec_select_blocks(q, bd, pos, blocks)
    o = torch.empty_like(q)
    gd.dec_block_decode_attn(q, k, v, pos, blocks, o)
    assert torch.all(o[:-1] == 0) and torch.all(blocks[:-1] == -1)
    for h in range(Hkv):
        assert torch.equal(bd[-1, h, -8:], R.bounds(k[-1, h], S - 1)[-8:])
    check_select(blocks[-1:].cpu(), q[-1:], bd[-1:], [S - 1], 8, 1, 1)
    check_attention(q[-1:], k[-1:], v[-1:], [S - 1], blocks[-1:].tolist(), o[-1:])
    assert gd.device_error(clear=True) == 0
