"""The long-cache calls refuse bad arguments on the host, before any GPU work
(through the C entry points with addresses that are never read, and through
the Python binding with CPU tensors)."""
import pytest
import torch

import long_refs as R

P = 0x1000  # an aligned address; nothing is launched


@pytest.fixture(scope="module")
def gd():
    import greedy_decode_step_gb300 as gd
    gd.build()
    return gd


def refused(gd, name, good, code, word, **change):
    """The call with `good`'s arguments and `change`'s in their place fails with this code and message."""
    unknown = set(change) - set(good)
    assert not unknown, unknown
    rc = getattr(gd.lib(), name)(*{**good, **change}.values())
    msg = gd.lib().dec_last_error().decode()
    assert rc == code and word in msg, (rc, msg)


Q = 0x2000
STORE = dict(k=P, v=P, bf16=0, sb=1024, st=512, sh=128, from_cache=0, src=4, pos=P, lens=None, T=4, kc=P, kp=P, vc=Q, vp=Q,
             B=2, Hkv=4, D=128, group=32, S=64, stream=None)
LOAD = dict(kc=P, kp=P, vc=P, vp=P, pos=P, lens=None, T=4, k=P, v=Q, bf16=1, sb=1024, st=512, sh=128, B=2, Hkv=4, D=128,
            group=32, S=64, stream=None)
ATTN = dict(q=P, kc=P, kp=P, vc=P, vp=P, pos=P, o=P, ws=P, ws_bytes=1 << 40, B=2, Hq=8, Hkv=4, D=128, group=32, S=64,
            stream=None)
BOUNDS = dict(k=P, pos=P, T=1, bounds=P, B=2, Hkv=4, D=128, S=64, stream=None)
SELECT = dict(q=P, bounds=P, pos=P, blocks=P, n=4, first=1, last=1, B=2, Hq=8, Hkv=4, D=128, S=640, stream=None)
BLOCK = dict(q=P, k=P, v=P, pos=P, blocks=P, n=4, o=P, ws=P, ws_bytes=1 << 40, B=2, Hq=8, Hkv=4, D=128, S=640, stream=None)
ALL = [("dec_kv4_store", STORE), ("dec_kv4_load", LOAD), ("dec_kv4_decode_attn", ATTN), ("dec_block_bounds", BOUNDS),
       ("dec_select_blocks", SELECT), ("dec_block_decode_attn", BLOCK)]


@pytest.mark.parametrize("name,good", ALL, ids=[n for n, _ in ALL])
def test_sizes(gd, name, good):
    refused(gd, name, good, gd.DEC_EUNSUPPORTED, "batch", B=0)
    refused(gd, name, good, gd.DEC_EUNSUPPORTED, "batch", B=1025)
    refused(gd, name, good, gd.DEC_EUNSUPPORTED, "Hkv", Hkv=0)
    refused(gd, name, good, gd.DEC_EUNSUPPORTED, "head_dim", D=96)
    refused(gd, name, good, gd.DEC_EINVAL, "S_max", S=0)
    refused(gd, name, good, gd.DEC_EUNSUPPORTED, "2^31", S=1 << 28)
    if "Hq" in good:
        refused(gd, name, good, gd.DEC_EINVAL, "multiple", Hq=6)
        refused(gd, name, good, gd.DEC_EINVAL, "multiple", Hq=0)
        refused(gd, name, good, gd.DEC_EUNSUPPORTED, "above 16", Hq=68)
    if "group" in good:
        refused(gd, name, good, gd.DEC_EUNSUPPORTED, "group", group=16)
        refused(gd, name, good, gd.DEC_EUNSUPPORTED, "group", group=128, D=64)


@pytest.mark.parametrize("name,good", ALL, ids=[n for n, _ in ALL])
def test_pointers(gd, name, good):
    for arg, x in good.items():
        if x in (P, Q):
            refused(gd, name, good, gd.DEC_EINVAL, "null", **{arg: None})
            refused(gd, name, good, gd.DEC_EINVAL, "aligned", **{arg: P + 2})
    if "lens" in good:
        refused(gd, name, good, gd.DEC_EINVAL, "lens", lens=P + 1)


def test_particular_arguments(gd):
    refused(gd, "dec_kv4_store", STORE, gd.DEC_EINVAL, "source has 3", src=3)
    refused(gd, "dec_kv4_store", STORE, gd.DEC_EINVAL, ">= 0", T=-1)
    refused(gd, "dec_kv4_load", LOAD, gd.DEC_EINVAL, ">= 0", T=-1)
    for s in ("sb", "st", "sh"):
        refused(gd, "dec_kv4_store", STORE, gd.DEC_EINVAL, "strides", **{s: 130})
        refused(gd, "dec_kv4_load", LOAD, gd.DEC_EINVAL, "strides", **{s: 132})  # 264 bytes of bf16
        refused(gd, "dec_kv4_load", LOAD, gd.DEC_EINVAL, "strides", **{s: -8})
        refused(gd, "dec_kv4_load", LOAD, gd.DEC_EINVAL, "share memory", **{s: 0})
    refused(gd, "dec_kv4_load", LOAD, gd.DEC_EINVAL, "must differ", v=P)
    refused(gd, "dec_kv4_store", STORE, gd.DEC_EINVAL, "of their own", vc=P)
    refused(gd, "dec_kv4_store", STORE, gd.DEC_EINVAL, "of their own", vp=P)
    for name, good in ALL[:2]:
        refused(gd, name, good, gd.DEC_EUNSUPPORTED, "2^30", T=(1 << 30) + 1, **({"src": 2 ** 31 - 1} if "src" in good else {}))
    need = gd.long_attn_workspace_size(8, 4, 128)
    refused(gd, "dec_kv4_decode_attn", ATTN, gd.DEC_EINVAL, "needs", ws_bytes=need - 1)
    refused(gd, "dec_block_decode_attn", BLOCK, gd.DEC_EINVAL, "needs", ws_bytes=need - 1)
    refused(gd, "dec_kv4_decode_attn", ATTN, gd.DEC_EINVAL, "256", ws=P + 16)
    refused(gd, "dec_block_bounds", BOUNDS, gd.DEC_EINVAL, "T = 65", T=65)
    refused(gd, "dec_block_bounds", BOUNDS, gd.DEC_EINVAL, "T = -1", T=-1)
    refused(gd, "dec_select_blocks", SELECT, gd.DEC_EINVAL, "n_select", n=0)
    refused(gd, "dec_select_blocks", SELECT, gd.DEC_EINVAL, "n_first", first=4, last=1)
    refused(gd, "dec_select_blocks", SELECT, gd.DEC_EINVAL, "n_first", first=-1)
    refused(gd, "dec_select_blocks", SELECT, gd.DEC_EINVAL, "n_first", last=2 ** 31 - 1)
    refused(gd, "dec_select_blocks", SELECT, gd.DEC_EUNSUPPORTED, "524288", S=524289)
    refused(gd, "dec_block_decode_attn", BLOCK, gd.DEC_EINVAL, "n_select", n=0)
    refused(gd, "dec_block_decode_attn", BLOCK, gd.DEC_EUNSUPPORTED, "2^28", n=1 << 27)


def test_no_tokens_is_no_work(gd):
    for name, good in ALL[:2] + [ALL[3]]:
        assert getattr(gd.lib(), name)(*{**good, "T": 0}.values()) == gd.DEC_OK


def test_workspace_size(gd):
    assert gd.long_attn_workspace_size(32, 8, 128) >= 2 * 2 * 152 * 4 * 130 * 4
    assert gd.long_attn_workspace_size(16, 1, 64) > 0
    for bad in ((0, 1, 64), (17, 1, 64), (4, 3, 64), (4, 2, 80), (4, 0, 64)):
        assert gd.long_attn_workspace_size(*bad) == 0


# ----------------------------------------------------------------------------- Python binding

def cache(B=2, Hkv=2, S=8, D=64, group=32):
    return [torch.zeros(B, Hkv, S, D // 2, dtype=torch.uint8), torch.zeros(B, Hkv, S, D // group, 2, dtype=torch.float16),
            torch.zeros(B, Hkv, S, D // 2, dtype=torch.uint8), torch.zeros(B, Hkv, S, D // group, 2, dtype=torch.float16)]


def test_binding_refuses_cpu_tensors(gd):
    pos, rows, q = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, 2, 64), torch.zeros(2, 4, 64)
    kv = torch.zeros(2, 2, 128, 64, dtype=torch.bfloat16)
    blocks, bd = torch.zeros(2, 2, 2, dtype=torch.int32), torch.zeros(2, 2, 2, 2, 64, dtype=torch.bfloat16)
    ws = torch.zeros(1 << 22, dtype=torch.uint8)
    for call in (lambda: gd.dec_kv4_store(rows, rows, pos, *cache()),
                 lambda: gd.dec_kv4_load(*cache(), pos, rows, rows),
                 lambda: gd.dec_kv4_decode_attn(q, *cache(), pos, q, ws=ws),
                 lambda: gd.dec_block_bounds(kv, pos, bd),
                 lambda: gd.dec_select_blocks(q, bd, pos, blocks),
                 lambda: gd.dec_block_decode_attn(q, kv, kv, pos, blocks, q, ws=ws)):
        with pytest.raises(gd.DecError, match="CUDA device"):
            call()


def test_binding_refuses_types_shapes_and_layouts(gd):
    pos, rows, q = torch.zeros(2, dtype=torch.int32), torch.zeros(2, 3, 2, 64), torch.zeros(2, 4, 64)
    with pytest.raises(TypeError, match="pos"):
        gd.dec_kv4_store(rows, rows, pos.long(), *cache())
    with pytest.raises(TypeError, match="k must be"):
        gd.dec_kv4_store(rows.double(), rows, pos, *cache())
    with pytest.raises(gd.DecError, match="one type"):
        gd.dec_kv4_store(rows, rows.bfloat16(), pos, *cache())
    with pytest.raises(gd.DecError, match="rows"):
        gd.dec_kv4_store(rows[:, :, :1], rows, pos, *cache())
    with pytest.raises(gd.DecError, match="contiguous values"):
        gd.dec_kv4_store(rows.transpose(2, 3).contiguous().transpose(2, 3), rows, pos, *cache())
    with pytest.raises(gd.DecError, match="strided alike"):
        gd.dec_kv4_store(rows, rows.transpose(1, 2).contiguous().transpose(1, 2), pos, *cache())
    bad = cache()
    bad[2] = bad[2][:, :, :7]
    with pytest.raises(gd.DecError, match="v_codes"):
        gd.dec_kv4_load(*bad, pos, rows, rows)
    bad = cache()
    bad[3] = bad[3].float()
    with pytest.raises(TypeError, match="v_params"):
        gd.dec_kv4_decode_attn(q, *bad, pos, q)
    with pytest.raises(gd.DecError, match="o must have shape"):
        gd.dec_kv4_decode_attn(q, *cache(), pos, q[:, :2], ws=torch.zeros(1 << 22, dtype=torch.uint8))
    with pytest.raises(gd.DecError):
        gd.dec_kv4_decode_attn(q[0], *cache(), pos, q)
    kv = torch.zeros(2, 2, 128, 64, dtype=torch.bfloat16)
    with pytest.raises(gd.DecError, match="bounds"):
        gd.dec_block_bounds(kv, pos, torch.zeros(2, 2, 3, 2, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous"):
        gd.dec_block_bounds(kv.transpose(1, 2).contiguous().transpose(1, 2), pos, torch.zeros(2, 2, 2, 2, 64).bfloat16())


# ----------------------------------------------------------------------------- the plain forms themselves

def test_plain_quantiser_is_within_its_step():
    x = torch.randn(200, 128, generator=torch.Generator().manual_seed(1)) * 3
    for group in (32, 64, 128):
        c, p = R.quantise(x, group)
        err = (R.values(R.pack(c), p) - x.double()).abs()
        # half a step, plus what rounding s and z to half may move the ends: 15 s 2^-11 + |z| 2^-11
        s, z = (p[..., i].double().repeat_interleave(group, -1) for i in (0, 1))
        assert (err <= 0.5 * s * (1 + 2 ** -9) + (15 * s + z.abs()) * 2 ** -11).all()


def test_selection_bound_covers_every_key():
    g = torch.Generator().manual_seed(2)
    k, q = torch.randn(300, 64, generator=g), torch.randn(3, 64, generator=g)
    bd = R.bounds(k, 280).double()
    score = torch.maximum(q.double()[:, None] * bd[:, 0], q.double()[:, None] * bd[:, 1]).sum(-1)
    for j in range(bd.shape[0]):
        keys = k[64 * j:min(281, 64 * j + 64)].double()
        assert ((q.double() @ keys.T).amax(-1) <= score[:, j] + 1e-9).all()
