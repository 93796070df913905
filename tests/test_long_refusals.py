"""Refusals of the long-cache calls that name their reason, on the host."""
import pytest
import torch

from test_long_args import gd  # noqa: F401


@pytest.mark.parametrize("sizes,word", [((4, 0, 64), "Hkv"), ((4, -2, 64), "Hkv"), ((4, 2, 80), "head_dim"),
                                        ((4, 2, 0), "head_dim"), ((5, 2, 64), "multiple"), ((34, 2, 64), "above 16")])
def test_a_workspace_size_of_zero_leaves_its_reason(gd, sizes, word):  # noqa: F811
    assert gd.lib().dec_add_rmsnorm(None, None, None, None, 1, 64, 0.0, None) != gd.DEC_OK  # another call's message
    assert gd.long_attn_workspace_size(*sizes) == 0
    assert word in gd.lib().dec_last_error().decode()


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,code,word", [
    (4, 2, 96, "DEC_EUNSUPPORTED", "head_dim"), (5, 2, 64, "DEC_EINVAL", "multiple"),
    (34, 2, 64, "DEC_EUNSUPPORTED", "above 16")])
def test_sizes_are_refused_alike_with_and_without_a_workspace(gd, Hq, Hkv, D, code, word):  # noqa: F811
    B, S = 2, 64
    q = torch.zeros(B, Hq, D, device="cuda")
    kv = torch.zeros(B, Hkv, S, D, dtype=torch.bfloat16, device="cuda")
    cache = [torch.zeros(B, Hkv, S, D // 2, dtype=torch.uint8, device="cuda") if i % 2 == 0 else
             torch.zeros(B, Hkv, S, D // 32, 2, dtype=torch.float16, device="cuda") for i in range(4)]
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    blocks = torch.zeros(B, Hkv, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(gd.DecError):  # another call's message
        gd.dec_block_bounds(kv, pos, torch.zeros(B, Hkv, 1, 2, D, dtype=torch.bfloat16, device="cuda"), tokens=S + 1)
    for ws in (None, torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")):
        for call in (lambda: gd.dec_kv4_decode_attn(q, *cache, pos, q.clone(), ws=ws),
                     lambda: gd.dec_block_decode_attn(q, kv, kv, pos, blocks, q.clone(), ws=ws)):
            with pytest.raises(gd.DecError, match=word) as e:
                call()
            assert e.value.code == getattr(gd, code)
