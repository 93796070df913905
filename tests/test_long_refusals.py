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


def test_selection_slots_that_do_not_match_the_bounds(gd):  # noqa: F811
    q, pos = torch.zeros(2, 4, 64), torch.zeros(2, dtype=torch.int32)
    bounds, blocks = torch.zeros(2, 2, 3, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 2, dtype=torch.int32)
    for slots in (128, 193, 0, -1):
        with pytest.raises(gd.DecError, match="slots"):
            gd.dec_select_blocks(q, bounds, pos, blocks, S_max=slots)
    with pytest.raises(gd.DecError, match="CUDA device"):  # these match
        gd.dec_select_blocks(q, bounds, pos, blocks, S_max=129)


@pytest.mark.gpu
def test_selection_refuses_positions_behind_the_cache(gd):  # noqa: F811
    """The cache's slots may end inside its last block: a position behind them is outside the cache."""
    S = 130
    q = torch.zeros(3, 4, 64, device="cuda")
    bounds = torch.zeros(3, 2, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    blocks = torch.full((3, 2, 3), -7, dtype=torch.int32, device="cuda")
    pos = torch.tensor([129, 130, 191], dtype=torch.int32, device="cuda")
    gd.dec_select_blocks(q, bounds, pos, blocks, S_max=S)
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 4
    assert blocks.tolist() == [[[0, 1, 2]] * 2] + [[[-7, -7, -7]] * 2] * 2
    gd.dec_select_blocks(q, bounds, pos, blocks)  # not told, every block counts as whole
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 0 and blocks.tolist() == [[[0, 1, 2]] * 2] * 3
