"""Weights that the launch right ahead of a call writes, whatever launch that is:
the call reads what was written, eager and replayed from a graph."""
import pytest
import torch

pytestmark = pytest.mark.gpu
gd = pytest.importorskip("greedy_decode_step_gb300")


@pytest.fixture(autouse=True)
def no_device_error():
    gd.lib()
    gd.device_error(clear=True)
    yield
    torch.cuda.synchronize()
    assert gd.device_error(clear=True) == 0


def normal(seed, *shape):
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def packed(x, rows):
    c = torch.zeros(x.shape, dtype=torch.uint8, device="cuda")
    s = torch.zeros(-(-x.shape[0] // rows), -(-x.shape[1] // 128), device="cuda")
    gd.dec_fp8_quant(x, c, s, block_rows=rows)
    return c, s


# a column of weights, few rows, tiles of 64 to 256 columns, pairs of CTAs
@pytest.mark.parametrize("M,N,K", [(1, 1, 4096), (1, 19456, 2560), (16, 1536, 8960), (64, 9728, 2560), (500, 6140, 1040),
                                   (2040, 9704, 2576)])
def test_product(M, N, K):
    x = packed(normal(1, M, K), 1)
    sets = [packed(0.05 * normal(2 + i, N, K), 128) for i in range(3)]
    want = []
    for w in sets:
        torch.cuda.synchronize()
        want.append(torch.zeros(M, N, device="cuda"))
        gd.dec_fp8_gemm(*x, *w, want[-1])
    assert not torch.equal(want[0], want[1]) and not torch.equal(want[1], want[2])
    wc, ws = torch.zeros_like(sets[0][0]), torch.zeros_like(sets[0][1])
    outs = [torch.zeros(M, N, device="cuda") for _ in range(9)]

    def run():
        for i, out in enumerate(outs):
            ws.copy_(sets[i % 3][1])
            wc.copy_(sets[i % 3][0])
            gd.dec_fp8_gemm(*x, wc, ws, out)

    torch.cuda.synchronize()
    run()
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 3])
        out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    g.replay()
    for i, out in enumerate(outs):
        assert torch.equal(out, want[i % 3])


@pytest.mark.parametrize("T,H,E,k", [(1, 256, 8, 2), (1, 2560, 64, 8), (16, 1536, 80, 10), (4, 16384, 1024, 16)])
def test_router(T, H, E, k):
    y = normal(11, T, H)
    sets = [(normal(12 + i, E, H) / H ** 0.5).bfloat16() for i in range(3)]
    new = lambda: (torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.zeros(T, k, device="cuda"))
    want = []
    for w in sets:
        torch.cuda.synchronize()
        want.append(new())
        gd.dec_moe_route(y, w, *want[-1])
    assert not torch.equal(want[0][1], want[1][1]) and not torch.equal(want[1][1], want[2][1])
    w, outs = torch.zeros_like(sets[0]), [new() for _ in range(9)]

    def run():
        for i, out in enumerate(outs):
            w.copy_(sets[i % 3])
            gd.dec_moe_route(y, w, *out)

    torch.cuda.synchronize()
    run()
    for i, out in enumerate(outs):
        assert torch.equal(out[0], want[i % 3][0]) and torch.equal(out[1], want[i % 3][1])
        out[1].zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    g.replay()
    for i, out in enumerate(outs):
        assert torch.equal(out[0], want[i % 3][0]) and torch.equal(out[1], want[i % 3][1])
