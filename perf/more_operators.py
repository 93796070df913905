"""Timing cases of the 8-bit weight operators and the mixture-of-experts layer.

Three groups of operators:

* ``pack``   quantising float rows or weights to e4m3 codes with a scale per
             1 x 128 or 128 x 128 block, and reading them back
             (``dec_fp8_quant``, ``dec_fp8_dequant``);
* ``lin``    a linear layer with 8-bit weights: the rows are quantised and
             multiplied, scale block by scale block (``dec_fp8_quant``,
             ``dec_fp8_gemm``);
* ``moe``    a mixture-of-experts layer for a decode step's tokens, bf16 or
             8-bit weights (``dec_moe_route``, ``dec_moe_experts``).

``run`` computes a case in elementary torch operations, or, with ``own`` set,
through the library's entry points.  A code c of a block with scale s stands
for c * s; the scale of a block is the smallest power of two s with
max |x| <= 448 s (weights from elsewhere may carry any float scale).
"""
import math

import torch

own = False

BLOCK = 128
TOP = 448.0  # the largest e4m3 value


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # the normed rows of 16 sequences ahead of an 8-bit projection: latency only
        dict(name="pack_rows_b16", op="pack", n=1, rows=16, K=2560, block_rows=1, bf16=False),
        # one projection of the smallest model: latency only
        dict(name="pack_weights_tiny", op="pack", n=1, rows=704, K=256, block_rows=128, bf16=True),
        # a layer's experts taken over from bf16, 64 matrices of an odd number of half blocks
        dict(name="pack_experts", op="pack", n=64, rows=1216, K=2560, block_rows=128, bf16=True),
        # the one-layer model's gate projection for one token
        dict(name="lin_tiny", op="lin", M=1, K=256, N=704, bf16=False, residual=False),
        # the 4B-class layer's gate and up projection in a decode step at batch 1
        dict(name="lin_b1", op="lin", M=1, K=2560, N=19456, bf16=False, residual=False),
        # a down projection into the residual, 16 sequences
        dict(name="lin_b16", op="lin", M=16, K=8960, N=1536, bf16=False, residual=True),
        # the fused query, key and value projection of one prompt of odd length
        dict(name="lin_prompt_509", op="lin", M=509, K=2560, N=6144, bf16=False, residual=False),
        # the gate and up projection of a long prompt, the largest product
        dict(name="lin_prompt_8k", op="lin", M=8191, K=2560, N=19456, bf16=True, residual=False),
        # a small layer, one token and two of eight experts: the smallest call
        dict(name="moe_tiny", op="moe", T=1, H=256, I=704, E=8, k=2, fp8=False, score="softmax", renorm=True, scale=1.0),
        # a 4B-class layer split into 64 experts of which 8 do the dense layer's work, batch 1
        dict(name="moe_b1", op="moe", T=1, H=2560, I=1216, E=64, k=8, fp8=False, score="softmax", renorm=True, scale=1.0),
        # 16 sequences, 10 of 80 small experts each
        dict(name="moe_b16", op="moe", T=16, H=1536, I=896, E=80, k=10, fp8=False, score="sigmoid", renorm=True, scale=2.5),
        # 16 sequences, 8 of 128 experts in 8 bits: the largest layer
        dict(name="moe_b16_fp8", op="moe", T=16, H=2560, I=1216, E=128, k=8, fp8=True, score="softmax", renorm=True,
             scale=1.0),
    ]


def draw(rng):
    def logint(a, b, step=1):
        v = math.exp(rng.uniform(math.log(a), math.log(b)))
        return max(-(-a // step), min(b // step, int(round(v / step)))) * step

    op = rng.choice(["pack", "lin", "lin", "lin", "moe", "moe", "moe"])
    if op == "pack":
        c = dict(op=op, n=rng.choice([1, 1, logint(2, 64)]), K=logint(64, 8960, 16), block_rows=rng.choice([1, 128]),
                 bf16=rng.random() < 0.5)
        c["rows"] = logint(1, max(1, min(20000, 64 * 1216 * 2560 // (2 * c["n"] * c["K"]))))
        return c
    if op == "lin":
        c = dict(op=op, K=logint(256, 9728, 16), N=logint(96, 19456), bf16=rng.random() < 0.3, residual=rng.random() < 0.4)
        # a decode step's few rows as often as a prompt's many
        most = max(1, min(8191, 8191 * 2560 * 19456 // (c["K"] * c["N"])))
        c["M"] = logint(1, 32) if rng.random() < 0.5 else logint(33, max(34, most))
        return c
    c = dict(op=op, T=rng.choice([1, 1, logint(2, 16)]), H=logint(256, 4096, 16), E=logint(4, 256), fp8=rng.random() < 0.5,
             score=rng.choice(["softmax", "sigmoid"]), renorm=rng.random() < 0.7, scale=rng.choice([1.0, 1.0, 2.5]))
    c["k"] = min(c["E"], logint(1, 10))
    most = 128 * 1216 * 2560 // (c["E"] * c["H"] * (1 if c["fp8"] else 2))
    c["I"] = logint(64, max(64, min(2048, most)), 16)
    return c


def distinct(c):
    """Expected number of distinct experts that T tokens choose, k of E each."""
    return c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** c["T"])


def work(c):
    if c["op"] == "pack":
        each = 2 if c["bf16"] else 4
        values = c["n"] * c["rows"] * c["K"]
        scales = c["n"] * -(-c["rows"] // c["block_rows"]) * -(-c["K"] // BLOCK)
        # values read, codes written, codes read, values written
        return dict(bytes=values * (2 * each + 2) + 8 * scales, flops=4 * values)
    if c["op"] == "lin":
        M, K, N = c["M"], c["K"], c["N"]
        return dict(bytes=M * K * (2 if c["bf16"] else 4) + N * K + 4 * -(-N // BLOCK) * -(-K // BLOCK) +
                    4 * M * N * (2 if c["residual"] else 1), flops=2 * M * K * N)
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    return dict(bytes=int(distinct(c) * 3 * H * I * (1 if c["fp8"] else 2)) + 2 * E * H + 12 * T * H,
                flops=6 * T * k * H * I + 2 * T * E * H)


# --------------------------------------------------------------------------- inputs

def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    def weights(*shape):  # [.., N, K] in bf16, rows and channels of unlike size
        w = normal(*shape).mul_(0.02)
        return w.mul_(torch.exp(0.3 * normal(*shape[:-1], 1))).bfloat16()

    def stored(n, N, K):
        """8-bit weights as a checkpoint holds them: any float scale, chosen so that the largest value is 448."""
        codes = torch.empty(n, N, K, device=dev, dtype=torch.float8_e4m3fn)
        scales = torch.empty(n, -(-N // BLOCK), -(-K // BLOCK), device=dev)
        for i in range(n):
            w = weights(N, K).float()
            scales[i] = block_amax(w, BLOCK) / TOP
            codes[i] = (w / spread(scales[i], N, K, BLOCK)).clamp(-TOP, TOP).to(codes.dtype)
        return codes, scales

    s = dict(c)
    if c["op"] == "pack":
        n, R, K = c["n"], c["rows"], c["K"]
        dtype = torch.bfloat16 if c["bf16"] else torch.float32
        s["x"] = torch.empty(n, R, K, device=dev, dtype=dtype)
        for i in range(n):
            s["x"][i] = weights(R, K) if c["bf16"] else normal(R, K) * torch.exp(0.5 * normal(K))
        s["codes"] = torch.zeros(n, R, K, device=dev, dtype=torch.float8_e4m3fn)
        s["scales"] = torch.zeros(n, -(-R // c["block_rows"]), -(-K // BLOCK), device=dev)
        s["back"] = torch.zeros_like(s["x"])
        return s
    if c["op"] == "lin":
        M, K, N = c["M"], c["K"], c["N"]
        codes, scales = stored(1, N, K)
        s["w"], s["w_scales"] = codes[0], scales[0]
        x = normal(M, K) * torch.exp(0.5 * normal(K))  # channels of unlike size, as normed rows have
        s["x"] = x.bfloat16() if c["bf16"] else x
        s["x_codes"] = torch.zeros(M, K, device=dev, dtype=torch.float8_e4m3fn)
        s["x_scales"] = torch.zeros(M, -(-K // BLOCK), device=dev)
        s["res"] = normal(M, N) if c["residual"] else None
        s["out"] = torch.zeros(M, N, device=dev)
        return s
    T, H, I, E, k = c["T"], c["H"], c["I"], c["E"], c["k"]
    s["y"] = normal(T, H) * torch.exp(0.3 * normal(H))
    s["router"] = (normal(E, H) / math.sqrt(H)).bfloat16()
    s["bias"] = 0.05 * normal(E) if c["score"] == "sigmoid" else None
    s["res"] = normal(T, H)
    s["scales"] = None
    if c["fp8"]:
        (s["wg"], a), (s["wu"], b), (s["wd"], d) = stored(E, I, H), stored(E, I, H), stored(E, H, I)
        s["scales"] = (a, b, d)
    else:
        s["wg"], s["wu"], s["wd"] = (torch.empty(E, *z, device=dev, dtype=torch.bfloat16) for z in ((I, H), (I, H), (H, I)))
        for e in range(E):
            s["wg"][e], s["wu"][e], s["wd"][e] = weights(I, H), weights(I, H), weights(H, I)
    s["ids"] = torch.zeros(T, k, device=dev, dtype=torch.int32)
    s["gates"] = torch.zeros(T, k, device=dev)
    s["out"] = torch.zeros(T, H, device=dev)
    return s


def block_amax(x, block_rows):
    """Largest magnitude of each block of [.., R, K], [.., blocks of R, blocks of K]."""
    R, K = x.shape[-2:]
    x = torch.nn.functional.pad(x.abs(), (0, -K % BLOCK, 0, -R % block_rows))
    return x.unflatten(-1, (-1, BLOCK)).unflatten(-3, (-1, block_rows)).amax((-3, -1))


def spread(scales, R, K, block_rows):
    """The scale of every value of [.., R, K]."""
    if block_rows > 1:
        scales = scales.repeat_interleave(block_rows, -2)[..., :R, :]
    return scales.repeat_interleave(BLOCK, -1)[..., :K]


# --------------------------------------------------------------------------- one pass

def run(s):
    return {"pack": run_pack, "lin": run_lin, "moe": run_moe}[s["op"]](s)


def quantise(x, block_rows):
    """Codes and scales of float32 [.., R, K]."""
    amax = block_amax(x, block_rows)
    mantissa, exponent = torch.frexp(amax)  # amax = mantissa 2^exponent, mantissa in [0.5, 1); 448 = 0.875 2^9
    exponent = exponent - 9 + (mantissa > 0.875).int()
    scale = ((exponent.clamp(min=-126) + 127) << 23).view(torch.float32)
    scale = torch.where(amax > 0, scale, 1.0)
    return (x / spread(scale, *x.shape[-2:], block_rows)).to(torch.float8_e4m3fn), scale


def run_pack(s):
    if own:
        import greedy_decode_step_gb300 as gd
        gd.dec_fp8_quant(s["x"], s["codes"], s["scales"], block_rows=s["block_rows"])
        gd.dec_fp8_dequant(s["codes"], s["scales"], s["back"], block_rows=s["block_rows"])
        return s["back"], s["scales"]
    for i in range(s["n"]):
        codes, scales = quantise(s["x"][i].float(), s["block_rows"])
        s["codes"][i], s["scales"][i] = codes, scales
        s["back"][i] = s["codes"][i].float() * spread(s["scales"][i], s["rows"], s["K"], s["block_rows"])
    return s["back"], s["scales"]


def run_lin(s):
    if own:
        import greedy_decode_step_gb300 as gd
        gd.dec_fp8_quant(s["x"], s["x_codes"], s["x_scales"])
        gd.dec_fp8_gemm(s["x_codes"], s["x_scales"], s["w"], s["w_scales"], s["out"], residual=s["res"])
        return s["out"]
    codes, scales = quantise(s["x"].float(), 1)
    x = codes.float() * spread(scales, s["M"], s["K"], 1)
    w = s["w"].float() * spread(s["w_scales"], s["N"], s["K"], BLOCK)
    out = x @ w.T
    s["out"].copy_(out + s["res"] if s["residual"] else out)
    return s["out"]


def run_moe(s):
    if own:
        import greedy_decode_step_gb300 as gd
        gd.dec_moe_route(s["y"], s["router"], s["ids"], s["gates"], bias=s["bias"], score=s["score"],
                         renormalise=s["renorm"], scale=s["scale"])
        # the workspace of the first call is kept, as a serving loop keeps it
        s["ws"] = gd.dec_moe_experts(s["y"], s["ids"], s["gates"], s["wg"], s["wu"], s["wd"], s["out"], residual=s["res"],
                                     scales=s["scales"], ws=s.get("ws"))
        return s["ids"], s["gates"], s["out"]
    y, k = s["y"], s["k"]
    z = y.double() @ s["router"].double().T  # in 64 bits, as experts are chosen by it
    if s["score"] == "softmax":
        p = torch.exp(z - z.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
        rank = z
    else:
        p = 1.0 / (1.0 + torch.exp(-z))
        rank = p + s["bias"].double()
    ids = rank.sort(dim=-1, descending=True, stable=True).indices[:, :k]  # ties: the lower id first
    gates = p.gather(1, ids)
    if s["renorm"]:
        gates = gates / gates.sum(-1, keepdim=True)
    s["ids"].copy_(ids)
    s["gates"].copy_(gates * s["scale"])

    def chosen(name, i, t):  # the chosen experts' matrices of token t, [k, ., .]
        w = s[name][ids[t]].float()
        if s["fp8"]:
            w *= spread(s["scales"][i][ids[t]], *w.shape[-2:], BLOCK)
        return w

    for t in range(s["T"]):
        gate, up = (chosen(n, i, t) @ y[t] for i, n in ((0, "wg"), (1, "wu")))  # [k, I]
        h = gate / (1.0 + torch.exp(-gate)) * up
        down = (chosen("wd", 2, t) @ h[..., None]).squeeze(-1)  # [k, H]
        s["out"][t] = s["res"][t] + (s["gates"][t, :, None] * down).sum(0)
    return s["ids"], s["gates"], s["out"]


# --------------------------------------------------------------------------- in 64 bits

def exact(c, seed):
    """The operators' definitions in 64 bits."""
    s = prepare(c, seed)
    f64 = torch.float64

    def blocks(x, rows):
        """(index of rows, index of columns) of every block of a matrix."""
        for i in range(0, x.shape[0], rows):
            for j in range(0, x.shape[1], BLOCK):
                yield slice(i, min(i + rows, x.shape[0])), slice(j, min(j + BLOCK, x.shape[1]))

    def held(x, rows):
        """What a matrix's codes stand for, and the scales, from the values alone."""
        x = x.to(f64)
        pad_r, pad_k = -x.shape[0] % rows, -x.shape[1] % BLOCK
        full = torch.zeros(x.shape[0] + pad_r, x.shape[1] + pad_k, dtype=f64, device=x.device)
        full[:x.shape[0], :x.shape[1]] = x
        tiles = full.reshape(full.shape[0] // rows, rows, full.shape[1] // BLOCK, BLOCK)
        top = tiles.abs().amax(3).amax(1)
        scale = torch.exp2(torch.ceil(torch.log2(torch.where(top > 0, top, TOP) / TOP)))
        # the logarithm may be off by its last place: the definition's bounds settle it
        scale = torch.where(scale * TOP < top, scale * 2, scale)
        scale = torch.where((scale / 2 * TOP >= top) & (top > 0), scale / 2, scale)
        v = tiles / scale[:, None, :, None]
        # nearest of a grid of 3 bits below the leading one, from 2^-9 on
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        v = torch.round(v / step) * step * scale[:, None, :, None]
        return v.reshape(full.shape)[:x.shape[0], :x.shape[1]], scale

    def decoded(codes, scales):
        w = codes.to(torch.float32).to(f64)
        for a, b in blocks(w, BLOCK):
            w[a, b] *= scales[a.start // BLOCK, b.start // BLOCK].to(f64)
        return w

    if c["op"] == "pack":
        parts = [held(s["x"][i], c["block_rows"]) for i in range(c["n"])]
        return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])
    if c["op"] == "lin":
        x, w = held(s["x"], 1)[0], decoded(s["w"], s["w_scales"])
        out = torch.einsum("mk,nk->mn", x, w)
        return out if s["res"] is None else out + s["res"].to(f64)
    T, k = c["T"], c["k"]
    ids = torch.zeros(T, k, dtype=torch.int32, device=s["y"].device)
    gates = torch.zeros(T, k, dtype=f64, device=s["y"].device)
    out = s["res"].to(f64)
    for t in range(T):
        y = s["y"][t].to(f64)
        z = torch.mv(s["router"].to(f64), y)
        p = torch.softmax(z, 0) if c["score"] == "softmax" else torch.sigmoid(z)
        key = (p if s["bias"] is None else p + s["bias"].to(f64)).tolist()
        take = sorted(range(c["E"]), key=lambda e: (-key[e], e))[:k]
        ids[t] = torch.tensor(take, dtype=torch.int32)
        gate = p[take]
        gates[t] = c["scale"] * (gate / gate.sum() if c["renorm"] else gate)
        for j, e in enumerate(take):
            wg, wu, wd = ((decoded(s[n][e], s["scales"][i][e]) if c["fp8"] else s[n][e].to(f64))
                          for i, n in enumerate(("wg", "wu", "wd")))
            a = torch.mv(wg, y)
            out[t] += gates[t, j] * torch.mv(wd, a * torch.sigmoid(a) * torch.mv(wu, y))
    return ids, gates, out
