"""Timing cases of the long-cache decode operators.

Three groups of operators, all on a decode step's KV cache:

* ``kv4``     quantising K/V rows into the 4-bit cache as they are written, and
              reading a range of it back (``dec_kv4_store``, ``dec_kv4_load``);
* ``kv4attn`` GQA decode attention over the 4-bit cache (``dec_kv4_decode_attn``);
* ``bounds``  per-block channel bounds of the bf16 key cache (``dec_block_bounds``);
* ``sparse``  attention over the blocks that the bounds' cheap score selects for
              each row and KV head (``dec_select_blocks``, ``dec_block_decode_attn``).

``run`` computes a case in elementary torch operations, or, with ``own`` set,
through the library's entry points.  The 4-bit cache holds, for each (row, KV
head, slot), D/2 bytes (dim 2i in the low, 2i + 1 in the high nibble of byte
i) and per group of dims a half-precision pair (scale s, middle z); a code c
stands for z + s * (c - 8).
"""
import math

import torch

own = False

BLOCK = 64  # keys of a selectable block


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token of the one-layer model (4 query, 2 KV heads of 64): the smallest call, latency only
        dict(name="kv4_one_token", op="kv4", src="rows", B=1, T=1, Hq=4, Hkv=2, D=64, group=32, S_max=160, lo=129, hi=129),
        # one new token of each of 16 sequences, from the fused projection's rows (12 query, 3 KV heads of 128)
        dict(name="kv4_step_b16", op="kv4", src="rows", B=16, T=1, Hq=12, Hkv=3, D=128, group=64, S_max=8320, lo=8192,
             hi=8192),
        # a prompt's bf16 cache taken over into 4 bits, eight padded sequences of odd lengths
        dict(name="kv4_prompt_b8", op="kv4", src="cache", B=8, T=4093, Hq=32, Hkv=8, D=128, group=32, S_max=4096, lo=1021,
             hi=4093),
        # the one-layer model's attention: two rows of about 128 keys
        dict(name="kv4attn_tiny", op="kv4attn", B=2, Hq=4, Hkv=2, D=64, group=64, S_max=160, lo=97, hi=129),
        # the 4B-class layer at batch 1 and a 4096-key cache, 32 query over 8 KV heads
        dict(name="kv4attn_b1_4k", op="kv4attn", B=1, Hq=32, Hkv=8, D=128, group=32, S_max=4096, lo=4095, hi=4095),
        # 16 sequences of 8192 keys, 12 query over 3 KV heads
        dict(name="kv4attn_b16_8k", op="kv4attn", B=16, Hq=12, Hkv=3, D=128, group=64, S_max=8320, lo=8193, hi=8193),
        # eight ragged sequences of 1024 to 32768 keys of the 4B-class layer: the largest cache read
        dict(name="kv4attn_b8_32k", op="kv4attn", B=8, Hq=32, Hkv=8, D=128, group=32, S_max=32768, lo=1024, hi=32768),
        # the block bounds after one decode step of 16 sequences
        dict(name="bounds_step_b16", op="bounds", B=16, T=1, Hq=12, Hkv=3, D=128, S_max=8320, lo=8120, hi=8261),
        # the block bounds of eight prompts' whole caches
        dict(name="bounds_prompt_b8", op="bounds", B=8, T=8191, Hq=32, Hkv=8, D=128, S_max=8192, lo=8191, hi=8191),
        # few heads (6 query over 3 KV heads), a short odd cache: selection and attention as latency
        dict(name="sparse_gqa6x3_b2", op="sparse", B=2, Hq=6, Hkv=3, D=128, S_max=2111, lo=1500, hi=2100, n_select=16),
        # one sequence of 32768 keys, 4096 of them attended
        dict(name="sparse_b1_32k", op="sparse", B=1, Hq=32, Hkv=8, D=128, S_max=32768, lo=32767, hi=32767, n_select=64),
        # eight ragged long sequences, 64 blocks each
        dict(name="sparse_b8_32k", op="sparse", B=8, Hq=32, Hkv=8, D=128, S_max=32768, lo=1024, hi=32768, n_select=64),
    ]


def draw(rng):
    def logint(a, b):
        return max(a, min(b, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))

    op = rng.choice(["kv4", "kv4attn", "kv4attn", "bounds", "sparse", "sparse"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, B=logint(1, 16), Hq=Hkv * rng.choice([1, 2, 3, 4, 4, 5, 8]), Hkv=Hkv, D=D)
    # keys of all rows and heads: at most those of the largest listed case of the kind
    most = {"kv4": 8 * 8 * 2048, "kv4attn": 8 * 8 * 16384, "bounds": 8 * 8 * 8192, "sparse": 8 * 8 * 16384}[op] // (c["B"] * Hkv)
    if op == "kv4":
        # one token each (a decode step) as often as a prompt
        c.update(src=rng.choice(["rows", "cache"]), group=rng.choice([32, 64, D]),
                 T=1 if rng.random() < 0.5 else logint(2, min(8192, most)))
        if c["T"] == 1:
            c["lo"] = c["hi"] = logint(1, min(8192, most))
        else:
            c["hi"] = c["T"]
            c["lo"] = logint(1, c["T"])
        c["S_max"] = c["hi"] + rng.randint(0, 70)
        return c
    hi = logint(1 if op != "sparse" else 500, min(32768, most))
    c.update(hi=hi, lo=logint(max(1, hi // 32), hi), S_max=hi + rng.randint(0, 70))
    if op == "kv4attn":
        c["group"] = rng.choice([32, 64, D])
    elif op == "bounds":
        c["T"] = 1 if rng.random() < 0.5 else logint(1, c["lo"])
    else:
        c["n_select"] = logint(4, 64)
    return c


def lengths(c):
    """Keys of each row once the call's tokens are in: spread evenly from lo to hi."""
    B = c["B"]
    return [c["lo"] + (c["hi"] - c["lo"]) * i // max(1, B - 1) for i in range(B)]


def work(c):
    B, Hq, Hkv, D, keys = c["B"], c["Hq"], c["Hkv"], c["D"], sum(lengths(c))
    if c["op"] == "kv4":
        rows = Hkv * (keys if c["T"] > 1 else B)
        held = D // 2 + 4 * (D // c["group"])
        # rows read, codes written, codes read back, bf16 rows written; K and V
        return dict(bytes=2 * rows * ((4 if c["src"] == "rows" else 2) * D + 2 * held + 2 * D), flops=2 * rows * D * 8)
    if c["op"] == "kv4attn":
        held = D // 2 + 4 * (D // c["group"])
        return dict(bytes=2 * keys * Hkv * held + 8 * B * Hq * D, flops=4 * keys * Hq * D)
    if c["op"] == "bounds":
        rows = blocks = 0
        for n in lengths(c):
            j0 = (n - c["T"]) // BLOCK
            rows += n - j0 * BLOCK
            blocks += (n + BLOCK - 1) // BLOCK - j0
        return dict(bytes=Hkv * D * (2 * rows + 4 * blocks), flops=2 * Hkv * D * rows)
    blocks = sum((n + BLOCK - 1) // BLOCK for n in lengths(c))
    chosen = sum(min(n, c["n_select"] * BLOCK) for n in lengths(c))
    return dict(bytes=Hkv * D * (4 * blocks + 4 * chosen) + 8 * B * Hq * D + 4 * B * Hkv * c["n_select"],
                flops=4 * Hkv * D * blocks + 4 * Hq * D * chosen)


# --------------------------------------------------------------------------- inputs

def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    B, Hq, Hkv, D, S = c["B"], c["Hq"], c["Hkv"], c["D"], c["S_max"]
    # the rows' order goes by the seed, their lengths by the case
    order = torch.randperm(B, generator=g, device=dev)
    lens = torch.tensor(lengths(c), device=dev, dtype=torch.int32)[order]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    # keys have channels of unlike size, as rotated projections do
    size = torch.exp(0.4 * normal(Hkv, 1, D))
    s = dict(c, lens=lens)
    if c["op"] == "kv4":
        T, NG = c["T"], D // c["group"]
        s["k_codes"], s["v_codes"] = (torch.zeros(B, Hkv, S, D // 2, device=dev, dtype=torch.uint8) for _ in range(2))
        s["k_params"], s["v_params"] = (torch.zeros(B, Hkv, S, NG, 2, device=dev, dtype=torch.float16) for _ in range(2))
        s["k_out"], s["v_out"] = (torch.zeros(B, T, Hkv, D, device=dev, dtype=torch.bfloat16) for _ in range(2))
        if T == 1:
            s["pos"], s["count"] = lens - 1, None
        else:  # padded sequences: row b brings lens[b] of T tokens, from slot 0 on
            s["pos"], s["count"] = torch.zeros_like(lens), lens
        if c["src"] == "rows":  # the fused projection's output, q | k | v in each row
            qkv = normal(B, T, (Hq + 2 * Hkv) * D)
            s["k"] = qkv[..., Hq * D:(Hq + Hkv) * D].unflatten(-1, (Hkv, D))
            s["v"] = qkv[..., (Hq + Hkv) * D:].unflatten(-1, (Hkv, D))
            s["k"] *= size.squeeze(1)
        else:  # the bf16 cache of the prompt pass
            s["k"] = torch.empty(B, Hkv, S, D, device=dev, dtype=torch.bfloat16)
            s["v"] = torch.empty_like(s["k"])
            for b in range(B):
                s["k"][b], s["v"][b] = size * normal(Hkv, S, D), normal(Hkv, S, D)
        return s
    s["pos"] = lens - 1
    s["q"] = normal(B, Hq, D)
    s["o"] = torch.zeros(B, Hq, D, device=dev)
    if c["op"] == "kv4attn":
        NG = D // c["group"]
        for n in "kv":
            s[n + "_codes"] = torch.zeros(B, Hkv, S, D // 2, device=dev, dtype=torch.uint8)
            s[n + "_params"] = torch.zeros(B, Hkv, S, NG, 2, device=dev, dtype=torch.float16)
            for b in range(B):
                x = normal(Hkv, S, D)
                s[n + "_codes"][b], s[n + "_params"][b] = quantise(x * size if n == "k" else x, c["group"])
        return s
    NB = (S + BLOCK - 1) // BLOCK
    s["k"] = torch.empty(B, Hkv, S, D, device=dev, dtype=torch.bfloat16)
    s["v"] = torch.empty_like(s["k"]) if c["op"] == "sparse" else None
    s["bounds"] = torch.zeros(B, Hkv, NB, 2, D, device=dev, dtype=torch.bfloat16)
    slot = torch.arange(NB * BLOCK, device=dev)
    for b in range(B):
        # neighbouring keys are alike: a slow walk under the noise gives the blocks unlike scores
        drift = normal(Hkv, NB, D).repeat_interleave(BLOCK, 1)[:, :S]
        s["k"][b] = size * (0.8 * drift + 0.6 * normal(Hkv, S, D))
        if c["op"] == "sparse":
            s["v"][b] = normal(Hkv, S, D)
            s["bounds"][b] = block_bounds(s["k"][b], slot, s["pos"][b])
    if c["op"] == "bounds":
        s["pos"] = lens - c["T"]  # the first of the T tokens just written
    else:
        s["blocks"] = torch.full((B, Hkv, c["n_select"]), -1, device=dev, dtype=torch.int32)
    return s


def quantise(x, group):
    """Codes and (scale, middle) pairs of fp32 rows [..., D]."""
    x = x.unflatten(-1, (-1, group))
    top, low = x.amax(-1), x.amin(-1)
    scale = ((top - low) / 15).clamp(max=65504.0).half()
    middle = (low + 8 * scale.float()).clamp(-65504.0, 65504.0).half()
    step, mid = scale.float()[..., None], middle.float()[..., None]
    c = torch.where(step > 0, torch.round((x - mid) / step) + 8, 8.0).clamp(0, 15)
    c = c.to(torch.uint8).flatten(-2)
    return c[..., 0::2] | (c[..., 1::2] << 4), torch.stack((scale, middle), -1)


def values(codes, params):
    """What a 4-bit cache stands for, in fp32 [..., D]."""
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8
    p = params.float()
    return (p[..., 1:] + p[..., :1] * c.unflatten(-1, (p.shape[-2], -1))).flatten(-2)


def block_bounds(k, slot, last):
    """Largest and smallest value of each channel over each block's keys up to `last`, [Hkv, NB, 2, D]."""
    pad = slot.numel() - k.shape[1]
    k = torch.nn.functional.pad(k, (0, 0, 0, pad)) if pad else k
    live = (slot <= last)[None, :, None]
    hi = k.masked_fill(~live, -math.inf).unflatten(1, (-1, BLOCK)).amax(2)
    lo = k.masked_fill(~live, math.inf).unflatten(1, (-1, BLOCK)).amin(2)
    return torch.stack((hi, lo), 2)


# --------------------------------------------------------------------------- one pass

def attend(q, k, v, live):
    """softmax(q k^T / sqrt(D)) v for q [.., G, D], k and v [.., n, D], live [.., n]."""
    x = (q @ k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    x = x.masked_fill(~live[..., None, :], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    v = v.masked_fill(~live[..., None], 0.0)
    return (p @ v) / p.sum(-1, keepdim=True)


def run(s):
    return {"kv4": run_kv4, "kv4attn": run_kv4attn, "bounds": run_bounds, "sparse": run_sparse}[s["op"]](s)


def run_kv4(s):
    if own:
        import greedy_decode_step_gb300 as gd
        cache = s["src"] == "cache"
        held = (s["k_codes"], s["k_params"], s["v_codes"], s["v_params"])
        k, v = (s[n].transpose(1, 2) if cache else s[n] for n in "kv")
        gd.dec_kv4_store(k, v, s["pos"], *held, tokens=s["T"], lens=s["count"], from_cache=cache)
        gd.dec_kv4_load(*held, s["pos"], s["k_out"], s["v_out"], lens=s["count"])
        return s["k_out"], s["v_out"]
    B, T = s["B"], s["T"]
    dev = s["pos"].device
    t = torch.arange(T, device=dev)
    slot = s["pos"].long()[:, None] + t  # [B, T]
    row = torch.arange(B, device=dev)[:, None].expand(B, T)
    if s["count"] is not None:
        live = t < s["count"][:, None]
        at, row, slot = live.nonzero(as_tuple=True), row[live], slot[live]
    else:
        at, row, slot = (row.reshape(-1), t.repeat(B)), row.reshape(-1), slot.reshape(-1)
    for n in "kv":
        x = s[n][row, :, slot] if s["src"] == "cache" else s[n][at]  # [rows, Hkv, D]
        codes, params = quantise(x.float(), s["group"])
        s[n + "_codes"][row, :, slot] = codes
        s[n + "_params"][row, :, slot] = params
        s[n + "_out"][at] = values(s[n + "_codes"][row, :, slot], s[n + "_params"][row, :, slot]).bfloat16()
    return s["k_out"], s["v_out"]


def run_kv4attn(s):
    if own:
        import greedy_decode_step_gb300 as gd
        # the workspace of the first call is kept, as a serving loop keeps it
        s["ws"] = gd.dec_kv4_decode_attn(s["q"], s["k_codes"], s["k_params"], s["v_codes"], s["v_params"], s["pos"], s["o"],
                                         ws=s.get("ws"))
        return s["o"]
    k, v = values(s["k_codes"], s["k_params"]), values(s["v_codes"], s["v_params"])
    live = torch.arange(s["S_max"], device=k.device) <= s["pos"][:, None]
    o = attend(s["q"].unflatten(1, (s["Hkv"], -1)), k, v, live[:, None].expand(-1, s["Hkv"], -1))
    s["o"].copy_(o.flatten(1, 2))
    return s["o"]


def run_bounds(s):
    if own:
        import greedy_decode_step_gb300 as gd
        gd.dec_block_bounds(s["k"], s["pos"], s["bounds"], tokens=s["T"])
        return s["bounds"]
    # blocks that the T tokens from pos on touch, each over its slots up to the last token
    dev, NB, S, T = s["k"].device, s["bounds"].shape[2], s["S_max"], s["T"]
    first, last = s["pos"].long() // BLOCK, s["pos"].long() + T - 1
    n = min(NB, (T + BLOCK - 2) // BLOCK + 1)
    j = first[:, None] + torch.arange(n, device=dev)  # [B, n]
    slot = j[..., None] * BLOCK + torch.arange(BLOCK, device=dev)  # [B, n, BLOCK]
    live = (slot <= last[:, None, None])[:, None, ..., None]
    row = torch.arange(s["B"], device=dev)
    k = s["k"][row[:, None, None], :, slot.clamp(max=S - 1)].permute(0, 3, 1, 2, 4)  # [B, Hkv, n, BLOCK, D]
    new = torch.stack((k.masked_fill(~live, -math.inf).amax(3), k.masked_fill(~live, math.inf).amin(3)), 3)
    touched = j * BLOCK <= last[:, None]
    at = touched.nonzero(as_tuple=True)
    s["bounds"][at[0], :, j[touched]] = new.transpose(1, 2)[at]
    return s["bounds"]


def run_sparse(s):
    if own:
        import greedy_decode_step_gb300 as gd
        gd.dec_select_blocks(s["q"], s["bounds"], s["pos"], s["blocks"])
        s["ws"] = gd.dec_block_decode_attn(s["q"], s["k"], s["v"], s["pos"], s["blocks"], s["o"], ws=s.get("ws"))
        return s["blocks"], s["o"]
    B, Hkv, D, S, n = s["B"], s["Hkv"], s["D"], s["S_max"], s["n_select"]
    dev, pos, bounds = s["k"].device, s["pos"].long(), s["bounds"]
    NB = bounds.shape[2]
    q = s["q"].unflatten(1, (Hkv, -1))
    # the group's sum of each block's largest possible scores; in 64 bits, as blocks are ranked by it
    w = torch.stack((q.double().clamp(min=0).sum(2), q.double().clamp(max=0).sum(2)), 2).flatten(2)  # [B, Hkv, 2 D]
    score = (bounds.double().flatten(3) @ w[..., None]).squeeze(-1)
    j = torch.arange(NB, device=dev)
    last = (pos // BLOCK)[:, None, None]
    score = score.masked_fill((j == 0) | (j == last), math.inf).masked_fill(j > last, -math.inf)
    top = score.sort(dim=-1, descending=True, stable=True).indices[..., :n]  # ties: the lower block first
    if top.shape[-1] < n:
        top = torch.nn.functional.pad(top, (0, n - top.shape[-1]), value=NB)
    top = top.masked_fill(top > last, NB).sort(-1).values
    s["blocks"].copy_(top.masked_fill(top == NB, -1))
    slot = (top[..., None] * BLOCK + torch.arange(BLOCK, device=dev)).flatten(2)  # [B, Hkv, n * BLOCK]
    live = slot <= pos[:, None, None]
    at = slot.clamp(max=S - 1)[..., None].expand(-1, -1, -1, D)
    k, v = s["k"].gather(2, at).float(), s["v"].gather(2, at).float()
    s["o"].copy_(attend(q, k, v, live).flatten(1, 2))
    return s["blocks"], s["o"]


# --------------------------------------------------------------------------- in 64 bits

def exact(c, seed):
    """The operators' definitions, row by row in 64 bits."""
    s = prepare(c, seed)
    B, Hkv, D = c["B"], c["Hkv"], c["D"]
    G = c["Hq"] // Hkv
    lens = s["lens"].tolist()

    def decode(codes, params):  # [n, D / 2], [n, NG, 2] -> [n, D]
        n = codes.shape[0]
        out = torch.empty(n, D, dtype=torch.float64, device=codes.device)
        out[:, 0::2] = (codes % 16).double()
        out[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
        size = D // params.shape[1]
        scale = params[:, :, 0].double().repeat_interleave(size, 1)
        middle = params[:, :, 1].double().repeat_interleave(size, 1)
        return middle + (out - 8.0) * scale

    def rows(q, k, v):  # [G, D], [n, D], [n, D]
        z = torch.einsum("gd,nd->gn", q, k) * D ** -0.5
        return torch.einsum("gn,nd->gd", torch.softmax(z, 1), v)

    if c["op"] == "kv4":
        res = []
        for n in "kv":
            out = torch.zeros(B, c["T"], Hkv, D, dtype=torch.float64, device=s["pos"].device)
            for b in range(B):
                m = c["T"] if s["count"] is None else lens[b]
                p = int(s["pos"][b])
                x = (s[n][b][:, p:p + m].transpose(0, 1) if c["src"] == "cache" else s[n][b, :m]).double()
                x = x.reshape(m, Hkv, D // c["group"], c["group"])
                low = x.min(3, keepdim=True).values
                step = ((x.max(3, keepdim=True).values - low) / 15).to(torch.float16).double()
                mid = (low + 8 * step).to(torch.float16).double()
                code = ((x - mid) / step).round().clamp(-8, 7)
                out[b, :m] = (mid + code * step).reshape(m, Hkv, D)
            res.append(out)
        return tuple(res)
    if c["op"] == "bounds":
        out = s["bounds"].double()
        for b in range(B):
            first = int(s["pos"][b])
            for j in range(first // BLOCK, (lens[b] - 1) // BLOCK + 1):
                part = s["k"][b, :, j * BLOCK:min(lens[b], (j + 1) * BLOCK)].double()
                out[b, :, j, 0], out[b, :, j, 1] = part.max(1).values, part.min(1).values
        return out
    o = torch.empty(B, c["Hq"], D, dtype=torch.float64, device=s["q"].device)
    if c["op"] == "kv4attn":
        for b in range(B):
            for h in range(Hkv):
                k, v = (decode(s[n + "_codes"][b, h, :lens[b]], s[n + "_params"][b, h, :lens[b]]) for n in "kv")
                o[b, h * G:(h + 1) * G] = rows(s["q"][b, h * G:(h + 1) * G].double(), k, v)
        return o
    ids = torch.full((B, Hkv, c["n_select"]), -1, dtype=torch.int32, device=s["q"].device)
    for b in range(B):
        last = (lens[b] - 1) // BLOCK
        for h in range(Hkv):
            q = s["q"][b, h * G:(h + 1) * G].double()
            hi, lo = s["bounds"][b, h, :last + 1, 0].double(), s["bounds"][b, h, :last + 1, 1].double()
            score = torch.maximum(q[:, None] * hi, q[:, None] * lo).sum((0, 2)).tolist()
            rank = sorted(range(last + 1), key=lambda j: (j not in (0, last), -score[j], j))
            take = sorted(rank[:c["n_select"]])
            ids[b, h, :len(take)] = torch.tensor(take, dtype=torch.int32)
            k, v = (torch.cat([s[n][b, h, j * BLOCK:min(lens[b], (j + 1) * BLOCK)] for j in take]).double() for n in "kv")
            o[b, h * G:(h + 1) * G] = rows(q, k, v)
    return ids, o
