"""What the operators of a decoding attention layer are measured on.

Four families, each in a plain form (elementary torch operations in 32 bits)
and as the calls a user makes of the library:

  rope    norms of the query and key heads with the position rotation, from the
          output of the QKV projection; and its gradient
  append  keys and values quantised into a paged cache as they are written
          (behind the norm and the rotation, or as they are), and the cached
          tokens read back
  attend  attention of one new token per sequence over the paged cache
  gemv    products of a few BF16 rows with 4-bit weights and block scales

The cache is one byte tensor [pages, kv_heads, page_size / 16, unit].  A unit
holds 16 tokens of one head: K codes, K scales, V codes, V scales, each in the
order that `cache_places` gives.
"""
import math

import torch

own = False

TYPES = ("bf16", "e4m3", "nvfp4")
CODE_BITS = {"bf16": 16, "e4m3": 8, "nvfp4": 4}
FLOOR = 2.0 ** -100          # smallest magnitude that an E4M3 vector's scale is taken from
EPS = 1e-6
MEASURED = 24.0              # largest magnitude that the NVFP4 global scales are calibrated for


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # a training batch through the projections of an attention layer: norms and rotation of queries and keys
        {"name": "rope train", "op": "rope", "t": 16384, "q": 32, "kv": 8, "d": 128, "r": 128, "norm": True, "interleaved": False, "padded": False},
        # a ragged prompt, wide heads of which a quarter turns, pairs next to each other, padding behind it
        {"name": "rope ragged", "op": "rope", "t": 1531, "q": 16, "kv": 2, "d": 256, "r": 64, "norm": True, "interleaved": True, "padded": True},
        # the gradient of the training batch, with that of the norms' weights
        {"name": "rope gradient", "op": "drope", "t": 16384, "q": 32, "kv": 8, "d": 128, "r": 128, "norm": True, "interleaved": False, "padded": False},
        # a short batch of narrow heads, each with a key of its own
        {"name": "rope gradient short", "op": "drope", "t": 777, "q": 16, "kv": 16, "d": 64, "r": 64, "norm": True, "interleaved": True, "padded": True},
        # 64 sequences append their new token, straight from the projection
        {"name": "append 64", "op": "append", "type": "e4m3", "t": 64, "back": 64, "q": 32, "kv": 8, "d": 128, "r": 128, "page": 16, "fused": True, "norm": True,
         "interleaved": False},
        # a chunk of a long prompt joins the cache, and the whole prefix comes back for the chunk's attention
        {"name": "append chunk", "op": "append", "type": "nvfp4", "t": 4096, "back": 32768, "q": 0, "kv": 8, "d": 128, "r": 0, "page": 64, "fused": False, "norm": False,
         "interleaved": False},
        # one user's token: latency
        {"name": "attend 1", "op": "attend", "type": "nvfp4", "b": 1, "len": 4096, "ragged": False, "q": 32, "kv": 8, "d": 128, "page": 16, "window": 0},
        # a serving batch of unevenly long sequences
        {"name": "attend 64", "op": "attend", "type": "e4m3", "b": 64, "len": 8192, "ragged": True, "q": 32, "kv": 8, "d": 128, "page": 64, "window": 0},
        # few long contexts
        {"name": "attend long", "op": "attend", "type": "nvfp4", "b": 4, "len": 131072, "ragged": False, "q": 64, "kv": 8, "d": 128, "page": 64, "window": 0},
        # an unquantised cache, a key head for each query head, the last thousand tokens only
        {"name": "attend window", "op": "attend", "type": "bf16", "b": 17, "len": 3001, "ragged": True, "q": 16, "kv": 16, "d": 64, "page": 32, "window": 1000},
        # one token through an attention projection: latency
        {"name": "gemv 1", "op": "gemv", "fmt": "nvfp4", "m": 1, "n": 4096, "k": 4096},
        # a few tokens through a large up-projection: streaming the weights
        {"name": "gemv 16", "op": "gemv", "fmt": "mxfp4", "m": 16, "n": 28672, "k": 8192},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("rope", "drope", "append", "append", "attend", "attend", "attend", "gemv", "gemv"))
    kv = rng.choice((1, 2, 4, 8, 8, 16))
    q = kv * rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    if op in ("rope", "drope"):
        d = rng.choice((64, 80, 96, 128, 128, 192, 256))
        r = d if rng.random() < 0.6 else 16 * rng.randint(1, d // 16)
        t = log_int(1, 32768)
        while t * (q + kv) * d > 16384 * 40 * 128:
            t = t // 2
        return {"op": op, "t": t, "q": q, "kv": kv, "d": d, "r": r, "norm": rng.random() < 0.7, "interleaved": rng.random() < 0.5, "padded": rng.random() < 0.5}
    d = rng.choice((64, 128, 128, 256))
    page = rng.choice((16, 32, 48, 64, 128))
    kind = rng.choice(TYPES)
    if op == "append":
        t = log_int(1, 8192)
        back = max(t, log_int(1, 65536))
        while (back + 2 * t) * kv * d > 32768 * 8 * 128:
            t, back = max(1, t // 2), max(1, back // 2)
        # behind a norm or a rotation the last bit of 32 decides at a code's border: four-bit codes, whose steps are wide, are compared as they are written alone
        fused = kind != "nvfp4" and rng.random() < 0.6
        return {"op": op, "type": kind, "t": t, "back": back, "q": q if fused else 0, "kv": kv, "d": d, "r": rng.choice((0, d // 2, d)) if fused else 0, "page": page, "fused": fused,
                "norm": fused and rng.random() < 0.7, "interleaved": fused and rng.random() < 0.3}
    if op == "attend":
        b, length = log_int(1, 256), log_int(1, 131072)
        while b * length * kv * d > 4 * 131072 * 8 * 128 // (CODE_BITS[kind] // 4) or b * length * q * d > 4 * 131072 * 64 * 128:
            b, length = max(1, b // 2), max(1, length // 2)
        return {"op": op, "type": kind, "b": b, "len": length, "ragged": rng.random() < 0.7, "q": q, "kv": kv, "d": d, "page": page,
                "window": rng.choice((0, 0, 0, max(1, length // 3)))}
    m, n, k = rng.randint(1, 16), log_int(64, 32768), 128 * log_int(1, 128)
    while n * k > 28672 * 8192:
        n = n // 2
    return {"op": op, "fmt": rng.choice(("nvfp4", "mxfp4")), "m": m, "n": n, "k": k}


def token_bytes(kind, d):
    """K and V of one token and head: codes and scales."""
    return 2 * (d * CODE_BITS[kind] // 8 + {"bf16": 0, "e4m3": 4, "nvfp4": d // 16}[kind])


def lengths_of(case):
    """Tokens that each sequence has in the cache, from the case alone: evenly spread, or from a sixteenth up."""
    b, top = case["b"], case["len"]
    if not case["ragged"]:
        return [top] * b
    return [max(1, round(top * (1 + 15 * ((7 * i) % b) / max(1, b - 1)) / 16)) for i in range(b)]


def work(case):
    op = case["op"]
    if op in ("rope", "drope"):
        heads = case["t"] * (case["q"] + case["kv"]) * case["d"]
        table = 4 * case["t"] * case["r"]
        return {"bytes": (4 if op == "rope" else 6) * heads + table, "flops": (8.0 if op == "rope" else 16.0) * heads}
    if op == "append":
        t, n, kv, d = case["t"], case["back"], case["kv"], case["d"]
        q = 4 * t * case["q"] * d if case["fused"] else 0
        return {"bytes": q + t * kv * (4 * d + token_bytes(case["type"], d)) + n * kv * (4 * d + token_bytes(case["type"], d)), "flops": 4.0 * (t + n) * kv * d}
    if op == "attend":
        seen = sum(min(n, case["window"]) if case["window"] else n for n in lengths_of(case))
        io = 4 * case["b"] * case["q"] * case["d"]
        return {"bytes": seen * case["kv"] * token_bytes(case["type"], case["d"]) + io, "flops": 4.0 * seen * case["q"] * case["d"]}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": n * k // 2 + n * k // (16 if case["fmt"] == "nvfp4" else 32) + 2 * m * (n + k), "flops": 2.0 * m * n * k}


# ---------------------------------------------------------- the cache's layout

def cache_places(kind, d):
    """Where a unit keeps what: (bytes of a unit, then for K codes, K scales, V
    codes and V scales the places of the bytes of [16 tokens, bytes of a token]).

    Token j of a unit, j = 8 h + 2 t + e with e in {0, 1}, t in 0..3, h in {0, 1}.
      K codes   a token's bytes in pieces of 64 (or all, where they are fewer);
                eight tokens' pieces side by side, by h, then piece
      V codes   a token's bytes in eight pieces p; the pieces p of tokens t make
                a string by (h, e), cut into sixteens; those lie by cut, p, t
      scales    NVFP4: K [token][block], V [block][t][h][e]; E4M3: fp32 [token]
    """
    def numbers(n):
        return torch.arange(n, device="cuda")

    row = d * CODE_BITS[kind] // 8
    j = numbers(16)[:, None]
    h, t, e = j // 8, j % 8 // 2, j % 2
    x = numbers(row)[None]
    piece = min(64, row)
    k = ((h * (row // piece) + x // piece) * 8 + j % 8) * piece + x % piece
    w = row // 8
    at = (2 * h + e) * w + x % w
    v = ((at // 16) * 32 + 4 * (x // w) + t) * 16 + at % 16
    if kind == "bf16":
        ks = vs = numbers(0).view(1, 0).expand(16, 0)
    elif kind == "e4m3":
        ks = vs = 4 * j + numbers(4)[None]
    else:
        block = numbers(d // 16)[None]
        ks, vs = j * (d // 16) + block, block * 16 + 4 * t + 2 * h + e
    codes, scales = 16 * row, 16 * ks.shape[1]
    unit = 2 * (codes + scales)
    return unit, k, codes + ks, codes + scales + v, 2 * codes + scales + vs


def gathered(cache, slots, page, kind, d):
    """(K codes, K scales, V codes, V scales) of the tokens at these slots, as bytes [.., heads, bytes]."""
    unit, *places = cache_places(kind, d)
    units = cache.view(cache.shape[0], cache.shape[1], -1, unit)
    rows = units[slots // page, :, slots % page // 16]                 # [.., heads, unit]
    j = slots % 16
    return [rows.gather(-1, p[j][..., None, :].expand(*rows.shape[:-1], p.shape[1])) for p in places]


def paged(cache, table, kind, d):
    """The same of every token of these pages [b, n]: bytes [b, heads, tokens, bytes]."""
    unit, *places = cache_places(kind, d)
    units = cache.view(cache.shape[0], cache.shape[1], -1, unit)[table].transpose(1, 2)     # [b, heads, n, units, unit]
    return [units[..., p].flatten(2, 4) for p in places]


def values_of(codes, scales, kind, gs):
    """fp32 values of bytes [.., row] and their scales' bytes."""
    if kind == "bf16":
        return codes.contiguous().view(torch.bfloat16).float()
    if kind == "e4m3":
        return codes.contiguous().view(torch.float8_e4m3fn).float() * scales.contiguous().view(torch.float32)
    return nibbles(codes) * (scales.contiguous().view(torch.float8_e4m3fn).float() * gs).repeat_interleave(16, -1)


def nibbles(codes):
    """E2M1 values of packed bytes, the low half first."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=codes.device)
    table = torch.cat([table, -table])
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return table[both.int()]


def stored(cache, slots, page, kind, x, gs, half):
    """Quantises x [t, heads, d] (fp32) and writes it as the K (half 0) or V (half 1) of these slots."""
    d = x.shape[-1]
    unit, *places = cache_places(kind, d)
    units = cache.view(cache.shape[0], cache.shape[1], -1, unit)
    heads = torch.arange(cache.shape[1], device="cuda")[None, :, None]
    codes, scales = quantized(x, kind, gs)
    for bytes_, place in zip((codes, scales), places[2 * half: 2 * half + 2]):
        if bytes_.shape[-1]:
            units[(slots // page)[:, None, None], heads, (slots % page // 16)[:, None, None], place[slots % 16][:, None, :]] = bytes_


def quantized(x, kind, gs):
    """(codes, scales) of [.., d], as bytes."""
    if kind == "bf16":
        return x.bfloat16().view(torch.uint8), x.new_zeros(*x.shape[:-1], 0).to(torch.uint8)
    if kind == "e4m3":
        amax = x.abs().amax(-1, keepdim=True).clamp(min=FLOOR)
        top = torch.full_like(amax, 448.0)      # a tensor: by a number, the quotient would be a product with its reciprocal
        return (x * (top / amax)).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), (amax / top).view(torch.uint8)
    return nvfp4(x, gs)


def nvfp4(x, gs):
    """Packed E2M1 codes and UE4M3 scale bytes, one per 16 elements."""
    blocks = x.unflatten(-1, (-1, 16))
    amax = blocks.abs().amax(-1)
    sf = (amax / torch.full_like(amax, 6.0) / gs).clamp(max=448).to(torch.float8_e4m3fn)
    s = (sf.float() * gs)[..., None]
    y = torch.where(s > 0, blocks / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(blocks))
    return packed(y.flatten(-2)), sf.view(torch.uint8)


def packed(y):
    """E2M1 codes of y, nearest with ties to the even code, two per byte."""
    a = y.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a * 0.5 + 4)).to(torch.uint8)
    code = code | (torch.signbit(y).to(torch.uint8) << 3)
    return code[..., 0::2] | (code[..., 1::2] << 4)


# --------------------------------------------------------------------- inputs

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def normal(g, *shape, sigma=1.0):
    return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, sigma, generator=g)


def heads_of(g, t, heads, d):
    """N(0, 1) with a few channels of every head far larger, as queries and keys have them."""
    x = torch.randn(t, heads, d, generator=g, device="cuda")
    channel = 1.0 + 5.0 * (torch.rand(heads, d, generator=g, device="cuda") < 0.03)
    return (x * channel).bfloat16()


def rotation_table(rows, r):
    """cos and sin of every position, angles in 64 bits, as a model keeps them: fp32 [rows, r]."""
    angle = torch.arange(rows, device="cuda", dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / max(1, r))
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def projected(case, g, v_heads):
    """Output of a QKV projection and what its queries and keys go through."""
    t, q, kv, d, r = case["t"], case["q"], case["kv"], case["d"], case["r"]
    s = {"qkv": heads_of(g, t, q + kv + v_heads, d).flatten(1)}
    rows = 32768
    s["cos_sin"] = rotation_table(rows, r) if r else None
    at = torch.randint(0, rows - t if rows > t else 1, (1,), generator=g, device="cuda", dtype=torch.int32)
    s["positions"] = at + torch.arange(t, device="cuda", dtype=torch.int32)
    if case.get("padded"):      # rows behind the last sequence
        s["positions"][t - t // 16:] = -1
    for name in ("q_weight", "k_weight"):
        s[name] = (1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).bfloat16() if case["norm"] else None
    return s


def prepare(case, seed):
    g, op = generator(seed), case["op"]
    s = {"case": case}
    if op in ("rope", "drope"):
        t, q, kv, d = case["t"], case["q"], case["kv"], case["d"]
        s |= projected(case, g, kv)
        if op == "rope":
            s["q_out"] = torch.zeros(t, q, d, dtype=torch.bfloat16, device="cuda")
            s["k_out"] = torch.zeros(t, kv, d, dtype=torch.bfloat16, device="cuda")
        else:
            s["dq"], s["dk"] = normal(g, t, q, d, sigma=1e-2), normal(g, t, kv, d, sigma=1e-2)
            s["dqkv"] = torch.zeros_like(s["qkv"])
            s["dq_weight"], s["dk_weight"] = (torch.zeros(d, device="cuda") if case["norm"] else None for _ in range(2))
            s["workspace"] = torch.zeros(8 << 20, dtype=torch.uint8, device="cuda")
        return s
    if op == "gemv":
        m, n, k, fmt = case["m"], case["n"], case["k"], case["fmt"]
        s["x"] = (torch.randn(m, k, generator=g, device="cuda") * torch.where(torch.rand(m, k, generator=g, device="cuda") < 0.01, 20.0, 1.0)).bfloat16()
        w = torch.randn(n, k, generator=g, device="cuda") * 0.02
        if fmt == "nvfp4":
            s["gs"] = w.abs().amax().view(1) / (6.0 * 448.0)
            s["w"], sf = nvfp4(w, s["gs"])
        else:
            s["gs"] = None
            s["w"], sf = mxfp4(w)
        s["w_sf"] = to_tiles(sf)
        s["d"] = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        return s
    kind, kv, d, page = case["type"], case["kv"], case["d"], case["page"]
    unit = 16 * token_bytes(kind, d)
    s["gs_k"], s["gs_v"] = (torch.tensor([MEASURED * f / (6.0 * 448.0)], device="cuda") if kind == "nvfp4" else None for f in (1.0, 0.5))
    if op == "append":
        t, back = case["t"], case["back"]
        pages = -(-back // page) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        token = torch.arange(back, device="cuda")
        slots = order[token // page] * page + token % page
        s["cache"] = torch.zeros(pages, kv, page // 16 * unit, dtype=torch.uint8, device="cuda")
        s["read"] = slots.int()
        s["slots"] = slots[back - t:].int().contiguous()
        old = slots[: back - t]
        if old.numel():
            stored(s["cache"], old, page, kind, heads_of(g, old.numel(), kv, d).float(), s["gs_k"], 0)
            stored(s["cache"], old, page, kind, normal(g, old.numel(), kv, d).float(), s["gs_v"], 1)
        if case["fused"]:
            s |= projected(case, g, kv)
            s["q_out"] = torch.zeros(t, case["q"], d, dtype=torch.bfloat16, device="cuda")
        else:
            s["k"], s["v"] = heads_of(g, t, kv, d), normal(g, t, kv, d)
        s["k_out"], s["v_out"] = (torch.zeros(back, kv, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        return s
    b, lens = case["b"], lengths_of(case)
    each = [-(-n // page) for n in lens]
    pages = sum(each) + 1
    order = torch.randperm(pages, generator=g, device="cuda").int()
    need = torch.tensor(each, device="cuda")
    first = need.cumsum(0) - need
    column = torch.arange(max(each), device="cuda")
    s["page_table"] = torch.where(column < need[:, None], order[(first[:, None] + column).clamp(max=pages - 1)], 0).int()
    s["lengths"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["cache"] = torch.zeros(pages, kv, page // 16 * unit, dtype=torch.uint8, device="cuda")
    for start in range(0, pages * page, 65536):         # in pieces: the plain quantiser's intermediate values are many times the cache
        slots = torch.arange(start, min(pages * page, start + 65536), device="cuda")
        stored(s["cache"], slots, page, kind, heads_of(g, slots.numel(), kv, d).float(), s["gs_k"], 0)
        stored(s["cache"], slots, page, kind, normal(g, slots.numel(), kv, d).float(), s["gs_v"], 1)
    s["q"] = heads_of(g, b, case["q"], d)
    s["scale"] = 1.0 / math.sqrt(d)
    s["out"] = torch.empty(b, case["q"], d, dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.empty(b, case["q"], device="cuda")
    s["workspace"] = torch.zeros(32 << 20, dtype=torch.uint8, device="cuda")
    return s


def mxfp4(w):
    blocks = w.unflatten(-1, (-1, 32))
    amax = blocks.abs().amax(-1)
    exponent = torch.frexp(amax / 6.0)[1]       # the smallest power of two that keeps the block in range
    scale = torch.exp2(exponent.float())
    return packed((blocks / scale[..., None]).flatten(-2)), (exponent + 127).clamp(0, 254).to(torch.uint8)


def to_tiles(sf):
    """Scale bytes [rows, cols] in the tensor cores' order: tiles of 128 rows x 4 columns."""
    rows, cols = sf.shape
    p = sf.new_zeros(-(-rows // 128) * 128, cols)
    p[:rows] = sf
    return p.view(-1, 4, 32, cols // 4, 4).permute(0, 3, 2, 1, 4).contiguous()


def from_tiles(tiles, rows):
    return tiles.permute(0, 3, 2, 1, 4).reshape(-1, tiles.shape[1] * 4)[:rows]


# ----------------------------------------------------------------- one pass

def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    from block_scaled_fp4_tcgen05_gb300 import qfp4
    c = s["case"]
    op = c["op"]
    if op == "rope":
        qfp4.qk_norm_rope(s["qkv"], c["q"], c["kv"], s["q_out"], s["k_out"], s["q_weight"], s["k_weight"], s["cos_sin"], s["positions"], eps=EPS,
                          interleaved=c["interleaved"])
        return {"q": s["q_out"], "k": s["k_out"]}
    if op == "drope":
        qfp4.qk_norm_rope_backward(s["qkv"], c["q"], c["kv"], s["dq"], s["dk"], s["dqkv"], s["dq_weight"], s["dk_weight"], s["workspace"], s["q_weight"],
                                   s["k_weight"], s["cos_sin"], s["positions"], eps=EPS, interleaved=c["interleaved"])
        return {"dqkv": s["dqkv"], "dq_weight": s["dq_weight"], "dk_weight": s["dk_weight"]}
    if op == "gemv":
        qfp4.gemv_nt({"nvfp4": qfp4.NVFP4, "mxfp4": qfp4.MXFP4}[c["fmt"]], s["x"], s["w"], s["w_sf"], s["gs"], s["d"])
        return s["d"]
    kind = {"bf16": qfp4.CACHE_BF16, "e4m3": qfp4.CACHE_E4M3, "nvfp4": qfp4.CACHE_NVFP4}[c["type"]]
    if op == "append":
        out = {"k": s["k_out"], "v": s["v_out"]}
        if c["fused"]:
            qfp4.qk_norm_rope_cache(s["qkv"], c["q"], c["kv"], s["q_out"], kind, s["cache"], c["page"], s["slots"], s["q_weight"], s["k_weight"], s["cos_sin"],
                                    s["positions"], s["gs_k"], s["gs_v"], eps=EPS, interleaved=c["interleaved"])
            out["q"] = s["q_out"]
        else:
            qfp4.kv_cache_write(kind, s["k"], s["v"], s["slots"], s["cache"], c["page"], s["gs_k"], s["gs_v"])
        qfp4.kv_cache_read(kind, s["cache"], c["page"], s["read"], s["k_out"], s["v_out"], s["gs_k"], s["gs_v"])
        return out
    qfp4.attention_decode(kind, s["q"], s["cache"], c["page"], s["page_table"], s["lengths"], s["scale"], s["out"], s["workspace"], s["gs_k"], s["gs_v"],
                          lse=s["lse"], window=c["window"])
    return {"out": s["out"], "lse": s["lse"]}


def run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "rope":
        q, k = plain_heads(s, c)
        return {"q": q.bfloat16(), "k": k.bfloat16()}
    if op == "drope":
        return plain_gradient(s, c)
    if op == "gemv":
        sf = from_tiles(s["w_sf"], c["n"])
        if c["fmt"] == "nvfp4":
            scale = (sf.contiguous().view(torch.float8_e4m3fn).float() * s["gs"]).repeat_interleave(16, 1)
        else:
            scale = torch.exp2(sf.float() - 127.0).repeat_interleave(32, 1)
        return (s["x"].float() @ (nibbles(s["w"]) * scale).t()).bfloat16()
    if op == "append":
        return plain_append(s, c)
    return plain_attend(s, c)


# --------------------------------------------------------------- plain forms

def rotated(z, cos, sin, interleaved, back=False):
    """The first 2 * cos.shape[-1] elements of each head turned by the angles (back: by their negatives)."""
    r = 2 * cos.shape[-1]
    sin = -sin if back else sin
    if interleaved:
        a, b = z[..., 0:r:2], z[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = z[..., : r // 2], z[..., r // 2: r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, z[..., r:]], -1)


def angles(s, c):
    rows = s["cos_sin"][s["positions"].clamp(min=0).long()][:, None, :]
    return rows[..., : c["r"] // 2], rows[..., c["r"] // 2:]


def plain_heads(s, c):
    """Queries and keys after norm and rotation, fp32; rows without a position are zeros."""
    x = s["qkv"].view(c["t"], -1, c["d"])[:, : c["q"] + c["kv"]].float()
    if c["norm"]:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        x = torch.cat([x[:, : c["q"]] * s["q_weight"].float(), x[:, c["q"]:] * s["k_weight"].float()], 1)
    if c["r"]:
        x = rotated(x, *angles(s, c), c["interleaved"])
    x = torch.where((s["positions"] >= 0)[:, None, None], x, 0.0)
    return x[:, : c["q"]], x[:, c["q"]:]


def plain_gradient(s, c):
    q, kv, d = c["q"], c["kv"], c["d"]
    alive = (s["positions"] >= 0)[:, None, None]
    dz = torch.where(alive, torch.cat([s["dq"], s["dk"]], 1).float(), 0.0)
    if c["r"]:
        dz = rotated(dz, *angles(s, c), c["interleaved"], back=True)
    out = {"dqkv": torch.zeros_like(s["qkv"])}
    if c["norm"]:
        x = s["qkv"].view(c["t"], -1, d)[:, : q + kv].float()
        rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        hat = x * rstd
        each = (dz * hat).double()
        out["dq_weight"], out["dk_weight"] = each[:, :q].sum((0, 1)).float(), each[:, q:].sum((0, 1)).float()
        g = torch.cat([dz[:, :q] * s["q_weight"].float(), dz[:, q:] * s["k_weight"].float()], 1)
        dz = rstd * (g - hat * (g * hat).mean(-1, keepdim=True))
    else:
        out["dq_weight"] = out["dk_weight"] = None
    out["dqkv"].view(c["t"], -1, d)[:, : q + kv] = dz.bfloat16()
    return out


def plain_append(s, c):
    kind, kv, d, page = c["type"], c["kv"], c["d"], c["page"]
    slots, out = s["slots"].long(), {}
    if c["fused"]:
        q, k = plain_heads(s, c)
        v = s["qkv"].view(c["t"], -1, d)[:, c["q"] + kv:].float()
        out["q"] = q.bfloat16()
    else:
        k, v = s["k"].float(), s["v"].float()
    stored(s["cache"], slots, page, kind, k, s["gs_k"], 0)
    stored(s["cache"], slots, page, kind, v, s["gs_v"], 1)
    kc, ks, vc, vs = gathered(s["cache"], s["read"].long(), page, kind, d)
    out["k"], out["v"] = values_of(kc, ks, kind, s["gs_k"]).bfloat16(), values_of(vc, vs, kind, s["gs_v"]).bfloat16()
    return out


def plain_attend(s, c):
    """Every sequence's cache laid out to the longest one's length, in 32 bits."""
    b, q, kv, d, page, kind = c["b"], c["q"], c["kv"], c["d"], c["page"], c["type"]
    kc, ks, vc, vs = paged(s["cache"], s["page_table"].long(), kind, d)
    token = torch.arange(kc.shape[2], device="cuda")
    seen = token < s["lengths"][:, None]
    if c["window"]:
        seen &= token >= s["lengths"][:, None] - c["window"]
    query = s["q"].float().view(b, kv, q // kv, d)
    keys = values_of(kc, ks, kind, s["gs_k"])           # [b, kv, tokens, d]
    logits = (query @ keys.transpose(2, 3)) * s["scale"]
    del keys, kc, ks
    logits = torch.where(seen[:, None, None, :], logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    values = values_of(vc, vs, kind, s["gs_v"])
    out = (p @ values) / total
    return {"out": out.view(b, q, d).bfloat16(), "lse": (top + torch.log(total)).view(b, q)}


# ------------------------------------------------------------ 64-bit results

def e2m1_exact(code):
    """Value of 4-bit codes: sign, two exponent bits, one mantissa bit."""
    e, m = (code >> 1 & 3).double(), (code & 1).double()
    size = torch.where(e > 0, (1 + m / 2) * 2 ** (e - 1), m / 2)
    return torch.where(code >= 8, -size, size)


def e4m3_exact(code):
    e, m = (code >> 3 & 15).double(), (code & 7).double()
    size = torch.where(e > 0, (1 + m / 8) * 2 ** (e - 7), m / 512)
    return torch.where(code >= 128, -size, size)


def exact_values(codes, scales, kind, gs):
    if kind == "bf16":
        return codes.contiguous().view(torch.bfloat16).double()
    if kind == "e4m3":
        return e4m3_exact(codes) * scales.contiguous().view(torch.float32).double()
    y = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device="cuda")
    y[..., 0::2], y[..., 1::2] = e2m1_exact(codes & 15), e2m1_exact(codes >> 4)
    return (y.unflatten(-1, (-1, 16)) * (e4m3_exact(scales) * gs.double())[..., None]).flatten(-2)


def exact_rounded(y, mantissa, least, top):
    """y to the nearest value with so many mantissa bits, smallest exponent and largest magnitude, ties to the even one."""
    exponent = (torch.frexp(y)[1] - 1).clamp(min=least).double()
    step = 2.0 ** (exponent - mantissa)
    return (torch.round(y / step) * step).clamp(-top, top)


def exact_stored(x, kind, gs):
    """What the cache gives back for x in 64 bits."""
    if kind == "bf16":
        return exact_rounded(x, 7, -126, 3.3e38)
    if kind == "e4m3":
        scale = x.abs().amax(-1, keepdim=True).clamp(min=FLOOR) / 448
        return exact_rounded(x / scale, 3, -6, 448.0) * scale
    blocks = x.unflatten(-1, (-1, 16))
    s = exact_rounded(blocks.abs().amax(-1, keepdim=True) / 6 / gs.double(), 3, -6, 448.0) * gs.double()
    return (exact_rounded(torch.where(s > 0, blocks / s.clamp(min=1e-300), 0.0), 1, 0, 6.0) * s).flatten(-2)


def exact_heads(case, s):
    q, kv, d, r = case["q"], case["kv"], case["d"], case["r"]
    x = s["qkv"].view(case["t"], -1, d)[:, : q + kv].double()
    if case["norm"]:
        x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
        x[:, :q] *= s["q_weight"].double()
        x[:, q:] *= s["k_weight"].double()
    if r:
        x = turned_exact(x, case, s, 1.0)
    return x * (s["positions"] >= 0).double()[:, None, None]


def turned_exact(x, case, s, sign):
    """Pairs as complex numbers times cos + i sin."""
    r = case["r"]
    table = s["cos_sin"].double()[s["positions"].clamp(min=0).long()][:, None]
    turn = torch.complex(table[..., : r // 2], sign * table[..., r // 2:])
    first, second = (slice(0, r, 2), slice(1, r, 2)) if case["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
    z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rope":
        x = exact_heads(case, s)
        return {"q": x[:, : case["q"]], "k": x[:, case["q"]:]}
    if op == "drope":
        q, kv, d = case["q"], case["kv"], case["d"]
        dz = torch.cat([s["dq"], s["dk"]], 1).double() * (s["positions"] >= 0).double()[:, None, None]
        if case["r"]:
            dz = turned_exact(dz, case, s, -1.0)
        full = torch.zeros(case["t"], q + 2 * kv, d, dtype=torch.float64, device="cuda")
        if not case["norm"]:
            full[:, : q + kv] = dz
            return {"dqkv": full.flatten(1), "dq_weight": None, "dk_weight": None}
        x = s["qkv"].view(case["t"], -1, d)[:, : q + kv].double()
        n = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)     # x / n is what the weight multiplies
        w = torch.cat([s["q_weight"].double().expand(q, d), s["k_weight"].double().expand(kv, d)])
        dw = (dz * x / n).sum(0)
        full[:, : q + kv] = w * dz / n - x * (w * dz * x).sum(-1, keepdim=True) / (d * n ** 3)
        return {"dqkv": full.flatten(1), "dq_weight": dw[:q].sum(0), "dk_weight": dw[q:].sum(0)}
    if op == "gemv":
        m, n, k = case["m"], case["n"], case["k"]
        y = torch.empty(m, n, dtype=torch.float64, device="cuda")
        x, sf = s["x"].double(), from_tiles(s["w_sf"], n)
        for lo in range(0, n, 4096):        # in pieces: 64-bit weights are sixteen times the codes
            codes, f = s["w"][lo:lo + 4096], sf[lo:lo + 4096]
            w = torch.empty(codes.shape[0], k, dtype=torch.float64, device="cuda")
            w[:, 0::2], w[:, 1::2] = e2m1_exact(codes & 15), e2m1_exact(codes >> 4)
            f = e4m3_exact(f) * s["gs"].double() if case["fmt"] == "nvfp4" else 2.0 ** (f.double() - 127)
            y[:, lo:lo + 4096] = x @ (w.view(w.shape[0], f.shape[1], -1) * f[..., None]).flatten(1).t()
        return y
    kind, kv, d, page = case["type"], case["kv"], case["d"], case["page"]
    if op == "append":
        t, out = case["t"], {}
        if case["fused"]:
            x = exact_heads(case, s)
            out["q"], k = x[:, : case["q"]], x[:, case["q"]:]
            v = s["qkv"].view(t, -1, d)[:, case["q"] + kv:].double()
        else:
            k, v = s["k"].double(), s["v"].double()
        kc, ks, vc, vs = gathered(s["cache"], s["read"].long(), page, kind, d)
        out["k"], out["v"] = exact_values(kc, ks, kind, s["gs_k"]), exact_values(vc, vs, kind, s["gs_v"])
        out["k"][case["back"] - t:], out["v"][case["back"] - t:] = exact_stored(k, kind, s["gs_k"]), exact_stored(v, kind, s["gs_v"])
        return out
    b, q, group = case["b"], case["q"], case["q"] // kv
    out, lse = torch.zeros(b, q, d, dtype=torch.float64, device="cuda"), torch.zeros(b, q, dtype=torch.float64, device="cuda")
    for i, n in enumerate(lengths_of(case)):
        token = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device="cuda")
        slots = s["page_table"][i, token // page].long() * page + token % page
        kc, ks, vc, vs = gathered(s["cache"], slots, page, kind, d)
        keys, values = exact_values(kc, ks, kind, s["gs_k"]), exact_values(vc, vs, kind, s["gs_v"])
        query = s["q"][i].double().view(kv, group, d)
        logits = torch.einsum("hgd,nhd->hgn", query, keys) * s["scale"]
        lse[i] = torch.logsumexp(logits, -1).flatten()
        out[i] = torch.einsum("hgn,nhd->hgd", torch.softmax(logits, -1), values).reshape(q, d)
    return {"out": out, "lse": lse}
