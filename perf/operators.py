"""What the 8-bit floating point product with block scales, its quantisers and the
mixture-of-experts router are measured on.

Three families of operators, each in a plain form (elementary torch operations
in 32 bits) and as the calls a user makes of the library:

  gemm    D = A B^T with E4M3 / E5M2 operands and one fp32 scale per 128
          elements of K: A one scale per row and K block, B one per 128 x 128
          block (weights) or one per row and K block (weight gradients); dense
          or one product per expert
  quant   BF16 -> 8-bit codes and scales, for the product along the rows, for
          its gradients along the columns, gathered into expert order, and
          128 x 128 blocks for weights with their transpose
  route   top-k experts per token, gates, per-expert counts, the row order of
          the experts' product and the balance loss; and its gradient

With tokens valid (v_t), logits l, p = softmax(l), n = sum v_t, c_e = how many
(token, choice) pairs chose expert e, P_e = sum_t v_t p_te / n:
  loss = E / (k n) * sum_e c_e P_e          (1 when both are uniform)
"""
import math

import torch

own = False

BLOCK = 128
TYPES = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
FLOOR = 2.0 ** -100          # smallest amax a block's scale is taken from
ROUTE_WORKSPACE = 1 << 20    # bytes that serve the router at every size


# ---------------------------------------------------------------------- cases

def listed():
    return [
        # one token through an attention projection: latency of the smallest product
        {"name": "gemm decode 1", "op": "gemm", "kind": "weight", "m": 1, "n": 4096, "k": 4096, "a": "e4m3", "b": "e4m3"},
        # a decode batch through the up-projection: streaming the weights
        {"name": "gemm decode 128", "op": "gemm", "kind": "weight", "m": 128, "n": 14336, "k": 4096, "a": "e4m3", "b": "e4m3"},
        # prefill through the down-projection
        {"name": "gemm prefill", "op": "gemm", "kind": "weight", "m": 4096, "n": 4096, "k": 14336, "a": "e4m3", "b": "e4m3"},
        # a ragged prompt, sizes no tile divides; E5M2 gradients against transposed weights (input gradient)
        {"name": "gemm ragged", "op": "gemm", "kind": "weight", "m": 1531, "n": 4100, "k": 2000, "a": "e5m2", "b": "e4m3"},
        # weight gradient of the up-projection over 4096 tokens: both operands scaled along the tokens, fp32 result
        {"name": "gemm wgrad", "op": "gemm", "kind": "wgrad", "m": 14336, "n": 4096, "k": 4096, "a": "e5m2", "b": "e4m3"},
        # the experts' up-projection: 4096 tokens, 2 of 8 experts each, unevenly loaded
        {"name": "gemm experts", "op": "gemm", "kind": "grouped", "m": 8192, "n": 14336, "k": 4096, "experts": 8, "a": "e4m3", "b": "e4m3"},
        # 64 decoding tokens sent to 2 experts each: gathered and quantised
        {"name": "quant dispatch 64", "op": "quant", "m": 128, "k": 4096, "tokens": 64, "type": "e4m3", "pow2": False, "rows": True, "cols": False},
        # a training batch: for the forward product and, transposed, for the weight gradient
        {"name": "quant train", "op": "quant", "m": 16384, "k": 4096, "tokens": 0, "type": "e4m3", "pow2": False, "rows": True, "cols": True},
        # a weight and its transpose for the input gradient, power-of-two scales
        {"name": "quant weight", "op": "qweight", "n": 14336, "k": 4096, "type": "e4m3", "pow2": True, "transpose": True},
        # 64 decoding tokens over 8 experts: latency of the router
        {"name": "route 64", "op": "route", "t": 64, "e": 8, "topk": 2, "logits": "fp32", "renorm": True, "padded": False, "masked": False},
        # a prefill batch over many experts, some rows padding, some experts masked
        {"name": "route 16384", "op": "route", "t": 16384, "e": 256, "topk": 8, "logits": "fp32", "renorm": True, "padded": True, "masked": True},
        # its gradient in a training batch, BF16 logits
        {"name": "route gradient", "op": "droute", "t": 16384, "e": 64, "topk": 6, "logits": "bf16", "renorm": True, "padded": True, "masked": False},
    ]


def draw(rng):
    def log_int(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(("gemm", "gemm", "gemm", "quant", "qweight", "route", "droute"))
    if op == "gemm":
        kind = rng.choice(("weight", "weight", "wgrad", "grouped"))
        while True:
            m, n, k = log_int(1, 16384), log_int(64, 16384), 16 * log_int(4, 1024)
            if kind == "wgrad":
                m = max(m, 64)
            if 2 * m * n * k <= 9.0e11 and (m * n + m * k + n * k) <= 4e8:
                break
        if rng.random() < 0.5:
            n = -(-n // 128) * 128
        c = {"op": "gemm", "kind": kind, "m": m, "n": n, "k": k, "a": rng.choice(("e4m3", "e5m2")), "b": rng.choice(("e4m3", "e4m3", "e5m2"))}
        if kind == "grouped":
            e = log_int(2, 64)
            while e * n * k > 5e8:
                e = max(1, e // 2)
                n = max(64, n // 2)
            c["experts"] = e
            c["n"] = n
        return c
    if op == "quant":
        m, k = log_int(1, 32768), 16 * log_int(1, 1024)
        while m * k > 16384 * 4096:
            m = m // 2
        kind = rng.choice(("rows", "cols", "both", "gather"))
        return {"op": "quant", "m": m, "k": k, "tokens": max(1, m // 2) if kind == "gather" else 0, "type": rng.choice(("e4m3", "e5m2")),
                "pow2": rng.random() < 0.5, "rows": kind != "cols", "cols": kind in ("cols", "both")}
    if op == "qweight":
        n, k = log_int(16, 16384), 16 * log_int(1, 1024)
        while n * k > 14336 * 4096:
            n = n // 2
        return {"op": "qweight", "n": n, "k": k, "type": "e4m3", "pow2": rng.random() < 0.5, "transpose": rng.random() < 0.5}
    e = rng.choice((8, 16, 60, 64, 128, 160, 256, rng.randint(2, 256)))
    t = log_int(1, 65536)
    while t * e > 16384 * 256:
        t = t // 2
    return {"op": op, "t": t, "e": e, "topk": rng.randint(1, min(8, e)), "logits": rng.choice(("fp32", "bf16")),
            "renorm": rng.random() < 0.5, "padded": rng.random() < 0.5, "masked": rng.random() < 0.3}


def work(case):
    op = case["op"]
    if op == "gemm":
        m, n, k, e = case["m"], case["n"], case["k"], case.get("experts", 1)
        kb = -(-k // BLOCK)
        b_scales = 4 * kb * (n if case["kind"] == "wgrad" else e * -(-n // BLOCK))
        out = m * n * (4 if case["kind"] == "wgrad" else 2)
        return {"bytes": m * k + e * n * k + 4 * m * kb + b_scales + out, "flops": 2.0 * m * n * k}
    if op == "quant":
        m, k = case["m"], case["k"]
        read = 2 * k * (min(m, case["tokens"]) if case["tokens"] else m)
        rows = m * k + 4 * m * -(-k // BLOCK) if case["rows"] else 0
        cols = k * (-(-m // 16) * 16) + 4 * k * -(-m // BLOCK) if case["cols"] else 0
        return {"bytes": read + rows + cols, "flops": 2.0 * m * k}
    if op == "qweight":
        n, k = case["n"], case["k"]
        return {"bytes": n * k * (4 if case["transpose"] else 3), "flops": 2.0 * n * k}
    t, e, k = case["t"], case["e"], case["topk"]
    size = 4 if case["logits"] == "fp32" else 2
    if op == "route":
        return {"bytes": t * e * size + t * k * 16 + 16 * e, "flops": 5.0 * t * e}
    return {"bytes": 2 * t * e * size + t * k * 8 + 4 * e, "flops": 8.0 * t * e}


# --------------------------------------------------------------------- inputs

def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def activations(g, rows, cols, sigma=1.0):
    """N(0, sigma) with one value in a hundred twenty times larger, as activations have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda") * sigma
    far = torch.rand(rows, cols, generator=g, device="cuda") < 0.01
    return torch.where(far, x * 20.0, x).bfloat16()


def loads(g, rows, experts):
    """Row offsets of unevenly loaded experts, some of them empty where there are many."""
    w = torch.empty(experts, device="cuda", dtype=torch.float64).exponential_(generator=g)
    cut = (w.cumsum(0) / w.sum() * rows).round().int()
    cut[-1] = rows
    return torch.cat([cut.new_zeros(1), cut])


def inputs(case, seed):
    """What the operator is given, in BF16 or fp32: the part exact() starts from too."""
    g = generator(seed)
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        gradient = case["a"] == "e5m2"
        a = activations(g, m, k, 1e-3 if gradient else 1.0)
        if case["kind"] == "wgrad":
            return {"a": a, "b": activations(g, n, k)}
        e = case.get("experts", 1)
        w = torch.empty(e * n, k, dtype=torch.bfloat16, device="cuda").normal_(0.0, 0.02, generator=g)
        return {"a": a, "b": w, "offsets": loads(g, m, e)} if case["kind"] == "grouped" else {"a": a, "b": w}
    if op == "quant":
        rows = case["tokens"] or case["m"]
        x = activations(g, rows, case["k"], 1e-3 if case["type"] == "e5m2" else 1.0)
        if not case["tokens"]:
            return {"x": x, "index": None}
        return {"x": x, "index": torch.randint(0, rows, (case["m"],), generator=g, device="cuda", dtype=torch.int32)}
    if op == "qweight":
        return {"x": torch.empty(case["n"], case["k"], dtype=torch.bfloat16, device="cuda").normal_(0.0, 0.02, generator=g)}
    t, e, k = case["t"], case["e"], case["topk"]
    l = torch.randn(t, e, generator=g, device="cuda") + 0.5 * torch.randn(e, generator=g, device="cuda")
    if case["masked"]:      # experts that this token may not use; the first k always stay open
        hide = torch.rand(t, e, generator=g, device="cuda") < 0.25
        hide[:, : k] = False
        l = l.masked_fill(hide, -math.inf)
    l = l if case["logits"] == "fp32" else l.bfloat16()
    valid = None
    if case["padded"]:
        valid = (torch.rand(t, generator=g, device="cuda") < 0.9375).to(torch.uint8)
    return {"logits": l, "valid": valid, "dgates": torch.randn(t, k, generator=g, device="cuda") * 1e-2,
            "dloss": torch.rand(1, generator=g, device="cuda") * 1e-2}


def prepare(case, seed):
    s = inputs(case, seed)
    s["case"] = case
    op = case["op"]
    if op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        s["qa"], s["sa"] = plain_quantize(s.pop("a"), case["a"], False)
        b = s.pop("b")
        if case["kind"] == "wgrad":
            s["qb"], s["sb"] = plain_quantize(b, case["b"], False)
        else:
            e = case.get("experts", 1)
            s["qb"], s["sb"] = plain_quantize_weight(b.view(e, n, k), case["b"], False)
        s["d"] = torch.empty(m, n, dtype=torch.float32 if case["kind"] == "wgrad" else torch.bfloat16, device="cuda")
    elif op == "quant":
        m, k, t = case["m"], case["k"], TYPES[case["type"]][0]
        s["out"] = {}
        if case["rows"]:
            s["out"]["q"] = torch.empty(m, k, dtype=t, device="cuda")
            s["out"]["sf"] = torch.empty(-(-k // BLOCK), m, device="cuda")
        if case["cols"]:
            s["out"]["q_t"] = torch.empty(k, -(-m // 16) * 16, dtype=t, device="cuda")
            s["out"]["sf_t"] = torch.empty(-(-m // BLOCK), k, device="cuda")
    elif op == "qweight":
        n, k, t = case["n"], case["k"], TYPES[case["type"]][0]
        s["out"] = {"q": torch.empty(n, k, dtype=t, device="cuda"), "sf": torch.empty(-(-n // BLOCK), -(-k // BLOCK), device="cuda")}
        if case["transpose"]:
            s["out"]["q_t"] = torch.empty(k, -(-n // 16) * 16, dtype=t, device="cuda")
            s["out"]["sf_t"] = torch.empty(-(-k // BLOCK), -(-n // BLOCK), device="cuda")
    elif op == "route":
        t, e, k = case["t"], case["e"], case["topk"]
        i32 = {"dtype": torch.int32, "device": "cuda"}
        s["out"] = {"ids": torch.empty(t, k, **i32), "gates": torch.empty(t, k, device="cuda"), "counts": torch.empty(e, **i32),
                    "row_offsets": torch.empty(e + 1, **i32), "dest": torch.empty(t, k, **i32), "src": torch.empty(t * k, **i32),
                    "n_valid": torch.empty(1, **i32), "mean_prob": torch.empty(e, device="cuda"), "loss": torch.empty(1, device="cuda")}
        s["workspace"] = torch.zeros(ROUTE_WORKSPACE, dtype=torch.uint8, device="cuda")
    else:
        forward = plain_route(s["logits"], s["valid"], case["topk"], case["renorm"])
        s["ids"], s["counts"], s["n_valid"] = forward["ids"], forward["counts"], forward["n_valid"]
        s["dlogits"] = torch.empty_like(s["logits"])
    return s


# ----------------------------------------------------------------- one pass

def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    from block_scaled_fp4_tcgen05_gb300 import qfp4
    c = s["case"]
    op = c["op"]
    code = {"e4m3": qfp4.E4M3, "e5m2": qfp4.E5M2}
    if op == "gemm":
        ta, tb = code[c["a"]], code[c["b"]]
        if c["kind"] == "grouped":
            qfp4.gemm_nt_fp8_grouped(ta, tb, s["offsets"], c["m"], 0, c["n"], c["k"], s["qa"], s["sa"], s["qb"], s["sb"], s["d"])
        elif c["kind"] == "wgrad":
            qfp4.gemm_nt_fp8(ta, tb, c["m"], c["n"], c["k"], s["qa"], s["sa"], s["qb"], s["sb"], s["d"], b_rows=1, out=qfp4.OUT_FP32)
        else:
            qfp4.gemm_nt_fp8(ta, tb, c["m"], c["n"], c["k"], s["qa"], s["sa"], s["qb"], s["sb"], s["d"])
        return s["d"]
    if op in ("quant", "qweight"):
        o = s["out"]
        mode = qfp4.SCALE_POW2 if c["pow2"] else qfp4.SCALE_FP32
        if op == "quant":
            qfp4.fp8_quantize(code[c["type"]], s["x"], o.get("q"), o.get("sf"), o.get("q_t"), o.get("sf_t"), scale=mode, row_index=s["index"])
        else:
            qfp4.fp8_quantize_weight(code[c["type"]], s["x"], o["q"], o["sf"], o.get("q_t"), o.get("sf_t"), scale=mode)
        return o
    if op == "route":
        o = s["out"]
        qfp4.moe_route(s["logits"], c["topk"], o["ids"], o["gates"], o["counts"], o["row_offsets"], o["dest"], o["src"], o["n_valid"], o["mean_prob"], o["loss"],
                       s["workspace"], valid=s["valid"], renorm=c["renorm"])
        return o
    qfp4.moe_route_backward(s["logits"], s["ids"], s["counts"], s["n_valid"], s["dgates"], s["dloss"], s["dlogits"], valid=s["valid"], renorm=c["renorm"])
    return s["dlogits"]


def run_plain(s):
    c = s["case"]
    op = c["op"]
    if op == "gemm":
        return plain_gemm(s, c)
    if op == "quant":
        x = s["x"] if s["index"] is None else s["x"][s["index"].long()]
        out = {}
        if c["rows"]:
            out["q"], out["sf"] = plain_quantize(x, c["type"], c["pow2"])
        if c["cols"]:
            out["q_t"], out["sf_t"] = plain_quantize(pad_cols(x.t(), 16), c["type"], c["pow2"])
        return out
    if op == "qweight":
        q, sf = plain_quantize_weight(s["x"][None], c["type"], c["pow2"])
        out = {"q": q[0], "sf": sf[0]}
        if c["transpose"]:
            out["q_t"] = pad_cols(q[0].view(torch.uint8).t(), 16).contiguous().view(q.dtype)
            out["sf_t"] = sf[0].t().contiguous()
        return out
    if op == "route":
        return plain_route(s["logits"], s["valid"], c["topk"], c["renorm"])
    return plain_route_backward(s, c)


# --------------------------------------------------------------- plain forms

def pad_cols(x, multiple):
    more = -x.shape[-1] % multiple
    return x if not more else torch.cat([x, x.new_zeros(*x.shape[:-1], more)], -1)


def block_scales(amax, kind, pow2):
    """(scale, factor that takes a value to its code) of blocks with this largest magnitude."""
    top = TYPES[kind][1]
    amax = amax.clamp(min=FLOOR)
    most = torch.full_like(amax, top)       # a tensor: by a number, the quotient would be a product with its reciprocal
    if not pow2:
        return amax / most, most / amax
    mantissa, exponent = torch.frexp(amax / most)
    exponent = torch.where(mantissa == 0.5, exponent - 1, exponent)     # smallest power of two not below
    return power_of_two(exponent), power_of_two(-exponent)


def power_of_two(n):
    return ((n + 127) << 23).int().view(torch.float32)


def plain_quantize(x, kind, pow2):
    """Codes [rows, cols] and scales [ceil(cols / 128), rows], one per 128 elements of a row."""
    rows, cols = x.shape
    p = pad_cols(x.float(), BLOCK).view(rows, -1, BLOCK)
    scale, factor = block_scales(p.abs().amax(2), kind, pow2)
    top = TYPES[kind][1]
    q = (p * factor[..., None]).clamp(-top, top).view(rows, -1)[:, :cols].to(TYPES[kind][0])
    return q.contiguous(), scale.t().contiguous()


def plain_quantize_weight(w, kind, pow2):
    """Codes [e, n, k] and scales [e, ceil(n / 128), ceil(k / 128)], one per 128 x 128 block."""
    e, n, k = w.shape
    p = pad_cols(pad_cols(w.float(), BLOCK).transpose(1, 2), BLOCK).transpose(1, 2)
    p = p.reshape(e, p.shape[1] // BLOCK, BLOCK, p.shape[2] // BLOCK, BLOCK)
    scale, factor = block_scales(p.abs().amax((2, 4)), kind, pow2)
    top = TYPES[kind][1]
    q = (p * factor[:, :, None, :, None]).clamp(-top, top).reshape(e, p.shape[1] * BLOCK, -1)[:, :n, :k]
    return q.to(TYPES[kind][0]).contiguous(), scale.contiguous()


def dequantize_rows(q, scale):
    return q.float() * scale.t().repeat_interleave(BLOCK, 1)[:, : q.shape[1]]


def plain_gemm(s, c):
    a = dequantize_rows(s["qa"], s["sa"])
    if c["kind"] == "wgrad":
        return a @ dequantize_rows(s["qb"], s["sb"]).t()
    n, k = c["n"], c["k"]
    scale = s["sb"].repeat_interleave(BLOCK, 1)[:, :n].repeat_interleave(BLOCK, 2)[:, :, :k]
    b = s["qb"].float() * scale
    if c["kind"] == "weight":
        return (a @ b[0].t()).bfloat16()
    cuts = s["offsets"].tolist()
    return torch.cat([a[lo:hi] @ w.t() for lo, hi, w in zip(cuts, cuts[1:], b)]).bfloat16()


def softmax(l):
    """Along the experts, in 64 bits; a row with no expert left has only zeros."""
    l = l.double()
    top = l.amax(1, keepdim=True)
    p = torch.exp(l - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    total = p.sum(1, keepdim=True)
    return p / torch.where(total > 0, total, torch.ones_like(total))


def plain_route(l, valid, k, renorm):
    t, e = l.shape
    alive = torch.ones(t, dtype=torch.bool, device=l.device) if valid is None else valid != 0
    order = torch.sort(l.float(), dim=1, descending=True, stable=True)[1][:, :k]
    takes = alive[:, None] & (l.gather(1, order) > -math.inf)
    p = softmax(l) * alive[:, None]
    gates = p.gather(1, order) * takes
    if renorm:
        total = gates.sum(1, keepdim=True)
        gates = gates / torch.where(total > 0, total, torch.ones_like(total))
    ids = torch.where(takes, order, -1).int()
    flat = torch.where(takes, order, e).view(-1)
    counts = torch.bincount(flat, minlength=e + 1)[:e]
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    sequence = torch.sort(flat, stable=True)[1]
    at = torch.empty_like(sequence)
    at[sequence] = torch.arange(t * k, device=l.device)
    dest = torch.where(takes.view(-1), at, -1).view(t, k).int()
    src = torch.where(torch.arange(t * k, device=l.device) < offsets[-1], sequence // k, -1).int()
    n_valid = alive.sum().view(1)
    n = n_valid.clamp(min=1)
    mean = p.sum(0) / n
    loss = (counts * mean).sum() * e / (k * n)
    return {"ids": ids, "gates": gates.float(), "counts": counts.int(), "row_offsets": offsets.int(), "dest": dest, "src": src,
            "n_valid": n_valid.int(), "mean_prob": mean.float(), "loss": loss.float().view(1)}


def plain_route_backward(s, c):
    """d/dlogits of (gates . dgates + loss * dloss)."""
    l, ids, k, e = s["logits"], s["ids"].long(), c["topk"], c["e"]
    t = l.shape[0]
    alive = torch.ones(t, 1, dtype=torch.bool, device=l.device) if s["valid"] is None else (s["valid"] != 0)[:, None]
    p = softmax(l)
    takes = ids >= 0
    safe = ids.clamp(min=0)
    dg = s["dgates"].double() * takes
    chosen = p.gather(1, safe) * takes
    if c["renorm"]:     # gate = p / sum of the chosen p
        total = chosen.sum(1, keepdim=True)
        total = torch.where(total > 0, total, torch.ones_like(total))
        dg = (dg - (dg * chosen).sum(1, keepdim=True) / total) / total * takes
    n = s["n_valid"].double().clamp(min=1)
    dp = (s["dloss"].double() * s["counts"].double() * e / (k * n * n)).expand(t, e).clone()
    dp.scatter_add_(1, safe, dg)
    d = p * (dp - (p * dp).sum(1, keepdim=True)) * alive
    return d.to(l.dtype)


# ------------------------------------------------------------ 64-bit results

def round_codes(y, kind):
    """Values y rounded to the nearest code of the type, ties to the even one, in 64 bits."""
    mantissa, least, top = (3, -6, 448.0) if kind == "e4m3" else (2, -14, 57344.0)
    y = y.clamp(-top, top)
    exponent = (torch.frexp(y)[1] - 1).clamp(min=least).long()
    step = ((exponent - mantissa + 1023) << 52).view(torch.float64)
    return torch.round(y / step) * step


def exact_scales(amax, kind, pow2):
    s = amax.clamp(min=FLOOR) / TYPES[kind][1]
    power = torch.ceil(torch.log2(s) - 1e-12).long()
    return ((power + 1023) << 52).view(torch.float64) if pow2 else s


def exact_rows(x, kind, pow2):
    rows, cols = x.shape
    blocks = -(-cols // BLOCK)
    q, sf = torch.empty(rows, cols, dtype=torch.float64, device=x.device), torch.empty(blocks, rows, dtype=torch.float64, device=x.device)
    for i in range(blocks):
        part = x[:, i * BLOCK:(i + 1) * BLOCK].double()
        sf[i] = exact_scales(part.abs().amax(1), kind, pow2)
        q[:, i * BLOCK:(i + 1) * BLOCK] = round_codes(part / sf[i][:, None], kind)
    return q, sf


def exact(case, seed):
    op = case["op"]
    if op == "gemm":
        s = prepare(case, seed)     # the product's inputs are the codes
        m, n, k, kind = case["m"], case["n"], case["k"], case["kind"]
        d = torch.zeros(m, n, dtype=torch.float64, device="cuda")
        cuts = s["offsets"].tolist() if kind == "grouped" else [0, m]
        for e in range(len(cuts) - 1):
            lo, hi = cuts[e], cuts[e + 1]
            for i in range(-(-k // BLOCK)):
                cols = slice(i * BLOCK, min(k, (i + 1) * BLOCK))
                a = s["qa"][lo:hi, cols].double() * s["sa"][i, lo:hi, None].double()
                if kind == "wgrad":
                    b = s["qb"][:, cols].double() * s["sb"][i][:, None].double()
                else:
                    row = torch.arange(n, device="cuda") // BLOCK
                    b = s["qb"][e, :, cols].double() * s["sb"][e, row, i][:, None].double()
                d[lo:hi] += a @ b.t()
        return d
    s = inputs(case, seed)
    if op == "quant":
        x = s["x"] if s["index"] is None else s["x"].index_select(0, s["index"].long())
        out = {}
        if case["rows"]:
            out["q"], out["sf"] = exact_rows(x, case["type"], case["pow2"])
        if case["cols"]:
            q, out["sf_t"] = exact_rows(x.t(), case["type"], case["pow2"])
            out["q_t"] = torch.zeros(q.shape[0], -(-q.shape[1] // 16) * 16, dtype=torch.float64, device="cuda")
            out["q_t"][:, : q.shape[1]] = q
        return out
    if op == "qweight":
        x = s["x"].double()
        n, k = x.shape
        q, sf = torch.empty_like(x), torch.empty(-(-n // BLOCK), -(-k // BLOCK), dtype=torch.float64, device="cuda")
        for i in range(sf.shape[0]):
            rows = x[i * BLOCK:(i + 1) * BLOCK]
            peak = rows.abs().amax(0)
            full = torch.zeros(sf.shape[1] * BLOCK, dtype=torch.float64, device="cuda")
            full[:k] = peak
            sf[i] = exact_scales(full.view(-1, BLOCK).amax(1), case["type"], case["pow2"])
            q[i * BLOCK:(i + 1) * BLOCK] = round_codes(rows / sf[i].repeat_interleave(BLOCK)[:k], case["type"])
        out = {"q": q, "sf": sf}
        if case["transpose"]:
            out["q_t"] = torch.zeros(k, -(-n // 16) * 16, dtype=torch.float64, device="cuda")
            out["q_t"][:, :n] = q.t()
            out["sf_t"] = sf.t().contiguous()
        return out
    return exact_route(case, s)


def exact_route(case, s):
    l, k, e, t = s["logits"].double(), case["topk"], case["e"], case["t"]
    alive = torch.ones(t, dtype=torch.float64, device="cuda") if s["valid"] is None else (s["valid"] != 0).double()
    p = torch.exp(l - torch.logsumexp(l, 1, keepdim=True)) * alive[:, None]
    left, picks = l.clone(), []
    for _ in range(k):          # the largest, then the largest of the rest; argmax of equal values: the lowest
        best = left.amax(1, keepdim=True)
        at = (left == best).to(torch.uint8).argmax(1)
        picks.append(torch.where(best[:, 0] > -math.inf, at, -1))
        left.scatter_(1, at[:, None], -math.inf)
    ids = torch.stack(picks, 1)
    here = (ids >= 0) & (alive[:, None] > 0)
    one_hot = torch.zeros(t, e, dtype=torch.float64, device="cuda").scatter_add_(1, ids.clamp(min=0), here.double())
    counts = one_hot.sum(0)
    n = max(1.0, float(alive.sum()))
    mean = p.sum(0) / n
    total = (p * one_hot).sum(1, keepdim=True) if case["renorm"] else torch.ones(t, 1, dtype=torch.float64, device="cuda")
    total = torch.where(total > 0, total, torch.ones_like(total))
    gates = p.gather(1, ids.clamp(min=0)) * here / total
    if case["op"] == "route":
        return {"ids": None, "gates": gates, "counts": None, "row_offsets": None, "dest": None, "src": None, "n_valid": None, "mean_prob": mean,
                "loss": (counts * mean).sum().view(1) * e / (k * n)}
    # f = sum_j dgates_j gate_j + dloss loss: df/dl_i = sum over the chosen + balance part, both through the softmax
    weight = torch.zeros_like(p).scatter_add_(1, ids.clamp(min=0), s["dgates"].double() * here)
    share = p * one_hot / total                      # the gates, at their experts
    if case["renorm"]:                               # gates are a softmax over the chosen experts alone
        d = share * (weight - (share * weight).sum(1, keepdim=True))
    else:
        d = share * weight - p * (share * weight).sum(1, keepdim=True)
    slope = s["dloss"].double() * counts * e / (k * n * n)
    return d + p * (slope - (p * slope).sum(1, keepdim=True))
