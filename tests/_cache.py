"""The paged cache in torch on the CPU or GPU: its types' rules and its layout as
the header states them, apart from the library."""
import torch

from block_scaled_fp4_tcgen05_gb300 import qfp4

TYPES = (qfp4.CACHE_BF16, qfp4.CACHE_E4M3, qfp4.CACHE_NVFP4)
ROW = {qfp4.CACHE_BF16: lambda D: 2 * D, qfp4.CACHE_E4M3: lambda D: D, qfp4.CACHE_NVFP4: lambda D: D // 2}
SCALE = {qfp4.CACHE_BF16: lambda D: 0, qfp4.CACHE_E4M3: lambda D: 4, qfp4.CACHE_NVFP4: lambda D: D // 16}
GRID = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def encode(type, x, gs):
    """(codes, scales, values) of fp32 x [.., D]: bytes, bytes and what they stand for, all in fp32 arithmetic."""
    if type == qfp4.CACHE_BF16:
        y = x.bfloat16()
        return y.contiguous().view(torch.uint8), x.new_zeros(*x.shape[:-1], 0).to(torch.uint8), y.float()
    if type == qfp4.CACHE_E4M3:
        a = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -100)
        top = torch.full_like(a, 448.0)
        s = a / top
        q = (x * (top / a)).clamp(-448, 448).to(torch.float8_e4m3fn)
        return q.view(torch.uint8), s.contiguous().view(torch.uint8), q.float() * s
    b = x.unflatten(-1, (-1, 16))
    amax = b.abs().amax(-1)
    sf = (amax / torch.full_like(amax, 6.0) / gs).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = (sf.float() * gs)[..., None]
    t = torch.where(s > 0, b / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(b)).flatten(-2)
    mid = (GRID[1:] + GRID[:-1]).to(x.device) / 2           # ties to the even code
    size = t.abs().contiguous()
    low, high = torch.bucketize(size, mid, right=False), torch.bucketize(size, mid, right=True)
    code = torch.where(low == high, low, torch.where(low % 2 == 0, low, high))
    signed = (code | (torch.signbit(t).long() << 3)).to(torch.uint8)
    value = torch.where(torch.signbit(t), -GRID.to(x.device)[code], GRID.to(x.device)[code]).unflatten(-1, (-1, 16)) * s
    return signed[..., 0::2] | (signed[..., 1::2] << 4), sf.view(torch.uint8), value.flatten(-2)


def places(type, D):
    """Offsets in a unit of [16, row] K codes, [16, scale] K scales, V codes, V scales."""
    row, sb = ROW[type](D), SCALE[type](D)
    out = [torch.zeros(16, n, dtype=torch.long) for n in (row, sb, row, sb)]
    p, w = min(64, row), row // 8
    for j in range(16):
        h, t, e = j // 8, j % 8 // 2, j % 2
        for x in range(row):
            out[0][j, x] = ((h * (row // p) + x // p) * 8 + j % 8) * p + x % p
            a = (2 * h + e) * w + x % w
            out[2][j, x] = 16 * (row + sb) + ((a // 16) * 32 + 4 * (x // w) + t) * 16 + a % 16
        for x in range(sb):
            out[1][j, x] = 16 * row + j * sb + x
            out[3][j, x] = 16 * (2 * row + sb) + (j * 4 + x if type == qfp4.CACHE_E4M3 else x * 16 + 4 * t + 2 * h + e)
    return out


def empty(type, pages, kv_heads, D, page_size, fill=0):
    n = qfp4.kv_cache_page_bytes(type, kv_heads, D, page_size) // kv_heads
    return torch.full((pages, kv_heads, n), fill, dtype=torch.uint8, device="cuda")


def put(type, cache, page_size, slots, k, v, gs_k, gs_v):
    """Writes k, v [T, heads, D] (fp32) by the stated layout; returns their values."""
    D, out = k.shape[-1], []
    at = [p.cuda() for p in places(type, D)]
    unit = 2 * 16 * (ROW[type](D) + SCALE[type](D))
    units = cache.view(cache.shape[0], cache.shape[1], -1, unit)
    slots = slots.long()
    heads = torch.arange(cache.shape[1], device="cuda")[None, :, None]
    for half, (x, gs) in enumerate(((k, gs_k), (v, gs_v))):
        codes, scales, value = encode(type, x, gs)
        for data, place in ((codes, at[2 * half]), (scales, at[2 * half + 1])):
            if data.shape[-1]:
                units[(slots // page_size)[:, None, None], heads, (slots % page_size // 16)[:, None, None], place[slots % 16][:, None]] = data
        out.append(value)
    return out
