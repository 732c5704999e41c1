"""A mixture-of-experts layer in 8-bit floating point, forward and backward, on
one GPU: router -> gather and quantise -> experts' up and down products ->
weighted sum, then the gradients of the router, of the weights and of the input.

    python examples/moe_fp8_layer.py [--tokens 4096] [--experts 8] [--topk 2]

Every product and quantiser and the router are the library's kernels; the
elementwise steps between them (SwiGLU, the weighted sum) are torch.  No step
needs the experts' loads on the host.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from block_scaled_fp4_tcgen05_gb300 import qfp4  # noqa: E402

BLOCK = 128


def up16(n: int) -> int:
    return -(-n // 16) * 16


def quantize(x, kind, rows=True, cols=False, index=None):
    """(Q, SF, Q_t, SF_t) of fp8_quantize, each None where not asked for."""
    M, K = (x.shape[0] if index is None else index.numel()), x.shape[1]
    t = torch.float8_e4m3fn if kind == qfp4.E4M3 else torch.float8_e5m2
    q = torch.empty(M, K, dtype=t, device=x.device) if rows else None
    sf = torch.empty(-(-K // BLOCK), M, device=x.device) if rows else None
    qt = torch.empty(K, up16(M), dtype=t, device=x.device) if cols else None
    sft = torch.empty(-(-M // BLOCK), K, device=x.device) if cols else None
    qfp4.fp8_quantize(kind, x, q, sf, qt, sft, row_index=index)
    return q, sf, qt, sft


class Experts:
    """Weights [E, N, K] of one projection: their codes and those of the transpose."""

    def __init__(self, w):
        E, N, K = w.shape
        self.shape = (E, N, K)
        new = dict(dtype=torch.float8_e4m3fn, device=w.device)
        nb, kb = -(-N // BLOCK), -(-K // BLOCK)
        self.q, self.sf = torch.empty(E, N, K, **new), torch.empty(E, nb, kb, device=w.device)
        self.qt, self.sft = torch.empty(E, K, up16(N), **new), torch.empty(E, kb, nb, device=w.device)
        qfp4.fp8_quantize_weight(qfp4.E4M3, w, self.q, self.sf, self.qt, self.sft)

    def forward(self, q, sf, offsets):
        E, N, K = self.shape
        d = torch.zeros(q.shape[0], N, dtype=torch.bfloat16, device=q.device)
        qfp4.gemm_nt_fp8_grouped(qfp4.E4M3, qfp4.E4M3, offsets, q.shape[0], 0, N, K, q, sf, self.q, self.sf, d)
        return d

    def input_gradient(self, dy, offsets):
        """dX = dY W: the transposed weights, gradients in E5M2 (N a multiple of 16 here)."""
        E, N, K = self.shape
        q, sf, _, _ = quantize(dy, qfp4.E5M2)
        d = torch.zeros(dy.shape[0], K, dtype=torch.bfloat16, device=dy.device)
        qfp4.gemm_nt_fp8_grouped(qfp4.E5M2, qfp4.E4M3, offsets, dy.shape[0], 0, K, N, q, sf, self.qt, self.sft, d)
        return d

    def weight_gradient(self, dy, x, offsets, index=None):
        """dW[e] = dY_e^T X_e, fp32, both operands scaled along the tokens; index
        gathers the rows of x into expert order."""
        E, N, K = self.shape
        rows = dy.shape[0]
        cols = qfp4.fp8_grouped_cols(rows, E)
        operands = []
        for t, kind, ix in ((dy, qfp4.E5M2, None), (x, qfp4.E4M3, index)):
            qt = torch.empty(t.shape[1], cols, dtype=torch.uint8, device=t.device)
            sft = torch.empty(cols // BLOCK, t.shape[1], device=t.device)
            qfp4.fp8_quantize_grouped(kind, t, offsets, qt, sft, row_index=ix)
            operands += [qt, sft]
        dw = torch.empty(E, N, K, device=x.device)
        qfp4.gemm_nt_fp8_kgrouped(qfp4.E5M2, qfp4.E4M3, offsets, rows, N, K, *operands, dw)
        return dw


def swiglu(h):
    gate, up = h.float().chunk(2, -1)
    return (torch.nn.functional.silu(gate) * up).bfloat16()


def layer(x, logits, up, down, topk, dy=None, balance=0.01, valid=None):
    """Output and balance loss of the layer, and with dy (the gradient of the
    output) those of x, of the logits and of both projections' weights."""
    T, E = logits.shape
    dev, i32 = x.device, dict(dtype=torch.int32, device=x.device)
    ids, dest, src = torch.empty(T, topk, **i32), torch.empty(T, topk, **i32), torch.empty(T * topk, **i32)
    counts, offsets, n = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(1, **i32)
    gates, mean, loss = torch.empty(T, topk, device=dev), torch.empty(E, device=dev), torch.empty(1, device=dev)
    ws = torch.empty(qfp4.moe_route_workspace_bytes(T, E, topk), dtype=torch.uint8, device=dev)
    qfp4.moe_route(logits, topk, ids, gates, counts, offsets, dest, src, n, mean, loss, ws, valid=valid)

    q, sf, _, _ = quantize(x, qfp4.E4M3, index=src)             # tokens in expert order
    h = up.forward(q, sf, offsets)
    a = swiglu(h)
    q2, sf2, _, _ = quantize(a, qfp4.E4M3)
    o = down.forward(q2, sf2, offsets)
    chosen = (dest >= 0).float()[..., None]
    rows = o[dest.clamp(min=0).long().view(-1)].view(T, topk, -1).float() * chosen
    y = (rows * gates[..., None]).sum(1)
    if dy is None:
        return y, loss
    dgates = (rows * dy[:, None]).sum(-1)
    at = dest.view(-1).long()
    keep = at >= 0
    do = torch.zeros_like(o)
    do[at[keep]] = (gates[..., None] * dy[:, None]).reshape(T * topk, -1)[keep].bfloat16()
    da = down.input_gradient(do, offsets).float()
    gate, uph = h.float().chunk(2, -1)
    s = torch.sigmoid(gate)
    dh = torch.cat([da * uph * s * (1 + gate * (1 - s)), da * gate * s], -1).bfloat16()
    dxe = up.input_gradient(dh, offsets)
    dx = (dxe[dest.clamp(min=0).long().view(-1)].view(T, topk, -1).float() * chosen).sum(1)
    dlogits = torch.empty_like(logits)
    qfp4.moe_route_backward(logits, ids, counts, n, dgates, torch.full((1,), balance, device=dev), dlogits, valid=valid)
    return y, loss, {"x": dx, "logits": dlogits, "up": up.weight_gradient(dh, x, offsets, src),
                     "down": down.weight_gradient(do, a, offsets)}


def plain(x, logits, w_up, w_down, topk, dy, balance):
    """The same layer in torch, fp32 weights and autograd."""
    T, E = logits.shape
    x, logits, w_up, w_down = (t.float().detach().requires_grad_() for t in (x, logits, w_up, w_down))
    p = torch.softmax(logits, -1)
    top, ids = p.topk(topk, -1)
    g = top / top.sum(-1, keepdim=True)
    y = torch.zeros(T, w_down.shape[1], device=x.device)
    for e in range(E):
        t, j = (ids == e).nonzero(as_tuple=True)
        gate, up = (x[t] @ w_up[e].t()).chunk(2, -1)
        y = y.index_add(0, t, (torch.nn.functional.silu(gate) * up @ w_down[e].t()) * g[t, j, None])
    counts = torch.bincount(ids.view(-1), minlength=E).float()
    loss = E / (topk * T) * (counts * p.mean(0)).sum()
    ((y * dy).sum() + balance * loss).backward()
    return y.detach(), loss.detach(), {"x": x.grad, "logits": logits.grad, "up": w_up.grad, "down": w_down.grad}


def inputs(T, E, D, H, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    def normal(*s):
        return torch.randn(*s, generator=g, device=device)
    return (normal(T, D).bfloat16(), normal(T, E), (normal(E, 2 * H, D) / D ** 0.5).bfloat16(),
            (normal(E, D, H) / H ** 0.5).bfloat16(), normal(T, D) * 1e-2)


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("tokens", 4096), ("experts", 8), ("topk", 2), ("model", 4096), ("hidden", 2048)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    x, logits, w_up, w_down, dy = inputs(a.tokens, a.experts, a.model, a.hidden)
    up, down = Experts(w_up), Experts(w_down)
    y, loss, grads = layer(x, logits, up, down, a.topk, dy)
    assert qfp4.poll_device_status() == 0
    want_y, want_loss, want = plain(x, logits, w_up, w_down, a.topk, dy, 0.01)
    print(f"balance loss {float(loss):.6f} (plain {float(want_loss):.6f})")
    for name, got, ref in (("output", y, want_y), *((k, grads[k], want[k]) for k in want)):
        print(f"{name:8s} relative difference to fp32 weights and activations: "
              f"{float((got.float() - ref).norm() / ref.norm()):.4f}")


if __name__ == "__main__":
    main()
