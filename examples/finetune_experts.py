"""Fine-tunes a routed expert layer, then serves it in four bits.

A student layer learns a random teacher's outputs: router, padded layout,
expert products, their gradients, clipping by the global norm and a plain
gradient step, all on the library's kernels (the activation between the two
products and the parameter update are elementary torch).  Then the learned
weights are quantised to MXFP4 and run in the two forms the library has for
them: 4-bit activations (ragged_gemm_mxfp4) and 8-bit ones (fused_experts).

    python examples/finetune_experts.py [steps]
"""
from __future__ import annotations

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch

import mixture_experts_ffn_align_gb300 as moe

M, H, I, E, TOPK = 512, 256, 512, 8, 2      # tokens, hidden, intermediate, experts
BLOCK = 16                                  # padding of an expert's rows in the layout


class ExpertLayer:
    """Buffers and plans of one layer for M tokens."""

    def __init__(self):
        self.p = moe.Problem(M=M, H=H, I=I, E=E, topk=TOPK, block_size=BLOCK)
        b = moe.stage_buffers(self.p)
        self.b, rows = b, b["x_perm"].shape[0]
        # the padded layout is a ragged one too: rows of expert e from expert_offsets[e]
        self.up = moe.Ragged(R=rows, N=2 * I, K=H, E=E)
        self.down = moe.Ragged(R=rows, N=H, K=I, E=E)
        n = max(moe.moe_ragged_workspace_bytes(self.up), moe.moe_ragged_workspace_bytes(self.down))
        self.ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.weights = torch.empty(M, TOPK, device="cuda")
        self.ids = torch.empty(M, TOPK, dtype=torch.int32, device="cuda")
        # what the kernels leave alone (rows past the last segment) stays zero
        self.h, self.dh = (torch.zeros(rows, 2 * I, dtype=torch.bfloat16, device="cuda")
                           for _ in range(2))
        self.y2, self.dy2 = (torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
                             for _ in range(2))
        self.dz = torch.zeros(rows, I, dtype=torch.bfloat16, device="cuda")
        self.y = torch.empty(M, H, dtype=torch.bfloat16, device="cuda")

    def route(self, x, logits):
        b = self.b
        moe.moe_topk_router(logits, TOPK, self.weights, self.ids)
        moe.moe_align_permute(self.p, x, self.ids, self.weights, b["sorted_ids"],
                              b["block_expert_ids"], b["expert_offsets"], b["num_post_padded"],
                              b["inv_perm"], b["x_perm"], None, b["align_ws"])
        item = b["sorted_ids"].long()
        live = item < M * TOPK
        self.token = torch.where(live, item // TOPK, 0)
        self.row_weight = torch.where(live, self.weights.flatten()[item.clamp(max=M * TOPK - 1)],
                                      0.0)

    def forward(self, w13, w2):
        b, off = self.b, self.b["expert_offsets"]
        moe.ragged_gemm(self.up, b["x_perm"], w13, off, self.h, self.ws)
        g, u = self.h.float().split(I, 1)
        self.z = (torch.nn.functional.silu(g) * u).bfloat16()
        moe.ragged_gemm(self.down, self.z, w2, off, self.y2, self.ws)
        moe.unpermute_reduce(self.p, self.y2, b["inv_perm"], self.weights, self.y)
        return self.y

    def backward(self, dy, w13, w2, dw13, dw2):
        """Gradients of w13 and w2 from dy, the gradient of the layer's output."""
        off = self.b["expert_offsets"]
        self.dy2.copy_(dy.float()[self.token] * self.row_weight[:, None])
        moe.ragged_gemm_wgrad(self.down, self.dy2, self.z, off, dw2, self.ws)
        moe.ragged_gemm_dgrad(self.down, self.dy2, w2, off, self.dz, self.ws)
        g, u = self.h.float().split(I, 1)
        s, dz = torch.sigmoid(g), self.dz.float()
        self.dh[:, :I] = dz * u * s * (1 + g * (1 - s))
        self.dh[:, I:] = dz * g * s
        moe.ragged_gemm_wgrad(self.up, self.dh, self.b["x_perm"], off, dw13, self.ws)


def mxfp4(w):
    """Codes, scales and packed scales of weights [E, N, K]."""
    n, k = w.shape[1:]
    codes = torch.empty(E * n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(E * n, k // 32, dtype=torch.uint8, device="cuda")
    moe.moe_mxfp4_quantize(w.view(E * n, k), codes, scales, scale_mode="ceil")
    codes, scales = codes.view(E, n, k // 2), scales.view(E, n, k // 32)
    packed = torch.empty_like(scales)
    moe.moe_mxfp4_pack_scales(scales, packed)
    return codes, scales, packed


def serve_w4a4(layer, q13, q2):
    """The layer's output with weights and activations in four bits."""
    b, off = layer.b, layer.b["expert_offsets"]

    def product(p, x, q, y):
        codes = torch.empty(p.R, p.K // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(p.R, p.K // 32, dtype=torch.uint8, device="cuda")
        moe.moe_mxfp4_quantize(x, codes, scales)
        moe.ragged_gemm_mxfp4(p, codes, scales, q[0], q[2], off, y, layer.ws)
        return y

    g, u = product(layer.up, b["x_perm"], q13, layer.h).float().split(I, 1)
    product(layer.down, (torch.nn.functional.silu(g) * u).bfloat16(), q2, layer.y2)
    y = torch.empty_like(layer.y)
    moe.unpermute_reduce(layer.p, layer.y2, b["inv_perm"], layer.weights, y)
    return y


def serve_w4a8(layer, x, q13, q2):
    """The same weights through fused_experts, with 8-bit activations."""
    p = moe.Problem(M=M, H=H, I=I, E=E, topk=TOPK, quant="mxfp4", act_scale_fmt="ue8m0")
    y = torch.empty_like(layer.y)
    ws = torch.empty(moe.moe_workspace_bytes(p), dtype=torch.uint8, device="cuda")
    moe.fused_experts(p, x, q13[0], q13[1], q2[0], q2[1], layer.weights, layer.ids, y, ws)
    return y


def main(steps: int = 60, lr: float = 2.0, max_norm: float = 1.0, verbose: bool = True):
    g = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale

    x, logits = randn(M, H).bfloat16(), randn(M, E)
    layer = ExpertLayer()
    layer.route(x, logits)
    target = layer.forward(randn(E, 2 * I, H, scale=0.06).bfloat16(),
                           randn(E, H, I, scale=0.06).bfloat16()).float().clone()
    masters = [randn(E, 2 * I, H, scale=0.06), randn(E, H, I, scale=0.06)]
    w13, w2 = (w.bfloat16() for w in masters)
    grads = [torch.empty(w.shape, device="cuda") for w in masters]      # float32
    norm = torch.empty((), device="cuda")
    ws = torch.empty(moe.moe_clip_workspace_bytes(), dtype=torch.uint8, device="cuda")
    losses, norms = [], []
    for step in range(steps):
        err = layer.forward(w13, w2).float() - target
        losses.append(err.square().mean())
        layer.backward(err * (2 / M), w13, w2, *grads)
        moe.moe_clip_grad_norm(grads, max_norm, norm, ws)
        norms.append(norm.clone())
        for w, m, d in zip((w13, w2), masters, grads):
            m.sub_(d, alpha=lr)
            w.copy_(m)
        if verbose and step % 10 == 0:
            print(f"step {step:3d}  loss {float(losses[-1]):.4f}  gradient norm {float(norm):.3f}")
    y = layer.forward(w13, w2).float().clone()
    q13, q2 = mxfp4(w13), mxfp4(w2)
    rms = float(y.square().mean().sqrt())

    def off(t):
        return float((t.float() - y).square().mean().sqrt()) / rms

    w4a4, w4a8 = off(serve_w4a4(layer, q13, q2)), off(serve_w4a8(layer, x, q13, q2))
    status = moe.moe_sync_status()
    if status != 0:
        raise RuntimeError(moe.moe_status_string(status))
    if verbose:
        print(f"loss {float(losses[0]):.4f} -> {float(losses[-1]):.4f}; error of the 4-bit "
              f"layer against bf16 (rms): 4-bit activations {w4a4:.3f}, 8-bit {w4a8:.3f}")
    return dict(losses=[float(v) for v in losses], norms=[float(v) for v in norms], w4a4=w4a4,
                w4a8=w4a8)


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:2]))
