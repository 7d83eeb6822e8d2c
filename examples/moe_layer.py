"""One mixture-of-experts layer on the library's calls: a training step and a serving step.

    python examples/moe_layer.py [--ranks 4 --tokens 256 --experts 32 --top-k 4 --hidden 512 --ffn 256]

Training: route -> plan -> prefetch -> dispatch -> product -> gated activation (8-bit checkpoint)
-> product -> combine, and the backward of each. What is kept from forward to backward is the
tokens, the plan, the checkpoint and the combine's input: the receive rows are dispatched again
and the activation comes out of the checkpoint's backward.
Serving: the experts' weights are quantised to 4 bits once; a step routes, plans, dispatches the
tokens in 4 bits, multiplies, quantises the activation, multiplies and combines.

The router's own product is a plain matrix product and is left to torch.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import moe_expert_dispatch_online_gb300 as bep  # noqa: E402


class MoELayer:
    """R ranks of S tokens, E experts of [H, 2F] and [F, H], K experts a token."""

    def __init__(self, R, S, E, K, H, F, route=bep.RouteConfig(), device="cuda"):
        self.R, self.S, self.E, self.K, self.H, self.F = R, S, E, K, H, F
        self.up = bep.Context(bep.Config(R, E, E // R, K, S, H, 2 * F, bep.BEP_TRAIN))
        self.down = bep.Context(bep.Config(R, E, E // R, K, S, F, H, bep.BEP_TRAIN))
        self.route = route
        self.buf = bep.Buffers(self.up.cfg, device)
        bf16 = dict(dtype=torch.bfloat16, device=device)
        rows = R * S * K
        self.topk = torch.empty((R, S, K), dtype=torch.int32, device=device)
        self.gates = torch.empty((R, S, K), dtype=torch.float32, device=device)
        self.load = torch.zeros(E, dtype=torch.int32, device=device)
        self.bias = torch.zeros(E, dtype=torch.float32, device=device)
        self.a = torch.empty((rows, F), **bf16)
        self.y = torch.empty((rows, H), **bf16)
        self.out = torch.empty((R, S, H), **bf16)
        self.ckpt = bep.ActCheckpoint(rows, F, device)
        self.w_router = torch.randn(H, E, device=device) * H ** -0.5
        self.w1 = (torch.randn(E, H, 2 * F, device=device) * H ** -0.5).bfloat16()
        self.w2 = (torch.randn(E, F, H, device=device) * F ** -0.5).bfloat16()
        self.slots1 = torch.empty((R, E // R, H, 2 * F), **bf16)
        self.slots2 = torch.empty((R, E // R, F, H), **bf16)

    def choose(self, x):
        """Router scores, experts, gates and the plan of this step."""
        buf = self.buf
        self.logits = x.float() @ self.w_router
        self.load.zero_()
        bep.bep_route(self.up, self.route, self.logits, self.topk, self.gates, bias=self.bias,
                      load=self.load)
        bep.bep_plan(self.up, self.topk, buf.cu_seqlens, buf.slot_expert, buf.dest, buf.maxvio)

    def balance(self, rate=1e-3):
        """Moves the choice towards the experts that got fewer tokens than the mean."""
        mean = self.R * self.S * self.K / self.E
        self.bias += rate * torch.sign(mean - self.load)

    def forward(self, x):
        buf = self.buf
        self.choose(x)
        bep.bep_prefetch_weight(self.up, buf.slot_expert, self.w1, self.slots1)
        bep.bep_prefetch_weight(self.down, buf.slot_expert, self.w2, self.slots2)
        bep.bep_dispatch(self.up, x, buf.dest, buf.recv)
        bep.bep_grouped_gemm(self.up, buf.cu_seqlens, buf.recv, self.w1, self.slots1, buf.y)
        bep.bep_swiglu(self.up, buf.y, self.a, self.ckpt.codes, self.ckpt.scales)
        bep.bep_grouped_gemm(self.down, buf.cu_seqlens, self.a, self.w2, self.slots2, self.y)
        bep.bep_combine(self.down, self.y, buf.dest, self.gates, self.out)
        return self.out

    def backward(self, x, dout):
        """Gradients of the tokens and of the three weights, for the last forward's x."""
        buf, R, E = self.buf, self.R, self.E
        dev = x.device
        dgates = torch.empty_like(self.gates)
        bep.bep_combine_dgates(self.down, dout, self.y, buf.dest, dgates)
        dy = torch.empty_like(self.y)
        bep.bep_combine_bwd(self.down, dout, buf.dest, self.gates, dy)
        da = torch.empty_like(self.a)
        bep.bep_grouped_gemm_dx(self.down, buf.cu_seqlens, dy, self.w2, self.slots2, da)
        dh = buf.y                                     # the forward's h is not needed any more
        bep.bep_swiglu_bwd(self.up, da, self.ckpt.codes, self.ckpt.scales, dh, self.a)
        g2 = torch.empty(self.w2.shape, dtype=torch.float32, device=dev)
        red2 = torch.empty((R, E // R) + g2.shape[1:], dtype=torch.float32, device=dev)
        bep.bep_grouped_gemm_dw_overwrite(self.down, buf.cu_seqlens, self.a, dy, g2, red2)
        self.fold(self.down, g2, red2)
        g1 = torch.empty(self.w1.shape, dtype=torch.float32, device=dev)
        red1 = torch.empty((R, E // R) + g1.shape[1:], dtype=torch.float32, device=dev)
        bep.bep_dispatch(self.up, x, buf.dest, buf.recv)
        bep.bep_grouped_gemm_dw_overwrite(self.up, buf.cu_seqlens, buf.recv, dh, g1, red1)
        self.fold(self.up, g1, red1)
        bep.bep_grouped_gemm_dx(self.up, buf.cu_seqlens, dh, self.w1, self.slots1, buf.recv)
        dx = torch.empty_like(x)
        bep.bep_dispatch_bwd(self.up, buf.recv, buf.dest, dx)
        dlogits = torch.empty_like(self.logits)
        bep.bep_route_bwd(self.up, self.route, self.logits, self.topk, dgates, dlogits)
        dx = (dx.float() + dlogits @ self.w_router.t()).bfloat16()
        g_router = x.float().view(-1, self.H).t() @ dlogits.view(-1, E)
        return dx, g_router, g1, g2

    def fold(self, ctx, g, red):
        """Replica gradients into their home rows; slots without tokens hold nothing to add."""
        cu = self.buf.cu_seqlens
        used = cu[:, self.E + 1:] > cu[:, self.E:-1]
        red.masked_fill_(~used.view(*used.shape, 1, 1), 0.0)
        bep.bep_reduce_grad(ctx, self.buf.slot_expert, g, red)

    def quantise(self):
        """4-bit weights, once before serving."""
        self.q1, self.q2 = bep.MxWeight(self.up), bep.MxWeight(self.down)
        bep.bep_mx_quantize_weight(self.up, self.w1, self.q1.codes, self.q1.scales)
        bep.bep_mx_quantize_weight(self.down, self.w2, self.q2.codes, self.q2.scales)
        rows = self.R * self.S * self.K
        self.rows1, self.rows2 = bep.MxRows(rows, self.H), bep.MxRows(rows, self.F)

    def serve(self, x):
        buf = self.buf
        self.choose(x)
        bep.bep_dispatch_mx(self.up, x, buf.dest, self.rows1.codes, self.rows1.scales)
        bep.bep_grouped_gemm_mx(self.up, buf.cu_seqlens, buf.slot_expert, self.rows1.codes,
                                self.rows1.scales, self.q1.codes, self.q1.scales, buf.y)
        bep.bep_swiglu_mx(self.up, buf.y, self.rows2.codes, self.rows2.scales)
        bep.bep_grouped_gemm_mx(self.down, buf.cu_seqlens, buf.slot_expert, self.rows2.codes,
                                self.rows2.scales, self.q2.codes, self.q2.scales, self.y)
        bep.bep_combine(self.down, self.y, buf.dest, self.gates, self.out)
        return self.out

    def check(self):
        for ctx in (self.up, self.down):
            st = bep.bep_status(ctx)
            if st:
                raise RuntimeError(bep.strerror(st))


def main():
    p = argparse.ArgumentParser()
    for name, value in (("ranks", 4), ("tokens", 256), ("experts", 32), ("top-k", 4), ("hidden", 512),
                        ("ffn", 256), ("steps", 5)):
        p.add_argument("--" + name, type=int, default=value)
    a = p.parse_args()
    torch.manual_seed(0)
    layer = MoELayer(a.ranks, a.tokens, a.experts, a.top_k, a.hidden, a.ffn,
                     bep.RouteConfig(score=bep.BEP_SCORE_SIGMOID, renorm=True))
    x = torch.randn(a.ranks, a.tokens, a.hidden, device="cuda").bfloat16()
    target = torch.randn_like(x)
    for step in range(a.steps):
        out = layer.forward(x)
        diff = out.float() - target.float()
        _, g_router, g1, g2 = layer.backward(x, (diff * (2 / diff.numel())).bfloat16())
        scale = 0.1 * diff.numel()
        layer.w_router -= scale * 0.01 * g_router
        layer.w1.copy_((layer.w1.float() - scale * 0.01 * g1).bfloat16())
        layer.w2.copy_((layer.w2.float() - scale * 0.01 * g2).bfloat16())
        layer.balance()
        print(f"step {step}: loss {diff.square().mean().item():.4f}, "
              f"largest load {layer.load.max().item()} of mean {layer.load.float().mean().item():.0f}")
    full = layer.forward(x).float()
    layer.quantise()
    served = layer.serve(x).float()
    layer.check()
    print(f"served in 4 bits: {((served - full).norm() / full.norm()).item():.3f} relative to bf16")


if __name__ == "__main__":
    main()
