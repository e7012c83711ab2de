"""Trains one pre-norm mixture block with the library's training calls, then
quantises it and runs the MXFP4 layer on the same tokens.

    h = x + residual,  n = layer_norm(h),  out = h + sum_j w_j expert_j(n)

Forward and backward go through moe_layer_norm, moe_router, moe_route,
moe_token_map, moe_permute, moe_unpermute and their gradients; the products of
an expert are torch matrix products over its rows (expert_offsets); moe_adamw
updates the fp32 parameters.  The target is another block of the same shape.

    python examples/train_block.py [--steps 40] [--mxfp8] [--tokens 512]
"""
import argparse
import dataclasses
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_mixture_experts_02_gb300 as moe  # noqa: E402


@dataclasses.dataclass
class BlockConfig:
    T: int = 512
    hidden: int = 512
    inter: int = 256
    experts: int = 16
    top_k: int = 4
    shared_scale: float = 0.5


class Block:
    """Parameters (fp32) and one forward and backward pass in bf16."""

    NAMES = ("norm_w", "norm_b", "router", "gate", "w1", "w2")

    def __init__(self, cfg: BlockConfig, seed: int):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        rnd = lambda s, *shape: torch.randn(shape, generator=g, device="cuda") * s  # noqa: E731
        H, I, E = cfg.hidden, cfg.inter, cfg.experts
        self.cfg = cfg
        self.norm_w, self.norm_b = torch.ones(H, device="cuda"), torch.zeros(H, device="cuda")
        self.router = rnd(H ** -0.5, E, H)
        self.gate = rnd(H ** -0.5, 1, H)                    # of the shared expert
        self.w1 = rnd(H ** -0.5, E + 1, 2 * I, H)           # gate rows, then up rows; the shared expert last
        self.w2 = rnd(I ** -0.5, E + 1, H, I)
        self.shape = moe.MoeTokenShape(cfg.T, E, E, 0, cfg.top_k, 1, H)
        self.layer = moe.MoeShape(cfg.T, cfg.T, E, E, 0, cfg.top_k, 1, H, I, 16, shared_scale=cfg.shared_scale)
        self.layer_ws = moe.workspace(self.layer)
        self.map_ws = moe.token_map_workspace(self.shape)
        self.norm_ws = moe.layer_norm_workspace(cfg.T, H)

    def params(self):
        return [getattr(self, n) for n in self.NAMES]

    def forward(self, x, residual):
        s = {}
        s["n"], s["h"], s["mean"], s["rstd"] = moe.moe_layer_norm(x, self.norm_w, self.norm_b, residual)
        s["router"], s["gate"] = self.router.bfloat16(), self.gate.bfloat16()
        logits = moe.moe_router(self.layer, s["n"], s["router"], self.layer_ws)
        s["z"] = s["n"] @ s["gate"].T
        s["ids"], s["w"] = moe.moe_route(self.layer, logits, s["z"])
        s["maps"] = moe.moe_token_map(self.shape, s["ids"], ws=self.map_ws)
        s["rows"] = moe.moe_permute(self.shape, s["n"], s["maps"])
        s["offsets"] = s["maps"].expert_offsets.tolist()
        s["w1"], s["w2"] = self.w1.bfloat16(), self.w2.bfloat16()
        s["gu"] = torch.empty((s["rows"].shape[0], 2 * self.cfg.inter), device=x.device, dtype=x.dtype)
        s["y"] = torch.empty_like(s["rows"])
        for e, (a, b) in enumerate(zip(s["offsets"], s["offsets"][1:])):
            torch.matmul(s["rows"][a:b], s["w1"][e].T, out=s["gu"][a:b])
            gate, up = s["gu"][a:b].chunk(2, dim=1)
            torch.matmul(torch.nn.functional.silu(gate) * up, s["w2"][e].T, out=s["y"][a:b])
        return s["h"] + moe.moe_unpermute(self.shape, s["y"], s["w"], s["maps"]), s

    def backward(self, s, dout):
        """(gradient of x and residual, gradients of params())."""
        dy, dw = moe.moe_unpermute_backward(self.shape, dout, s["y"], s["w"], s["maps"])
        dw1, dw2 = torch.zeros_like(self.w1), torch.zeros_like(self.w2)
        drows = torch.empty_like(s["rows"])
        for e, (a, b) in enumerate(zip(s["offsets"], s["offsets"][1:])):
            gate, up = s["gu"][a:b].float().chunk(2, dim=1)
            sig = torch.sigmoid(gate)
            act = gate * sig
            dact = (dy[a:b] @ s["w2"][e]).float()
            dw2[e] = dy[a:b].T @ (act * up).to(dy.dtype)
            dgu = torch.cat([dact * up * (sig + act * (1 - sig)), dact * act], 1).to(dy.dtype)
            dw1[e] = dgu.T @ s["rows"][a:b]
            drows[a:b] = dgu @ s["w1"][e]
        dlogits, dz = moe.moe_route_backward(self.shape, s["ids"], s["w"], dw, s["z"], self.cfg.shared_scale)
        dn = moe.moe_permute_backward(self.shape, drows, s["maps"]).float()
        dn += dlogits @ s["router"].float() + dz @ s["gate"].float()
        n = s["n"].float()
        dx, dnw, dnb = moe.moe_layer_norm_backward(dn.to(s["n"].dtype), s["h"], s["mean"], s["rstd"], self.norm_w,
                                                   dh=dout, ws=self.norm_ws)
        return dx, [dnw, dnb, dlogits.T @ n, dz.T @ n, dw1, dw2]


def train(cfg: BlockConfig, steps: int, mxfp8: bool, seed: int = 0):
    """The losses of `steps` steps, the trained block and the last batch."""
    teacher, block = Block(cfg, seed + 1), Block(cfg, seed + 2)
    grads = [torch.zeros_like(p) for p in block.params()]
    tensors = moe.adamw_tensors(block.params(), grads, mxfp8=mxfp8)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 3)
    losses = []
    x, r = (torch.randn((cfg.T, cfg.hidden), generator=g, device="cuda").bfloat16() for _ in range(2))
    want = teacher.forward(x, r)[0].float()
    for step in range(1, steps + 1):
        out, saved = block.forward(x, r)
        err = out.float() - want
        losses.append(err.square().mean())
        _, new = block.backward(saved, (err * (2.0 / err.numel() * 1024)).bfloat16())  # scaled past bf16's small end
        for have, got in zip(grads, new):
            have.copy_(got)
        norm = torch.stack([v.norm() for v in grads]).norm()
        # the scale is taken out again, the norm kept at 1 or below, on the device
        scale = (1.0 / 1024) * torch.clamp(1024.0 / norm, max=1.0)
        moe.moe_adamw(tensors, step, lr=2e-3, weight_decay=0.01, grad_scale=scale.view(1), seed=step)
    return torch.stack(losses).tolist(), block, (x, r)


def serve(block: Block, x, residual):
    """The trained block's output with its experts in MXFP4, by the fused layer."""
    weights = moe.quantize_expert_weights(block.w1, block.w2)
    n, h, _, _ = moe.moe_layer_norm(x, block.norm_w, block.norm_b, residual)
    out = moe.moe_layer_router(block.layer, block.router.bfloat16(), n @ block.gate.bfloat16().T, n, weights,
                               block.layer_ws)[0]
    return h + out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--mxfp8", action="store_true", help="optimizer states in MXFP8 instead of fp32")
    a = ap.parse_args()
    losses, block, (x, r) = train(BlockConfig(T=a.tokens), a.steps, a.mxfp8)
    for i in range(0, len(losses), max(1, len(losses) // 8)):
        print("step %4d  loss %.5f" % (i + 1, losses[i]))
    print("step %4d  loss %.5f" % (len(losses), losses[-1]))
    y, _ = block.forward(x, r)
    q = serve(block, x, r)
    print("MXFP4 layer against the trained block: relative difference %.3f" %
          float((q.float() - y.float()).norm() / y.float().norm()))


if __name__ == "__main__":
    main()
