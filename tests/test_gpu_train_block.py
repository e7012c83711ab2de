"""The training calls together, as examples/train_block.py uses them: a whole
block's gradients against automatic differentiation in 64 bits, a run whose
loss falls, and the trained block through the MXFP4 layer."""
import os
import sys

import pytest
import torch

import mxfp4_mixture_experts_02_gb300 as moe
from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import train_block as ex  # noqa: E402

pytestmark = pytest.mark.gpu


def plain(block, params, x, residual, ids):
    """The block in 64 bits with the given picks."""
    norm_w, norm_b, router, gate, w1, w2 = params
    cfg = block.cfg
    h = x + residual
    d = h - h.mean(1, keepdim=True)
    n = d / torch.sqrt(d.square().mean(1, keepdim=True) + 1e-5) * norm_w + norm_b
    k = cfg.top_k
    picks = ids[:, :k].long()
    w = torch.softmax((n @ router.T).gather(1, picks), 1)
    w = torch.cat([w, torch.sigmoid(n @ gate.T) * cfg.shared_scale], 1)
    out = h
    for j in range(k + 1):
        e = picks[:, j] if j < k else torch.full_like(picks[:, 0], cfg.experts)
        gu = torch.einsum("th,tih->ti", n, w1[e])
        g, u = gu.chunk(2, dim=1)
        out = out + w[:, j:j + 1] * torch.einsum("ti,thi->th", g * torch.sigmoid(g) * u, w2[e])
    return out


def rel(a, b):
    return float((a.double() - b).norm() / b.norm())


def test_block_gradients_against_automatic_differentiation():
    cfg = ex.BlockConfig(T=96, hidden=512, inter=128, experts=8, top_k=2)
    block = ex.Block(cfg, 3)
    # matrices that bf16 holds exactly, so both sides differentiate the same function
    for p in block.params():
        p.copy_(p.bfloat16().float())
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x, r, dout = (torch.randn((cfg.T, 512), generator=g, device="cuda").bfloat16() for _ in range(3))
    out, s = block.forward(x, r)
    dx, grads = block.backward(s, dout)
    leaves = [p.double().requires_grad_() for p in block.params()]
    xd = x.double().requires_grad_()
    want = plain(block, leaves, xd, r.double(), s["ids"])
    want.backward(dout.double())
    # a dozen bf16 roundings (2^-9 each, root mean square below) along the longest path, sums averaging them
    tol = 12 ** 0.5 * 2 ** -8
    assert rel(out, want.detach()) <= tol
    assert rel(dx, xd.grad) <= tol
    for name, got, leaf in zip(block.NAMES, grads, leaves):
        assert rel(got, leaf.grad) <= tol, (name, rel(got, leaf.grad))


@pytest.mark.parametrize("mxfp8", [False, True])
def test_training_lowers_the_loss_and_the_layer_serves_the_result(mxfp8):
    losses, block, (x, r) = ex.train(ex.BlockConfig(T=256, inter=128, experts=8), 30, mxfp8)
    assert losses[-1] < 0.5 * losses[0], losses
    assert all(torch.isfinite(p).all() for p in block.params())
    y, _ = block.forward(x, r)
    q = ex.serve(block, x, r)
    torch.cuda.synchronize()
    assert moe.moe_get_status(block.layer_ws) == (0, 0)
    # E2M1 keeps one mantissa bit: about a tenth of the experts' part of the output
    assert rel(q, y.double()) <= 0.15
