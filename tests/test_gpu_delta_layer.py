"""The example block of layer norm, queries and keys of norm 1 and the gated delta rule: a training step's gradients against the
block in 64 bits, and serving against one pass.

Tolerances. On the way to a gradient lie 22 roundings to BF16 at most (the norm's output, weights, projection, q and k, g, beta,
o's three, y; dy, do, the rule's five, q's and k's norm, the gates, the projection's gradient, the product with its weights),
each off by half a step, 2^-8, at most, 2^-8 / sqrt(3) rms; each rounded quantity enters a gradient twice at most:
2 sqrt(22 / 3) 2^-8. A token's output, by a step of its own and in one pass: eight such roundings differ,
2 sqrt(8 / 3) 2^-8."""

import math
import os
import sys

import pytest
import torch

from decay_reference import BF16, rel_l2
from delta_reference import delta_scan, layer_norm

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_attention_gated_gb300 import build
    build.build()


def plain_step(block, x, target, spans):
    w = {n: t.double().requires_grad_() for n, t in block.weights.items()}
    x = x.double().requires_grad_()
    q, k, v, z, b, _ = (layer_norm(x, w["norm"], w["bias"], 1e-5)[0] @ w["in"]).split(block.split, -1)
    q, k = (t.unflatten(-1, (block.hqk, D)) for t in (q, k))
    q, k = (t / (t.square().mean(-1, keepdim=True) + 1e-6).sqrt() * f for t, f in ((q, 1.0), (k, D ** -0.5)))
    g, beta = -torch.nn.functional.softplus(z - 2.0), torch.sigmoid(b)
    h0 = torch.zeros(len(spans), block.hv, D, D, dtype=torch.float64, device=x.device)
    o, _ = delta_scan(q[0], k[0], v[0].unflatten(-1, (block.hv, D)), g[0], beta[0], h0, spans, D ** -0.5)
    loss = (x[0] + o.flatten(1) @ w["out"] - target[0].double()).square().mean()
    grads = torch.autograd.grad(loss, list(w.values()) + [x])
    return loss, dict(zip(w, grads)), grads[-1]


@pytest.mark.parametrize("lens,hqk,hv", [((130, 1, 67), 1, 2), ((40,), 2, 2), ((64, 65), 1, 3)])
def test_step_gradients(lens, hqk, hv):
    from delta_layer import DeltaBlock, packed
    block = DeltaBlock(256, hqk, hv, seed=3)
    r = torch.Generator("cuda").manual_seed(4)
    x, target = (torch.randn(1, sum(lens), 256, generator=r, device="cuda").bfloat16() for _ in range(2))
    cu, cu_cpu = packed(lens)
    loss, grads, dx = block.step(x, target, cu, cu_cpu)
    block.context.status()
    c = cu_cpu.tolist()
    want_loss, want, want_dx = plain_step(block, x, target, list(zip(c[:-1], c[1:])))
    bar = 2 * math.sqrt(22 / 3) * BF16
    assert abs(loss.item() - want_loss.item()) <= bar * want_loss.item()
    for n in want:
        assert rel_l2(grads[n], want[n]) <= bar, (n, rel_l2(grads[n], want[n]))
    assert rel_l2(dx, want_dx) <= bar


def test_example_trains_and_serves():
    from delta_layer import main
    losses, rel = main(width=256, lens=(300, 1, 64, 29), steps=6)
    assert len(losses) == 6 and all(math.isfinite(x) for x in losses)
    assert rel <= 2 * math.sqrt(8 / 3) * BF16, rel
