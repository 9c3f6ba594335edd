"""The example layer of norm, rotation and attention with a decay for each head: a training step's
gradients against the layer in 64 bits, and serving against one pass.

Tolerances. About 16 roundings to BF16 lie on the way to a weight's gradient (weights, projection, q, k, g,
o's three, y, and as many backwards), each off by half a step, 2^-8, at most, 2^-8 / sqrt(3) rms; each
rounded quantity enters a gradient twice at most: 2 sqrt(16 / 3) 2^-8. A token's output, by a step of its own
and in one pass: eight such roundings differ, 2 sqrt(8 / 3) 2^-8."""

import math
import os
import sys

import pytest
import torch

from decay_reference import BF16, norm_rope, rel_l2, scan

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
D = 128


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_attention_gated_gb300 import build
    build.build()


def plain_step(layer, x, target, positions, spans):
    w = {n: t.double().requires_grad_() for n, t in layer.weights.items()}
    q, k, v, z, _ = (x.double() @ w["in"]).split(layer.split, -1)
    q, k = (norm_rope(t.unflatten(-1, (layer.hqk, D)), w[n], positions, layer.inv_freq, 1e-6, False)
            for n, t in (("q", q), ("k", k)))
    g = -torch.nn.functional.softplus(z - 2.0)
    h0 = torch.zeros(len(spans), layer.hv, D, D, dtype=torch.float64, device=x.device)
    o, _ = scan(q[0], k[0], v[0].unflatten(-1, (layer.hv, D)), g[0], h0, spans, D ** -0.5)
    loss = (o.flatten(1) @ w["out"] - target[0].double()).square().mean()
    return loss, dict(zip(w, torch.autograd.grad(loss, list(w.values()))))


@pytest.mark.parametrize("lens,hqk,hv", [((130, 1, 67), 1, 2), ((40,), 2, 2)])
def test_step_gradients(lens, hqk, hv):
    from decay_layer import DecayLayer, packed
    layer = DecayLayer(256, hqk, hv, seed=3)
    r = torch.Generator("cuda").manual_seed(4)
    x, target = (torch.randn(1, sum(lens), 256, generator=r, device="cuda").bfloat16() for _ in range(2))
    cu, cu_cpu, positions = packed(lens)
    loss, grads = layer.step(x, target, positions, cu, cu_cpu)
    layer.context.status()
    c = cu_cpu.tolist()
    want_loss, want = plain_step(layer, x, target, positions, list(zip(c[:-1], c[1:])))
    bar = 2 * math.sqrt(16 / 3) * BF16
    assert abs(loss.item() - want_loss.item()) <= bar * want_loss.item()
    for n in want:
        assert rel_l2(grads[n], want[n]) <= bar, (n, rel_l2(grads[n], want[n]))


def test_example_trains_and_serves():
    from decay_layer import main
    losses, rel = main(width=256, lens=(300, 1, 64, 29), steps=30)
    assert all(math.isfinite(x) for x in losses)
    assert losses[-1] < 0.5 * losses[0]
    assert rel <= 2 * math.sqrt(8 / 3) * BF16, rel
