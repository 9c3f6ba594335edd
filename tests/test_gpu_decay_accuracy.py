"""FP32 states of the linear attention with a decay for each head, on the GPU, to their last bits.

Tolerances. What enters a state is a product of one factor in two BF16 parts, hi + lo, and one in BF16. With half a step
2^-8 relative to a value in [1, 2), lo is uniform in +-2^-8 and its own half step is 2^-17 with chance 1/2, 2^-18 with
1/4 and so on: an rms of 2^-17 sqrt((1/2) / (1 - 1/8) / 3) = 0.436 2^-17 of the value at most. A chunk's products are
added in eight steps of the tensor core, each off by one FP32 step, 2^-23, at most.
"""

import math

import pytest
import torch

from decay_reference import FP32, rel_l2
from test_gpu_decay import D, library, make, reference, run  # noqa: F401

pytestmark = pytest.mark.gpu

STATE_REL = 0.436 * 2.0 ** -17 + 8 * 2 * FP32


@pytest.mark.parametrize("lens,hqk,hv,gate,slow", [
    ((200, 64, 1000), 1, 2, "token", 1.0), ((200, 64, 1000), 1, 2, "token", 0.02), ((333, 1), 2, 2, "head", 1.0),
    ((5000, 70), 1, 1, "token", 0.02),  # the first is cut into segments
], ids=str)
def test_states(lens, hqk, hv, gate, slow):
    x = make(lens, hqk, hv, gate, seed=31)
    x["g"] = (x["g"].float() * slow).to(x["g"].dtype)
    got, _ = run(x)
    ref = reference(x, device="cuda")
    for n in ("hT", "dh0"):
        assert rel_l2(got[n], ref[n]) <= STATE_REL, (n, rel_l2(got[n], ref[n]))


@pytest.mark.parametrize("gate", ["head", "token"])
@pytest.mark.parametrize("lens", [(98304,), (98304,) + (0,) * 520], ids=["cut", "whole"])
def test_slow_decays_over_a_long_sequence(lens, gate):
    """A state that nothing is added to, over 1536 chunks: h0 exp(T g). Each chunk rounds the state once, independently,
    2^-24 / sqrt(3) rms; a decay's logarithm is rounded ten times at most (products with log2 e and ln 2, a sum of 64); eight
    roundings for the factors themselves. (More than 512 sequences are not cut into segments.)"""
    from linear_attention_gated_gb300 import kda_decay_attn_bwd, kda_decay_attn_fwd
    T = lens[0]
    gen = torch.Generator("cuda").manual_seed(1)
    g = -torch.tensor([3e-6, 1e-5, 1.7e-5, 4e-5, 1e-4], device="cuda")
    if gate == "token":
        g = g.bfloat16()
    hv, N = g.numel(), len(lens)
    z = torch.zeros(1, T, hv, D, dtype=torch.bfloat16, device="cuda")
    h0, dhT = (torch.randn(N, hv, D, D, generator=gen, device="cuda") for _ in range(2))
    cu = torch.tensor([0, *lens]).cumsum(0)
    decays = g if gate == "head" else g.expand(1, T, hv).contiguous()
    _, hT, ctx = kda_decay_attn_fwd(z, z, z, decays, h0, cu.cuda(), cu_seqlens_cpu=cu)
    dh0 = kda_decay_attn_bwd(ctx, z, dhT)[4]
    ctx.status()
    for h in range(hv):
        total = T * g[h].double()
        bar = (math.sqrt(T / 64 / 3) + 8 + 10 * abs(total.item())) * FP32
        for n, got, start in (("hT", hT, h0), ("dh0", dh0, dhT)):
            off = rel_l2(got[0, h], start[0, h].double() * total.exp())
            assert off <= bar, (n, g[h].item(), off, bar)
    assert torch.equal(hT[1:], h0[1:]) and torch.equal(dh0[1:], dhT[1:])
