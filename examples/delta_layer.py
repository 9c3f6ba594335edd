"""A block of the gated delta rule, trained and served.

y = x + o W_out: a layer norm (kda_layer_norm), one fused projection that gives queries, keys, values, the heads' decays and
step sizes, keys brought to norm 1 and queries to sqrt(128) (kda_qk_norm_rope without a rotation), and the gated delta rule with a state per
sequence (kda_gated_delta). Training goes over packed sequences with the kernels' own backward passes; serving prefills
prompts into a state pool and then takes one token a sequence at a time. The projections are plain matrix products of torch.

    python examples/delta_layer.py
"""

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_gated_gb300 import (kda_gated_delta_bwd, kda_gated_delta_decode, kda_gated_delta_fwd,  # noqa: E402
                                          kda_gated_delta_prefill, kda_layer_norm_bwd, kda_layer_norm_fwd,
                                          kda_qk_norm_rope_bwd, kda_qk_norm_rope_fwd)

D = 128
UNIT = D ** -0.5  # a norm's weight that leaves a head's vector with norm 1


class DeltaBlock:
    """Hqk query/key heads, Hv value heads, of a model of `width` values a token."""

    def __init__(self, width, hqk, hv, seed=0, device="cuda"):
        r = torch.Generator("cpu").manual_seed(seed)
        self.hqk, self.hv = hqk, hv
        self.split = [hqk * D, hqk * D, hv * D, hv, hv, -2 * hv % 8]  # (rows of the projection stay multiples of 16 bytes)
        w_in = torch.randn(width, sum(self.split), generator=r) * width ** -0.5
        w_out = torch.randn(hv * D, width, generator=r) * (hv * D) ** -0.5
        self.weights = {"in": w_in.to(device), "out": w_out.to(device),  # FP32 masters; products run in BF16
                        "norm": torch.ones(width, device=device), "bias": torch.zeros(width, device=device)}
        self.unit = torch.full((D,), UNIT, device=device)
        self.one = torch.ones(D, device=device)
        self.context = None

    def _inputs(self, x):
        """[B, T, width] -> what the norm gave, the projection's views, and the gated delta rule's inputs."""
        w = self.weights
        normed = kda_layer_norm_fwd(x, w["norm"], w["bias"])
        q, k, v, z, b, _ = (normed[0] @ w["in"].bfloat16()).split(self.split, -1)
        q, k = (t.unflatten(-1, (self.hqk, D)) for t in (q, k))  # views: the kernels take their strides
        v = v.unflatten(-1, (self.hv, D))
        g = -F.softplus(z.float() - 2.0).bfloat16()  # log decays <= 0, about 0.88 a token at the start
        beta = torch.sigmoid(b.float()).bfloat16()
        qn, kn = kda_qk_norm_rope_fwd(q, k, self.one, self.unit, None, None)
        return normed, (q, k, z, b), (qn, kn, v, g, beta)

    def step(self, x, target, cu, cu_cpu, rate=0.0):
        """One training step on packed sequences [1, T, width]: the loss, the weights' gradients, which `rate` times are taken
        off the weights, and the input's."""
        w = self.weights
        (xn, mean, rstd), (q, k, z, b), tokens = self._inputs(x)
        o, _, self.context = kda_gated_delta_fwd(*tokens, cu_seqlens=cu, cu_seqlens_cpu=cu_cpu, context_out=self.context)
        flat = o.flatten(2)
        diff = x.float() + (flat @ w["out"].bfloat16()).float() - target.float()
        loss = diff.square().mean()

        dy = (diff * (2.0 / diff.numel())).bfloat16()
        d_out = flat[0].T @ dy[0]
        do = (dy @ w["out"].bfloat16().T).unflatten(-1, (self.hv, D))
        dqn, dkn, dv, dg, dbeta, _ = kda_gated_delta_bwd(self.context, do)
        dq, dk, _, _ = kda_qk_norm_rope_bwd(dqn, dkn, q, k, self.one, self.unit, None, None)
        dz = -torch.sigmoid(z.float() - 2.0) * dg.float()
        s = torch.sigmoid(b.float())
        db = s * (1 - s) * dbeta.float()
        d_proj = F.pad(torch.cat([dq.flatten(2), dk.flatten(2), dv.flatten(2), dz.bfloat16(), db.bfloat16()], -1), (0, self.split[-1]))
        d_in = xn[0].T @ d_proj[0]
        dx, d_norm, d_bias = kda_layer_norm_bwd(d_proj @ w["in"].bfloat16().T, x, w["norm"], mean, rstd)
        grads = {"in": d_in.float(), "out": d_out.float(), "norm": d_norm, "bias": d_bias}
        if rate:
            for n, t in grads.items():
                w[n] -= rate * t
        return loss, grads, dx.float() + dy.float()

    def state_pool(self, slots, dtype=torch.float32):
        return torch.zeros(slots, self.hv, D, D, dtype=dtype, device=self.unit.device)

    def prefill(self, x, pool, slots, slots_cpu, cu, cu_cpu):
        """Prompts [1, T, width], packed: their outputs; each one's state is left in its slot of the pool."""
        _, _, tokens = self._inputs(x)
        o = kda_gated_delta_prefill(*tokens, pool, cu, slots, cu_seqlens_cpu=cu_cpu, state_indices_cpu=slots_cpu)
        return x + o.flatten(2) @ self.weights["out"].bfloat16()

    def decode(self, x, pool, slots, slots_cpu):
        """One token [N, 1, width] of each sequence."""
        _, _, tokens = self._inputs(x)
        o = kda_gated_delta_decode(*tokens, pool, slots, state_indices_cpu=slots_cpu)
        return x + o.flatten(2) @ self.weights["out"].bfloat16()


def packed(lens, device="cuda"):
    """Offsets (device, CPU) of packed sequences."""
    cu = torch.tensor([0, *lens], dtype=torch.int64).cumsum(0)
    return cu.to(device), cu


def train(block, teacher, lens, width, steps, rate, seed=1):
    """Losses of `steps` steps towards another block's outputs."""
    r = torch.Generator("cuda").manual_seed(seed)
    cu, cu_cpu = packed(lens)
    slots = torch.arange(len(lens), dtype=torch.int32)
    losses = []
    for _ in range(steps):
        x = torch.randn(1, sum(lens), width, generator=r, device="cuda").bfloat16()
        target = teacher.prefill(x, teacher.state_pool(len(lens)), slots.cuda(), slots, cu, cu_cpu)
        losses.append(block.step(x, target, cu, cu_cpu, rate)[0])
    return torch.stack(losses).tolist()


def serve(block, prompts, tokens, width, seed=2):
    """Prefills prompts of these lengths, decodes `tokens` more for each, and returns the outputs of these tokens and
    those of one prefill over the whole sequences."""
    r = torch.Generator("cuda").manual_seed(seed)
    N = len(prompts)
    xs = [torch.randn(1, n + tokens, width, generator=r, device="cuda").bfloat16() for n in prompts]
    slots_cpu = torch.arange(N, dtype=torch.int32).flip(0).contiguous()  # any order, and a slot that stays unused
    slots = slots_cpu.cuda()
    pool = block.state_pool(N + 1)
    block.prefill(torch.cat([x[:, :n] for x, n in zip(xs, prompts)], 1), pool, slots, slots_cpu, *packed(prompts))
    stepped = torch.cat([block.decode(torch.cat([x[:, n + t:n + t + 1] for x, n in zip(xs, prompts)]), pool, slots, slots_cpu)
                         for t in range(tokens)], 1)
    cu, cu_cpu = packed([n + tokens for n in prompts])
    whole = block.prefill(torch.cat(xs, 1), block.state_pool(N + 1), slots, slots_cpu, cu, cu_cpu)
    ends = cu_cpu[1:].tolist()
    return stepped, torch.cat([whole[:, e - tokens:e] for e in ends])


def main(width=512, hqk=2, hv=4, lens=(700, 1, 260, 63), steps=60, rate=30.0):
    block, teacher = (DeltaBlock(width, hqk, hv) for _ in range(2))
    for n, t in DeltaBlock(width, hqk, hv, seed=7).weights.items():  # starts next to what it is to learn
        if n in ("in", "out"):
            block.weights[n] += 0.3 * t
    losses = train(block, teacher, lens, width, steps, rate)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    stepped, whole = serve(block, (130, 1, 64, 7), 12, width)
    rel = ((stepped.float() - whole.float()).norm() / whole.float().norm()).item()
    print(f"token by token against one prefill: relative difference {rel:.1e}")
    return losses, rel


if __name__ == "__main__":
    main()
