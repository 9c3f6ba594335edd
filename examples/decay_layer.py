"""A layer of linear attention with a decay for each head, trained and served.

One fused projection gives queries, keys, values and the heads' decays; queries and keys are
normalised per head and rotated by position (kda_qk_norm_rope), the attention carries a state per
sequence (kda_decay_attn), and an output projection closes the layer. Training goes over packed
sequences with the kernels' own backward passes; serving prefills prompts into a state pool and then
takes one token a sequence at a time. The projections are plain matrix products of torch.

    python examples/decay_layer.py
"""

import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from linear_attention_gated_gb300 import (kda_decay_attn_bwd, kda_decay_attn_decode, kda_decay_attn_fwd,  # noqa: E402
                                          kda_decay_attn_prefill, kda_qk_norm_rope_bwd, kda_qk_norm_rope_fwd)

D = 128


class DecayLayer:
    """y = o W_out, o the attention's output for q, k, v, g from x W_in; Hqk query/key heads, Hv value heads."""

    def __init__(self, width, hqk, hv, rotated=64, theta=10000.0, seed=0, device="cuda"):
        r = torch.Generator("cpu").manual_seed(seed)
        self.hqk, self.hv = hqk, hv
        self.split = [hqk * D, hqk * D, hv * D, hv, -hv % 8]  # (rows of the projection stay multiples of 16 bytes)
        w_in = torch.randn(width, sum(self.split), generator=r) * width ** -0.5
        w_out = torch.randn(hv * D, width, generator=r) * (hv * D) ** -0.5
        self.weights = {"in": w_in.to(device), "out": w_out.to(device),  # FP32 masters; products run in BF16
                        "q": torch.ones(D, device=device), "k": torch.ones(D, device=device)}
        self.inv_freq = theta ** (-torch.arange(0, rotated, 2, dtype=torch.float64, device=device) / rotated)
        self.context = None

    def _inputs(self, x, positions):
        """[B, T, width] -> the projection's views, normalised and rotated q and k, and the log decays."""
        B, T, _ = x.shape
        q, k, v, z, _ = (x @ self.weights["in"].bfloat16()).split(self.split, -1)
        q, k = (t.unflatten(-1, (self.hqk, D)) for t in (q, k))  # views: the kernels take their strides
        v = v.unflatten(-1, (self.hv, D))
        g = -F.softplus(z.float() - 2.0).bfloat16()  # log decays <= 0, about 0.88 a token at the start
        qr, kr = kda_qk_norm_rope_fwd(q, k, self.weights["q"], self.weights["k"], positions, self.inv_freq)
        return q, k, v, z, g, qr, kr

    def step(self, x, target, positions, cu, cu_cpu, rate=0.0):
        """One training step on packed sequences [1, T, width]: the loss and the weights' gradients, which
        `rate` times are taken off the weights."""
        w = self.weights
        q, k, v, z, g, qr, kr = self._inputs(x, positions)
        o, _, self.context = kda_decay_attn_fwd(qr, kr, v, g, cu_seqlens=cu, cu_seqlens_cpu=cu_cpu, context_out=self.context)
        flat = o.flatten(2)
        y = flat @ w["out"].bfloat16()
        diff = y.float() - target.float()
        loss = diff.square().mean()

        dy = (diff * (2.0 / diff.numel())).bfloat16()
        d_out = flat[0].T @ dy[0]
        do = (dy @ w["out"].bfloat16().T).unflatten(-1, (self.hv, D))
        dqr, dkr, dv, dg, _ = kda_decay_attn_bwd(self.context, do)
        dq, dk, d_q, d_k = kda_qk_norm_rope_bwd(dqr, dkr, q, k, w["q"], w["k"], positions, self.inv_freq)
        dz = (-torch.sigmoid(z.float() - 2.0) * dg.float()).bfloat16()
        d_proj = F.pad(torch.cat([dq.flatten(2), dk.flatten(2), dv.flatten(2), dz], -1), (0, self.split[-1]))
        d_in = x[0].T @ d_proj[0]
        grads = {"in": d_in.float(), "out": d_out.float(), "q": d_q, "k": d_k}
        if rate:
            for n, t in grads.items():
                w[n] -= rate * t
        return loss, grads

    def state_pool(self, slots, dtype=torch.float32):
        return torch.zeros(slots, self.hv, D, D, dtype=dtype, device=self.inv_freq.device)

    def prefill(self, x, positions, pool, slots, slots_cpu, cu, cu_cpu):
        """Prompts [1, T, width], packed: their outputs; each one's state is left in its slot of the pool."""
        _, _, v, _, g, qr, kr = self._inputs(x, positions)
        o = kda_decay_attn_prefill(qr, kr, v, g, pool, cu, slots, cu_seqlens_cpu=cu_cpu, state_indices_cpu=slots_cpu)
        return o.flatten(2) @ self.weights["out"].bfloat16()

    def decode(self, x, positions, pool, slots, slots_cpu):
        """One token [N, 1, width] of each sequence."""
        _, _, v, _, g, qr, kr = self._inputs(x, positions)
        o = kda_decay_attn_decode(qr, kr, v, g, pool, slots, state_indices_cpu=slots_cpu)
        return o.flatten(2) @ self.weights["out"].bfloat16()


def packed(lens, device="cuda"):
    """Offsets (device, CPU) and positions of packed sequences."""
    cu = torch.tensor([0, *lens], dtype=torch.int64).cumsum(0)
    positions = torch.cat([torch.arange(n) for n in lens])[None]
    return cu.to(device), cu, positions.to(device)


def train(layer, teacher, lens, width, steps, rate, seed=1):
    """Losses of `steps` steps towards another layer's outputs."""
    r = torch.Generator("cuda").manual_seed(seed)
    cu, cu_cpu, positions = packed(lens)
    losses = []
    for _ in range(steps):
        x = torch.randn(1, sum(lens), width, generator=r, device="cuda").bfloat16()
        slots = torch.arange(len(lens), dtype=torch.int32)
        target = teacher.prefill(x, positions, teacher.state_pool(len(lens)), slots.cuda(), slots, cu, cu_cpu)
        losses.append(layer.step(x, target, positions, cu, cu_cpu, rate)[0])
    return torch.stack(losses).tolist()


def serve(layer, prompts, tokens, width, seed=2):
    """Prefills prompts of these lengths, decodes `tokens` more for each, and returns the outputs of these tokens and
    those of one prefill over the whole sequences."""
    r = torch.Generator("cuda").manual_seed(seed)
    N = len(prompts)
    xs = [torch.randn(1, n + tokens, width, generator=r, device="cuda").bfloat16() for n in prompts]
    slots_cpu = torch.arange(N, dtype=torch.int32).flip(0).contiguous()  # any order, and a slot that stays unused
    slots = slots_cpu.cuda()
    pool = layer.state_pool(N + 1)
    cu, cu_cpu, positions = packed(prompts)
    layer.prefill(torch.cat([x[:, :n] for x, n in zip(xs, prompts)], 1), positions, pool, slots, slots_cpu, cu, cu_cpu)
    at = torch.tensor(prompts, device="cuda")[:, None]
    stepped = torch.cat([layer.decode(torch.cat([x[:, n + t:n + t + 1] for x, n in zip(xs, prompts)]), at + t, pool, slots,
                                      slots_cpu) for t in range(tokens)], 1)
    cu, cu_cpu, positions = packed([n + tokens for n in prompts])
    whole = layer.prefill(torch.cat(xs, 1), positions, layer.state_pool(N + 1), slots, slots_cpu, cu, cu_cpu)
    ends = cu_cpu[1:].tolist()
    return stepped, torch.cat([whole[:, e - tokens:e] for e in ends])


def main(width=512, hqk=2, hv=4, lens=(700, 1, 260, 63), steps=60, rate=2.0):
    layer, teacher = (DecayLayer(width, hqk, hv) for _ in range(2))
    for n, t in DecayLayer(width, hqk, hv, seed=7).weights.items():  # starts next to what it is to learn
        layer.weights[n] += 0.3 * t
    losses = train(layer, teacher, lens, width, steps, rate)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} in {steps} steps")
    stepped, whole = serve(layer, (130, 1, 64, 7), 12, width)
    rel = ((stepped.float() - whole.float()).norm() / whole.float().norm()).item()
    print(f"token by token against one prefill: relative difference {rel:.1e}")
    return losses, rel


if __name__ == "__main__":
    main()
