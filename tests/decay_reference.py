"""Plain 64-bit forms of the linear attention with a decay for each head and of the norm and
position rotation of its queries and keys; gradients by autograd of the same few lines."""

import torch

BF16 = 2.0 ** -8   # half a step of each type, relative to the value
FP16 = 2.0 ** -11
FP32 = 2.0 ** -24


def scan(q, k, v, g, h0, spans, scale):
    """Token by token. q, k [Ttot, Hqk, 128], v [Ttot, Hv, 128], g [Ttot, Hv], h0 [N, Hv, 128, 128];
    spans: (first, end) of each sequence. Returns o [Ttot, Hv, 128], final states."""
    r = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    decay = g.exp()
    outs, states = [], []
    for n, (a, b) in enumerate(spans):
        S = h0[n]
        for t in range(a, b):
            S = decay[t][:, None, None] * S + v[t][:, :, None] * k[t][:, None, :]
            outs.append(scale * (S @ q[t][:, :, None])[:, :, 0])
        states.append(S)
    return (torch.stack(outs) if outs else v.new_zeros(v.shape)), torch.stack(states)


def norm_rope(x, w, pos, inv_freq, eps, interleaved):
    """x [B, T, H, D]."""
    n = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        n = n * w
    if inv_freq is None:
        return n
    R = 2 * inv_freq.numel()
    a = pos.to(torch.float64)[:, :, None, None] * inv_freq
    c, s = a.cos(), a.sin()
    if interleaved:
        x0, x1 = n[..., 0:R:2], n[..., 1:R:2]
        rot = torch.stack([x0 * c - x1 * s, x1 * c + x0 * s], -1).flatten(-2)
    else:
        x0, x1 = n[..., :R // 2], n[..., R // 2:R]
        rot = torch.cat([x0 * c - x1 * s, x1 * c + x0 * s], -1)
    return torch.cat([rot, n[..., R:]], -1)


def rel_l2(x, ref):
    x, ref = x.double().cpu(), ref.double().cpu()
    norm = ref.norm().item()
    return (x - ref).norm().item() / norm if norm else (x - ref).norm().item()


def check(name, x, ref, rel, step):
    """Relative L2 at most rel; no value further off than half a step of its own and six of the rms of
    its row's tensor (values that cancel carry the roundings of what they were summed from)."""
    x, ref = x.double().cpu(), ref.double().cpu()
    assert x.shape == ref.shape, (name, x.shape, ref.shape)
    assert torch.isfinite(x).all(), name
    if ref.numel() == 0:
        return
    assert rel_l2(x, ref) <= rel, (name, rel_l2(x, ref), rel)
    rms = ref.square().mean().sqrt()
    bad = (x - ref).abs() > step * ref.abs() + 6 * step * torch.maximum(rms, ref.abs())
    assert not bad.any(), (name, int(bad.sum()))
