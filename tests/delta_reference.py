"""Plain 64-bit forms of the gated delta rule and of layer norm; gradients by autograd of the same few lines."""

import torch


def delta_scan(q, k, v, g, beta, h0, spans, scale):
    """Token by token. q, k [Ttot, Hqk, 128], v [Ttot, Hv, 128], g, beta [Ttot, Hv], h0 [N, Hv, 128, 128];
    spans: (first, end) of each sequence. Returns o [Ttot, Hv, 128], final states."""
    r = v.shape[1] // q.shape[1]
    q, k = q.repeat_interleave(r, 1), k.repeat_interleave(r, 1)
    decay = g.exp()
    outs, states = [], []
    for n, (a, b) in enumerate(spans):
        S = h0[n]
        for t in range(a, b):
            S = decay[t][:, None, None] * S
            u = v[t] - (S @ k[t][:, :, None])[:, :, 0]
            S = S + (beta[t][:, None] * u)[:, :, None] * k[t][:, None, :]
            outs.append(scale * (S @ q[t][:, :, None])[:, :, 0])
        states.append(S)
    return (torch.stack(outs) if outs else v.new_zeros(v.shape)), torch.stack(states)


def layer_norm(x, w, b, eps):
    """x [..., width]; y, mean, rstd."""
    mean = x.mean(-1, keepdim=True)
    rstd = 1 / ((x - mean).square().mean(-1, keepdim=True) + eps).sqrt()
    y = (x - mean) * rstd
    y = y if w is None else y * w
    return (y if b is None else y + b), mean[..., 0], rstd[..., 0]
