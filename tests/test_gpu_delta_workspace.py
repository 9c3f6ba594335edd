"""What the workspace of a training step of the gated delta rule holds, on the GPU: before the forward, and where it is not the
forward's any more."""

import pytest
import torch

from test_gpu_delta import D, GRADS, library, make, run  # noqa: F401
from test_gpu_delta_forms import NAMES, TOKENS, same

pytestmark = pytest.mark.gpu
PACKET = (26 << 10) + (8 << 10)  # bytes of a (chunk, head) in front of the list of chunks


@pytest.mark.parametrize("entry", [lambda i, T: (T - 1, 64), lambda i, T: (T, 3), lambda i, T: (T + 40, 64), lambda i, T: (-1, 64),
                                   lambda i, T: (-40, 20), lambda i, T: (i, 1 << 30), lambda i, T: (7, -5),
                                   lambda i, T: (-(1 << 31), (1 << 31) - 1), lambda i, T: ((1 << 31) - 1, 64),
                                   lambda i, T: ((-1, 64) if i % 2 else (0, 64))])
@pytest.mark.parametrize("hqk,hv", [(1, 1), (16, 32)])
def test_a_list_of_chunks_that_is_not_the_forwards(entry, hqk, hv):
    """Chunks that begin outside of the tensors, end there or have too many tokens: nothing around the gradients changes, and the
    next step is right. (With 32 heads a CTA has several units, whose chunks are asked for ahead.)"""
    from linear_attention_gated_gb300 import kda_gated_delta_bwd, kda_gated_delta_fwd
    x = make((300, 0, 70, 400), hqk, hv, seed=50)
    T, slots = 770, 770 // 64 + 4
    want, _ = run(x)
    d = {n: t.cuda() for n, t in x.items()}
    room = {n: torch.full((want[n].numel() + 2 * 64 * hv * D,), 3.0, dtype=want[n].dtype, device="cuda") for n in GRADS}
    mine = {n: room[n][64 * hv * D:-64 * hv * D].view(want[n].shape) for n in GRADS}

    def step(change):
        o, hT, ctx = kda_gated_delta_fwd(*(d[n] for n in TOKENS), d["h0"], d["cu"], cu_seqlens_cpu=x["cu"])
        if change:
            at = slots * hv * PACKET
            ctx.workspace[at:at + 8 * slots].copy_(torch.tensor([entry(i, T) for i in range(slots)], dtype=torch.int32).view(torch.uint8).flatten())
        kda_gated_delta_bwd(ctx, d["do"], d["dhT"], out=tuple(mine[n] for n in GRADS))
        ctx.status()
        return dict(o=o, hT=hT, **mine)

    step(True)
    for n in GRADS:
        assert (room[n][:64 * hv * D] == 3).all() and (room[n][-64 * hv * D:] == 3).all(), n
    for n in d:
        assert torch.equal(d[n].cpu(), x[n]), n
    same(want, step(False))


@pytest.mark.parametrize("lens,hqk,hv,gate", [((90, 0, 40, 1), 2, 4, True), ((3100, 0, 20), 1, 1, True), ((3100, 70), 1, 2, False),
                                              ((0, 0), 1, 2, True)], ids=str)
@pytest.mark.parametrize("fill", [0xff, 0x7f, 1])
def test_what_a_contexts_workspace_held_does_not_matter(lens, hqk, hv, gate, fill):
    """A step on a used context whose workspace was overwritten before its forward: NaN in all types, the largest numbers, ones.
    Places of no chunk, segments' maps that are known to be zero and the last segments' stay unwritten."""
    x = make(lens, hqk, hv, seed=51, gate=gate)
    if gate and len(lens) == 3:  # resets: the first head's maps are zero
        x["g"][:, 700::500] = -float("inf")
    want, ctx = run(x)
    ctx.workspace.fill_(fill)
    same(want, run(x, ctx=ctx)[0])


def test_contexts_of_growing_and_shrinking_lengths():
    """Steps whose backward follows a refused forward, and steps of other lengths on one context."""
    from linear_attention_gated_gb300 import KdaError, kda_gated_delta_bwd, kda_gated_delta_fwd
    even, long = make([512] * 16, 1, 1, seed=52), make([7680] + [34] * 14 + [36], 1, 1, seed=53)
    first, ctx = run(even)
    d = {n: t.cuda() for n, t in even.items()}
    e = {n: t.cuda() for n, t in long.items()}
    before = ctx.workspace
    for error, wrong in ((ValueError, dict(out=e["v"][:, :5])), (KdaError, dict(out=e["v"]))):  # (of another shape, and over an input)
        kda_gated_delta_fwd(*(d[n] for n in TOKENS), d["h0"], d["cu"], context_out=ctx, cu_seqlens_cpu=even["cu"])
        with pytest.raises(error):
            kda_gated_delta_fwd(*(e[n] for n in TOKENS), e["h0"], e["cu"], context_out=ctx, cu_seqlens_cpu=long["cu"], **wrong)
        assert ctx.workspace is before
        got = kda_gated_delta_bwd(ctx, d["do"], d["dhT"])
        same({n: first[n] for n in GRADS}, dict(zip(GRADS, got)))
    alone, _ = run(long)
    same(alone, run(long, ctx=ctx)[0])
    assert ctx.workspace is not before
    same(first, run(even, ctx=ctx)[0])
