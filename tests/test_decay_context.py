"""What the Python context of kda_decay_attn_fwd / _bwd keeps and passes on: no GPU needed. The library's kernels are not
called: the tensors are on the CPU, and the calls are caught where they would enter the library."""

import ctypes

import pytest
import torch

D = 128


@pytest.fixture(scope="module", autouse=True)
def library():
    from linear_attention_gated_gb300 import build
    build.build()


class Call:
    """One caught call: its arguments, and what the offsets and the workspace were when it was made."""

    def __init__(self, f, args):
        self.name, self.args = f.__name__, args
        cu, n = args[7], args[8]
        self.cu = None if cu is None else list((ctypes.c_int64 * (n + 1)).from_address(cu))
        at = {"kda_decay_attn_fwd": 18, "kda_decay_attn_bwd": 24}[self.name]
        self.workspace, self.workspace_bytes = args[at], args[at + 1]


@pytest.fixture
def calls(monkeypatch):
    from linear_attention_gated_gb300 import decay
    made = []
    monkeypatch.setattr(decay, "_call", lambda f, device, *args: made.append(Call(f, args)))
    return made


def inputs(T, hv=1):
    x = [torch.zeros(1, T, hv, D, dtype=torch.bfloat16) for _ in range(3)]
    return x + [torch.zeros(1, T, hv, dtype=torch.bfloat16)]


def offsets(lens):
    return torch.tensor([0, *lens]).cumsum(0)


EVEN, LONG = [512] * 16, [7680] + [34] * 14 + [36]  # the second is cut into segments, the first is not


def need(lens, hv=1):
    from linear_attention_gated_gb300 import decay_workspace_bytes
    return decay_workspace_bytes(1, sum(lens), hv, hv, offsets(lens))


def test_lengths_differ_in_what_they_need():
    assert need(LONG) > need(EVEN)


def test_backward_goes_by_the_lengths_of_its_forward(calls):
    """A mirror that is filled again for the next batch before the backward."""
    from linear_attention_gated_gb300 import kda_decay_attn_bwd, kda_decay_attn_fwd
    x, mirror = inputs(8192), offsets(LONG)
    *_, ctx = kda_decay_attn_fwd(*x, cu_seqlens=mirror.clone(), cu_seqlens_cpu=mirror)
    mirror.copy_(offsets(EVEN))
    kda_decay_attn_bwd(ctx, x[2])
    assert [c.cu for c in calls] == [offsets(LONG).tolist()] * 2


def test_a_mirror_filled_again_gets_the_workspace_it_needs(calls):
    from linear_attention_gated_gb300 import kda_decay_attn_fwd
    x, mirror = inputs(8192), offsets(EVEN)
    cu = mirror.clone()
    *_, ctx = kda_decay_attn_fwd(*x, cu_seqlens=cu, cu_seqlens_cpu=mirror)
    mirror.copy_(offsets(LONG))
    cu.copy_(mirror)
    kda_decay_attn_fwd(*x, cu_seqlens=cu, cu_seqlens_cpu=mirror, context_out=ctx)
    assert [c.cu for c in calls] == [offsets(EVEN).tolist(), offsets(LONG).tolist()]
    assert calls[0].workspace_bytes == need(EVEN) and calls[1].workspace_bytes >= need(LONG)


def test_reuse_between_fixed_and_packed(calls):
    from linear_attention_gated_gb300 import kda_decay_attn_fwd
    x, cu = inputs(64), offsets([64])
    *_, ctx = kda_decay_attn_fwd(*x)
    kda_decay_attn_fwd(*x, cu_seqlens=cu, cu_seqlens_cpu=cu, context_out=ctx)
    kda_decay_attn_fwd(*x, context_out=ctx)
    assert [c.cu for c in calls] == [None, [0, 64], None]


def test_a_workspace_that_was_too_small_lives_as_long_as_the_context(calls):
    """A captured graph, or work in flight, may still write to it."""
    import weakref

    from linear_attention_gated_gb300 import kda_decay_attn_fwd
    x = inputs(8192)
    *_, ctx = kda_decay_attn_fwd(*x, cu_seqlens=offsets(EVEN), cu_seqlens_cpu=offsets(EVEN))
    first = weakref.ref(ctx.workspace)
    kda_decay_attn_fwd(*x, cu_seqlens=offsets(LONG), cu_seqlens_cpu=offsets(LONG), context_out=ctx)
    assert ctx.workspace.numel() >= need(LONG)
    assert first() is not None and first().data_ptr() == calls[0].workspace
    second = ctx.workspace.data_ptr()
    kda_decay_attn_fwd(*x, cu_seqlens=offsets(EVEN), cu_seqlens_cpu=offsets(EVEN), context_out=ctx)
    assert calls[2].workspace == second  # the largest serves all
    del ctx
    assert first() is None


def test_reuse_on_another_stream_is_refused(calls, monkeypatch):
    """Two steps at once would share one workspace."""
    from linear_attention_gated_gb300 import KdaError, decay, kda_decay_attn_fwd
    x = inputs(64)
    on = [5]
    monkeypatch.setattr(decay, "_stream", lambda device: on[0], raising=False)
    *_, ctx = kda_decay_attn_fwd(*x)
    on[0] = 6
    with pytest.raises(KdaError, match="stream"):
        kda_decay_attn_fwd(*x, context_out=ctx)
    on[0] = 5
    kda_decay_attn_fwd(*x, context_out=ctx)
    assert len(calls) == 2
