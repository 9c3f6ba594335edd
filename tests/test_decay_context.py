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


def test_writes_into_the_callers_tensors_count_as_changes(monkeypatch):
    """Tensors that a call writes get a new version, those that it reads keep theirs."""
    import linear_attention_gated_gb300 as lib
    from linear_attention_gated_gb300 import decay
    monkeypatch.setattr(decay, "_call", lambda *args: None)
    x = inputs(1, hv=2)
    q, k, v, g = x
    f32 = {n: torch.zeros(1, 2, D, D) for n in ("h0", "hT", "pool", "dh0", "dhT")}
    o, dq, dk, dv, dg, do, q2, k2 = (torch.zeros_like(t) for t in (v, q, k, v, g, v, q, k))
    pos, freq = torch.zeros(1, 1, dtype=torch.int64), torch.ones(64, dtype=torch.float64)

    def changed(f, *written):
        every = [*x, *f32.values(), o, dq, dk, dv, dg, do, q2, k2, pos, freq]
        before = [t._version for t in every]
        got = f()
        for t, b in zip(every, before):
            assert (t._version != b) == any(t is w for w in written), (t.shape, t._version - b)
        return got

    pool = f32["pool"]
    *_, ctx = changed(lambda: lib.kda_decay_attn_fwd(*x, f32["h0"], out=o, final_state_out=f32["hT"]), o, f32["hT"])
    changed(lambda: lib.kda_decay_attn_bwd(ctx, do, f32["dhT"], out=(dq, dk, dv, dg, f32["dh0"])), dq, dk, dv, dg, f32["dh0"])
    changed(lambda: lib.kda_decay_attn_fwd(*x, f32["h0"]))
    changed(lambda: lib.kda_decay_attn_prefill(*x, pool, out=o), o, pool)
    changed(lambda: lib.kda_decay_attn_prefill(*x, pool), pool)
    changed(lambda: lib.kda_decay_attn_decode(*x, pool, out=o), o, pool)
    changed(lambda: lib.kda_qk_norm_rope_fwd(q, k, None, None, pos, freq, q_out=q, k_out=k2), q, k2)
    changed(lambda: lib.kda_qk_norm_rope_bwd(dq, dk, q, k, None, None, pos, freq, out=(dq, k2)), dq, k2)
    changed(lambda: lib.kda_qk_norm_rope_bwd(dq, dk, q, k, None, None, pos, freq))
    with torch.inference_mode():  # tensors without versions
        lib.kda_decay_attn_decode(*x, torch.zeros(1, 2, D, D), out=torch.zeros_like(v))


def test_backward_notices_inputs_that_the_package_changed(calls):
    from linear_attention_gated_gb300 import (KdaError, kda_decay_attn_bwd, kda_decay_attn_fwd, kda_qk_norm_rope_fwd)
    x, shared = inputs(64), torch.zeros(1, 1, D, D)
    fixed = x[:3] + [torch.zeros(1)]
    do, dhT = x[2], torch.zeros(1, 1, D, D)
    *_, first = kda_decay_attn_fwd(*x, final_state_out=shared)
    *_, other = kda_decay_attn_fwd(*fixed, final_state_out=shared)
    *_, last = kda_decay_attn_fwd(*x, final_state_out=shared)
    with pytest.raises(KdaError):  # the decays' gradient would read another layer's final state
        kda_decay_attn_bwd(first, do, dhT)
    kda_decay_attn_bwd(first, do)  # (it is not read here,
    kda_decay_attn_bwd(other, do, dhT)  # nor here)
    kda_decay_attn_bwd(last, do, dhT)
    made = len(calls)
    # in place on a query that the forward had
    from linear_attention_gated_gb300 import decay
    caught, decay._call = decay._call, lambda *args: None
    try:
        kda_qk_norm_rope_fwd(x[0], x[1], None, None, None, None, q_out=x[0], k_out=torch.empty_like(x[1]))
    finally:
        decay._call = caught
    with pytest.raises(KdaError):
        kda_decay_attn_bwd(last, do)
    assert len(calls) == made


def test_a_training_pair_in_inference_mode(calls):
    """Tensors made there have no versions to check."""
    from linear_attention_gated_gb300 import kda_decay_attn_bwd, kda_decay_attn_fwd
    outside = inputs(64)
    with torch.inference_mode():
        for x in (outside, inputs(64)):
            *_, ctx = kda_decay_attn_fwd(*x)
            kda_decay_attn_bwd(ctx, x[2], torch.zeros(1, 1, D, D))
    assert len(calls) == 4


def test_prefill_without_a_workspace_is_for_sequences_that_are_never_cut():
    """The length up to which the binding does not ask the library, against the library."""
    from linear_attention_gated_gb300 import decay, decay_workspace_bytes
    for hv in (1, 2, 8, 96):
        for B in (1, 3, 40):
            assert decay_workspace_bytes(B, decay._UNCUT, hv, hv, training=False) == 0
        for lens in ([decay._UNCUT], [decay._UNCUT - 1, 1], [1] * 100 + [decay._UNCUT - 100]):
            assert decay_workspace_bytes(1, sum(lens), hv, hv, offsets(lens), training=False) == 0
    assert decay_workspace_bytes(1, decay._UNCUT + 1, 1, 1, training=False) > 0
