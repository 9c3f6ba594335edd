"""What the Python context of kda_gated_delta_fwd / _bwd keeps and passes on, and which tensors get a new version: no GPU
needed. The library's kernels are not called: the tensors are on the CPU, and the calls are caught where they would enter the
library."""

import ctypes
import weakref

import pytest
import torch

D = 128


@pytest.fixture(scope="module", autouse=True)
def library():
    from linear_attention_gated_gb300 import build
    build.build()


class Call:
    """One caught call: its name, what its offsets were when it was made, and its workspace."""

    def __init__(self, f, args):
        at_cu, at_ws = {"kda_gated_delta_fwd": (7, 18), "kda_gated_delta_bwd": (6, 23)}[f.__name__]
        cu, n = args[at_cu], args[at_cu + 1]
        self.cu = None if cu is None else list((ctypes.c_int64 * (n + 1)).from_address(cu))
        self.workspace, self.workspace_bytes = args[at_ws], args[at_ws + 1]


@pytest.fixture
def calls(monkeypatch):
    from linear_attention_gated_gb300 import delta
    made = []
    monkeypatch.setattr(delta, "_call", lambda f, device, *args: made.append(Call(f, args)))
    return made


def inputs(T, hv=1):
    x = [torch.zeros(1, T, hv, D, dtype=torch.bfloat16) for _ in range(3)]
    return x + [torch.zeros(1, T, hv, dtype=torch.bfloat16) for _ in range(2)]


def offsets(lens):
    return torch.tensor([0, *lens]).cumsum(0)


EVEN, LONG = [512] * 16, [7680] + [34] * 14 + [36]  # the second is cut into segments, the first is not


def need(lens):
    from linear_attention_gated_gb300 import gated_delta_workspace_bytes
    return gated_delta_workspace_bytes(1, sum(lens), 1, 1, offsets(lens))


def test_backward_goes_by_the_lengths_of_its_forward(calls):
    """A mirror that is filled again for the next batch before the backward."""
    from linear_attention_gated_gb300 import kda_gated_delta_bwd, kda_gated_delta_fwd
    x, mirror = inputs(8192), offsets(LONG)
    *_, ctx = kda_gated_delta_fwd(*x, cu_seqlens=mirror.clone(), cu_seqlens_cpu=mirror)
    mirror.copy_(offsets(EVEN))
    kda_gated_delta_bwd(ctx, x[2])
    assert [c.cu for c in calls] == [offsets(LONG).tolist()] * 2
    assert calls[0].workspace == calls[1].workspace and calls[0].workspace_bytes == calls[1].workspace_bytes


def test_a_workspace_that_was_too_small_lives_as_long_as_the_context(calls):
    """A captured graph, or work in flight, may still write to it."""
    from linear_attention_gated_gb300 import kda_gated_delta_fwd
    assert need(LONG) > need(EVEN)
    x, mirror = inputs(8192), offsets(EVEN)
    cu = mirror.clone()
    *_, ctx = kda_gated_delta_fwd(*x, cu_seqlens=cu, cu_seqlens_cpu=mirror)
    first = weakref.ref(ctx.workspace)
    mirror.copy_(offsets(LONG))
    cu.copy_(mirror)
    kda_gated_delta_fwd(*x, cu_seqlens=cu, cu_seqlens_cpu=mirror, context_out=ctx)
    assert [c.cu for c in calls] == [offsets(EVEN).tolist(), offsets(LONG).tolist()]
    assert calls[0].workspace_bytes >= need(EVEN) and calls[1].workspace_bytes >= need(LONG)
    assert first() is not None and first().data_ptr() == calls[0].workspace
    kda_gated_delta_fwd(*x, cu_seqlens=offsets(EVEN), cu_seqlens_cpu=offsets(EVEN), context_out=ctx)
    assert calls[2].workspace == calls[1].workspace  # the largest serves all
    del ctx
    assert first() is None


def test_a_refused_forward_leaves_the_one_before_as_it_was(calls):
    """A forward on a used context that needs a larger workspace and is refused, by the binding or by the library: the backward of the
    forward before still gets that forward's workspace and offsets."""
    from linear_attention_gated_gb300 import KdaError, delta, kda_gated_delta_bwd, kda_gated_delta_fwd
    x = inputs(8192)
    *_, ctx = kda_gated_delta_fwd(*x, cu_seqlens=offsets(EVEN), cu_seqlens_cpu=offsets(EVEN))
    more = dict(cu_seqlens=offsets(LONG), cu_seqlens_cpu=offsets(LONG), context_out=ctx)

    def refused(error, **kw):
        with pytest.raises(error):
            kda_gated_delta_fwd(*x, **more, **kw)
        made = len(calls)
        kda_gated_delta_bwd(ctx, x[2])
        assert len(calls) == made + 1
        assert (calls[-1].workspace, calls[-1].workspace_bytes, calls[-1].cu) == (calls[0].workspace, calls[0].workspace_bytes, calls[0].cu)

    refused(ValueError, out=x[0][:, :5])
    refused(ValueError, final_state_out=torch.zeros(1, 1, D, D))
    caught = delta._call

    def overlap(f, device, *args):
        if f.__name__ == "kda_gated_delta_fwd":
            raise KdaError(3, "an output overlaps an input or another output")
        caught(f, device, *args)

    with pytest.MonkeyPatch.context() as m:
        m.setattr(delta, "_call", overlap)
        refused(KdaError)
    kda_gated_delta_fwd(*x, **more)  # and the larger one is taken when the call goes through
    assert calls[-1].workspace_bytes >= need(LONG) > calls[0].workspace_bytes


def test_a_forward_that_failed_on_its_way_has_no_backward(calls, monkeypatch):
    """Its first launches may have written to the workspace: neither its own backward nor that of the forward before is right."""
    from linear_attention_gated_gb300 import KdaError, delta, kda_gated_delta_bwd, kda_gated_delta_fwd
    x = inputs(64)
    *_, ctx = kda_gated_delta_fwd(*x)
    caught = delta._call

    def fails(*args):
        raise KdaError(5, "a launch failed")

    monkeypatch.setattr(delta, "_call", fails)
    with pytest.raises(KdaError, match="launch"):
        kda_gated_delta_fwd(*x, context_out=ctx)
    monkeypatch.setattr(delta, "_call", caught)
    with pytest.raises(KdaError, match="no forward"):
        kda_gated_delta_bwd(ctx, x[2])
    kda_gated_delta_fwd(*x, context_out=ctx)
    kda_gated_delta_bwd(ctx, x[2])
    assert len(calls) == 3

    def unversioned(tensors):
        raise RuntimeError("an inference tensor outside of inference mode")

    monkeypatch.setattr(delta, "_written", unversioned)
    with pytest.raises(RuntimeError, match="inference"):
        kda_gated_delta_fwd(*x, context_out=ctx)
    with pytest.raises(KdaError, match="no forward"):
        kda_gated_delta_bwd(ctx, x[2])


def test_reuse_that_is_refused(calls, monkeypatch):
    """Another stream (two steps at once would share one workspace), other shapes, a context of another operator."""
    from linear_attention_gated_gb300 import KdaError, delta, kda_gated_delta_bwd, kda_gated_delta_fwd
    from linear_attention_gated_gb300.decay import DecayContext
    x = inputs(64)
    on = [5]
    monkeypatch.setattr(delta, "_stream", lambda device: on[0])
    *_, ctx = kda_gated_delta_fwd(*x)
    on[0] = 6
    with pytest.raises(KdaError, match="stream"):
        kda_gated_delta_fwd(*x, context_out=ctx)
    on[0] = 5
    with pytest.raises(KdaError):
        kda_gated_delta_fwd(*inputs(65), context_out=ctx)
    other = DecayContext(ctx.key, 256, ctx.device, 5)
    with pytest.raises(KdaError):
        kda_gated_delta_fwd(*x, context_out=other)
    with pytest.raises(KdaError):
        kda_gated_delta_bwd(other, x[2])
    kda_gated_delta_fwd(*x, context_out=ctx)
    assert len(calls) == 2


def test_backward_notices_inputs_that_changed(calls):
    from linear_attention_gated_gb300 import KdaError, kda_gated_delta_bwd, kda_gated_delta_fwd
    for i in range(5):
        x, h0 = inputs(64), torch.zeros(1, 1, D, D)
        *_, ctx = kda_gated_delta_fwd(*x, h0)
        kda_gated_delta_bwd(ctx, x[2].clone())
        x[i].zero_()
        with pytest.raises(KdaError):
            kda_gated_delta_bwd(ctx, x[2].clone())
    *_, ctx = kda_gated_delta_fwd(*x, h0, final_state_out=(hT := torch.zeros_like(h0)))
    hT.zero_()
    kda_gated_delta_bwd(ctx, x[2].clone(), hT)  # (the final state is not read again)


def test_a_training_pair_in_inference_mode(calls):
    """Tensors made there have no versions to check."""
    from linear_attention_gated_gb300 import kda_gated_delta_bwd, kda_gated_delta_fwd
    outside = inputs(64)
    with torch.inference_mode():
        for x in (outside, inputs(64)):
            *_, ctx = kda_gated_delta_fwd(*x)
            kda_gated_delta_bwd(ctx, x[2], torch.zeros(1, 1, D, D))
    assert len(calls) == 4


def test_writes_into_the_callers_tensors_count_as_changes(monkeypatch):
    """Tensors that a call writes get a new version, those that it reads keep theirs."""
    import linear_attention_gated_gb300 as lib
    from linear_attention_gated_gb300 import delta, norm
    for m in (delta, norm):
        monkeypatch.setattr(m, "_call", lambda *args: None)
    x = inputs(1, hv=2)
    q, k, v, g, beta = x
    f32 = {n: torch.zeros(1, 2, D, D) for n in ("h0", "hT", "pool", "dh0", "dhT")}
    o, dq, dk, dv, dg, db, do, y, dx = (torch.zeros_like(t) for t in (v, q, k, v, g, beta, v, q, q))
    w, mean, rstd = torch.ones(D), torch.zeros(1, 1, 2), torch.ones(1, 1, 2)

    def changed(f, *written):
        every = [*x, *f32.values(), o, dq, dk, dv, dg, db, do, y, dx, w, mean, rstd]
        before = [t._version for t in every]
        got = f()
        for t, b in zip(every, before):
            assert (t._version != b) == any(t is z for z in written), (t.shape, t._version - b)
        return got

    pool = f32["pool"]
    *_, ctx = changed(lambda: lib.kda_gated_delta_fwd(*x, f32["h0"], out=o, final_state_out=f32["hT"]), o, f32["hT"])
    out = (dq, dk, dv, dg, db, f32["dh0"])
    changed(lambda: lib.kda_gated_delta_bwd(ctx, do, f32["dhT"], out=out), *out)
    changed(lambda: lib.kda_gated_delta_fwd(*x, f32["h0"]))
    changed(lambda: lib.kda_gated_delta_prefill(*x, pool, out=o), o, pool)
    changed(lambda: lib.kda_gated_delta_decode(*x, pool, out=o), o, pool)
    changed(lambda: lib.kda_layer_norm_fwd(q, w, w))
    changed(lambda: lib.kda_layer_norm_fwd(q, w, w, out=y), y)
    changed(lambda: lib.kda_layer_norm_bwd(do, q, w, mean, rstd))
    changed(lambda: lib.kda_layer_norm_bwd(do, q, w, mean, rstd, out=dx), dx)


def test_no_decays(calls):
    from linear_attention_gated_gb300 import kda_gated_delta_bwd, kda_gated_delta_fwd
    q, k, v, g, beta = inputs(64)
    *_, ctx = kda_gated_delta_fwd(q, k, v, None, beta)
    assert kda_gated_delta_bwd(ctx, v)[3] is None
    with pytest.raises(ValueError):
        kda_gated_delta_bwd(ctx, v, out=(q, k, v, g, beta, None))
    with pytest.raises(ValueError):
        kda_gated_delta_bwd(ctx, v, out=(q, k, v, None, beta))
