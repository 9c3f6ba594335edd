"""The gated delta rule with a decay and a step size for each token and head (Python binding of the
``kda_gated_delta_*`` entry points of include/kda.h).

Argument marshalling only: torch provides device memory and the current CUDA stream; all arithmetic
runs in libkda.so's kernels, and there is no CPU fallback. Every call enqueues on the current stream
of its tensors' device.
"""

from __future__ import annotations

import ctypes

import torch

from .decay import (_BF16, _F32, _I32, _NAN, DecayContext, _all_strides, _call, _offsets, _p, _pool, _slots, _stream, _typed,
                    _want, _written)
from .kda import KdaError, _check, load_library


def _inputs(q, k, v, log_decay, beta):
    """Checks of the token tensors; (B, T, Hqk, Hv, D, strides)."""
    for name, t in (("q", q), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a [B, T, H, 128] tensor")
    B, T, Hqk, D = q.shape
    Hv = v.shape[2]
    dev = q.device
    _typed(q, "q", _BF16, q.shape, dev)
    _typed(k, "k", _BF16, q.shape, dev)
    _typed(v, "v", _BF16, (B, T, Hv, D), dev)
    if log_decay is not None:
        _want(log_decay, "log_decay", _BF16, (B, T, Hv), dev)
    _want(beta, "beta", _BF16, (B, T, Hv), dev)
    flat = q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
    return B, T, Hqk, Hv, D, None if flat else _all_strides(("q", q), ("k", k), ("v", v))


def gated_delta_workspace_bytes(B, T, Hqk, Hv, cu_seqlens_cpu=None, training=True) -> int:
    """Device bytes that kda_gated_delta_fwd and _bwd (or, training False, kda_gated_delta_prefill)
    need for this problem."""
    lib = load_library()
    out = ctypes.c_size_t(0)
    n = 0 if cu_seqlens_cpu is None else cu_seqlens_cpu.numel() - 1
    _check(lib.kda_gated_delta_workspace_bytes(B, T, Hqk, Hv, _p(cu_seqlens_cpu), n, int(training), ctypes.byref(out)))
    return out.value


class DeltaContext(DecayContext):
    """What the backward of one forward call needs: the borrowed inputs with their tensor versions (they must not
    change before the backward), and a workspace that holds each chunk's system, start state and u. Passing it
    back as ``context_out`` uses the workspace again for another call of the same shapes on the same stream, whose
    backward is then the only one it has. A captured graph of calls on a context needs the context for as long as it
    is replayed."""


def kda_gated_delta_fwd(q, k, v, log_decay, beta, initial_state=None, cu_seqlens=None, scale=None, out=None,
                        final_state_out=None, context_out=None, *, cu_seqlens_cpu=None):
    """Training forward of the gated delta rule: S' = exp(g_t) S_{t-1}, u_t = v_t - S' k_t,
    S_t = S' + beta_t u_t k_t^T, o_t = scale S_t q_t, per sequence and value head (head h reads query/key
    head h // (Hv / Hqk)). Returns (o, final_state, ctx).

    q, k [B, T, Hqk, 128] and v [B, T, Hv, 128] BF16, contiguous or views with whole heads contiguous
    (slices of one projection); log_decay BF16 [B, T, Hv], or None for the delta rule without decays;
    beta BF16 [B, T, Hv]; initial_state FP32 [N, Hv, 128, 128] value-first, None for zeros. Keys are taken as they
    are: of norm 1, with beta in [0, 2], they keep the state bounded. Packed sequences (B = 1) have
    cu_seqlens int64 [N + 1] on the device and its CPU mirror; sequences may be empty. scale defaults to
    1 / sqrt(128). ctx goes to kda_gated_delta_bwd; as ``context_out`` of a later call of the same shapes
    on the same stream its workspace is used again."""
    lib = load_library()
    B, T, Hqk, Hv, D, strides = _inputs(q, k, v, log_decay, beta)
    dev = q.device
    cu_host = _offsets(cu_seqlens, cu_seqlens_cpu, dev, True)
    N = B if cu_host is None else cu_host.numel() - 1
    if initial_state is not None:
        _want(initial_state, "initial_state", _F32, (N, Hv, D, D), dev)
    ctx = context_out
    key = (B, T, Hqk, Hv, N)
    stream = _stream(dev)
    if ctx is not None and (not isinstance(ctx, DeltaContext) or ctx.key != key or ctx.device != dev or ctx.stream != stream):
        raise KdaError(4, "context reuse needs the same shapes, device and stream")
    if cu_host is not None:
        known = ctx is not None and ctx.cu is not None and torch.equal(cu_host, ctx.cu)
        cu_host = ctx.cu if known else cu_host.clone()
    if out is None:
        out = torch.empty((B, T, Hv, D), dtype=_BF16, device=dev)
    else:
        _want(out, "out", _BF16, (B, T, Hv, D), dev)
    if final_state_out is None:
        final_state_out = torch.empty((N, Hv, D, D), dtype=_F32, device=dev)
    else:
        _want(final_state_out, "final_state_out", _F32, (N, Hv, D, D), dev)
    if ctx is None:
        ctx = DeltaContext(key, gated_delta_workspace_bytes(B, T, Hqk, Hv, cu_host), dev, stream)
    ws = ctx.workspace
    if context_out is not None and cu_host is not None and not known:
        nbytes = gated_delta_workspace_bytes(B, T, Hqk, Hv, cu_host)  # other lengths may need more
        if nbytes > ws.numel():  # (the context keeps its own until the call has gone through: the last forward's backward needs it)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    s = _NAN if scale is None else float(scale)
    shape = (_p(cu_seqlens), _p(cu_host), N, B, T, Hqk, Hv, D, s, strides)
    tokens = (q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(log_decay), beta.data_ptr())
    last, ctx.inputs = ctx.inputs, ()
    try:
        _call(lib.kda_gated_delta_fwd, dev, *tokens, _p(initial_state), *shape, out.data_ptr(), final_state_out.data_ptr(),
              ws.data_ptr(), ws.numel(), ctx.device_status.data_ptr())
    except KdaError as e:
        if e.status != 5:  # refused before any launch: the last forward stands (after a CUDA error the workspace may hold a part of this one)
            ctx.inputs = last
        raise
    _written((out, final_state_out))
    if ws is not ctx.workspace:
        ctx.outgrown.append(ctx.workspace)
        ctx.workspace = ws
    # (the final state is not read again)
    ctx._snapshot((q, k, v, log_decay, beta, initial_state, cu_seqlens, None), tokens + shape, cu_host,
                  (q.shape, v.shape, (N, Hv, D, D), log_decay is not None))
    return out, final_state_out, ctx


def kda_gated_delta_bwd(ctx: DeltaContext, do, dfinal_state=None, out=None):
    """Training backward from the context of kda_gated_delta_fwd. Returns
    (dq, dk, dv, dlog_decay, dbeta, dinitial_state): BF16 but for dinitial_state FP32; dlog_decay is None
    without decays and dinitial_state None where there was no initial state. ``out``: six tensors (or None
    in those two places) in that order."""
    lib = load_library()
    if not isinstance(ctx, DeltaContext):
        raise KdaError(4, "not a forward context")
    ctx.check_unchanged(False)
    qs, vs, ss, decays = ctx.shapes
    dev = ctx.device
    _want(do, "do", _BF16, vs, dev)
    if dfinal_state is not None:
        _want(dfinal_state, "dfinal_state", _F32, ss, dev)
    shapes = (qs, qs, vs, vs[:3] if decays else None, vs[:3], ss if ctx.inputs[5] is not None else None)
    if out is None:
        out = tuple(None if s is None else torch.empty(s, dtype=_F32 if i == 5 else _BF16, device=dev)
                    for i, s in enumerate(shapes))
    else:
        if len(out) != 6:
            raise ValueError("out must hold six gradient tensors in return order")
        for i, (t, s) in enumerate(zip(out, shapes)):
            if s is None:
                if t is not None:
                    raise ValueError("out holds a tensor for a gradient that this call does not have")
            else:
                _want(t, ("dq", "dk", "dv", "dlog_decay", "dbeta", "dinitial_state")[i], _F32 if i == 5 else _BF16, s, dev)
    ws = ctx.workspace
    _call(lib.kda_gated_delta_bwd, dev, *ctx.call, do.data_ptr(), _p(dfinal_state), *[_p(t) for t in out],
          ws.data_ptr(), ws.numel(), ctx.device_status.data_ptr())
    _written([t for t in out if t is not None])
    return tuple(out)


def kda_gated_delta_prefill(q, k, v, log_decay, beta, state, cu_seqlens=None, state_indices=None, scale=None, out=None,
                            device_status=None, workspace=None, *, cu_seqlens_cpu=None, state_indices_cpu=None):
    """Inference prefill of the gated delta rule from a state pool: returns o; every sequence starts from its
    slot of ``state`` (BF16 or FP32 [num_slots, Hv, 128, 128], slot n without state_indices) and leaves its
    final state there. Token tensors as for kda_gated_delta_fwd. The ``*_cpu`` keywords pass trusted CPU
    mirrors of the device index tensors; without them the mirrors are copied from the device, which waits
    for it. ``workspace``: a uint8 tensor of gated_delta_workspace_bytes(..., training=False); None takes
    one for the call."""
    lib = load_library()
    B, T, Hqk, Hv, D, strides = _inputs(q, k, v, log_decay, beta)
    dev = q.device
    cu_host = _offsets(cu_seqlens, cu_seqlens_cpu, dev, False)
    N = B if cu_host is None else cu_host.numel() - 1
    idx_host = _slots(state_indices, state_indices_cpu, N, dev)
    sdt = _pool(state, Hv, D, dev)
    if out is None:
        out = torch.empty((B, T, Hv, D), dtype=_BF16, device=dev)
    else:
        _want(out, "out", _BF16, (B, T, Hv, D), dev)
    if device_status is not None:
        _want(device_status, "device_status", _I32, device_status.shape, dev)
    if workspace is None:
        nbytes = gated_delta_workspace_bytes(B, T, Hqk, Hv, cu_host, False)
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    else:
        _want(workspace, "workspace", torch.uint8, workspace.shape, dev)
    _call(lib.kda_gated_delta_prefill, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(log_decay), beta.data_ptr(),
          _p(cu_seqlens), _p(cu_host), N, B, T, Hqk, Hv, D, _NAN if scale is None else float(scale), strides, state.data_ptr(),
          sdt, _p(state_indices), _p(idx_host), state.shape[0], out.data_ptr(), _p(workspace),
          0 if workspace is None else workspace.numel(), _p(device_status))
    _written((state, out))
    return out


def kda_gated_delta_decode(q, k, v, log_decay, beta, state, state_indices=None, scale=None, out=None, *, state_indices_cpu=None):
    """One decode step (T = 1) of the gated delta rule: updates ``state`` (BF16 or FP32 [num_slots, Hv, 128, 128])
    in place at slot state_indices[n] (int32 [N], slot n when None) and returns o. q, k [N, 1, Hqk, 128],
    v [N, 1, Hv, 128], log_decay (or None) and beta [N, 1, Hv] BF16. ``state_indices_cpu``, a trusted CPU copy of
    state_indices, is what the library validates; without it the indices are copied to the host, which
    waits for the device. One launch."""
    lib = load_library()
    N, T, Hqk, Hv, D, strides = _inputs(q, k, v, log_decay, beta)
    if T != 1:
        raise ValueError("decode takes one token per sequence (T = 1)")
    dev = q.device
    sdt = _pool(state, Hv, D, dev)
    idx_host = _slots(state_indices, state_indices_cpu, N, dev)
    if out is None:
        out = torch.empty_like(v) if v.is_contiguous() else torch.empty((N, 1, Hv, D), dtype=_BF16, device=dev)
    else:
        _want(out, "out", _BF16, (N, 1, Hv, D), dev)
    _call(lib.kda_gated_delta_decode, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(log_decay), beta.data_ptr(),
          state.data_ptr(), sdt, _p(state_indices), _p(idx_host), state.shape[0], N, Hqk, Hv, D,
          _NAN if scale is None else float(scale), strides, out.data_ptr())
    _written((state, out))
    return out
