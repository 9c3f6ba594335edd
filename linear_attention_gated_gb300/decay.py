"""Linear attention with a decay for each head, and the norm and position rotation of its queries
and keys (Python binding of the ``kda_decay_attn_*`` and ``kda_qk_norm_rope_*`` entry points of
include/kda.h).

Argument marshalling only: torch provides device memory and the current CUDA stream; all arithmetic
runs in libkda.so's kernels, and there is no CPU fallback. Every call enqueues on the current stream
of its tensors' device.
"""

from __future__ import annotations

import ctypes

import torch

from .kda import KdaError, _check, load_library

DIM = 128
_NAN = float("nan")
_UNCUT = 1536  # sequences up to this long are never cut into segments (24 chunks in csrc/kda_decay_pass.cu): prefill needs no workspace for them
_BF16, _F32, _F64, _I32, _I64 = torch.bfloat16, torch.float32, torch.float64, torch.int32, torch.int64
_STATE = {torch.bfloat16: 0, torch.float32: 1}
_ROPE_WORKSPACE = {}  # head_dim -> bytes
_ROPE_TYPES = {torch.bfloat16: 0, torch.float32: 1, torch.float16: 2}


_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None
# Tensors that a call wrote get a new version, as torch's own writes in place give them: _written((t, ...))
_written = getattr(torch._C, "_increment_version", torch.autograd.graph.increment_version)
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _stream(device):
    """The current stream of `device` (0 for the CPU, whose tensors _call refuses)."""
    if device.type != "cuda":
        return 0
    return torch.cuda.current_stream(device.index).cuda_stream if _raw_stream is None else _raw_stream(device.index)


def _call(f, device, *args):
    """f(*args, stream) with `device` current, its status checked. (The small calls are host-bound: torch's stream and
    device objects would cost as much as the launch.)"""
    if device.type != "cuda":
        raise ValueError("tensors must be CUDA tensors")
    index = device.index
    stream = torch.cuda.current_stream(index).cuda_stream if _raw_stream is None else _raw_stream(index)
    if _current_device() == index:
        rc = f(*args, stream)
    else:
        with torch.cuda.device(index):
            rc = f(*args, stream)
    if rc:
        _check(rc)


def _typed(t, name, dtype, shape, device):
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == device:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}")


def _want(t, name, dtype, shape, device):
    _typed(t, name, dtype, shape, device)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _strides(t, name):
    """Token and head strides of a [B, T, H, D] tensor whose heads are contiguous rows."""
    B, T, H, D = t.shape
    sb, st, sh, sd = t.stride()
    if D > 1 and sd != 1:
        raise ValueError(f"{name} must be contiguous in its last dimension")
    if H == 1:
        sh = D
    if T == 1:
        st = sb if B > 1 else H * sh
    elif B > 1 and sb != T * st:
        raise ValueError(f"{name}: batch rows must be T token strides apart")
    return st, sh


def _all_strides(*named):
    """Token and head strides of all as a C array. (Not needed where all are contiguous.)"""
    flat = [s for name, t in named for s in (_strides(t, name) if t.numel() else (t.shape[2] * t.shape[3], t.shape[3]))]
    return (ctypes.c_int64 * len(flat))(*flat)


def _decay_inputs(q, k, v, log_decay):
    """Checks of the token tensors; (B, T, Hqk, Hv, per_token, strides)."""
    for name, t in (("q", q), ("v", v)):
        if not isinstance(t, torch.Tensor) or t.dim() != 4:
            raise ValueError(f"{name} must be a [B, T, H, 128] tensor")
    B, T, Hqk, D = q.shape
    Hv = v.shape[2]
    dev = q.device
    _typed(q, "q", _BF16, q.shape, dev)
    _typed(k, "k", _BF16, q.shape, dev)
    _typed(v, "v", _BF16, (B, T, Hv, D), dev)
    per_token = not (isinstance(log_decay, torch.Tensor) and log_decay.dim() == 1)
    if per_token:
        _want(log_decay, "log_decay", _BF16, (B, T, Hv), dev)
    else:
        _want(log_decay, "log_decay", _F32, (Hv,), dev)
    flat = q.is_contiguous() and k.is_contiguous() and v.is_contiguous()
    return B, T, Hqk, Hv, D, int(per_token), None if flat else _all_strides(("q", q), ("k", k), ("v", v))


def _offsets(cu_seqlens, cu_seqlens_cpu, dev, need_mirror):
    if cu_seqlens is None:
        if cu_seqlens_cpu is not None:
            raise ValueError("cu_seqlens_cpu given without cu_seqlens")
        return None
    if cu_seqlens_cpu is None:
        if need_mirror:
            raise ValueError("packed input requires cu_seqlens_cpu, a trusted CPU mirror of cu_seqlens")
        cu_seqlens_cpu = cu_seqlens.cpu()
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be a 1-D tensor of N + 1 offsets")
    _want(cu_seqlens, "cu_seqlens", _I64, cu_seqlens.shape, dev)
    _want(cu_seqlens_cpu, "cu_seqlens_cpu", _I64, cu_seqlens.shape, torch.device("cpu"))
    return cu_seqlens_cpu


def _slots(state_indices, state_indices_cpu, N, dev):
    if state_indices is None:
        if state_indices_cpu is not None:
            raise ValueError("state_indices_cpu given without state_indices")
        return None
    _want(state_indices, "state_indices", _I32, (N,), dev)
    if state_indices_cpu is None:
        return state_indices.cpu()
    _want(state_indices_cpu, "state_indices_cpu", _I32, (N,), torch.device("cpu"))
    return state_indices_cpu


def _pool(state, Hv, D, dev):
    if not isinstance(state, torch.Tensor) or state.dtype not in _STATE:
        raise TypeError("state must be a bfloat16 or float32 tensor")
    if state.dim() != 4 or state.shape[1:] != (Hv, D, D) or not state.is_contiguous():
        raise ValueError(f"state must be contiguous [num_slots, {Hv}, {D}, {D}]")
    if state.device != dev:
        raise ValueError(f"state must be on {dev}")
    return _STATE[state.dtype]


def _versions(tensors):
    """Their versions, as far as they have some (tensors made in inference mode have none)."""
    return tuple(None if t is None or t.is_inference() else t._version for t in tensors)


def _p(t):
    return None if t is None else t.data_ptr()


def decay_workspace_bytes(B, T, Hqk, Hv, cu_seqlens_cpu=None, per_token=True, training=True) -> int:
    """Device bytes that kda_decay_attn_fwd and _bwd (or, training False, kda_decay_attn_prefill)
    need for this problem, with decays for each token or fixed for each head."""
    lib = load_library()
    out = ctypes.c_size_t(0)
    n = 0 if cu_seqlens_cpu is None else cu_seqlens_cpu.numel() - 1
    _check(lib.kda_decay_attn_workspace_bytes(B, T, Hqk, Hv, _p(cu_seqlens_cpu), n, int(per_token), int(training), ctypes.byref(out)))
    return out.value


class DecayContext:
    """What the backward of one forward call needs: the borrowed inputs and final state with their tensor
    versions (they must not change before the backward), and a workspace. Passing it back as
    ``context_out`` uses the workspace again for another call of the same shapes on the same stream; sequences of
    other lengths may need a larger one. (A backward on another stream shares that workspace: the caller orders it
    after the forward and before the context's next call.) A captured graph of calls on a context needs the context
    for as long as it is replayed."""

    def __init__(self, key, nbytes, device, stream):
        self.key = key
        self.device = device
        self.stream = stream
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
        self.outgrown = []  # smaller ones from before: a captured graph may still write to them
        self.device_status = torch.zeros(1, dtype=_I32, device=device)
        self.inputs = ()
        self.versions = ()
        self.cu = None  # the context's own copy of the offsets: the caller's mirror may be filled again before the backward

    def _snapshot(self, inputs, call, cu, shapes):
        self.inputs = inputs
        self.versions = _versions(inputs)
        self.call, self.cu, self.shapes = call, cu, shapes

    def check_unchanged(self, final_state=True):
        """final_state: it is read again too (by the decays' gradient, with an adjoint of its own)."""
        if not self.inputs:
            raise KdaError(4, "the context holds no forward")
        now = _versions(self.inputs)
        if self.versions[:-1] != now[:-1] or (final_state and self.versions[-1] != now[-1]):
            raise KdaError(4, "an input or the final state of the forward was modified before the backward")

    def status(self):
        """Waits for the device and raises if a bounded device wait of these calls gave up."""
        if int(self.device_status.item()) & 1:
            raise KdaError(6, "a device-side wait gave up; the outputs are incomplete")


def kda_decay_attn_fwd(q, k, v, log_decay, initial_state=None, cu_seqlens=None, scale=None, out=None,
                       final_state_out=None, context_out=None, *, cu_seqlens_cpu=None):
    """Training forward of linear attention with a decay for each head:
    S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = scale S_t q_t, per sequence and value head (head h reads
    query/key head h // (Hv / Hqk)). Returns (o, final_state, ctx).

    q, k [B, T, Hqk, 128] and v [B, T, Hv, 128] BF16, contiguous or views with whole heads contiguous
    (slices of one projection); log_decay FP32 [Hv], fixed for each head, or BF16 [B, T, Hv];
    initial_state FP32 [N, Hv, 128, 128] value-first, None for zeros. Packed sequences (B = 1) have
    cu_seqlens int64 [N + 1] on the device and its CPU mirror; sequences may be empty. scale defaults to
    1 / sqrt(128). ctx goes to kda_decay_attn_bwd; as ``context_out`` of a later call of the same shapes
    on the same stream its workspace is used again."""
    lib = load_library()
    B, T, Hqk, Hv, D, per_token, strides = _decay_inputs(q, k, v, log_decay)
    dev = q.device
    cu_host = _offsets(cu_seqlens, cu_seqlens_cpu, dev, True)
    N = B if cu_host is None else cu_host.numel() - 1
    if initial_state is not None:
        _want(initial_state, "initial_state", _F32, (N, Hv, D, D), dev)
    ctx = context_out
    key = (B, T, Hqk, Hv, N, per_token)
    stream = _stream(dev)
    if ctx is not None and (ctx.key != key or ctx.device != dev or ctx.stream != stream):
        raise KdaError(4, "context reuse needs the same shapes, kind of decay, device and stream")
    if cu_host is not None:
        known = ctx is not None and ctx.cu is not None and torch.equal(cu_host, ctx.cu)
        cu_host = ctx.cu if known else cu_host.clone()
    if ctx is None:
        ctx = DecayContext(key, decay_workspace_bytes(B, T, Hqk, Hv, cu_host, per_token), dev, stream)
    elif cu_host is not None and not known:
        nbytes = decay_workspace_bytes(B, T, Hqk, Hv, cu_host, per_token)  # other lengths may need more
        if nbytes > ctx.workspace.numel():
            ctx.outgrown.append(ctx.workspace)
            ctx.workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    o = torch.empty((B, T, Hv, D), dtype=_BF16, device=dev) if out is None else out
    hT = torch.empty((N, Hv, D, D), dtype=_F32, device=dev) if final_state_out is None else final_state_out
    if out is not None:
        _want(out, "out", _BF16, (B, T, Hv, D), dev)
    if final_state_out is not None:
        _want(final_state_out, "final_state_out", _F32, (N, Hv, D, D), dev)
    s = _NAN if scale is None else float(scale)
    call = (q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), per_token, _p(initial_state), _p(cu_seqlens),
            _p(cu_host), N, B, T, Hqk, Hv, D, s, strides)
    ws = ctx.workspace
    _call(lib.kda_decay_attn_fwd, dev, *call, o.data_ptr(), hT.data_ptr(), ws.data_ptr(), ws.numel(),
          ctx.device_status.data_ptr())
    _written((o, hT))
    ctx._snapshot((q, k, v, log_decay, initial_state, cu_seqlens, hT), call, cu_host,
                  (q.shape, v.shape, (N, Hv, D, D), per_token))
    return o, hT, ctx


def kda_decay_attn_bwd(ctx: DecayContext, do, dfinal_state=None, out=None):
    """Training backward from the context of kda_decay_attn_fwd. Returns
    (dq, dk, dv, dlog_decay, dinitial_state): BF16 but for dinitial_state FP32; dlog_decay is None
    for decays fixed for each head and dinitial_state None where there was no initial state.
    ``out``: five tensors (or None in those two places) in that order."""
    lib = load_library()
    if not isinstance(ctx, DecayContext):
        raise KdaError(4, "not a forward context")
    ctx.check_unchanged(dfinal_state is not None and bool(ctx.inputs) and ctx.shapes[3])
    qs, vs, ss, per_token = ctx.shapes
    dev = ctx.device
    _want(do, "do", _BF16, vs, dev)
    if dfinal_state is not None:
        _want(dfinal_state, "dfinal_state", _F32, ss, dev)
    shapes = (qs, qs, vs, vs[:3] if per_token else None, ss if ctx.inputs[4] is not None else None)
    if out is None:
        out = tuple(None if s is None else torch.empty(s, dtype=_F32 if i == 4 else _BF16, device=dev)
                    for i, s in enumerate(shapes))
    else:
        if len(out) != 5:
            raise ValueError("out must hold five gradient tensors in return order")
        for i, (t, s) in enumerate(zip(out, shapes)):
            if s is None:
                if t is not None:
                    raise ValueError("out holds a tensor for a gradient that this call does not have")
            else:
                _want(t, ("dq", "dk", "dv", "dlog_decay", "dinitial_state")[i], _F32 if i == 4 else _BF16, s, dev)
    ws = ctx.workspace
    _call(lib.kda_decay_attn_bwd, dev, *ctx.call, ctx.inputs[6].data_ptr(), do.data_ptr(), _p(dfinal_state),
          *[_p(t) for t in out], ws.data_ptr(), ws.numel(), ctx.device_status.data_ptr())
    _written([t for t in out if t is not None])
    return tuple(out)


def kda_decay_attn_prefill(q, k, v, log_decay, state, cu_seqlens=None, state_indices=None, scale=None, out=None,
                           device_status=None, workspace=None, *, cu_seqlens_cpu=None, state_indices_cpu=None):
    """Inference prefill of linear attention with a decay for each head, from a state pool: returns o;
    every sequence starts from its slot of ``state`` (BF16 or FP32 [num_slots, Hv, 128, 128], slot n
    without state_indices) and leaves its final state there. Token tensors as for kda_decay_attn_fwd.
    The ``*_cpu`` keywords pass trusted CPU mirrors of the device index tensors; without them the mirrors
    are copied from the device, which waits for it. ``workspace``: a uint8 tensor of
    decay_workspace_bytes(..., training=False); None takes one for the call."""
    lib = load_library()
    B, T, Hqk, Hv, D, per_token, strides = _decay_inputs(q, k, v, log_decay)
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
        if T > _UNCUT:
            nbytes = decay_workspace_bytes(B, T, Hqk, Hv, cu_host, per_token, False)
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    else:
        _want(workspace, "workspace", torch.uint8, workspace.shape, dev)
    _call(lib.kda_decay_attn_prefill, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), per_token,
          _p(cu_seqlens), _p(cu_host), N, B, T, Hqk, Hv, D, _NAN if scale is None else float(scale), strides, state.data_ptr(),
          sdt, _p(state_indices), _p(idx_host), state.shape[0], out.data_ptr(), _p(workspace),
          0 if workspace is None else workspace.numel(), _p(device_status))
    _written((state, out))
    return out


def kda_decay_attn_decode(q, k, v, log_decay, state, state_indices=None, scale=None, out=None, *, state_indices_cpu=None):
    """One decode step (T = 1) of linear attention with a decay for each head: updates ``state`` (BF16 or
    FP32 [num_slots, Hv, 128, 128]) in place at slot state_indices[n] (int32 [N], slot n when None) and
    returns o. q, k [N, 1, Hqk, 128], v [N, 1, Hv, 128] BF16; log_decay BF16 [N, 1, Hv] or FP32 [Hv].
    ``state_indices_cpu``, a trusted CPU copy of state_indices, is what the library validates; without it
    the indices are copied to the host, which waits for the device. One launch."""
    lib = load_library()
    N, T, Hqk, Hv, D, per_token, strides = _decay_inputs(q, k, v, log_decay)
    if T != 1:
        raise ValueError("decode takes one token per sequence (T = 1)")
    dev = q.device
    sdt = _pool(state, Hv, D, dev)
    idx_host = _slots(state_indices, state_indices_cpu, N, dev)
    if out is None:
        out = torch.empty_like(v) if v.is_contiguous() else torch.empty((N, 1, Hv, D), dtype=_BF16, device=dev)
    else:
        _want(out, "out", _BF16, (N, 1, Hv, D), dev)
    _call(lib.kda_decay_attn_decode, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), per_token,
          state.data_ptr(), sdt, _p(state_indices), _p(idx_host), state.shape[0], N, Hqk, Hv, D,
          _NAN if scale is None else float(scale), strides, out.data_ptr())
    _written((state, out))
    return out


def _rope_inputs(q, k, q_weight, k_weight, positions, inv_freq):
    if not isinstance(q, torch.Tensor) or q.dim() != 4 or not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("q and k must be [B, T, H, D] tensors")
    if q.dtype not in _ROPE_TYPES:
        raise TypeError("q must be bfloat16, float16 or float32")
    B, T, Hq, D = q.shape
    Hk = k.shape[2]
    dev = q.device
    _typed(k, "k", q.dtype, (B, T, Hk, D), dev)
    if q_weight is not None:
        _want(q_weight, "q_weight", _F32, (D,), dev)
    if k_weight is not None:
        _want(k_weight, "k_weight", _F32, (D,), dev)
    if inv_freq is None:
        return B, T, Hq, Hk, D, 0, dev, None, None
    R = 2 * inv_freq.numel()
    _want(inv_freq, "inv_freq", _F64, (R // 2,), dev)
    _want(positions, "positions", _I64, (B, T), dev)
    if R == 0:
        return B, T, Hq, Hk, D, 0, dev, None, None
    return B, T, Hq, Hk, D, R, dev, positions.data_ptr(), inv_freq.data_ptr()


def kda_qk_norm_rope_fwd(q, k, q_weight, k_weight, positions, inv_freq, eps=1e-6, interleaved=False, q_out=None, k_out=None):
    """RMS norm of every query and key head and the rotation by position, in one pass: returns
    (q_out, k_out). q [B, T, Hq, D] and k [B, T, Hk, D] of one type (BF16, FP16 or FP32), contiguous or views
    with whole heads contiguous; q_weight, k_weight FP32 [D] or None; positions int64 [B, T]; inv_freq
    FP64 [R / 2], the angle of a pair per position: pairs are (d, d + R / 2) of the first R dimensions, or
    (2d, 2d + 1) when interleaved; None for the norm alone. D and R are multiples of 16, D up to 256.
    q_out and k_out may be q and k."""
    lib = load_library()
    B, T, Hq, Hk, D, R, dev, pos, freq = _rope_inputs(q, k, q_weight, k_weight, positions, inv_freq)
    flat_q, flat_k = q.is_contiguous(), k.is_contiguous()
    fresh = q_out is None and k_out is None
    if q_out is None:
        q_out = torch.empty_like(q) if flat_q else torch.empty((B, T, Hq, D), dtype=q.dtype, device=dev)
    else:
        _typed(q_out, "q_out", q.dtype, q.shape, dev)
        flat_q = flat_q and q_out.is_contiguous()
    if k_out is None:
        k_out = torch.empty_like(k) if flat_k else torch.empty((B, T, Hk, D), dtype=q.dtype, device=dev)
    else:
        _typed(k_out, "k_out", q.dtype, k.shape, dev)
        flat_k = flat_k and k_out.is_contiguous()
    strides = None if flat_q and flat_k else _all_strides(("q", q), ("k", k), ("q_out", q_out), ("k_out", k_out))
    _call(lib.kda_qk_norm_rope_fwd, dev, q.data_ptr(), k.data_ptr(), _ROPE_TYPES[q.dtype], _p(q_weight), _p(k_weight),
          pos, freq, B * T, Hq, Hk, D, R, eps, 1 if interleaved else 0, strides, q_out.data_ptr(), k_out.data_ptr())
    if not fresh:
        _written((q_out, k_out))
    return q_out, k_out


def kda_qk_norm_rope_bwd(dq, dk, q, k, q_weight, k_weight, positions, inv_freq, eps=1e-6, interleaved=False, out=None,
                         workspace=None):
    """Gradients of kda_qk_norm_rope_fwd from those of its outputs (dq, dk) and its inputs: returns
    (dq_in, dk_in, dq_weight, dk_weight), the last two FP32 [D], summed over all tokens and heads, or None
    where there is no weight. ``out``: (dq_in, dk_in) buffers, which may be dq and dk. ``workspace``: a uint8
    tensor for the weights' partial sums (kda_qk_norm_rope_workspace_bytes); None takes one for the call."""
    lib = load_library()
    B, T, Hq, Hk, D, R, dev, pos, freq = _rope_inputs(q, k, q_weight, k_weight, positions, inv_freq)
    _typed(dq, "dq", q.dtype, q.shape, dev)
    _typed(dk, "dk", q.dtype, k.shape, dev)
    flat_q, flat_k = q.is_contiguous(), k.is_contiguous()
    if out is None:
        gq = torch.empty_like(q) if flat_q else torch.empty((B, T, Hq, D), dtype=q.dtype, device=dev)
        gk = torch.empty_like(k) if flat_k else torch.empty((B, T, Hk, D), dtype=q.dtype, device=dev)
        flat = flat_q and flat_k
    else:
        gq, gk = out
        _typed(gq, "out[0]", q.dtype, q.shape, dev)
        _typed(gk, "out[1]", q.dtype, k.shape, dev)
        flat = flat_q and flat_k and gq.is_contiguous() and gk.is_contiguous()
    flat = flat and dq.is_contiguous() and dk.is_contiguous()
    gqw = None if q_weight is None else torch.empty_like(q_weight)
    gkw = None if k_weight is None else torch.empty_like(k_weight)
    if workspace is None:
        if gqw is not None or gkw is not None:
            nbytes = _ROPE_WORKSPACE.get(D)
            if nbytes is None:
                n = ctypes.c_size_t(0)
                _check(lib.kda_qk_norm_rope_workspace_bytes(D, ctypes.byref(n)))
                nbytes = _ROPE_WORKSPACE[D] = n.value
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    else:
        _want(workspace, "workspace", torch.uint8, workspace.shape, dev)
    strides = None if flat else _all_strides(("q", q), ("k", k), ("out[0]", gq), ("out[1]", gk), ("dq", dq), ("dk", dk))
    _call(lib.kda_qk_norm_rope_bwd, dev, dq.data_ptr(), dk.data_ptr(), q.data_ptr(), k.data_ptr(), _ROPE_TYPES[q.dtype],
          _p(q_weight), _p(k_weight), pos, freq, B * T, Hq, Hk, D, R, eps, 1 if interleaved else 0, strides,
          gq.data_ptr(), gk.data_ptr(), _p(gqw), _p(gkw), _p(workspace),
          0 if workspace is None else workspace.numel())
    if out is not None:
        _written((gq, gk))
    return gq, gk, gqw, gkw
