"""Refusals of the entry points for linear attention with a decay for each head and the norm and rotation
of its queries and keys, and their plain 64-bit form against differences: no GPU needed (the addresses
below are made up and never read; every refusal comes before any launch)."""

import ctypes
import math

import pytest
import torch

from decay_reference import norm_rope, scan

P = ctypes.c_void_p
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    from linear_attention_gated_gb300 import build as b
    b.build()
    from linear_attention_gated_gb300 import kda
    return kda.load_library()


def at(i):
    return (1 << 40) + i * (1 << 34)


def arr(values, kind=ctypes.c_int64):
    return None if values is None else (kind * len(values))(*values)


def ws_bytes(lib, B=1, T=64, hqk=2, hv=4, cu=None, training=1):
    n = ctypes.c_size_t(0)
    rc = lib.kda_decay_attn_workspace_bytes(B, T, hqk, hv, arr(cu), 0 if cu is None else len(cu) - 1, 1, training, ctypes.byref(n))
    return rc, n.value


def fwd(lib, B=1, T=64, hqk=2, hv=4, cu=None, cu_dev=0, per_token=1, head_dim=128, scale=NAN, strides=None, less=0, **at_):
    a = dict(q=at(0), k=at(1), v=at(2), g=at(3), h0=at(4), cu=at(5) if cu else None, o=at(6), hT=at(7), ws=at(8))
    a.update(at_)
    rc, n = ws_bytes(lib, max(B, 1), max(T, 0), 1, max(hv, 1))
    n = max(n, 1 << 30)
    rc = lib.kda_decay_attn_fwd(a["q"], a["k"], a["v"], a["g"], per_token, a["h0"], a["cu"], arr(cu),
                                0 if cu is None else len(cu) - 1, B, T, hqk, hv, head_dim, scale, arr(strides), a["o"],
                                a["hT"], a["ws"], 0 if less else n, None, None)
    return rc, lib.kda_last_error_message().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(hqk=0), 1), (dict(hqk=3, hv=4), 1),
    (dict(head_dim=64), 2), (dict(per_token=2), 1), (dict(scale=float("inf")), 1),
    (dict(q=None), 1), (dict(g=None), 1), (dict(o=None), 1), (dict(hT=None), 1),
    (dict(q=at(0) + 2), 1), (dict(h0=at(4) + 8), 1), (dict(ws=at(8) + 16), 1), (dict(less=1, hqk=2, hv=4), 7),
    (dict(cu=[0, 30, 60]), 1), (dict(cu=[1, 30, 64]), 1), (dict(cu=[0, 40, 30, 64]), 1), (dict(cu=[0]), 1),
    (dict(cu=[0, 64], B=2), 1), (dict(cu=[0, 64], cu_dev=1, o=at(0)), 3),
    (dict(o=at(2) + 1024), 3), (dict(hT=at(4)), 3), (dict(ws=at(6)), 3),
    (dict(strides=[256, 64, 256, 128, 512, 128]), 1),    # heads overlap
    (dict(strides=[128, 128, 256, 128, 512, 128]), 1),   # tokens overlap
    (dict(strides=[260, 128, 256, 128, 512, 128]), 1),   # not a multiple of 8
    (dict(T=1 << 41), 2), (dict(hv=1 << 21, hqk=1), 2),
])
def test_forward_refuses(lib, kw, status):
    rc, msg = fwd(lib, **kw)
    assert rc == status, (rc, msg)
    assert msg


def test_valid_forwards_reach_the_device_check(lib):
    for kw in (dict(), dict(cu=[0, 0, 64]), dict(cu=[0, 10, 10, 64]), dict(T=0, q=None, k=None, v=None, g=None, o=None), dict(h0=None),
               dict(strides=[1024, 128, 1024, 128, 1024, 128])):
        rc, msg = fwd(lib, **kw)
        assert rc in (2, 5) and ("sm_103a" in msg or "CUDA" in msg.upper()), (kw, rc, msg)


@pytest.mark.parametrize("kw,status", [
    (dict(dq=None), 1), (dict(dg=at(13), per_token=0), 2), (dict(dv=at(9)), 3), (dict(dh0=at(12)), 3), (dict(dq=at(10) + 2), 1),
    (dict(ws=None), 7), (dict(hT=None), 1), (dict(hT=at(15)), 3),
])
def test_backward_refuses(lib, kw, status):
    per_token = kw.pop("per_token", 1)
    a = dict(hT=at(17), do=at(9), dhT=at(14), dq=at(10), dk=at(11), dv=at(12), dg=at(13) if per_token else None, dh0=at(15), ws=at(16))
    a.update(kw)
    rc = lib.kda_decay_attn_bwd(at(0), at(1), at(2), at(3), per_token, at(4), None, None, 0, 1, 64, 2, 4, 128, NAN, None,
                                a["hT"], a["do"], a["dhT"], a["dq"], a["dk"], a["dv"], a["dg"], a["dh0"], a["ws"], 1 << 30, None, None)
    assert rc == status, lib.kda_last_error_message()


def slots_call(lib, what, host=(0, 1), slots=4, dtype=1, **kw):
    a = dict(state=at(5), idx=at(6), o=at(7))
    a.update(kw)
    h = arr(host, ctypes.c_int32)
    if what == "decode":
        return lib.kda_decay_attn_decode(at(0), at(1), at(2), at(3), 1, a["state"], dtype, a["idx"], h, slots, 2, 2, 4, 128, NAN,
                                         None, a["o"], None)
    return lib.kda_decay_attn_prefill(at(0), at(1), at(2), at(3), 1, None, None, 0, 2, 64, 2, 4, 128, NAN, None, a["state"], dtype,
                                      a["idx"], h, slots, a["o"], at(9), 1 << 30, None, None)


@pytest.mark.parametrize("what", ["decode", "prefill"])
@pytest.mark.parametrize("kw,status", [
    (dict(host=(0, 4)), 1), (dict(host=(-1, 0)), 1), (dict(host=(2, 2)), 1), (dict(host=None), 1), (dict(idx=None), 1),
    (dict(idx=None, host=None, slots=1), 1), (dict(dtype=2), 1), (dict(state=None), 1), (dict(state=at(5) + 4), 1),
    (dict(o=at(5)), 3), (dict(state=at(2)), 3), (dict(slots=1 << 33), 2), (dict(idx=at(5)), 3),
])
def test_pool_refusals(lib, what, kw, status):
    assert slots_call(lib, what, **kw) == status, lib.kda_last_error_message()


def test_valid_pool_calls_reach_the_device_check(lib):
    for what in ("decode", "prefill"):
        assert slots_call(lib, what) in (2, 5)
        assert "sm_103a" in lib.kda_last_error_message().decode() or "CUDA" in lib.kda_last_error_message().decode().upper()


def rope(lib, n=8, hq=4, hk=2, dim=128, rot=128, eps=1e-6, inter=0, dtype=0, strides=None, bwd=False, **kw):
    a = dict(q=at(0), k=at(1), qw=at(2), kw=at(3), pos=at(4), freq=at(5), qo=at(6), ko=at(7), dq=at(8), dk=at(9), dqw=at(10),
             dkw=at(11), ws=at(12), wsb=1 << 24)
    a.update(kw)
    if not bwd:
        return lib.kda_qk_norm_rope_fwd(a["q"], a["k"], dtype, a["qw"], a["kw"], a["pos"], a["freq"], n, hq, hk, dim, rot, eps, inter,
                                        arr(strides), a["qo"], a["ko"], None)
    return lib.kda_qk_norm_rope_bwd(a["dq"], a["dk"], a["q"], a["k"], dtype, a["qw"], a["kw"], a["pos"], a["freq"], n, hq, hk, dim,
                                    rot, eps, inter, arr(strides), a["qo"], a["ko"], a["dqw"], a["dkw"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(hq=0), 1), (dict(dim=72), 2), (dict(dim=272), 2), (dict(rot=24), 2), (dict(rot=144), 2),
    (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(inter=2), 1), (dict(dtype=3), 1), (dict(q=None), 1), (dict(pos=None), 1),
    (dict(freq=None), 1), (dict(q=at(0) + 8), 1), (dict(qo=at(0) + 256), 3), (dict(qo=at(1)), 3), (dict(ko=at(6)), 3),
    (dict(qo=at(4)), 3), (dict(n=1 << 41), 2),
    (dict(strides=[512, 64, 256, 128, 512, 128, 256, 128]), 1), (dict(strides=[516, 128, 256, 128, 512, 128, 256, 128]), 1),
    (dict(bwd=True, dqw=None), 1), (dict(bwd=True, ws=None), 1), (dict(bwd=True, wsb=64), 7), (dict(bwd=True, qo=at(9)), 3),
])
def test_rope_refuses(lib, kw, status):
    assert rope(lib, **kw) == status, lib.kda_last_error_message()


def test_valid_rope_calls_reach_the_device_check(lib):
    fused = [768, 128] * 2
    for kw in (dict(), dict(qo=at(0), ko=at(1)), dict(rot=0, pos=None, freq=None), dict(qw=None), dict(n=0, q=None),
               dict(k=at(0) + 4 * 128 * 2, qo=at(0), ko=at(0) + 4 * 128 * 2, strides=fused * 2), dict(bwd=True),
               dict(bwd=True, qo=at(8), ko=at(9))):
        assert rope(lib, **kw) in (2, 5), (kw, lib.kda_last_error_message())


def test_python_checks():
    from linear_attention_gated_gb300 import kda_decay_attn_decode, kda_decay_attn_fwd, kda_qk_norm_rope_fwd
    q = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    g = torch.zeros(2)
    with pytest.raises(TypeError):
        kda_decay_attn_fwd(q.float(), q, q, g)
    with pytest.raises(ValueError):
        kda_decay_attn_fwd(q, q[:, :3], q, g)
    with pytest.raises(TypeError):
        kda_decay_attn_fwd(q, q, q, torch.zeros(1, 4, 2))  # per token decays are BF16
    with pytest.raises(ValueError):
        kda_decay_attn_fwd(q, q, q, g, cu_seqlens=torch.tensor([0, 4]))  # no mirror
    with pytest.raises(ValueError):
        kda_decay_attn_fwd(q.transpose(1, 2).contiguous().transpose(1, 2).transpose(2, 3), q, q, g)
    with pytest.raises(ValueError):
        kda_decay_attn_fwd(q, q, q, g)  # CPU tensors
    with pytest.raises(ValueError):
        kda_decay_attn_decode(q, q, q, g, torch.zeros(1, 2, 128, 128))  # four tokens
    with pytest.raises(TypeError):
        kda_qk_norm_rope_fwd(q.double(), q.double(), None, None, None, None)
    with pytest.raises(ValueError):
        kda_qk_norm_rope_fwd(q, q, None, None, torch.zeros(1, 3, dtype=torch.int64), torch.zeros(8, dtype=torch.float64))


def test_plain_forms_against_differences():
    """Autograd of the plain forms, which the GPU's gradients are held to, against central differences."""
    gen = torch.Generator().manual_seed(0)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64)

    leaves = [rnd(5, 1, 128), rnd(5, 1, 128), rnd(5, 2, 128), -rnd(5, 2).abs(), rnd(2, 2, 128, 128)]
    do, dh = rnd(5, 2, 128), rnd(2, 2, 128, 128)

    def loss(*x):
        o, h = scan(*x, [(0, 3), (3, 5)], 1 / math.sqrt(128))
        return (o * do).sum() + (h * dh).sum()

    def rope_loss(x, w):
        return (norm_rope(x, w, torch.arange(3).reshape(1, 3) * 1000, torch.tensor([1.0, 0.1, 0.01], dtype=torch.float64), 1e-6,
                          True) * rdo).sum()

    rdo = rnd(1, 3, 2, 16)
    for f, xs in ((loss, leaves), (rope_loss, [rnd(1, 3, 2, 16), rnd(16)])):
        xs = [x.requires_grad_() for x in xs]
        grads = torch.autograd.grad(f(*xs), xs)
        with torch.no_grad():
            for i, gr in enumerate(grads):
                step = rnd(*gr.shape)
                e = 1e-5
                up, down = ([x + (s * e * step if j == i else 0) for j, x in enumerate(xs)] for s in (1, -1))
                want = (f(*up) - f(*down)) / (2 * e)
                assert abs((gr * step).sum() - want) <= 1e-6 * (gr * step).norm().clamp_min(1.0)
