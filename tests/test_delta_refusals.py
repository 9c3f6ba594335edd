"""Refusals of the entry points of the gated delta rule and of layer norm, and their plain 64-bit forms against differences:
no GPU needed (the addresses are made up and never read; every refusal comes before any launch)."""

import ctypes
import math

import pytest
import torch

from delta_reference import delta_scan, layer_norm
from test_decay_refusals import NAN, arr, at, lib  # noqa: F401

W = 256  # a width


def fwd(lib, B=1, T=64, hqk=2, hv=4, cu=None, head_dim=128, scale=NAN, strides=None, less=0, **kw):  # noqa: F811
    a = dict(q=at(0), k=at(1), v=at(2), g=at(3), beta=at(9), h0=at(4), cu=at(5) if cu else None, o=at(6), hT=at(7), ws=at(8))
    a.update(kw)
    rc = lib.kda_gated_delta_fwd(a["q"], a["k"], a["v"], a["g"], a["beta"], a["h0"], a["cu"], arr(cu), 0 if cu is None else len(cu) - 1,
                                 B, T, hqk, hv, head_dim, scale, arr(strides), a["o"], a["hT"], a["ws"], 0 if less else 1 << 30, None, None)
    return rc, lib.kda_last_error_message().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(B=0), 1), (dict(T=-1), 1), (dict(hqk=0), 1), (dict(hqk=3, hv=4), 1), (dict(head_dim=64), 2), (dict(scale=float("inf")), 1),
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(beta=None), 1), (dict(o=None), 1), (dict(hT=None), 1),
    (dict(q=at(0) + 2), 1), (dict(h0=at(4) + 8), 1), (dict(o=at(6) + 8), 1), (dict(ws=at(8) + 16), 1), (dict(less=1), 7), (dict(ws=None), 7),
    (dict(cu=[0, 30, 60]), 1), (dict(cu=[1, 30, 64]), 1), (dict(cu=[0, 40, 30, 64]), 1), (dict(cu=[0]), 1), (dict(cu=[0, 64], B=2), 1),
    (dict(cu=[0, 64], o=at(0)), 3), (dict(cu=[0, 64], hT=at(5)), 3),
    (dict(o=at(2) + 1024), 3), (dict(hT=at(4)), 3), (dict(ws=at(6)), 3), (dict(o=at(9)), 3), (dict(ws=at(9) - 256), 3), (dict(hT=at(3)), 3),
    (dict(strides=[256, 64, 256, 128, 512, 128]), 1),    # heads overlap
    (dict(strides=[128, 128, 256, 128, 512, 128]), 1),   # tokens overlap
    (dict(strides=[260, 128, 256, 128, 512, 128]), 1),   # not a multiple of 8
    (dict(T=1 << 41), 2), (dict(T=1 << 31), 2), (dict(hv=1 << 21, hqk=1), 2), (dict(T=1 << 30, hv=1 << 9, hqk=1), 2),
    (dict(strides=[256, 128, 256, 128, 1 << 50, 128]), 2),
])
def test_forward_refuses(lib, kw, status):  # noqa: F811
    rc, msg = fwd(lib, **kw)
    assert rc == status, (rc, msg)
    assert msg


def test_valid_forwards_reach_the_device_check(lib):  # noqa: F811
    for kw in (dict(), dict(g=None), dict(cu=[0, 0, 64]), dict(cu=[0, 10, 10, 64]), dict(h0=None),
               dict(T=0, q=None, k=None, v=None, g=None, beta=None, o=None, ws=None), dict(strides=[1024, 128, 1024, 128, 1024, 128])):
        rc, msg = fwd(lib, **kw)
        assert rc in (2, 5) and ("sm_103a" in msg or "CUDA" in msg.upper()), (kw, rc, msg)


@pytest.mark.parametrize("kw,status", [
    (dict(dq=None), 1), (dict(dk=None), 1), (dict(dv=None), 1), (dict(db=None), 1), (dict(do=None), 1), (dict(g=None), 1),
    (dict(dv=at(9)), 3), (dict(dh0=at(12)), 3), (dict(dk=at(10)), 3), (dict(db=at(13)), 3), (dict(db=at(18)), 3), (dict(dg=at(3)), 3),
    (dict(ws=at(14)), 3), (dict(dh0=at(14)), 3), (dict(dq=at(10) + 2), 1), (dict(dh0=at(15) + 4), 1), (dict(ws=None), 7), (dict(wsb=4096), 7),
])
def test_backward_refuses(lib, kw, status):  # noqa: F811
    a = dict(g=at(3), do=at(9), dhT=at(14), dq=at(10), dk=at(11), dv=at(12), dg=at(13), db=at(17), dh0=at(15), ws=at(16), wsb=1 << 30)
    a.update(kw)
    rc = lib.kda_gated_delta_bwd(at(0), at(1), at(2), a["g"], at(18), None, None, 0, 1, 64, 2, 4, 128, NAN, None, a["do"], a["dhT"],
                                 a["dq"], a["dk"], a["dv"], a["dg"], a["db"], a["dh0"], a["ws"], a["wsb"], None, None)
    assert rc == status, lib.kda_last_error_message()


def slots_call(lib, what, host=(0, 1), slots=4, dtype=1, **kw):  # noqa: F811
    a = dict(state=at(5), idx=at(6), o=at(7), beta=at(10), g=at(3))
    a.update(kw)
    h = arr(host, ctypes.c_int32)
    if what == "decode":
        return lib.kda_gated_delta_decode(at(0), at(1), at(2), a["g"], a["beta"], a["state"], dtype, a["idx"], h, slots, 2, 2, 4, 128, NAN,
                                          None, a["o"], None)
    return lib.kda_gated_delta_prefill(at(0), at(1), at(2), a["g"], a["beta"], None, None, 0, 2, 64, 2, 4, 128, NAN, None, a["state"],
                                       dtype, a["idx"], h, slots, a["o"], at(9), 1 << 30, None, None)


@pytest.mark.parametrize("what", ["decode", "prefill"])
@pytest.mark.parametrize("kw,status", [
    (dict(host=(0, 4)), 1), (dict(host=(-1, 0)), 1), (dict(host=(2, 2)), 1), (dict(host=None), 1), (dict(idx=None), 1),
    (dict(idx=None, host=None, slots=1), 1), (dict(dtype=2), 1), (dict(state=None), 1), (dict(state=at(5) + 4), 1), (dict(beta=None), 1),
    (dict(o=at(5)), 3), (dict(state=at(2)), 3), (dict(slots=1 << 33), 2), (dict(idx=at(5)), 3), (dict(o=at(10)), 3), (dict(o=at(3)), 3),
    (dict(o=at(7) + 8), 1),
])
def test_pool_refusals(lib, what, kw, status):  # noqa: F811
    assert slots_call(lib, what, **kw) == status, lib.kda_last_error_message()


def test_valid_pool_calls_reach_the_device_check(lib):  # noqa: F811
    for what in ("decode", "prefill"):
        for kw in (dict(), dict(g=None), dict(dtype=0), dict(idx=None, host=None)):
            assert slots_call(lib, what, **kw) in (2, 5)
            msg = lib.kda_last_error_message().decode()
            assert "sm_103a" in msg or "CUDA" in msg.upper()


def ws_bytes(lib, B=1, T=64, hqk=2, hv=4, cu=None, training=1):  # noqa: F811
    n = ctypes.c_size_t(0)
    rc = lib.kda_gated_delta_workspace_bytes(B, T, hqk, hv, arr(cu), 0 if cu is None else len(cu) - 1, training, ctypes.byref(n))
    return rc, n.value


def test_workspace_sizes(lib):  # noqa: F811
    chunk, trained = 26 << 10, (26 << 10) + (8 << 10) + (32 << 10) * 2 + (16 << 10)  # bytes of a (chunk, head)
    for hv in (1, 4, 96):
        for T in (1, 63, 64, 65, 1000):
            places = (T // 64 + 1) * hv
            assert places * chunk <= ws_bytes(lib, T=T, hqk=1, hv=hv, training=0)[1] < places * chunk + 1024
            assert places * trained <= ws_bytes(lib, T=T, hqk=1, hv=hv)[1] < places * trained + 1024
    assert ws_bytes(lib, T=0) == (0, 0) and ws_bytes(lib, cu=[0, 0], T=0) == (0, 0)
    assert ws_bytes(lib, T=-1)[0] == 1 and ws_bytes(lib, hv=3)[0] == 1 and ws_bytes(lib, T=1 << 31)[0] == 2
    assert lib.kda_gated_delta_workspace_bytes(1, 64, 1, 1, None, 0, 1, None) == 1
    # a long sequence of one head is cut, its states are kept; so is one among short ones
    for cu in (None, [0, 1, 32001]):
        n = ws_bytes(lib, T=32001, hqk=1, hv=1, cu=cu, training=0)[1]
        assert n > 502 * chunk + 2 * 8 * 65536


def norm(lib, rows=8, width=W, stride=None, eps=1e-5, dtype=0, bwd=False, dys=None, **kw):  # noqa: F811
    a = dict(x=at(0), w=at(1), b=at(2), y=at(3), mean=at(4), rstd=at(5), dy=at(6), dx=at(7), dw=at(8), db=at(9), ws=at(10), wsb=1 << 24)
    a.update(kw)
    s = width if stride is None else stride
    if not bwd:
        return lib.kda_layer_norm_fwd(a["x"], dtype, a["w"], a["b"], rows, width, s, eps, a["y"], a["mean"], a["rstd"], None)
    return lib.kda_layer_norm_bwd(a["dy"], a["x"], dtype, a["w"], a["mean"], a["rstd"], rows, width, width if dys is None else dys, s,
                                  a["dx"], a["dw"], a["db"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(width=0), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(eps=-1.0), 1), (dict(eps=NAN), 1),
    (dict(eps=float("inf")), 1), (dict(x=None), 1), (dict(y=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1), (dict(stride=W - 1), 1),
    (dict(x=at(0) + 1), 1), (dict(w=at(1) + 2), 1), (dict(mean=at(4) + 2), 1),
    (dict(width=(1 << 24) + 1), 2), (dict(rows=1 << 31), 2), (dict(rows=1 << 30, width=1 << 11), 2), (dict(stride=1 << 60), 2),
    (dict(y=at(0) + 2), 3), (dict(y=at(0), stride=W + 8), 3), (dict(y=at(1)), 3), (dict(mean=at(0)), 3), (dict(rstd=at(4)), 3),
    (dict(mean=at(3)), 3), (dict(rstd=at(2) + 4), 3),
    (dict(bwd=True, dys=W - 1), 1), (dict(bwd=True, dy=None), 1), (dict(bwd=True, dx=None), 1), (dict(bwd=True, mean=None), 1),
    (dict(bwd=True, ws=None), 7), (dict(bwd=True, wsb=8 * 8 * W - 1), 7), (dict(bwd=True, dx=at(6), dys=2 * W), 3),
    (dict(bwd=True, dx=at(0), stride=2 * W), 3), (dict(bwd=True, dx=at(0), width=12296, wsb=1 << 30), 3),
    (dict(bwd=True, dx=at(6), width=8200, dtype=1, wsb=1 << 30), 3), (dict(bwd=True, dw=at(0)), 3), (dict(bwd=True, db=at(6)), 3),
    (dict(bwd=True, dw=at(1)), 3), (dict(bwd=True, db=at(8)), 3), (dict(bwd=True, ws=at(7)), 3), (dict(bwd=True, ws=at(5)), 3),
    (dict(bwd=True, dx=at(0) + 2 * W), 3), (dict(bwd=True, ws=at(10) + 2), 1), (dict(bwd=True, dw=at(8) + 1), 1),
])
def test_layer_norm_refuses(lib, kw, status):  # noqa: F811
    assert norm(lib, **kw) == status, lib.kda_last_error_message()


def test_valid_layer_norms_reach_the_device_check(lib):  # noqa: F811
    for kw in (dict(), dict(y=at(0)), dict(w=None, b=None), dict(rows=0, x=None, y=None, mean=None, rstd=None), dict(stride=4 * W),
               dict(width=1), dict(eps=0.0), dict(bwd=True), dict(bwd=True, dx=at(6)), dict(bwd=True, dx=at(0)),
               dict(bwd=True, dw=None, db=None, ws=None, wsb=0), dict(bwd=True, w=None, dw=None), dict(bwd=True, rows=0, ws=None, wsb=0)):
        assert norm(lib, **kw) in (2, 5), (kw, lib.kda_last_error_message())


def test_layer_norm_workspace(lib):  # noqa: F811
    n = ctypes.c_size_t(0)
    assert lib.kda_layer_norm_workspace_bytes(5, 100, ctypes.byref(n)) == 0 and n.value == 8 * 5 * 100
    assert lib.kda_layer_norm_workspace_bytes(1 << 20, 100, ctypes.byref(n)) == 0 and n.value == 8 * 152 * 100
    assert lib.kda_layer_norm_workspace_bytes(0, 100, ctypes.byref(n)) == 0 and n.value == 0
    assert lib.kda_layer_norm_workspace_bytes(5, 0, ctypes.byref(n)) == 1
    assert lib.kda_layer_norm_workspace_bytes(5, 100, None) == 1


def test_python_checks():
    import linear_attention_gated_gb300 as m
    q = torch.zeros(1, 4, 2, 128, dtype=torch.bfloat16)
    g = torch.zeros(1, 4, 2, dtype=torch.bfloat16)
    cases = [
        (TypeError, lambda: m.kda_gated_delta_fwd(q.float(), q, q, g, g)), (ValueError, lambda: m.kda_gated_delta_fwd(q, q[:, :3], q, g, g)),
        (TypeError, lambda: m.kda_gated_delta_fwd(q, q, q, g.float(), g)), (TypeError, lambda: m.kda_gated_delta_fwd(q, q, q, g, g.float())),
        (ValueError, lambda: m.kda_gated_delta_fwd(q, q, q, g[:, :3], g)), (ValueError, lambda: m.kda_gated_delta_fwd(q, q, q, None, g[..., :1])),
        (ValueError, lambda: m.kda_gated_delta_fwd(q, q, q, g, g, cu_seqlens=torch.tensor([0, 4]))),  # no mirror
        (ValueError, lambda: m.kda_gated_delta_fwd(q, q, q, g, g)),  # CPU tensors
        (ValueError, lambda: m.kda_gated_delta_decode(q, q, q, g, g, torch.zeros(1, 2, 128, 128))),  # four tokens
        (m.KdaError, lambda: m.kda_gated_delta_bwd(None, q)),
        (TypeError, lambda: m.kda_layer_norm_fwd(q.double())), (ValueError, lambda: m.kda_layer_norm_fwd(q, torch.zeros(127))),
        (TypeError, lambda: m.kda_layer_norm_fwd(q, torch.zeros(128, dtype=torch.bfloat16))), (ValueError, lambda: m.kda_layer_norm_fwd(q.transpose(2, 3))),
        (ValueError, lambda: m.kda_layer_norm_fwd(q[:, :, :, ::2])), (ValueError, lambda: m.kda_layer_norm_fwd(q[..., :0])),
        (ValueError, lambda: m.kda_layer_norm_fwd(q[0, ::3, :, :])),  # rows that are not evenly apart
        (ValueError, lambda: m.kda_layer_norm_bwd(q[:, :2], q, None, torch.zeros(1, 4, 2), torch.zeros(1, 4, 2))),
        (ValueError, lambda: m.kda_layer_norm_bwd(q, q, None, torch.zeros(1, 4), torch.zeros(1, 4, 2))),
    ]
    for i, (error, call) in enumerate(cases):
        with pytest.raises(error):
            call()
            pytest.fail(f"case {i} was not refused")


def test_plain_forms_against_differences():
    """Autograd of the plain forms, which the GPU's gradients are held to, against central differences."""
    gen = torch.Generator().manual_seed(0)

    def rnd(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64)

    def unit(x):
        return x / x.norm(dim=-1, keepdim=True)

    leaves = [rnd(6, 1, 128), unit(rnd(6, 1, 128)), rnd(6, 2, 128), -rnd(6, 2).abs(), torch.sigmoid(rnd(6, 2)), rnd(2, 2, 128, 128)]
    do, dh, dy = rnd(6, 2, 128), rnd(2, 2, 128, 128), rnd(3, 50)

    def loss(*x):
        o, h = delta_scan(*x, [(0, 2), (2, 6)], 1 / math.sqrt(128))
        return (o * do).sum() + (h * dh).sum()

    def norm_loss(x, w, b):
        return (layer_norm(x, w, b, 1e-3)[0] * dy).sum()

    for f, xs in ((loss, leaves), (norm_loss, [rnd(3, 50), rnd(50), rnd(50)])):
        xs = [x.requires_grad_() for x in xs]
        grads = torch.autograd.grad(f(*xs), xs)
        with torch.no_grad():
            for i, gr in enumerate(grads):
                step, e = rnd(*gr.shape), 1e-5
                up, down = ([x + (s * e * step if j == i else 0) for j, x in enumerate(xs)] for s in (1, -1))
                want = (f(*up) - f(*down)) / (2 * e)
                assert abs((gr * step).sum() - want) <= 1e-6 * (gr * step).norm().clamp_min(1.0)
