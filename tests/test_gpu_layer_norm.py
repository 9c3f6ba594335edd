"""Layer norm and its gradients, on the GPU, against the formula in 64 bits.

Tolerances. Outputs of 16 bits are rounded once, from FP32 values: half a step of their own, and eight FP32 steps (2^-24
relative to the largest factor of a product) for the mean, the deviation, the norm, weight and bias. FP32 ones: a sum of n
terms in any order of the threads' and warps' partial sums is off by at most (n_s + 8) 2^-24 of the terms' absolute
sum, n_s the longest chain of additions: 32 within a thread, 5 in a warp, 16 over warps; over rows, one a row of a CTA.
"""

import pytest
import torch

from decay_reference import BF16, FP16, FP32
from delta_reference import layer_norm

pytestmark = pytest.mark.gpu

STEP = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_attention_gated_gb300 import build
    build.build()
    from linear_attention_gated_gb300 import kda
    kda.load_library()


def make(shape, dtype, seed, wide=0, offset=0, shift=0.5, affine="both"):
    gen = torch.Generator("cuda").manual_seed(seed)
    def randn(*s):
        return torch.randn(s, generator=gen, device="cuda")
    width = shape[-1]
    x = (randn(*shape[:-1], width + wide + offset) + shift * randn(*shape[:-1], 1)).to(dtype)[..., offset:offset + width]
    w = 1 + 0.2 * randn(width) if affine != "none" else None
    b = 0.2 * randn(width) if affine == "both" else None
    return x, w, b, randn(*shape).to(dtype)


def check_all(x, w, b, dy, out=None, eps=EPS):
    from linear_attention_gated_gb300 import kda_layer_norm_bwd, kda_layer_norm_fwd
    y, mean, rstd = kda_layer_norm_fwd(x, w, b, eps)
    dx, dw, db = kda_layer_norm_bwd(dy, x, w, mean, rstd, bias=b is not None)
    torch.cuda.synchronize()
    leaves = [t.double().detach().clone().requires_grad_() for t in (x, w, b) if t is not None]
    args = iter(leaves)
    xd = next(args)
    ry, rm, rr = layer_norm(xd, None if w is None else next(args), None if b is None else next(args), eps)
    grads = iter(torch.autograd.grad(ry, leaves, dy.double()) if x.numel() else [torch.zeros_like(t) for t in leaves])
    width, step = x.shape[-1], STEP[x.dtype]
    size = x.double().abs().amax(-1) if x.numel() else rm
    sum_error = (32 + 5 + 16 + 8) * FP32
    assert ((mean - rm).abs() <= sum_error * x.double().abs().mean(-1) + 2 * FP32 * size).all()
    # the deviation: two errors of the mean and one of the sum of squares, half of it for the root
    assert ((rstd - rr).abs() <= rr * (sum_error + 8 * FP32 + 4 * FP32 * (size * rr) ** 2)).all()
    wd = 1.0 if w is None else w.double().abs()
    n = ((x.double() - rm[..., None]) * rr[..., None]).abs()
    scale = n * wd + (0 if b is None else b.double().abs()) + (size * rr)[..., None] * wd
    off = (y.double() - ry).abs()
    assert (off <= step * ry.abs() + (sum_error + 8 * FP32) * scale + (2.0 ** -25 if x.dtype == torch.float16 else 0)).all(), (off / (step * scale)).max()
    rdx = next(grads)
    t = dy.double().abs() * wd
    parts = rr[..., None] * (t + t.mean(-1, keepdim=True) + n * (t * n).mean(-1, keepdim=True))
    off = (dx.double() - rdx).abs()
    assert (off <= step * rdx.abs() + (2 * sum_error + 16 * FP32) * parts * (1 + (size * rr)[..., None]) + (2.0 ** -25 if x.dtype == torch.float16 else 0)).all()
    rows = x.numel() // width
    per = -(-rows // 152) + 64 + 8 + 8  # additions in a CTA, then over CTAs' parts
    flat = (lambda z: z.reshape(-1, width))
    if w is not None:
        bar = (per * FP32 + sum_error) * (flat(dy.double().abs()) * (flat(n) + (size * rr).reshape(-1, 1))).sum(0)
        assert ((dw - next(grads)).abs() <= bar + 1e-30).all()
    if b is not None:
        assert ((db - next(grads)).abs() <= per * FP32 * flat(dy.double().abs()).sum(0) + 1e-30).all()
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("rows,width", [(1, 1), (3, 7), (5, 128), (33, 129), (70, 512), (9, 1001), (200, 2048), (3, 4095), (40, 4096),
                                        (7, 8192), (5, 8200), (4, 12288), (3, 12296), (2, 16384), (3, 16400), (1, 40001)])
def test_sizes(dtype, rows, width):
    check_all(*make((rows, width), TYPES[dtype], seed=rows + width))


@pytest.mark.parametrize("affine", ["weight", "none"])
@pytest.mark.parametrize("width", [96, 1000, 20000])
def test_without_weight_or_bias(affine, width):
    got = check_all(*make((17, width), torch.bfloat16, seed=1, affine=affine))
    assert (got[4] is None) == (affine == "none") and got[5] is None


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("wide,offset", [(64, 0), (5, 0), (64, 8), (3, 1)])
def test_columns_of_a_wider_tensor(dtype, wide, offset):
    check_all(*make((4, 11, 264), TYPES[dtype], seed=2, wide=wide, offset=offset))


def test_many_rows():
    check_all(*make((40000, 64), torch.bfloat16, seed=3))
    check_all(*make((8192, 1024), torch.float16, seed=4))


def test_far_mean_and_constant_rows():
    """A mean a thousand times the deviation, and rows without any (rstd = 1 / sqrt(eps), y = bias)."""
    x, w, b, dy = make((32, 1024), torch.float32, seed=5)
    check_all(x + 1000.0, w, b, dy)
    x[3] = 2.0
    y, _, rstd, *_ = check_all(x, w, b, dy)
    assert torch.equal(y[3], b) and abs(rstd[3].item() * EPS ** 0.5 - 1) < 4 * FP32


@pytest.mark.parametrize("width", [64, 1000, 12288])
def test_outputs_over_inputs(width):
    from linear_attention_gated_gb300 import kda_layer_norm_bwd, kda_layer_norm_fwd
    x, w, b, dy = make((300, width), torch.bfloat16, seed=6)
    y, mean, rstd = kda_layer_norm_fwd(x, w, b)
    dx, dw, db = kda_layer_norm_bwd(dy, x, w, mean, rstd)
    for over in ("dy", "x"):
        xi, di = x.clone(), dy.clone()
        got = kda_layer_norm_bwd(di, xi, w, mean, rstd, out=di if over == "dy" else xi)
        assert all(torch.equal(a, c) for a, c in zip(got, (dx, dw, db)))
    xi = x.clone()
    assert torch.equal(kda_layer_norm_fwd(xi, w, b, out=xi)[0], y) and torch.equal(xi, y)


def test_no_rows():
    got = check_all(*make((0, 64), torch.bfloat16, seed=7))
    assert got[0].shape == (0, 64) and not got[4].any() and not got[5].any()


def test_bad_values_stay_in_their_row():
    from linear_attention_gated_gb300 import kda_layer_norm_bwd, kda_layer_norm_fwd
    x, w, b, dy = make((64, 96), torch.bfloat16, seed=8)
    good = kda_layer_norm_fwd(x, w, b)[0].clone()
    x[5, 7], x[9, 0] = float("nan"), float("inf")
    y, mean, rstd = kda_layer_norm_fwd(x, w, b)
    keep = [i for i in range(64) if i not in (5, 9)]
    assert torch.equal(y[keep], good[keep]) and y[5].isnan().all() and y[9].isnan().all()
    dx = kda_layer_norm_bwd(dy, x, w, mean, rstd)[0]
    assert dx[keep].isfinite().all()


def test_captured_and_on_another_stream():
    from linear_attention_gated_gb300 import kda_layer_norm_bwd, kda_layer_norm_fwd
    x, w, b, dy = make((100, 1024), torch.bfloat16, seed=9)
    want = kda_layer_norm_fwd(x, w, b)
    wantg = kda_layer_norm_bwd(dy, x, w, want[1], want[2])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    xs = torch.zeros_like(x)
    with torch.cuda.graph(g, stream=s):
        got = kda_layer_norm_fwd(xs, w, b)
        gotg = kda_layer_norm_bwd(dy, xs, w, got[1], got[2])
    xs.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(got + gotg, want + wantg))


def test_rows_past_32_bit_offsets():
    """The last 100 rows of a tensor of 4 GiB, as alone."""
    from linear_attention_gated_gb300 import kda_layer_norm_bwd, kda_layer_norm_fwd
    width, before = 4096, 2 ** 31 // 4096 + 7
    x, w, b, dy = make((100, width), torch.bfloat16, seed=10)
    big, bigd = (torch.zeros(before + 100, width, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    big[before:], bigd[before:] = x, dy
    y, mean, rstd = kda_layer_norm_fwd(big, w, b)
    want = kda_layer_norm_fwd(x, w, b)
    for got, alone in zip((y, mean, rstd), want):
        assert torch.equal(got[before:], alone)
    assert torch.equal(y[:before:997], b.bfloat16().expand(y[:before:997].shape))
    dx = kda_layer_norm_bwd(bigd, big, w, mean, rstd)[0]
    assert torch.equal(dx[before:], kda_layer_norm_bwd(dy, x, w, *want[1:])[0]) and not dx[:before].any()


@pytest.mark.parametrize("width,dtype", [(96, torch.bfloat16), (4096, torch.bfloat16), (1001, torch.float32), (12296, torch.bfloat16)], ids=str)
def test_a_workspace_of_the_caller(width, dtype):
    """Of the documented size, used for two numbers of rows in turn (fewer and more than there are SMs): what it held does not
    matter, and what lies behind it stays."""
    import ctypes

    from linear_attention_gated_gb300 import KdaError, kda_layer_norm_bwd, kda_layer_norm_fwd
    from linear_attention_gated_gb300.kda import load_library

    def need(rows):
        n = ctypes.c_size_t(0)
        assert load_library().kda_layer_norm_workspace_bytes(rows, width, ctypes.byref(n)) == 0
        return n.value

    room = torch.full((need(700) + 4096,), 255, dtype=torch.uint8, device="cuda")
    for rows in (700, 5, 151, 153, 700):
        x, w, b, dy = make((rows, width), dtype, seed=rows)
        _, mean, rstd = kda_layer_norm_fwd(x, w, b)
        want = kda_layer_norm_bwd(dy, x, w, mean, rstd)
        got = kda_layer_norm_bwd(dy, x, w, mean, rstd, workspace=room[:need(rows)])
        assert all(torch.equal(a, c) for a, c in zip(got, want)), rows
        assert (room[need(700):] == 255).all()
        with pytest.raises(KdaError):
            kda_layer_norm_bwd(dy, x, w, mean, rstd, workspace=room[:need(rows) - 1])
