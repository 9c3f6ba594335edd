"""Norm and position rotation of queries and keys, on the GPU, against 64 bits.

Tolerances: FP32 arithmetic (a dozen roundings and a sum of D squares, 16 * 2^-24 relative) and one
rounding to the type: values are off by half a step of their own, and a value that the rotation cancels
by FP32 errors of its pair's size. Relative L2: half a step / sqrt(3) at most from the rounding.
"""

import math

import pytest
import torch

from decay_reference import BF16, FP16, FP32, norm_rope, rel_l2

pytestmark = pytest.mark.gpu

STEP = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_attention_gated_gb300 import build
    build.build()
    from linear_attention_gated_gb300 import kda
    kda.load_library()


def make(B, T, hq, hk, dim, rot, dtype, seed, far=0):
    gen = torch.Generator().manual_seed(seed)
    x = {n: torch.randn(B, T, h, dim, generator=gen).to(dtype) for n, h in (("q", hq), ("k", hk), ("dq", hq), ("dk", hk))}
    x["qw"], x["kw"] = (1 + 0.2 * torch.randn(dim, generator=gen) for _ in range(2))
    x["pos"] = torch.randint(0, far + 1, (B, 1), generator=gen) + torch.arange(T)
    x["freq"] = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2)) if rot else None
    return x


def reference(x, interleaved, eps=1e-6, weights=True):
    out = {}
    for n in ("q", "k"):
        v = x[n].double().requires_grad_()
        w = x[n + "w"].double().requires_grad_() if weights else None
        y = norm_rope(v, w, x["pos"], x["freq"], eps, interleaved)
        gr = torch.autograd.grad((y * x["d" + n].double()).sum(), [v] + ([w] if weights else []), allow_unused=True)
        out[n], out["d" + n] = y.detach(), gr[0]
        out["d" + n + "w"] = gr[1] if weights else None
    return out


def check(name, got, ref, dtype):
    got, ref = got.cpu().double(), ref.double()
    assert got.shape == ref.shape and torch.isfinite(got).all(), name
    row = ref.square().mean(-1, keepdim=True).sqrt()
    off = (got - ref).abs()
    bad = off > STEP[dtype] * ref.abs() + 64 * FP32 * torch.maximum(row, ref.abs()) * 4
    assert not bad.any(), (name, int(bad.sum()), off.max().item())
    assert rel_l2(got, ref) <= STEP[dtype] / math.sqrt(3) + 32 * FP32, name


def run(x, interleaved, weights=True, eps=1e-6):
    from linear_attention_gated_gb300 import kda_qk_norm_rope_bwd, kda_qk_norm_rope_fwd
    d = {n: t.cuda() if t is not None else None for n, t in x.items()}
    w = (d["qw"], d["kw"]) if weights else (None, None)
    q, k = kda_qk_norm_rope_fwd(d["q"], d["k"], *w, d["pos"], d["freq"], eps, interleaved)
    g = kda_qk_norm_rope_bwd(d["dq"], d["dk"], d["q"], d["k"], *w, d["pos"], d["freq"], eps, interleaved)
    return dict(zip(("q", "k", "dq", "dk", "dqw", "dkw"), (q, k) + g))


def compare(got, ref, dtype, rows):
    for n in ("q", "k", "dq", "dk"):
        assert got[n].dtype == dtype
        check(n, got[n], ref[n], dtype)
    for n in ("dqw", "dkw"):
        assert (got[n] is None) == (ref[n] is None)
        if got[n] is not None:  # a sum of `rows` products, added in at most a hundred steps of FP32
            assert rel_l2(got[n], ref[n]) <= 128 * FP32, n


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32], ids=str)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 64), (64, 64), (96, 48), (192, 96), (256, 256), (80, 16), (16, 16), (48, 0)])
def test_types_and_widths(dtype, interleaved, dim, rot):
    x = make(2, 7, 5, 2, dim, rot, dtype, seed=dim + rot)
    compare(run(x, interleaved), reference(x, interleaved), dtype, 70)


@pytest.mark.parametrize("B,T,hq,hk", [(1, 1, 1, 1), (3, 1, 64, 8), (1, 65, 1, 3), (1, 333, 17, 96), (2, 1000, 8, 1)])
def test_shapes(B, T, hq, hk):
    x = make(B, T, hq, hk, 128, 128, torch.bfloat16, seed=T)
    compare(run(x, False), reference(x, False), torch.bfloat16, B * T * max(hq, hk))


@pytest.mark.parametrize("far", [100_000, 10_000_000, 2**40])
def test_far_positions(far):
    """The 64-bit reference itself is off by far * 2^-53 radians of its angle."""
    x = make(4, 3, 2, 2, 64, 64, torch.float32, seed=1, far=far)
    from linear_attention_gated_gb300 import kda_qk_norm_rope_fwd
    d = {n: t.cuda() for n, t in x.items()}
    q, _ = kda_qk_norm_rope_fwd(d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["freq"])
    assert rel_l2(q, reference(x, False)["q"]) <= 32 * FP32 + 4 * far * 2.0 ** -53


def test_negative_positions_and_no_weights():
    x = make(2, 9, 3, 3, 64, 32, torch.bfloat16, seed=2)
    x["pos"] -= 5
    compare(run(x, True, weights=False), reference(x, True, weights=False), torch.bfloat16, 54)


def test_zero_rows_and_eps():
    x = make(1, 5, 2, 2, 64, 64, torch.float32, seed=3)
    x["q"][:, 2] = 0
    got, ref = run(x, False, eps=1e-2), reference(x, False, eps=1e-2)
    assert (got["q"][:, 2] == 0).all()
    compare(got, ref, torch.float32, 10)


def test_views_in_place_and_empty():
    from linear_attention_gated_gb300 import KdaError, kda_qk_norm_rope_bwd, kda_qk_norm_rope_fwd
    x = make(2, 33, 6, 2, 128, 128, torch.bfloat16, seed=4)
    want = run(x, False)
    d = {n: t.cuda() for n, t in x.items()}
    fused = torch.cat([d["q"], d["k"], torch.full_like(d["k"], 7.0)], 2)
    q, k = fused[:, :, :6], fused[:, :, 6:8]
    rest = (d["qw"], d["kw"], d["pos"], d["freq"])
    a, b = kda_qk_norm_rope_fwd(q, k, *rest)
    assert torch.equal(a, want["q"]) and torch.equal(b, want["k"])
    g = kda_qk_norm_rope_bwd(d["dq"], d["dk"], q, k, *rest)
    for t, n in zip(g, ("dq", "dk", "dqw", "dkw")):
        assert torch.equal(t, want[n]), n
    g = kda_qk_norm_rope_bwd(d["dq"], d["dk"], q, k, *rest, out=(d["dq"], d["dk"]))  # over the adjoints
    assert torch.equal(g[0], want["dq"]) and torch.equal(g[1], want["dk"])
    with pytest.raises(KdaError):  # over the other tensor
        kda_qk_norm_rope_fwd(q, k, *rest, q_out=q, k_out=fused[:, :, 4:6])
    kda_qk_norm_rope_fwd(q, k, *rest, q_out=q, k_out=k)
    assert torch.equal(q, want["q"]) and torch.equal(k, want["k"]) and (fused[:, :, 8:] == 7).all()
    e = torch.empty(1, 0, 6, 128, dtype=torch.bfloat16, device="cuda")
    none = torch.empty(1, 0, dtype=torch.int64, device="cuda")
    a, _ = kda_qk_norm_rope_fwd(e, e, d["qw"], d["kw"], none, d["freq"])
    assert a.shape == e.shape
    g = kda_qk_norm_rope_bwd(e, e, e, e, d["qw"], d["kw"], none, d["freq"])
    assert (g[2] == 0).all() and (g[3] == 0).all()


def test_repeatable():
    x = make(1, 700, 9, 3, 128, 128, torch.bfloat16, seed=5)
    a, b = run(x, False), run(x, False)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_difference():
    """The gradient along a direction against the forward's central difference, in FP32."""
    from linear_attention_gated_gb300 import kda_qk_norm_rope_bwd, kda_qk_norm_rope_fwd
    x = make(1, 8, 2, 2, 64, 64, torch.float32, seed=6)
    d = {n: t.cuda() for n, t in x.items()}
    rest = (d["qw"], d["kw"], d["pos"], d["freq"])
    g = kda_qk_norm_rope_bwd(d["dq"], d["dk"], d["q"], d["k"], *rest)[0]
    step = torch.randn(d["q"].shape, generator=torch.Generator().manual_seed(1)).cuda()
    e = 2.0 ** -7

    def loss(q):
        return (kda_qk_norm_rope_fwd(q, d["k"], *rest)[0].double() * d["dq"].double()).sum().item()

    want = (loss(d["q"] + e * step) - loss(d["q"] - e * step)) / (2 * e)
    size = (g.double() * step.double()).norm().item()
    # the difference's own error: e^2 / 6 of a third derivative of a few times the gradient
    assert abs((g.double() * step.double()).sum().item() - want) <= 2e-3 * size


@pytest.mark.parametrize("dtype,T,hq,hk,dim,rot,interleaved", [
    (torch.bfloat16, 40001, 7, 3, 64, 64, False),  # rows enough for several runs of angles a block, heads that no run divides
    (torch.bfloat16, 30011, 1, 17, 128, 96, True),
    (torch.float32, 12007, 3, 1, 256, 256, False),
])
def test_many_rows(dtype, T, hq, hk, dim, rot, interleaved):
    x = make(1, T, hq, hk, dim, rot, dtype, seed=T)
    got = run(x, interleaved)
    ref = reference({n: t.cuda() if t is not None else None for n, t in x.items()}, interleaved)
    compare(got, {n: t.cpu() for n, t in ref.items()}, dtype, T * max(hq, hk))


def test_a_stream_of_its_own_and_a_graph():
    """Forward and backward on a side stream, captured and replayed with other inputs."""
    from linear_attention_gated_gb300 import kda_qk_norm_rope_bwd, kda_qk_norm_rope_fwd
    x, y = make(2, 130, 6, 2, 128, 64, torch.bfloat16, seed=7), make(2, 130, 6, 2, 128, 64, torch.bfloat16, seed=8, far=1000)
    d = {n: t.cuda() for n, t in x.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        rest = (d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["freq"])
        return kda_qk_norm_rope_fwd(*rest) + kda_qk_norm_rope_bwd(d["dq"], d["dk"], *rest)

    with torch.cuda.stream(s):
        out = step()
    torch.cuda.synchronize()
    compare(dict(zip(("q", "k", "dq", "dk", "dqw", "dkw"), out)), reference(x, False), torch.bfloat16, 1560)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out = step()
    for n in d:
        d[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    compare(dict(zip(("q", "k", "dq", "dk", "dqw", "dkw"), out)), reference(y, False), torch.bfloat16, 1560)
