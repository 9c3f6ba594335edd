"""Linear attention with a decay for each head, on the GPU, against its recurrence in 64 bits.

Tolerances. BF16 outputs: each operand that is rounded to BF16 on the way (the state or its adjoint, the
masked product of queries and keys, the output itself) adds an independent relative error of at most
half a step, 2^-8, so of rms at most 2^-8 / sqrt(3): three of them for o (relative L2 2^-8), four for a
gradient (2^-8 sqrt(4 / 3)). FP32 states: operands in two BF16 parts, 2^-16 relative, and FP32 sums.
"""

import math

import pytest
import torch

from decay_reference import BF16, check, rel_l2, scan

pytestmark = pytest.mark.gpu

O_REL = BF16
GRAD_REL = BF16 * math.sqrt(4 / 3)
STATE_REL = 2.0 ** -16 + 64 * 2.0 ** -24
D = 128
SCALE = 1 / math.sqrt(128)


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_attention_gated_gb300 import build
    build.build()
    from linear_attention_gated_gb300 import kda
    kda.load_library()


def make(lens, hqk, hv, gate, seed, packed=True, state=0.05):
    """Inputs on the CPU; lens of the packed sequences, or B equal ones."""
    gen = torch.Generator().manual_seed(seed)
    B, T = (1, sum(lens)) if packed else (len(lens), lens[0])
    x = dict(q=torch.randn(B, T, hqk, D, generator=gen), k=torch.randn(B, T, hqk, D, generator=gen),
             v=torch.randn(B, T, hv, D, generator=gen), do=torch.randn(B, T, hv, D, generator=gen))
    x = {n: t.bfloat16() for n, t in x.items()}
    if gate == "head":
        x["g"] = -torch.exp2(-8.0 * torch.arange(1, hv + 1) / hv)
    else:
        x["g"] = (-torch.rand(B, T, hv, generator=gen) * torch.rand(1, 1, hv, generator=gen)).bfloat16()
    N = len(lens)
    x["h0"] = state * torch.randn(N, hv, D, D, generator=gen)
    x["dhT"] = state * torch.randn(N, hv, D, D, generator=gen)
    if packed:
        x["cu"] = torch.tensor([0] + list(lens)).cumsum(0)
    return x


def spans_of(x):
    if "cu" in x:
        cu = x["cu"].tolist()
        return list(zip(cu[:-1], cu[1:]))
    B, T = x["v"].shape[:2]
    return [(b * T, (b + 1) * T) for b in range(B)]


def reference(x, scale=SCALE, grads=True, device="cpu", with_state=True, with_dstate=True):
    f = {n: x[n].to(device).double().flatten(0, 1) for n in ("q", "k", "v", "do")}
    g = x["g"].to(device).double()
    g = g.flatten(0, 1) if g.dim() == 3 else g.expand(f["v"].shape[0], -1)
    h0 = x["h0"].to(device).double() * (1 if with_state else 0)
    leaves = [f["q"], f["k"], f["v"], g, h0]
    if grads:
        leaves = [t.clone().requires_grad_() for t in leaves]
    o, hT = scan(*leaves, spans_of(x), scale)
    shape = x["v"].shape
    out = dict(o=o.detach().reshape(shape), hT=hT.detach())
    if grads:
        loss = (o * f["do"]).sum() + ((hT * x["dhT"].to(device).double()).sum() if with_dstate else 0)
        gr = torch.autograd.grad(loss, leaves, allow_unused=True)
        gr = [torch.zeros_like(t) if d is None else d for d, t in zip(gr, leaves)]
        qs = x["q"].shape
        out.update(dq=gr[0].reshape(qs), dk=gr[1].reshape(qs), dv=gr[2].reshape(shape), dg=gr[3].reshape(shape[:3]), dh0=gr[4])
    return out


def run(x, grads=True, scale=None, ctx=None, with_state=True, with_dstate=True):
    from linear_attention_gated_gb300 import kda_decay_attn_bwd, kda_decay_attn_fwd
    d = {n: t.cuda() for n, t in x.items()}
    o, hT, ctx = kda_decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"] if with_state else None, d.get("cu"), scale,
                                    context_out=ctx, cu_seqlens_cpu=x.get("cu"))
    out = dict(o=o, hT=hT)
    if grads:
        out.update(zip(("dq", "dk", "dv", "dg", "dh0"), kda_decay_attn_bwd(ctx, d["do"], d["dhT"] if with_dstate else None)))
    torch.cuda.synchronize()
    ctx.status()
    return out, ctx


def compare(got, ref):
    for n, t in got.items():
        if t is None:
            continue
        if n in ("hT", "dh0"):
            assert rel_l2(t, ref[n]) <= STATE_REL, (n, rel_l2(t, ref[n]))
        else:
            assert t.dtype == torch.bfloat16
            check(n, t, ref[n], O_REL if n == "o" else GRAD_REL, BF16)


@pytest.mark.parametrize("lens", [(1,), (2, 1), (15, 17, 16), (63, 64, 65), (127, 1, 128, 129), (200, 31, 260)], ids=str)
@pytest.mark.parametrize("hqk,hv,gate", [(1, 1, "token"), (2, 4, "token"), (3, 3, "head"), (1, 5, "head")])
def test_packed(lens, hqk, hv, gate):
    x = make(lens, hqk, hv, gate, seed=len(lens) * 10 + hv)
    got, _ = run(x)
    assert (got["dg"] is None) == (gate == "head")
    compare(got, reference(x))


@pytest.mark.parametrize("B,T", [(2, 1), (3, 64), (2, 193)])
def test_fixed_layout_and_scale(B, T):
    x = make([T] * B, 2, 2, "token", seed=T, packed=False)
    got, _ = run(x, scale=0.25)
    compare(got, reference(x, scale=0.25))


def test_without_states():
    x = make((70, 140), 1, 2, "token", seed=3)
    got, _ = run(x, with_state=False, with_dstate=False)
    assert got.pop("dh0") is None
    compare(got, reference(x, with_state=False, with_dstate=False))


def test_empty_sequences_pass_their_state_on():
    x = make((0, 5, 0, 130, 0), 1, 2, "token", seed=4)
    got, _ = run(x)
    compare(got, reference(x))
    for n in (0, 2, 4):
        assert torch.equal(got["hT"][n].cpu(), x["h0"][n]) and torch.equal(got["dh0"][n].cpu(), x["dhT"][n])


def test_no_tokens():
    x = make((0, 0), 1, 2, "token", seed=5)
    got, _ = run(x)
    assert got["o"].shape == (1, 0, 2, D) and got["dq"].shape == (1, 0, 1, D)
    assert torch.equal(got["hT"].cpu(), x["h0"]) and torch.equal(got["dh0"].cpu(), x["dhT"])


@pytest.mark.parametrize("value", [0.0, -20.0, -90.0, -float("inf")])
def test_extreme_decays(value):
    """No decay, ones that leave nothing after a few tokens, and resets in the middle of a chunk."""
    x = make((150, 67), 1, 2, "token", seed=6)
    x["g"][:, ::(1 if value == 0.0 else 5)] = value
    ref = reference(x)
    if math.isinf(value):
        ref["dg"][:, ::5] = 0.0  # exp has no slope there; autograd multiplies 0 by what it scaled
    compare(run(x)[0], ref)


def test_head_decays_of_zero_and_reset():
    x = make((130,), 1, 3, "head", seed=7)
    x["g"] = torch.tensor([0.0, -float("inf"), -3.0])
    compare(run(x)[0], reference(x))


def test_non_finite_values_stay_in_their_sequence():
    """Tiles reach over a sequence's end; what they find there must not matter."""
    x = make((70, 61, 130), 1, 2, "token", seed=8)
    clean, _ = run(x)
    for bad in (float("nan"), float("inf")):
        y = dict(x)
        for n in ("q", "k", "v", "do"):
            y[n] = x[n].clone()
            y[n][:, 70:131] = bad
        got, _ = run(y)
        keep = torch.ones(261, dtype=torch.bool)
        keep[70:131] = False
        for n in ("o", "dq", "dk", "dv", "dg"):
            assert torch.equal(got[n].cpu()[:, keep], clean[n].cpu()[:, keep]), (n, bad)
        for n in ("hT", "dh0"):
            assert torch.equal(got[n][[0, 2]], clean[n][[0, 2]]), (n, bad)


def test_views_of_one_projection():
    from linear_attention_gated_gb300 import kda_decay_attn_bwd, kda_decay_attn_fwd
    x = make((100, 90), 2, 4, "token", seed=9)
    want, _ = run(x)
    fused = torch.full((1, 190, 9, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, :, 0:2], fused[:, :, 2:4], fused[:, :, 5:9] = x["q"].cuda(), x["k"].cuda(), x["v"].cuda()
    q, k, v = fused[:, :, 0:2], fused[:, :, 2:4], fused[:, :, 5:9]
    o, hT, ctx = kda_decay_attn_fwd(q, k, v, x["g"].cuda(), x["h0"].cuda(), x["cu"].cuda(), cu_seqlens_cpu=x["cu"])
    grads = kda_decay_attn_bwd(ctx, x["do"].cuda(), x["dhT"].cuda())
    got = dict(zip(("o", "hT", "dq", "dk", "dv", "dg", "dh0"), (o, hT) + grads))
    for n, t in want.items():
        assert torch.equal(t, got[n]), n


@pytest.mark.parametrize("T,gate", [(4097, "token"), (9000, "head")])
def test_long_sequences(T, gate):
    x = make((T, 70), 1, 2, gate, seed=10)
    compare(run(x)[0], reference(x, device="cuda"))


def test_many_heads_and_sequences():
    """More units than can run at once."""
    x = make((130, 7, 64, 1, 200, 90, 66, 33), 8, 64, "token", seed=11)
    compare(run(x)[0], reference(x, device="cuda"))


def test_more_sequences_than_are_put_in_order():
    """600 sequences of 0 to 5 tokens (512 at most are run longest first)."""
    lens = [(7 * i) % 6 for i in range(600)]
    x = make(lens, 1, 2, "head", seed=23)
    compare(run(x)[0], reference(x))


def test_runs_of_empty_sequences():
    """More empty units in a row than a running block's ring of units has places, before, between and after others."""
    lens = [0] * 40 + [70] + [0] * 300 + [1] + [0] * 60
    x = make(lens, 2, 8, "token", seed=25)
    compare(run(x)[0], reference(x, device="cuda"))


def test_long_sequences_among_short_ones():
    """Some sequences are cut into segments, others not, out of order."""
    x = make((3, 3100, 0, 64, 5000, 1, 200), 1, 1, "token", seed=24)
    got, _ = run(x)
    compare(got, reference(x, device="cuda"))
    again, _ = run(x)
    for n, t in got.items():
        assert torch.equal(t, again[n]), n


def test_context_reuse_and_repeatability():
    from linear_attention_gated_gb300 import KdaError, kda_decay_attn_bwd
    x, y = make((90, 40), 1, 2, "token", seed=12), make((40, 90), 1, 2, "token", seed=13)
    a, ctx = run(x)
    b, ctx2 = run(y, ctx=ctx)  # same shapes, other lengths
    assert ctx2 is ctx
    compare(b, reference(y))
    c, _ = run(x, ctx=ctx)
    for n, t in a.items():
        assert torch.equal(t, c[n]), n
    ctx.inputs[0].zero_()
    with pytest.raises(KdaError):
        kda_decay_attn_bwd(ctx, y["do"].cuda())


def test_differences_of_the_final_state():
    """dh0 and dv of a loss on the final state alone, against differences of the forward: it is linear in
    both, so a whole step differs from the gradient by the roundings only. The decays are slow (0.5 % a
    token), so that the first token still counts in the last state."""
    from linear_attention_gated_gb300 import kda_decay_attn_bwd, kda_decay_attn_fwd
    x = make((150,), 1, 1, "token", seed=22)
    x["g"] = (x["g"].float() * 0.02).bfloat16()
    d = {n: t.cuda() for n, t in x.items()}
    gen = torch.Generator().manual_seed(1)
    step, dirv = torch.randn(d["h0"].shape, generator=gen).cuda(), torch.randn(d["v"].shape, generator=gen).bfloat16().cuda()

    def final(v, h0):
        return kda_decay_attn_fwd(d["q"], d["k"], v, d["g"], h0, d["cu"], cu_seqlens_cpu=x["cu"])[1:]

    hT, ctx = final(d["v"], d["h0"])
    _, _, dv, _, dh0 = kda_decay_attn_bwd(ctx, torch.zeros_like(d["do"]), d["dhT"])
    dh = d["dhT"].double()

    def slope(a, b):
        return ((a.double() - b.double()) * dh).sum().item()

    hT2, _ = final(d["v"], d["h0"] + step)
    terms = dh0.double() * step.double()
    assert abs(terms.sum().item() - slope(hT2, hT)) <= 6 * STATE_REL * (terms.norm().item() + 2 * (hT.double() * dh).norm().item())
    h1, _ = final(dirv, torch.zeros_like(d["h0"]))
    terms = dv.double() * dirv.double()
    assert abs(terms.sum().item() - slope(h1, torch.zeros_like(h1))) <= 6 * GRAD_REL * terms.norm().item()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("lens,hqk,hv,gate", [((1, 64, 65), 1, 2, "token"), ((130, 300), 2, 2, "head"), ((5000,), 1, 1, "head")],
                         ids=str)
def test_prefill_from_a_pool(dtype, lens, hqk, hv, gate):
    from linear_attention_gated_gb300 import kda_decay_attn_prefill
    x = make(lens, hqk, hv, gate, seed=15)
    N = len(lens)
    idx = torch.randperm(N + 3, generator=torch.Generator().manual_seed(N))[:N].int()
    pool = torch.randn(N + 3, hv, D, D, generator=torch.Generator().manual_seed(5)).mul(0.05).to(dtype)
    x["h0"] = pool[idx.long()].float()
    ref = reference(x, grads=False, device="cuda")
    st = pool.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = kda_decay_attn_prefill(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), st, x["cu"].cuda(), idx.cuda(),
                               device_status=status, cu_seqlens_cpu=x["cu"], state_indices_cpu=idx)
    assert status.item() == 0
    check("o", o, ref["o"], O_REL, BF16)
    after = st.cpu()
    rest = [i for i in range(N + 3) if i not in idx.tolist()]
    assert torch.equal(after[rest], pool[rest])
    if dtype == torch.float32:
        assert rel_l2(after[idx.long()], ref["hT"]) <= STATE_REL
    else:
        check("pool", after[idx.long()], ref["hT"], BF16 * math.sqrt(1 / 3) + STATE_REL, BF16)


def test_prefill_reports_a_device_slot_outside_the_pool():
    from linear_attention_gated_gb300 import kda_decay_attn_prefill
    x = make((40, 50), 1, 1, "head", seed=16)
    st = torch.zeros(2, 1, D, D, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kda_decay_attn_prefill(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), st, x["cu"].cuda(),
                           torch.tensor([0, 7], dtype=torch.int32, device="cuda"), device_status=status,
                           cu_seqlens_cpu=x["cu"], state_indices_cpu=torch.tensor([0, 1], dtype=torch.int32))
    assert status.item() == 4
    assert (st[1] == 0).all() and (st[0] != 0).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("N,hqk,hv,gate", [(1, 1, 1, "token"), (5, 2, 6, "head"), (7, 3, 3, "token"), (40, 8, 64, "token")])
def test_decode(dtype, N, hqk, hv, gate):
    from linear_attention_gated_gb300 import kda_decay_attn_decode
    x = make((1,) * N, hqk, hv, gate, seed=17, packed=False)
    if gate == "token" and N > 1:
        x["g"][1] = -float("inf")
    idx = torch.randperm(N + 2, generator=torch.Generator().manual_seed(N))[:N].int()
    pool = torch.randn(N + 2, hv, D, D, generator=torch.Generator().manual_seed(6)).mul(0.05).to(dtype)
    x["h0"] = pool[idx.long()].float()
    ref = reference(x, grads=False)
    st = pool.cuda()
    o = kda_decay_attn_decode(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), st, idx.cuda(), state_indices_cpu=idx)
    check("o", o, ref["o"], BF16, BF16)
    after = st.cpu()
    rest = [i for i in range(N + 2) if i not in idx.tolist()]
    assert torch.equal(after[rest], pool[rest])
    if dtype == torch.float32:
        assert rel_l2(after[idx.long()], ref["hT"]) <= 2.0 ** -22  # two roundings and exp2f
    else:
        check("pool", after[idx.long()], ref["hT"], BF16, BF16)


def test_decode_follows_prefill_and_views():
    """A prompt by prefill, then tokens one by one, equals the whole sequence; tokens read as views."""
    from linear_attention_gated_gb300 import kda_decay_attn_decode, kda_decay_attn_prefill
    N, T, more = 2, 70, 5
    x = make([T + more] * N, 2, 4, "token", seed=18, packed=False, state=0.0)
    ref = reference(x, grads=False)
    fused = torch.cat([x["q"], x["k"], x["v"]], 2).cuda()
    q, k, v = fused[:, :, 0:2], fused[:, :, 2:4], fused[:, :, 4:8]
    g = x["g"].cuda()
    st = torch.zeros(N, 4, D, D, device="cuda")
    outs = [kda_decay_attn_prefill(q[:, :T].contiguous(), k[:, :T].contiguous(), v[:, :T].contiguous(), g[:, :T].contiguous(), st)]
    for t in range(T, T + more):
        outs.append(kda_decay_attn_decode(q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1], g[:, t:t + 1].contiguous(), st))
    check("o", torch.cat(outs, 1), ref["o"], O_REL, BF16)
    assert rel_l2(st, ref["hT"]) <= STATE_REL


def test_decode_bad_device_slot_gives_nan():
    from linear_attention_gated_gb300 import kda_decay_attn_decode
    x = make((1, 1), 1, 1, "head", seed=19, packed=False)
    st = torch.ones(2, 1, D, D, device="cuda")
    o = kda_decay_attn_decode(x["q"].cuda(), x["k"].cuda(), x["v"].cuda(), x["g"].cuda(), st,
                              torch.tensor([1, 9], dtype=torch.int32, device="cuda"),
                              state_indices_cpu=torch.tensor([1, 0], dtype=torch.int32))
    assert torch.isnan(o[1]).all() and torch.isfinite(o[0]).all()
    assert (st[0] == 1).all()


def test_decode_of_nothing():
    from linear_attention_gated_gb300 import kda_decay_attn_decode
    e = torch.empty(0, 1, 2, D, dtype=torch.bfloat16, device="cuda")
    o = kda_decay_attn_decode(e, e, e, torch.zeros(2, device="cuda"), torch.zeros(1, 2, D, D, device="cuda"))
    assert o.shape == (0, 1, 2, D)


def test_a_stream_of_its_own_and_a_graph():
    """The whole step on a side stream, captured and replayed with other inputs."""
    from linear_attention_gated_gb300 import kda_decay_attn_bwd, kda_decay_attn_fwd
    x, y = make((90, 140), 1, 2, "token", seed=20), make((90, 140), 1, 2, "token", seed=21)
    d = {n: t.cuda() for n, t in x.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step(ctx):
        o, hT, ctx = kda_decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["cu"], context_out=ctx, cu_seqlens_cpu=x["cu"])
        return (o, hT) + kda_decay_attn_bwd(ctx, d["do"], d["dhT"]), ctx

    with torch.cuda.stream(s):
        _, ctx = step(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, ctx = step(ctx)
    for n in d:
        d[n].copy_(y[n])
    graph.replay()
    torch.cuda.synchronize()
    compare(dict(zip(("o", "hT", "dq", "dk", "dv", "dg", "dh0"), out)), reference(y))
