"""Less usual inputs and forms of the gated delta rule, on the GPU: decays that leave nothing and resets, step sizes of 0 and 2,
keys that are alike, values that are not finite, views, buffers of the caller, contexts used again, captured graphs, other
streams, device offsets and lengths beyond the usual. Tolerances as in test_gpu_delta.py."""

import math

import pytest
import torch

from decay_reference import BF16, FP32, rel_l2
from test_gpu_delta import (D, GRAD_REL, GRADS, O_REL, SCALE, STATE_REL, check_rows, compare, library, make, reference,  # noqa: F401
                            run)

pytestmark = pytest.mark.gpu
NAMES = ("o", "hT") + GRADS
TOKENS = ("q", "k", "v", "g", "beta")


def same(a, b):
    for n, t in a.items():
        assert (t is None and b[n] is None) or torch.equal(t, b[n]), n


@pytest.mark.parametrize("value", [0.0, -1.5, -20.0, -90.0, -float("inf")])
def test_extreme_decays(value):
    """No decay, ones that leave nothing after a few tokens (chunks of factors too far apart for one product), and resets
    in the middle of a chunk."""
    x = make((150, 67, 64), 1, 2, seed=6)
    x["g"][:, ::(1 if value > -2 else 5)] = value
    ref = reference(x)
    if math.isinf(value):
        ref["dg"][:, ::5] = 0.0  # exp has no slope there; autograd multiplies 0 by what it scaled
    compare(run(x)[0], ref)


@pytest.mark.parametrize("beta", [0.0, 1.0, 2.0])
def test_step_sizes(beta):
    """0: the values do not count; 1: a key's old value is forgotten; 2: it is turned round."""
    x = make((130, 64, 5), 1, 2, seed=7)
    x["beta"].fill_(beta)
    got, ref = run(x)[0], reference(x)
    for n in ("dk", "dv") if beta == 0 else ():
        assert not ref[n].any() and not got.pop(n).any(), n
    compare(got, ref)


@pytest.mark.parametrize("beta", [1.0, 2.0])
def test_keys_that_are_alike(beta):
    """One direction for all keys but 5 %.
    With beta 1 then u_t = v_t - v_t-1, nearly: sums of up to 64 terms, rms sqrt 2, come out at rms 1, so errors relative to the
    terms are sqrt(2 64) times as large relative to the sum, and a state keeps the errors of its chunks.
    With beta 2 all A_ij are near 2, u is as large as the state's value along the keys, and T's entries are 2 and -2 in turn.
    A taken in two parts, off by 2 0.436 2^-17 rms a value, moves u_i by sum_kl T_ik dA_kl u_l: over the 64 63 / 2 pairs of a
    chunk 2 sqrt(2016) times that, relative to u and to the state; it is added once a chunk."""
    x = make((200,), 1, 2, seed=8, gate=False, alike=20.0)
    x["beta"].fill_(beta)
    got, _ = run(x)
    ref = reference(x)
    sums, chunks = math.sqrt(2 * 64), math.sqrt(200 / 64 + 1)
    for n in NAMES:
        if n in ("hT", "dh0"):
            bar = (STATE_REL[n] * sums if beta == 1 else 2 * math.sqrt(2016) * 2 * 0.436 * 2.0 ** -17) * chunks
            assert rel_l2(got[n], ref[n]) <= bar, (n, rel_l2(got[n], ref[n]))
        elif got[n] is not None:
            off = rel_l2(got[n], ref[n])
            assert off <= (O_REL if n == "o" else GRAD_REL) * sums, (n, off)


def test_values_that_are_not_finite_stay_in_their_sequence():
    """Tiles reach over a sequence's end; what they find there must not matter."""
    x = make((70, 61, 130), 1, 2, seed=9)
    clean, _ = run(x)
    keep = torch.ones(261, dtype=torch.bool)
    keep[70:131] = False
    for bad in (float("nan"), float("inf")):
        y = dict(x)
        for n in TOKENS + ("do",):
            y[n] = x[n].clone()
            y[n][:, 70:131] = bad
        got, _ = run(y)
        for n in NAMES:
            if n in ("hT", "dh0"):
                assert torch.equal(got[n][[0, 2]], clean[n][[0, 2]]), (n, bad)
            else:
                assert torch.equal(got[n].cpu()[:, keep], clean[n].cpu()[:, keep]), (n, bad)


@pytest.mark.parametrize("name", TOKENS)
def test_a_nan_does_not_go_back_in_time(name):
    """What a chunk has that is not finite is in its outputs and those after it."""
    x = make((200,), 1, 1, seed=10)
    clean, _ = run(x, grads=False)
    y = dict(x)
    y[name] = x[name].clone()
    y[name][:, 70] = float("nan")
    got, _ = run(y, grads=False)
    assert torch.equal(got["o"][:, :64], clean["o"][:, :64])
    assert got["o"][:, 70].isnan().all()
    if name != "q":
        assert got["hT"].isnan().any()


def test_views_of_one_projection():
    from linear_attention_gated_gb300 import kda_gated_delta_bwd, kda_gated_delta_fwd
    x = make((100, 90), 2, 4, seed=11)
    want, _ = run(x)
    fused = torch.full((1, 190, 9, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, :, 0:2], fused[:, :, 2:4], fused[:, :, 5:9] = x["q"].cuda(), x["k"].cuda(), x["v"].cuda()
    q, k, v = fused[:, :, 0:2], fused[:, :, 2:4], fused[:, :, 5:9]
    o, hT, ctx = kda_gated_delta_fwd(q, k, v, x["g"].cuda(), x["beta"].cuda(), x["h0"].cuda(), x["cu"].cuda(), cu_seqlens_cpu=x["cu"])
    grads = kda_gated_delta_bwd(ctx, x["do"].cuda(), x["dhT"].cuda())
    same(want, dict(zip(NAMES, (o, hT) + grads)))


@pytest.mark.parametrize("hqk,hv", [(2, 6), (1, 5), (2, 12), (1, 7)])
def test_groups_of_heads(hqk, hv):
    x = make((70, 33, 65), hqk, hv, seed=12)
    compare(run(x)[0], reference(x))


def test_fixed_layout_cut_into_segments():
    from linear_attention_gated_gb300 import gated_delta_workspace_bytes
    B, T = 2, 3100
    assert gated_delta_workspace_bytes(B, T, 1, 1, training=False) > (B * T // 64 + B) * 26624 + 256  # the segments' states
    x = make([T] * B, 1, 1, seed=13, packed=False)
    compare(run(x)[0], reference(x, device="cuda"))


def test_long_sequences_among_short_ones():
    """Some sequences are cut into segments, others not, out of order."""
    x = make((3, 3100, 0, 64, 4000, 1, 200), 1, 1, seed=14)
    got, _ = run(x)
    compare(got, reference(x, device="cuda"))
    same(got, run(x)[0])


def test_segments_of_resets():
    """A sequence that is cut, whose state is reset now and then: the segments' maps are zero."""
    x = make((3300,), 1, 1, seed=15)
    x["g"][:, 1000::500] = -float("inf")
    ref = reference(x, device="cuda")
    ref["dg"][:, 1000::500] = 0.0
    compare(run(x)[0], ref)


def test_a_nan_in_a_state_outlives_resets():
    """A reset multiplies by zero, and that leaves NaN: in the state's row alone, over segments whose maps are zero, too."""
    x = make((3300,), 1, 1, seed=40)
    x["g"][:, 1000::500] = -float("inf")
    clean, _ = run(x, grads=False)
    x["h0"][0, 0, 5, 7] = float("nan")
    got, _ = run(x, grads=False)
    rows = torch.arange(D) != 5
    assert got["o"][..., 5].isnan().all() and got["hT"][0, 0, 5].isnan().all()
    assert torch.equal(got["o"][..., rows], clean["o"][..., rows]) and torch.equal(got["hT"][0, 0, rows], clean["hT"][0, 0, rows])


def test_many_heads_and_sequences():
    """More units than can run at once."""
    x = make((130, 7, 64, 1, 200, 90, 66, 33), 8, 64, seed=16)
    got, _ = run(x)
    compare(got, reference(x, device="cuda"))
    same(got, run(x)[0])


def test_more_sequences_than_are_put_in_order():
    """600 sequences of 0 to 5 tokens (512 at most are run longest first, or cut)."""
    x = make([(7 * i) % 6 for i in range(600)], 1, 2, seed=17)
    compare(run(x)[0], reference(x))


def test_runs_of_empty_sequences():
    """More empty units in a row than a running block's ring of units has places, before, between and after others."""
    x = make([0] * 40 + [70] + [0] * 300 + [1] + [0] * 60, 2, 8, seed=18)
    compare(run(x)[0], reference(x, device="cuda"))


def test_buffers_of_the_caller():
    from linear_attention_gated_gb300 import kda_gated_delta_bwd, kda_gated_delta_fwd
    x = make((90, 40), 2, 4, seed=19)
    want, _ = run(x)
    d = {n: t.cuda() for n, t in x.items()}
    mine = {n: torch.full_like(t, float("nan")) for n, t in want.items()}
    o, hT, ctx = kda_gated_delta_fwd(*(d[n] for n in TOKENS), d["h0"], d["cu"], out=mine["o"], final_state_out=mine["hT"],
                                     cu_seqlens_cpu=x["cu"])
    got = kda_gated_delta_bwd(ctx, d["do"], d["dhT"], out=tuple(mine[n] for n in GRADS))
    assert o is mine["o"] and hT is mine["hT"] and all(a is mine[n] for a, n in zip(got, GRADS))
    same(want, mine)


def test_gradients_that_are_not_wanted():
    """At the C interface the decays' gradient and the start state's may be left out; the others are the same."""
    from linear_attention_gated_gb300 import kda_gated_delta_fwd
    from linear_attention_gated_gb300.decay import _call
    from linear_attention_gated_gb300.kda import load_library
    x = make((90, 40), 2, 4, seed=45)
    want, _ = run(x)
    d = {n: t.cuda() for n, t in x.items()}
    ctx = kda_gated_delta_fwd(*(d[n] for n in TOKENS), d["h0"], d["cu"], cu_seqlens_cpu=x["cu"])[2]
    got = {n: torch.full_like(want[n], float("nan")) for n in ("dq", "dk", "dv", "dbeta")}
    ws = ctx.workspace
    _call(load_library().kda_gated_delta_bwd, ctx.device, *ctx.call, d["do"].data_ptr(), d["dhT"].data_ptr(), got["dq"].data_ptr(),
          got["dk"].data_ptr(), got["dv"].data_ptr(), None, got["dbeta"].data_ptr(), None, ws.data_ptr(), ws.numel(),
          ctx.device_status.data_ptr())
    torch.cuda.synchronize()
    ctx.status()
    same(got, want)


@pytest.mark.parametrize("lens", [(90, 40), (3100, 20)], ids=str)
def test_what_a_workspace_held_does_not_matter(lens):
    """Prefill in a workspace of all ones bits (NaN), and one that is too small."""
    from linear_attention_gated_gb300 import KdaError, gated_delta_workspace_bytes, kda_gated_delta_prefill
    x = make(lens, 1, 1, seed=20)
    d = {n: t.cuda() for n, t in x.items()}
    nbytes = gated_delta_workspace_bytes(1, sum(lens), 1, 1, x["cu"], False)
    outs = []
    for ws in (None, torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")):
        pool = d["h0"].clone()
        o = kda_gated_delta_prefill(*(d[n] for n in TOKENS), pool, d["cu"], workspace=ws, cu_seqlens_cpu=x["cu"])
        outs.append((o, pool))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    with pytest.raises(KdaError):
        kda_gated_delta_prefill(*(d[n] for n in TOKENS), pool, d["cu"], workspace=ws[:nbytes - 256], cu_seqlens_cpu=x["cu"])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_prefill_cut_into_segments(dtype):
    """From and to slots of a pool, in any order; the short sequences beside the long one are not cut."""
    from linear_attention_gated_gb300 import kda_gated_delta_prefill
    x = make((20, 3000, 0, 66), 1, 2, seed=41)
    idx = torch.tensor([5, 0, 3, 2], dtype=torch.int32)
    pool = (0.05 * torch.randn(6, 2, D, D, generator=torch.Generator().manual_seed(42))).to(dtype)
    x["h0"] = pool[idx.long()].float()
    ref = reference(x, grads=False, device="cuda")
    got = pool.cuda()
    o = kda_gated_delta_prefill(*(x[n].cuda() for n in TOKENS), got, x["cu"].cuda(), idx.cuda(), cu_seqlens_cpu=x["cu"],
                                state_indices_cpu=idx)
    check_rows("o", o, ref["o"], O_REL)
    assert rel_l2(got[idx.long().cuda()], ref["hT"]) <= STATE_REL["hT"] + (0 if dtype == torch.float32 else BF16)
    assert torch.equal(got[[1, 4]].cpu(), pool[[1, 4]]) and torch.equal(got[3].cpu(), pool[3])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_prefill_of_nothing(dtype):
    """Sequences without tokens leave their states as they are."""
    from linear_attention_gated_gb300 import kda_gated_delta_prefill
    pool = torch.randn(5, 2, D, D, generator=torch.Generator().manual_seed(43)).to(dtype)
    got, cu, idx = pool.cuda(), torch.zeros(4, dtype=torch.int64), torch.tensor([4, 0, 1], dtype=torch.int32)
    e = torch.empty(1, 0, 2, D, dtype=torch.bfloat16, device="cuda")
    o = kda_gated_delta_prefill(e, e, e, None, e[..., 0].contiguous(), got, cu.cuda(), idx.cuda(), cu_seqlens_cpu=cu, state_indices_cpu=idx)
    assert o.shape == (1, 0, 2, D) and torch.equal(got.cpu(), pool)


def test_context_reuse_and_repeatability():
    from linear_attention_gated_gb300 import KdaError, kda_gated_delta_bwd
    x, y = make((90, 3140), 1, 1, seed=21), make((1600, 1630), 1, 1, seed=22)  # both are cut into segments, at other places
    b, ctx = run(y)
    a, _ = run(x)
    c, ctx2 = run(x, ctx=ctx)
    assert ctx2 is ctx
    same(a, c)
    same(b, run(y, ctx=ctx)[0])
    ctx.inputs[0].zero_()
    with pytest.raises(KdaError):
        kda_gated_delta_bwd(ctx, y["do"].cuda())


def test_two_contexts_at_once():
    """Two forwards before their backwards, on two streams."""
    from linear_attention_gated_gb300 import kda_gated_delta_bwd, kda_gated_delta_fwd
    xs = [make((90, 140), 1, 2, seed=23 + i) for i in range(2)]
    want = [run(x)[0] for x in xs]
    d = [{n: t.cuda() for n, t in x.items()} for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    fwd, got = [], []
    for s, x, y in zip(streams, xs, d):
        with torch.cuda.stream(s):
            fwd.append(kda_gated_delta_fwd(*(y[n] for n in TOKENS), y["h0"], y["cu"], cu_seqlens_cpu=x["cu"]))
    for s, f, y in zip(streams, fwd, d):
        with torch.cuda.stream(s):
            got.append(kda_gated_delta_bwd(f[2], y["do"], y["dhT"]))
    torch.cuda.synchronize()
    for w, f, g in zip(want, fwd, got):
        f[2].status()
        same(w, dict(zip(NAMES, f[:2] + g)))


@pytest.mark.parametrize("lens", [(90, 140), (3100, 70)], ids=str)
def test_a_training_step_in_a_graph(lens):
    """On a side stream, captured and replayed with other inputs; an eager step of the same inputs in between changes nothing."""
    from linear_attention_gated_gb300 import kda_gated_delta_bwd, kda_gated_delta_fwd
    x, y = make(lens, 1, 1, seed=25), make(lens, 1, 1, seed=26)
    want, _ = run(y)
    d = {n: t.cuda() for n, t in x.items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step(ctx):
        o, hT, ctx = kda_gated_delta_fwd(*(d[n] for n in TOKENS), d["h0"], d["cu"], context_out=ctx, cu_seqlens_cpu=x["cu"])
        return (o, hT) + kda_gated_delta_bwd(ctx, d["do"], d["dhT"]), ctx

    with torch.cuda.stream(s):
        _, ctx = step(None)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        out, ctx = step(ctx)
    for n in d:
        d[n].copy_(y[n])
    eager, _ = step(None)
    graph.replay()
    torch.cuda.synchronize()
    ctx.status()
    same(want, dict(zip(NAMES, out)))
    same(want, dict(zip(NAMES, eager)))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_serving_in_graphs(dtype):
    """A prefill and a decode step, captured and replayed with other inputs and slots."""
    from linear_attention_gated_gb300 import kda_gated_delta_decode, kda_gated_delta_prefill
    lens, hqk, hv, slots = (70, 1, 33), 2, 4, 5
    prompts = [make(lens, hqk, hv, seed=27 + i) for i in range(2)]
    tokens = [make((1,) * 3, hqk, hv, seed=29 + i, packed=False) for i in range(2)]
    order = [torch.tensor(i, dtype=torch.int32) for i in ((4, 0, 2), (1, 3, 0))]
    pools = [torch.randn(slots, hv, D, D, generator=torch.Generator().manual_seed(31 + i)).mul(0.05).to(dtype) for i in range(2)]
    p, t = ({n: v.cuda() for n, v in x[0].items()} for x in (prompts, tokens))
    idx, pool = order[0].cuda(), pools[0].cuda()

    def step():
        o = kda_gated_delta_prefill(*(p[n] for n in TOKENS), pool, p["cu"], idx, cu_seqlens_cpu=prompts[0]["cu"], state_indices_cpu=order[0])
        return o, kda_gated_delta_decode(*(t[n] for n in TOKENS), pool, idx, state_indices_cpu=order[0])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        o, o1 = step()
    for x, y in ((p, prompts[1]), (t, tokens[1])):
        for n in x:
            x[n].copy_(y[n])
    idx.copy_(order[1])
    pool.copy_(pools[1])
    graph.replay()
    torch.cuda.synchronize()
    at = order[1].long()
    prompts[1]["h0"] = pools[1][at].float()
    ref = reference(prompts[1], grads=False)
    check_rows("o", o, ref["o"], O_REL)
    tokens[1]["h0"] = ref["hT"].to(dtype).double()  # (rounded to the pool's type between the two)
    ref = reference(tokens[1], grads=False)
    check_rows("o", o1, ref["o"], O_REL)
    after = pool.cpu()
    rest = [i for i in range(slots) if i not in at.tolist()]
    assert torch.equal(after[rest], pools[1][rest])
    assert rel_l2(after[at], ref["hT"]) <= STATE_REL["hT"] + (0 if dtype == torch.float32 else 2 * BF16)  # (rounded twice)


@pytest.mark.parametrize("bad", [[0, 70, 3170], [0, 5000, -4], [-9, 1 << 40, 1 << 62], [3170, 0, 3170], [3170, 3170, 3170]], ids=str)
def test_device_offsets_that_disagree_with_the_mirror(bad):
    """They are held inside the tensors: nothing around the outputs changes, and the next call is right."""
    from linear_attention_gated_gb300 import kda_gated_delta_bwd, kda_gated_delta_fwd
    x = make((3100, 70), 1, 1, seed=33)  # the first is cut into segments
    want, _ = run(x)
    d = {n: t.cuda() for n, t in x.items()}
    room = {n: torch.full((want[n].numel() + 2 * 4096,), 3.0, dtype=want[n].dtype, device="cuda") for n in NAMES}
    mine = {n: room[n][4096:-4096].view(want[n].shape) for n in NAMES}

    def step(cu):
        _, _, ctx = kda_gated_delta_fwd(*(d[n] for n in TOKENS), d["h0"], cu, out=mine["o"], final_state_out=mine["hT"],
                                        cu_seqlens_cpu=x["cu"])
        kda_gated_delta_bwd(ctx, d["do"], d["dhT"], out=tuple(mine[n] for n in GRADS))
        ctx.status()

    step(torch.tensor(bad, device="cuda"))
    for n in NAMES:
        assert (room[n][:4096] == 3).all() and (room[n][-4096:] == 3).all(), n
    for n in ("q", "h0", "g", "beta"):
        assert torch.equal(d[n].cpu(), x[n]), n
    step(d["cu"])
    same(want, mine)


def test_differences_of_the_final_state():
    """Gradients of a loss on the final state alone, against differences of the forward. It is linear in h0 and v, so that a whole
    step differs by the roundings only; in k, g and beta central differences of step e are off by e^2 / 6 of the third
    derivative. Inputs are BF16: the steps taken are those that the rounded inputs make."""
    from linear_attention_gated_gb300 import kda_gated_delta_bwd, kda_gated_delta_fwd
    x = make((150,), 1, 1, seed=34)
    x["g"] = (x["g"].float() * 0.02).bfloat16()  # (slow: the first token still counts in the last state)
    d = {n: t.cuda() for n, t in x.items()}
    gen = torch.Generator().manual_seed(1)

    def final(**kw):
        y = {**d, **kw}
        return kda_gated_delta_fwd(*(y[n] for n in TOKENS), y["h0"], y["cu"], cu_seqlens_cpu=x["cu"])[1:]

    hT, ctx = final()
    grads = dict(zip(GRADS, kda_gated_delta_bwd(ctx, torch.zeros_like(d["do"]), d["dhT"])))
    assert not grads["dq"].any()
    dh = d["dhT"].double()
    noise = 6 * STATE_REL["hT"] * 2 * (hT.double() * dh).norm().item()

    def check(name, up, down, third):
        step = up[name].double() - down[name].double()
        terms = grads["d" + name].double() * step
        a, b = final(**up)[0], final(**down)[0]
        slope = ((a.double() - b.double()) * dh).sum().item()
        rel = STATE_REL["dh0"] if name == "h0" else GRAD_REL
        assert abs(terms.sum().item() - slope) <= 6 * rel * terms.norm().item() + noise + third * abs(slope), (name, slope)

    def along(name, e):
        t = d[name]
        r = torch.randn(t.shape, generator=gen).cuda() * (t.float().abs() if name in ("g", "beta") else t.float().square().mean().sqrt())
        return [{name: (t.float() + s * e * r).to(t.dtype)} for s in (1, -1)]

    check("h0", {"h0": d["h0"] + torch.randn(d["h0"].shape, generator=gen).cuda()}, {"h0": d["h0"]}, 0)
    check("v", *along("v", 1.0), 0)
    for name in ("k", "g", "beta"):
        up, down = along(name, 2.0 ** -5)
        # the middle of the two rounded inputs is off the point itself by a rounding: a slope's change of 2^-8 of the step's
        # size in relation to the values, twice, and the cubic term (2^-5)^2
        check(name, up, down, 2.0 ** -7 + 2.0 ** -10)


@pytest.mark.parametrize("T", [4500])
def test_slow_decays_over_a_long_sequence(T):
    """States that forget little over 70 chunks, some cut into segments: errors add up as the values do."""
    x = make((T, 60), 1, 2, seed=35)
    x["g"] = (x["g"].float() * 0.002).bfloat16()
    got, _ = run(x)
    ref = reference(x, device="cuda")
    compare(got, ref)


def test_decode_reset_and_no_decay():
    """-inf leaves the new token's update alone; g of 0 and no g are the same."""
    from linear_attention_gated_gb300 import kda_gated_delta_decode
    x = make((1,) * 4, 1, 2, seed=36, packed=False)
    d = {n: t.cuda() for n, t in x.items()}
    outs = []
    for g in (torch.full_like(d["g"], -float("inf")), torch.zeros_like(d["g"]), None):
        pool = d["h0"].clone()
        outs.append((kda_gated_delta_decode(d["q"], d["k"], d["v"], g, d["beta"], pool), pool))
    k, v, beta = (x[n].double() for n in ("k", "v", "beta"))
    new = beta[:, 0, :, None, None] * v[:, 0, :, :, None] * k[:, 0, :, None, :]
    assert rel_l2(outs[0][1], new) <= 4 * FP32
    assert torch.equal(outs[1][0], outs[2][0]) and torch.equal(outs[1][1], outs[2][1])


def test_decode_of_nothing():
    from linear_attention_gated_gb300 import kda_gated_delta_decode
    e = torch.empty(0, 1, 2, D, dtype=torch.bfloat16, device="cuda")
    o = kda_gated_delta_decode(e, e, e, None, e[..., 0].contiguous(), torch.zeros(1, 2, D, D, device="cuda"))
    assert o.shape == (0, 1, 2, D)


def test_a_pool_past_32_bit_offsets():
    """Slots whose first byte lies past 2^32 of a BF16 pool."""
    from linear_attention_gated_gb300 import kda_gated_delta_decode, kda_gated_delta_prefill
    hv = 64
    slots = 2 ** 32 // (hv * D * D * 2) + 40
    pool = torch.zeros(slots, hv, D, D, dtype=torch.bfloat16, device="cuda")
    idx = torch.tensor([slots - 1, 3, slots - 30], dtype=torch.int32)
    x = make((5, 66, 1), hv, hv, seed=37)
    t = make((1,) * 3, hv, hv, seed=38, packed=False)
    small = torch.zeros(3, hv, D, D, dtype=torch.bfloat16, device="cuda")
    outs = []
    for p, i in ((pool, idx), (small, None)):
        di = None if i is None else i.cuda()
        o = kda_gated_delta_prefill(*(x[n].cuda() for n in TOKENS), p, x["cu"].cuda(), di, cu_seqlens_cpu=x["cu"], state_indices_cpu=i)
        outs.append((o, kda_gated_delta_decode(*(t[n].cuda() for n in TOKENS), p, di, state_indices_cpu=i)))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert torch.equal(pool[idx.long().cuda()], small)
    used = torch.zeros(slots, dtype=torch.bool)
    used[idx.long()] = True
    assert not pool[~used.cuda()].any()


def test_tokens_past_32_bit_offsets():
    """A sequence of 100 tokens behind one whose values take 4 GiB: as alone, in training and in prefill."""
    from linear_attention_gated_gb300 import kda_gated_delta_bwd, kda_gated_delta_fwd, kda_gated_delta_prefill
    hv = 64
    before = 2 ** 32 // (hv * D * 2) + 130
    small = make((100,), 1, hv, seed=44)
    cu = torch.tensor([0, before, before + 100])
    big = {n: torch.zeros(1, before + 100, *small[n].shape[2:], dtype=torch.bfloat16, device="cuda") for n in TOKENS + ("do",)}
    for n in big:
        big[n][:, before:] = small[n].cuda()
    d = {n: t.cuda() for n, t in small.items()}
    h0, dhT = (torch.cat([torch.zeros_like(d[n]), d[n]]) for n in ("h0", "dhT"))
    o, hT, ctx = kda_gated_delta_fwd(*(big[n] for n in TOKENS), h0, cu.cuda(), cu_seqlens_cpu=cu)
    got = (o, hT) + kda_gated_delta_bwd(ctx, big["do"], dhT)
    ctx.status()
    want, _ = run(small)
    for n, t in zip(NAMES, got):
        assert torch.equal(t[1:] if n in ("hT", "dh0") else t[:, before:], want[n]), n
    assert not got[0][:, :before].any()
    del got, ctx, o
    pool = h0.clone()
    o = kda_gated_delta_prefill(*(big[n] for n in TOKENS), pool, cu.cuda(), cu_seqlens_cpu=cu)
    alone = d["h0"].clone()
    assert torch.equal(o[:, before:], kda_gated_delta_prefill(*(d[n] for n in TOKENS), alone, d["cu"], cu_seqlens_cpu=small["cu"]))
    assert torch.equal(pool[1:], alone)
