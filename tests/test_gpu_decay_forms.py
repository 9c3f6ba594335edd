"""Forms of the calls of the linear attention with a decay for each head and of the norm and rotation that stand beside the
usual ones: groups of other sizes, sequences of a fixed layout cut into segments, buffers of the caller, captured graphs,
device offsets that disagree with their mirror. On the GPU; tolerances as for the usual forms."""

import math

import pytest
import torch

import test_gpu_qk_norm_rope as rope
from decay_reference import BF16, check, rel_l2
from test_gpu_decay import (D, O_REL, STATE_REL, compare, library, make, reference, run)  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hqk,hv", [(2, 6), (1, 5), (2, 12), (1, 7)])
def test_groups_of_heads(hqk, hv):
    """Sums over 3, 5, 6 and 7 value heads, and what crosses each of them."""
    x = make((70, 33, 65), hqk, hv, "token", seed=41)
    compare(run(x)[0], reference(x))


@pytest.mark.parametrize("gate", ["token", "head"])
def test_fixed_layout_cut_into_segments(gate):
    from linear_attention_gated_gb300 import decay_workspace_bytes
    B, T = 2, 3100
    assert decay_workspace_bytes(B, T, 1, 2, training=False) > 0  # the segments' states
    x = make([T] * B, 1, 2, gate, seed=42, packed=False)
    compare(run(x)[0], reference(x, device="cuda"))


def test_buffers_of_the_caller():
    from linear_attention_gated_gb300 import kda_decay_attn_bwd, kda_decay_attn_fwd
    x = make((90, 40), 2, 4, "token", seed=43)
    want, _ = run(x)
    d = {n: t.cuda() for n, t in x.items()}
    mine = {n: torch.full_like(t, float("nan")) for n, t in want.items()}
    o, hT, ctx = kda_decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], d["cu"], out=mine["o"], final_state_out=mine["hT"],
                                    cu_seqlens_cpu=x["cu"])
    grads = tuple(mine[n] for n in ("dq", "dk", "dv", "dg", "dh0"))
    got = kda_decay_attn_bwd(ctx, d["do"], d["dhT"], out=grads)
    assert o is mine["o"] and hT is mine["hT"] and all(a is b for a, b in zip(got, grads))
    for n, t in want.items():
        assert torch.equal(t, mine[n]), n


def test_prefill_with_a_workspace():
    from linear_attention_gated_gb300 import KdaError, decay_workspace_bytes, kda_decay_attn_prefill
    x = make((5000, 30), 1, 1, "head", seed=44)
    d = {n: t.cuda() for n, t in x.items()}
    nbytes = decay_workspace_bytes(1, 5030, 1, 1, x["cu"], per_token=False, training=False)
    outs = []
    for ws in (None, torch.full((nbytes,), 255, dtype=torch.uint8, device="cuda")):
        pool = d["h0"].clone()
        o = kda_decay_attn_prefill(d["q"], d["k"], d["v"], d["g"], pool, d["cu"], workspace=ws, cu_seqlens_cpu=x["cu"])
        outs.append((o, pool))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    with pytest.raises(KdaError):
        kda_decay_attn_prefill(d["q"], d["k"], d["v"], d["g"], pool, d["cu"], workspace=ws[:nbytes - 256], cu_seqlens_cpu=x["cu"])


def test_norm_backward_with_a_workspace():
    from linear_attention_gated_gb300 import kda_qk_norm_rope_bwd
    x = rope.make(2, 77, 5, 2, 128, 64, torch.bfloat16, seed=45)
    want = rope.run(x, False)
    d = {n: t.cuda() for n, t in x.items()}
    ws = torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
    mine = torch.empty_like(d["q"]), torch.empty_like(d["k"])
    got = kda_qk_norm_rope_bwd(d["dq"], d["dk"], d["q"], d["k"], d["qw"], d["kw"], d["pos"], d["freq"], out=mine, workspace=ws)
    for n, t in zip(("dq", "dk", "dqw", "dkw"), got):
        assert torch.equal(t, want[n]), n


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_serving_in_graphs(dtype):
    """A prefill and a decode step, captured and replayed with other inputs and slots."""
    from linear_attention_gated_gb300 import kda_decay_attn_decode, kda_decay_attn_prefill
    lens, hqk, hv, slots = (70, 1, 33), 2, 4, 5
    prompts = [make(lens, hqk, hv, "token", seed=46 + i) for i in range(2)]
    tokens = [make((1,) * 3, hqk, hv, "token", seed=48 + i, packed=False) for i in range(2)]
    order = [torch.tensor(i, dtype=torch.int32) for i in ((4, 0, 2), (1, 3, 0))]
    pools = [torch.randn(slots, hv, D, D, generator=torch.Generator().manual_seed(50 + i)).mul(0.05).to(dtype) for i in range(2)]
    p, t = ({n: v.cuda() for n, v in x[0].items()} for x in (prompts, tokens))
    idx, pool = order[0].cuda(), pools[0].cuda()

    def step():
        o = kda_decay_attn_prefill(p["q"], p["k"], p["v"], p["g"], pool, p["cu"], idx, cu_seqlens_cpu=prompts[0]["cu"],
                                   state_indices_cpu=order[0])
        return o, kda_decay_attn_decode(t["q"], t["k"], t["v"], t["g"], pool, idx, state_indices_cpu=order[0])

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
    check("o", o, ref["o"], O_REL, BF16)
    tokens[1]["h0"] = ref["hT"].to(dtype).double()  # (rounded to the pool's type between the two)
    ref = reference(tokens[1], grads=False)
    check("o1", o1, ref["o"], O_REL, BF16)
    after = pool.cpu()
    rest = [i for i in range(slots) if i not in at.tolist()]
    assert torch.equal(after[rest], pools[1][rest])
    if dtype == torch.float32:
        assert rel_l2(after[at], ref["hT"]) <= STATE_REL
    else:
        check("pool", after[at], ref["hT"], BF16 * math.sqrt(2 / 3) + STATE_REL, BF16)


@pytest.mark.parametrize("bad", [[0, 70, 3170], [0, 5000, -4], [-9, 1 << 40, 1 << 62], [3170, 0, 3170], [3170, 3170, 3170]], ids=str)
def test_device_offsets_that_disagree_with_the_mirror(bad):
    """They are held inside the tensors: nothing around the outputs changes, and the next call is right."""
    from linear_attention_gated_gb300 import kda_decay_attn_bwd, kda_decay_attn_fwd
    x = make((3100, 70), 1, 2, "token", seed=47)  # the first is cut into segments
    want, _ = run(x)
    d = {n: t.cuda() for n, t in x.items()}
    names = ("o", "hT", "dq", "dk", "dv", "dg", "dh0")
    room = {n: torch.full((want[n].numel() + 2 * 4096,), 3.0, dtype=want[n].dtype, device="cuda") for n in names}
    mine = {n: room[n][4096:-4096].view(want[n].shape) for n in names}

    def step(cu):
        _, _, ctx = kda_decay_attn_fwd(d["q"], d["k"], d["v"], d["g"], d["h0"], cu, out=mine["o"], final_state_out=mine["hT"],
                                       cu_seqlens_cpu=x["cu"])
        kda_decay_attn_bwd(ctx, d["do"], d["dhT"], out=tuple(mine[n] for n in names[2:]))
        ctx.status()

    step(torch.tensor(bad, device="cuda"))
    for n in names:
        assert (room[n][:4096] == 3).all() and (room[n][-4096:] == 3).all(), n
    for n, t in (("q", d["q"]), ("h0", d["h0"]), ("g", d["g"])):
        assert torch.equal(t.cpu(), x[n]), n
    step(d["cu"])
    for n in names:
        assert torch.equal(mine[n], want[n]), n
