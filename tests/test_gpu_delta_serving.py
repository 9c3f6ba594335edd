"""Prefill and decode of the gated delta rule on a state pool, on the GPU, against its recurrence in 64 bits. Tolerances as in
test_gpu_delta.py; a decode step is FP32 throughout but for o's rounding (and a BF16 pool's), with sums of 128 products in
8 + 4 additions."""

import pytest
import torch

from decay_reference import BF16, FP32, rel_l2
from delta_reference import delta_scan
from test_gpu_delta import D, O_REL, SCALE, STATE_REL, check_rows, library, make, spans_of  # noqa: F401

pytestmark = pytest.mark.gpu


def serve(lens, hqk, hv, dtype, seed, gate=True, spare=2, indices=True):
    x = make(lens, hqk, hv, seed=seed, gate=gate)
    N, gen = len(lens), torch.Generator().manual_seed(seed)
    slots = N + spare
    pool = (0.05 * torch.randn(slots, hv, D, D, generator=gen)).to(dtype)
    idx = torch.randperm(slots, generator=gen)[:N].to(torch.int32) if indices else None
    return x, pool, idx


def reference(x, pool, idx, lens, device="cuda"):
    f = {n: x[n].to(device).double().flatten(0, 1) for n in ("q", "k", "v", "beta")}
    g = x["g"].to(device).double().flatten(0, 1) if "g" in x else torch.zeros_like(f["beta"])
    at = torch.arange(len(lens)) if idx is None else idx.long()
    o, S = delta_scan(f["q"], f["k"], f["v"], g, f["beta"], pool.to(device).double()[at], spans_of(x), SCALE)
    return o.reshape(x["v"].shape), S


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("lens,hqk,hv,gate", [((1,), 1, 1, True), ((64, 0, 65, 300), 2, 4, True), ((7, 200), 3, 3, False), ((1000, 30), 1, 2, True)])
def test_prefill(lens, hqk, hv, gate, dtype):
    from linear_attention_gated_gb300 import kda_gated_delta_prefill
    x, pool, idx = serve(lens, hqk, hv, dtype, seed=sum(lens) + hv, gate=gate)
    ref_o, ref_S = reference(x, pool, idx, lens)
    d = {n: t.cuda() for n, t in x.items()}
    got, di = pool.cuda(), idx.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o = kda_gated_delta_prefill(d["q"], d["k"], d["v"], d.get("g"), d["beta"], got, d["cu"], di, device_status=status,
                                cu_seqlens_cpu=x["cu"], state_indices_cpu=idx)
    check_rows("o", o, ref_o, O_REL)
    S = got[idx.long().cuda()]
    rounding = 0 if dtype is torch.float32 else BF16
    assert rel_l2(S, ref_S) <= STATE_REL["hT"] + rounding
    rest = [i for i in range(len(pool)) if i not in idx.tolist()]
    assert torch.equal(got[rest].cpu(), pool[rest]) and status.item() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("N,hqk,hv,gate,indices", [(1, 1, 1, True, True), (5, 2, 6, True, True), (33, 4, 4, False, False)])
def test_decode(N, hqk, hv, gate, indices, dtype):
    from linear_attention_gated_gb300 import kda_gated_delta_decode
    x, pool, idx = serve((1,) * N, hqk, hv, dtype, seed=N + hv, gate=gate, indices=indices)
    ref_o, ref_S = reference(x, pool, idx, (1,) * N)
    step = {n: x[n].cuda().reshape(N, 1, *x[n].shape[2:]) for n in ("q", "k", "v", "beta", "g") if n in x}
    got = pool.cuda()
    o = kda_gated_delta_decode(step["q"], step["k"], step["v"], step.get("g"), step["beta"], got,
                               None if idx is None else idx.cuda(), state_indices_cpu=idx)
    at = torch.arange(N) if idx is None else idx.long()
    # o: half a step of its own, and FP32 sums of 128 products (rms of the terms' sum: at most some ten times o's)
    off = (o.reshape(ref_o.shape).double() - ref_o).abs()
    assert (off <= BF16 * ref_o.abs() + 128 * FP32 * 10 * ref_o.square().mean().sqrt()).all()
    rounding = 0 if dtype is torch.float32 else BF16
    assert rel_l2(got[at.cuda()], ref_S) <= rounding + 16 * FP32
    rest = [i for i in range(len(pool)) if i not in at.tolist()]
    assert torch.equal(got[rest].cpu(), pool[rest])


def test_prefill_then_decode_is_one_sequence():
    """Chunks of a prompt, then tokens one by one, on one pool: as the whole sequence at once."""
    from linear_attention_gated_gb300 import kda_gated_delta_decode, kda_gated_delta_prefill
    T, hqk, hv = 150, 2, 4
    x, pool, _ = serve((T,), hqk, hv, torch.float32, seed=1, spare=0, indices=False)
    ref_o, ref_S = reference(x, pool, None, (T,))
    d = {n: t.cuda() for n, t in x.items()}
    got, outs = pool.cuda(), []
    for a, b in ((0, 70), (70, 71), (71, 140)):
        outs.append(kda_gated_delta_prefill(*(d[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "beta")), got))
    for t in range(140, T):
        outs.append(kda_gated_delta_decode(*(d[n][:, t:t + 1].contiguous() for n in ("q", "k", "v", "g", "beta")), got))
    check_rows("o", torch.cat(outs, 1), ref_o, O_REL)
    assert rel_l2(got, ref_S) <= STATE_REL["hT"]


def test_views_of_one_projection():
    from linear_attention_gated_gb300 import kda_gated_delta_decode, kda_gated_delta_prefill
    x, pool, _ = serve((90,), 2, 4, torch.float32, seed=2, spare=0, indices=False)
    d = {n: t.cuda() for n, t in x.items()}
    fused = torch.cat([d["q"], d["k"], d["v"]], 2)
    q, k, v = fused.split([2, 2, 4], 2)
    a, b = pool.cuda(), pool.cuda()
    assert torch.equal(kda_gated_delta_prefill(q, k, v, d["g"], d["beta"], a), kda_gated_delta_prefill(d["q"], d["k"], d["v"], d["g"], d["beta"], b))
    assert torch.equal(a, b)
    step = [t[:, :1] for t in (q, k, v)]
    gates = [d[n][:, :1].contiguous() for n in ("g", "beta")]
    assert torch.equal(kda_gated_delta_decode(*step, *gates, a), kda_gated_delta_decode(*(t.contiguous() for t in step), *gates, b))
    assert torch.equal(a, b)


def test_replayed_indices_outside_the_pool():
    """A captured step whose device indices were rewritten: a bad one touches nothing and reads NaN (prefill: sets bit 4)."""
    from linear_attention_gated_gb300 import kda_gated_delta_decode, kda_gated_delta_prefill
    N, hv = 3, 2
    x, pool, idx = serve((1,) * N, 1, hv, torch.float32, seed=3)
    d = {n: x[n].cuda() for n in ("q", "k", "v", "g", "beta", "cu")}
    step = [d[n].reshape(N, 1, *d[n].shape[2:]) for n in ("q", "k", "v", "g", "beta")]
    got, di = pool.cuda(), idx.cuda()
    di[1] = len(pool) + 5
    o = kda_gated_delta_decode(*step, got, di, state_indices_cpu=idx)
    assert o[1].isnan().all() and o[[0, 2]].isfinite().all()
    touched = [idx[0].item(), idx[2].item()]
    rest = [i for i in range(len(pool)) if i not in touched]
    assert torch.equal(got[rest].cpu(), pool[rest])
    got, status = pool.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda")
    kda_gated_delta_prefill(*(d[n] for n in ("q", "k", "v", "g", "beta")), got, d["cu"], di, device_status=status,
                            cu_seqlens_cpu=x["cu"], state_indices_cpu=idx)
    assert status.item() == 4 and torch.equal(got[rest].cpu(), pool[rest])
