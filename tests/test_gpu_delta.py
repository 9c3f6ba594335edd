"""The gated delta rule, on the GPU, against its recurrence in 64 bits.

Tolerances. BF16 outputs: each operand that is rounded to BF16 on the way (the state or its adjoint, u, rho, the
masked products, the output itself) adds an independent relative error of at most half a step, 2^-8, so of rms at
most 2^-8 / sqrt(3): three of them for a term of o and its rounding (relative L2 2^-8), five for a gradient.
FP32 states: an operand in two BF16 parts is off by an rms of 0.436 2^-17 at most (lo is uniform in +-2^-8 of a value in
[1, 2), and its own half step 2^-17 with chance 1/2, 2^-18 with 1/4 and so on). Four of them feed a state (S, x, T, u)
and five its adjoint (G, P, d, T, rho), and solving the triangular system of keys of norm 1 doubles an error's square.

Single values: every operand's error is relative to the operand, and all operands of a value belong to its own token (its
row of 128 values): with u or rho ten times the usual length in a token, the roundings of that token's gradients are ten
times the usual too, also in the values that happen to be small. So a value is held to half a step of its own and six
of its row's rms (or the tensor's, where that is more); tokens' scalars to their head's (or the tensor's): a head's numbers come
from its own states, and those of slow decays are larger than the others'. A scalar is a sum of products that
may come out far smaller than they are: dg has <G, S>, 128^2 products of two states' values, rms 128 STATE^2, and dbeta
u . (G k), 128 products of values of 1 and of STATE, rms sqrt(128) STATE. Few scalars are held to the rms that such sums have.
"""

import math

import pytest
import torch

from decay_reference import BF16, FP32, rel_l2
from delta_reference import delta_scan

pytestmark = pytest.mark.gpu

O_REL = BF16
GRAD_REL = BF16 * math.sqrt(5 / 3)
STATE_REL = {"hT": 0.436 * 2.0 ** -17 * math.sqrt(2 * 4) + 16 * FP32, "dh0": 0.436 * 2.0 ** -17 * math.sqrt(2 * 5) + 16 * FP32}
D = 128
STATE = 0.05  # rms of a state's values
SCALAR = {"dg": 128 * STATE ** 2, "dbeta": math.sqrt(128) * STATE}
SCALE = 1 / math.sqrt(128)
GRADS = ("dq", "dk", "dv", "dg", "dbeta", "dh0")


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from linear_attention_gated_gb300 import build
    build.build()
    from linear_attention_gated_gb300 import kda
    kda.load_library()


def make(lens, hqk, hv, seed, gate=True, packed=True, state=STATE, alike=0.0):
    """Inputs on the CPU; lens of the packed sequences, or B equal ones. alike: how much all keys have in common."""
    gen = torch.Generator().manual_seed(seed)
    B, T = (1, sum(lens)) if packed else (len(lens), lens[0])
    x = dict(q=torch.randn(B, T, hqk, D, generator=gen), k=torch.randn(B, T, hqk, D, generator=gen))
    x["k"] = x["k"] + alike * torch.randn(1, 1, hqk, D, generator=gen)
    x = {n: t / t.norm(dim=-1, keepdim=True) for n, t in x.items()}
    x.update(v=torch.randn(B, T, hv, D, generator=gen), do=torch.randn(B, T, hv, D, generator=gen),
             beta=torch.sigmoid(torch.randn(B, T, hv, generator=gen)))
    if gate:
        x["g"] = -torch.rand(B, T, hv, generator=gen) * torch.rand(1, 1, hv, generator=gen)
    x = {n: t.bfloat16() for n, t in x.items()}
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
    f = {n: x[n].to(device).double().flatten(0, 1) for n in ("q", "k", "v", "do", "beta")}
    g = x["g"].to(device).double().flatten(0, 1) if "g" in x else torch.zeros_like(f["beta"])
    h0 = x["h0"].to(device).double() * (1 if with_state else 0)
    leaves = [f["q"], f["k"], f["v"], g, f["beta"], h0]
    if grads:
        leaves = [t.clone().requires_grad_() for t in leaves]
    o, hT = delta_scan(*leaves, spans_of(x), scale)
    qs, shape = x["q"].shape, x["v"].shape
    out = dict(o=o.detach().reshape(shape), hT=hT.detach())
    if grads:
        loss = (o * f["do"]).sum() + ((hT * x["dhT"].to(device).double()).sum() if with_dstate else 0)
        gr = torch.autograd.grad(loss, leaves, allow_unused=True)
        gr = [torch.zeros_like(t) if d is None else d for d, t in zip(gr, leaves)]
        for n, d, s in zip(GRADS, gr, (qs, qs, shape, shape[:3], shape[:3], h0.shape)):
            out[n] = d.reshape(s)
    return out


def run(x, grads=True, scale=None, ctx=None, with_state=True, with_dstate=True):
    from linear_attention_gated_gb300 import kda_gated_delta_bwd, kda_gated_delta_fwd
    d = {n: t.cuda() for n, t in x.items()}
    o, hT, ctx = kda_gated_delta_fwd(d["q"], d["k"], d["v"], d.get("g"), d["beta"], d["h0"] if with_state else None, d.get("cu"), scale,
                                     context_out=ctx, cu_seqlens_cpu=x.get("cu"))
    out = dict(o=o, hT=hT)
    if grads:
        out.update(zip(GRADS, kda_gated_delta_bwd(ctx, d["do"], d["dhT"] if with_dstate else None)))
    torch.cuda.synchronize()
    ctx.status()
    return out, ctx


def check_rows(name, x, ref, rel):
    x, ref = x.double().cpu(), ref.double().cpu()
    assert x.shape == ref.shape and torch.isfinite(x).all(), name
    if ref.numel() == 0:
        return
    size = ref.square().mean().sqrt().clamp(min=SCALAR.get(name, 0))
    off = (x - ref).square().mean().sqrt() / size
    assert off <= rel, (name, off.item(), rel)
    if ref.dim() == 4:
        size = torch.maximum(size, ref.square().mean(-1, keepdim=True).sqrt())
    elif name in SCALAR:
        size = torch.maximum(size, ref.square().mean((0, 1), keepdim=True).sqrt())
    bad = (x - ref).abs() > BF16 * ref.abs() + 6 * BF16 * torch.maximum(size, ref.abs())
    assert not bad.any(), (name, int(bad.sum()))


def compare(got, ref):
    for n, t in got.items():
        if t is None:
            continue
        if n in STATE_REL:
            assert rel_l2(t, ref[n]) <= STATE_REL[n], (n, rel_l2(t, ref[n]))
        else:
            assert t.dtype == torch.bfloat16
            check_rows(n, t, ref[n], O_REL if n == "o" else GRAD_REL)


@pytest.mark.parametrize("lens", [(1,), (2, 1), (15, 17, 16), (63, 64, 65), (127, 1, 128, 129), (200, 31, 260)], ids=str)
@pytest.mark.parametrize("hqk,hv,gate", [(1, 1, True), (2, 4, True), (3, 3, False), (1, 5, True)])
def test_packed(lens, hqk, hv, gate):
    x = make(lens, hqk, hv, seed=len(lens) * 10 + hv, gate=gate)
    got, _ = run(x)
    assert (got["dg"] is None) == (not gate)
    compare(got, reference(x))


@pytest.mark.parametrize("B,T", [(2, 1), (3, 64), (2, 193)])
def test_fixed_layout_and_scale(B, T):
    x = make([T] * B, 2, 2, seed=T, packed=False)
    got, _ = run(x, scale=0.25)
    compare(got, reference(x, scale=0.25))


def test_without_states():
    x = make((70, 140), 1, 2, seed=3)
    got, _ = run(x, with_state=False, with_dstate=False)
    assert got.pop("dh0") is None
    compare(got, reference(x, with_state=False, with_dstate=False))


def test_empty_sequences_pass_their_state_on():
    x = make((0, 5, 0, 130, 0), 1, 2, seed=4)
    got, _ = run(x)
    compare(got, reference(x))
    for n in (0, 2, 4):
        assert torch.equal(got["hT"][n].cpu(), x["h0"][n]) and torch.equal(got["dh0"][n].cpu(), x["dhT"][n])


def test_no_tokens():
    x = make((0, 0), 1, 2, seed=5)
    got, _ = run(x)
    assert got["o"].shape == (1, 0, 2, D) and got["dq"].shape == (1, 0, 1, D)
    assert torch.equal(got["hT"].cpu(), x["h0"]) and torch.equal(got["dh0"].cpu(), x["dhT"])


@pytest.mark.parametrize("lens,hqk,hv,gate", [((3100,), 1, 1, True), ((2900, 0, 77, 3400), 1, 2, False)], ids=str)
def test_sequences_cut_into_segments(lens, hqk, hv, gate):
    """Long sequences of few heads: each is cut, and the segments' states are chained."""
    from linear_attention_gated_gb300 import gated_delta_workspace_bytes
    x = make(lens, hqk, hv, seed=11, gate=gate)
    places = (sum(lens) // 64 + len(lens)) * hv
    assert gated_delta_workspace_bytes(1, sum(lens), hqk, hv, x["cu"], False) > places * 26624 + 256  # (what uncut ones take)
    if gate:  # decays that leave something of the state over a segment
        x["g"] = (x["g"].float() * 0.02).bfloat16()
    got, _ = run(x)
    compare(got, reference(x, device="cuda"))
