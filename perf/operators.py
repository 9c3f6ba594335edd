"""Cases that measure the linear attention with a decay for each head and the norm and position
rotation of its queries and keys: one pass through an operator of the package (``own`` true), or the
same mathematics in elementary torch operations (``own`` false).

Per value head h (it reads query/key head h // (Hv // Hqk)), with a value-first state S [128, 128]:

    S_t = exp(g_t) S_{t-1} + v_t k_t^T,    o_t = s S_t q_t,    s = 1 / sqrt(128)

g is a fixed FP32 number per head or a BF16 number per token and head. Queries and keys are
normalised per head, y = R(pos) (x w / sqrt(mean(x^2) + eps)), where R turns pairs of the first
2 * len(inv_freq) dimensions by pos * inv_freq.
"""

import math
import random

import torch

own = False

DIM = 128
SCALE = 1.0 / math.sqrt(DIM)
CHUNK = 128  # tokens of one chunk in the plain form
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # queries and keys of one decode step: 16 requests, 32 heads, positions deep in their contexts
        dict(name="rope_step", op="rope_fwd", B=16, T=1, hq=32, hk=32, D=128, rot=128, pairs="half", dtype="bf16", fused=False,
             far=100000),
        # a prompt of odd length, 64 query and 8 key heads read from one fused projection, half of each head rotated
        dict(name="rope_prompt_fused", op="rope_fwd", B=1, T=8191, hq=64, hk=8, D=128, rot=64, pairs="half", dtype="bf16",
             fused=True, far=0),
        # gradients of the norm and rotation in a training step of 4 x 2048 tokens, 16 query and 16 key heads
        dict(name="rope_train_bwd", op="rope_bwd", B=4, T=2048, hq=16, hk=16, D=128, rot=128, pairs="half", dtype="bf16",
             fused=False, far=0),
        # the same for a short ragged batch of 64-wide heads in FP16, neighbouring dimensions paired
        dict(name="rope_bwd_narrow", op="rope_bwd", B=1, T=1537, hq=40, hk=10, D=64, rot=64, pairs="neighbours", dtype="fp16",
             fused=False, far=0),
        # the shortest prompt: one request of 64 tokens, two heads
        dict(name="prefill_64", op="prefill", lens="fixed", N=1, T=64, hqk=2, hv=2, gate="head", pool="fp32", spare=1),
        # 8 prompts of 1024 tokens, 96 heads, a BF16 state pool
        dict(name="prefill_8x1024_h96", op="prefill", lens="fixed", N=8, T=1024, hqk=96, hv=96, gate="head", pool="bf16", spare=4),
        # 24 prompts of 1 to 4000 tokens, 8 key heads for 64 value heads, a decay for each token
        dict(name="prefill_24mixed_hqk8_hv64", op="prefill", lens="mixed", N=24, T=4000, hqk=8, hv=64, gate="token", pool="fp32",
             spare=4),
        # one long prompt of odd length: few rows, a long axis
        dict(name="prefill_32771_h32", op="prefill", lens="fixed", N=1, T=32771, hqk=16, hv=32, gate="head", pool="fp32", spare=1),
        # a training step (forward and gradients), 4 x 2048 tokens, 16 key heads for 32 value heads, a decay for each token
        dict(name="train_4x2048_hqk16_hv32", op="train", lens="fixed", N=4, T=2048, hqk=16, hv=32, gate="token"),
        # a training step on packed sequences of 1 to 2000 tokens, 32 heads, fixed decays
        dict(name="train_8mixed_h32", op="train", lens="mixed", N=8, T=2000, hqk=32, hv=32, gate="head"),
        # one token of one request, 32 heads
        dict(name="decode_1xh32", op="decode", N=1, hqk=32, hv=32, gate="token", pool="fp32", spare=3),
        # one token of 256 requests, 96 heads, a BF16 state pool
        dict(name="decode_256xh96", op="decode", N=256, hqk=96, hv=96, gate="token", pool="bf16", spare=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope_fwd", "rope_bwd", "prefill", "prefill", "train", "decode"])
    if op in ("rope_fwd", "rope_bwd"):
        D = rng.choice([64, 96, 128, 192, 256])
        hq = rng.choice([1, 5, 8, 16, 32, 64])
        hk = max(1, hq // rng.choice([1, 1, 4, 8]))
        most = (8191 * 72 * 128 if op == "rope_fwd" else 8192 * 32 * 128) // ((hq + hk) * D)
        T = _log_int(rng, 1, min(most, 20000))
        B = rng.randint(1, max(1, min(16, most // T)))
        return dict(op=op, B=B, T=T, hq=hq, hk=hk, D=D, rot=rng.choice([0, D // 2 // 16 * 16, D]),
                    pairs=rng.choice(["half", "neighbours"]), dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    fused=rng.random() < 0.5, far=rng.choice([0, 0, 1000000]))
    hv = rng.choice([1, 2, 6, 16, 32, 48, 64, 96])
    hqk = rng.choice([d for d in (1, 2, 3, 8, 16, 32, 96) if hv % d == 0])
    gate = rng.choice(["head", "token"])
    pool = rng.choice(["fp32", "bf16"])
    if op == "decode":
        N = _log_int(rng, 1, min(300, 256 * 96 // hv // (2 if pool == "fp32" else 1)))
        return dict(op=op, N=N, hqk=hqk, hv=hv, gate=gate, pool=pool, spare=rng.randint(0, 5))
    most = (8 * 1024 * 96 if op == "prefill" else 4 * 2048 * 32) // hv
    lens = rng.choice(["fixed", "mixed"])
    T = _log_int(rng, 1, min(most, 33000))
    N = rng.randint(1, max(1, min(24, most // T)))
    case = dict(op=op, lens=lens, N=N, T=T, hqk=hqk, hv=hv, gate=gate)
    return dict(case, pool=pool, spare=rng.randint(0, 5)) if op == "prefill" else case


def _lengths(case):
    if case["lens"] == "fixed":
        return [case["T"]] * case["N"]
    rng = random.Random(1000003 * case["N"] + case["T"])
    return [rng.randint(1, case["T"]) for _ in range(case["N"])]


def work(case):
    if case["op"] in ("rope_fwd", "rope_bwd"):
        values = case["B"] * case["T"] * (case["hq"] + case["hk"]) * case["D"]
        size = DTYPES[case["dtype"]].itemsize
        moved = 2 if case["op"] == "rope_fwd" else 3
        return dict(bytes=moved * values * size + 8 * case["B"] * case["T"], flops=(8 if case["op"] == "rope_fwd" else 16) * values)
    N, hqk, hv = case["N"], case["hqk"], case["hv"]
    Ttot = N if case["op"] == "decode" else sum(_lengths(case))
    gate = 2 * Ttot * hv if case["gate"] == "token" else 4 * hv
    q, v, state = 2 * Ttot * hqk * DIM, 2 * Ttot * hv * DIM, N * hv * DIM * DIM
    step = 2 * Ttot * hv * DIM * DIM  # flops of one product of the state with a vector for each token
    if case["op"] == "train":  # reads q, k, v, g, do, h0, dhT; writes o, hT, dq, dk, dv, dg, dh0
        return dict(bytes=4 * q + 4 * v + (2 if case["gate"] == "token" else 1) * gate + 4 * 4 * state, flops=7 * step)
    size = DTYPES[case["pool"]].itemsize
    return dict(bytes=2 * q + 2 * v + gate + 2 * size * state, flops=2 * step)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16, by=1.0):
        return (by * torch.randn(shape, generator=gen, device="cuda")).to(dtype)

    s = dict(case)
    if case["op"] in ("rope_fwd", "rope_bwd"):
        B, T, hq, hk, D, dt = case["B"], case["T"], case["hq"], case["hk"], case["D"], DTYPES[case["dtype"]]
        if case["fused"]:  # queries and keys are views of one projection that holds the values too
            x = randn(B, T, hq + 2 * hk, D, dtype=dt)
            s["q"], s["k"] = x[:, :, :hq], x[:, :, hq:hq + hk]
        else:
            s["q"], s["k"] = randn(B, T, hq, D, dtype=dt), randn(B, T, hk, D, dtype=dt)
        s["qw"], s["kw"] = 1 + randn(D, dtype=torch.float32, by=0.1), 1 + randn(D, dtype=torch.float32, by=0.1)
        first = torch.randint(0, case["far"] + 1, (B, 1), generator=gen, device="cuda")
        s["pos"] = (first + torch.arange(T, device="cuda")).contiguous()
        half = case["rot"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half) if half else None
        if case["op"] == "rope_bwd":
            s["dq"], s["dk"] = randn(B, T, hq, D, dtype=dt), randn(B, T, hk, D, dtype=dt)
        return s
    N, hqk, hv = case["N"], case["hqk"], case["hv"]
    if case["op"] == "decode":
        B, T = N, 1
    elif case["lens"] == "fixed":
        B, T = N, case["T"]
    else:
        B, T = 1, sum(_lengths(case))
        s["cu_cpu"] = torch.tensor([0] + _lengths(case), dtype=torch.int64).cumsum(0)
        s["cu"] = s["cu_cpu"].cuda()
    s["q"], s["k"] = randn(B, T, hqk, DIM), randn(B, T, hqk, DIM)
    s["v"] = randn(B, T, hv, DIM)
    if case["gate"] == "head":  # decays from about 0.4 to 0.996 a token
        s["g"] = -torch.exp2(-8.0 * torch.arange(1, hv + 1, device="cuda") / hv) * (1 + 0.1 * torch.rand(hv, generator=gen, device="cuda"))
    else:  # a step size for each token, a rate for each head
        rate = 1 + 15 * torch.rand(hv, generator=gen, device="cuda")
        s["g"] = (-rate * torch.exp(math.log(0.001) + math.log(100.0) * torch.rand((B, T, hv), generator=gen, device="cuda"))).bfloat16()
    if case["op"] == "train":
        s["h0"], s["dhT"] = (randn(N, hv, DIM, DIM, dtype=torch.float32, by=0.05) for _ in range(2))
        s["do"] = randn(B, T, hv, DIM)
        return s
    slots = N + case["spare"]
    s["pool"] = randn(slots, hv, DIM, DIM, dtype=DTYPES[case["pool"]], by=0.05)
    cpu = torch.Generator("cpu").manual_seed(seed)
    s["idx_cpu"] = torch.randperm(slots, generator=cpu)[:N].to(torch.int32)
    s["idx"] = s["idx_cpu"].cuda()
    return s


def run(s):
    return (_run_own if own else _run_plain)(s)


# ---- the package's operators


def _run_own(s):
    import linear_attention_gated_gb300 as lib

    op = s["op"]
    if op == "rope_fwd":
        return lib.kda_qk_norm_rope_fwd(s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["inv_freq"], eps=EPS,
                                        interleaved=s["pairs"] == "neighbours")
    if op == "rope_bwd":
        return lib.kda_qk_norm_rope_bwd(s["dq"], s["dk"], s["q"], s["k"], s["qw"], s["kw"], s["pos"], s["inv_freq"], eps=EPS,
                                        interleaved=s["pairs"] == "neighbours")
    if op == "decode":
        o = lib.kda_decay_attn_decode(s["q"], s["k"], s["v"], s["g"], s["pool"], s["idx"], state_indices_cpu=s["idx_cpu"])
        return o, s["pool"]
    if op == "prefill":
        o = lib.kda_decay_attn_prefill(s["q"], s["k"], s["v"], s["g"], s["pool"], s.get("cu"), s["idx"],
                                       cu_seqlens_cpu=s.get("cu_cpu"), state_indices_cpu=s["idx_cpu"])
        return o, s["pool"]
    # the context (workspace) is kept from step to step
    o, hT, s["ctx"] = lib.kda_decay_attn_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], s.get("cu"), context_out=s.get("ctx"),
                                             cu_seqlens_cpu=s.get("cu_cpu"))
    dq, dk, dv, dg, dh0 = lib.kda_decay_attn_bwd(s["ctx"], s["do"], s["dhT"])
    return dict(o=o, hT=hT, dq=dq, dk=dk, dv=dv, dh0=dh0, **({} if dg is None else {"dg": dg}))


# ---- the plain form


def _run_plain(s):
    op = s["op"]
    if op == "rope_fwd":
        cos, sin = _angles(s)
        return tuple(_rotate(_normed(s[x])[0] * s[x + "w"], cos, sin, s).to(s[x].dtype) for x in ("q", "k"))
    if op == "rope_bwd":
        cos, sin = _angles(s)
        dq, dwq = _norm_rope_grads(s["dq"], s["q"], s["qw"], cos, sin, s)
        dk, dwk = _norm_rope_grads(s["dk"], s["k"], s["kw"], cos, sin, s)
        return dq, dk, dwq, dwk
    if op == "decode":
        idx, r = s["idx"].long(), s["hv"] // s["hqk"]
        q, k = (s[x][:, 0].float().repeat_interleave(r, dim=1) for x in ("q", "k"))
        g = s["g"][:, 0].float() if s["gate"] == "token" else s["g"]
        S = s["pool"][idx].float() * g.exp()[..., None, None] + s["v"][:, 0].float()[..., :, None] * k[..., None, :]
        s["pool"][idx] = S.to(s["pool"].dtype)
        return (SCALE * (S * q[..., None, :]).sum(-1)).to(torch.bfloat16)[:, None], s["pool"]
    if op == "prefill":
        idx = s["idx"].long()
        c = _chunks(s)
        o, hT = _forward(c, s["pool"][idx].float())[:2]
        s["pool"][idx] = hT.to(s["pool"].dtype)
        return _tokens(o, c).to(torch.bfloat16), s["pool"]
    return _train(s)


def _angles(s):
    """cos and sin of pos * inv_freq [B, T, 1, R / 2]: the angles of far positions need 64 bits."""
    if s["inv_freq"] is None:
        return None, None
    a = s["pos"].double()[..., None, None] * s["inv_freq"]
    return a.cos().float(), a.sin().float()


def _normed(x):
    x = x.float()
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return x * r, r


def _rotate(n, cos, sin, s):
    if cos is None:
        return n
    rot, tail = n[..., :s["rot"]], n[..., s["rot"]:]
    if s["pairs"] == "half":
        a, b = rot.chunk(2, dim=-1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin, tail], dim=-1)
    a, b = rot[..., 0::2], rot[..., 1::2]
    return torch.cat([torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2), tail], dim=-1)


def _norm_rope_grads(dy, x, w, cos, sin, s):
    dn = _rotate(dy.float(), cos, None if sin is None else -sin, s)
    n, r = _normed(x)
    t = dn * w
    dx = r * (t - n * (t * n).mean(-1, keepdim=True))
    return dx.to(x.dtype), (dn * n).sum((0, 1, 2))


def _chunks(s):
    """The tokens in chunks of one sequence each, heads first, and what the chunks' decays come to."""
    N, hv, C = s["N"], s["hv"], CHUNK
    dev, Ttot = s["v"].device, s["v"].shape[0] * s["v"].shape[1]
    cu = s["cu"] if "cu" in s else torch.arange(N + 1, device=dev) * s["T"]
    lens = cu[1:] - cu[:-1]
    per = (lens + C - 1) // C
    seq = torch.repeat_interleave(torch.arange(N, device=dev), per)  # [NC] the sequence of each chunk
    number = torch.arange(len(seq), device=dev) - (per.cumsum(0) - per)[seq]  # its place in it
    at = number[:, None] * C + torch.arange(C, device=dev)
    tok = torch.where(at < lens[seq][:, None], cu[:-1][seq][:, None] + at, Ttot)  # [NC, C], Ttot where there is none
    c = dict(seq=seq, tok=tok, hv=hv, Ttot=Ttot, N=N, like=s["v"].shape)

    def heads_first(x):  # [B, T, H, ...] -> [Hv, NC, C, ...] in 32 bits, zeros where there is no token
        x = x.reshape(Ttot, *x.shape[2:])
        x = torch.cat([x, x.new_zeros(1, *x.shape[1:])])[tok].float()
        x = x.movedim(2, 0)
        return x.repeat_interleave(hv // x.shape[0], dim=0)

    c["heads_first"] = heads_first
    c["q"], c["k"], c["v"] = (heads_first(s[x]) for x in ("q", "k", "v"))
    g = s["g"] if s["gate"] == "token" else s["g"].expand(1, Ttot, hv)
    g = heads_first(g).double()
    b = g.cumsum(-1)  # [Hv, NC, C]
    last = b[..., -1]
    total = last.cumsum(-1)  # over chunks of all sequences: only differences within one are used
    same = seq[:, None] == seq[None, :]
    order = torch.arange(len(seq), device=dev)
    ends = per.cumsum(0) - 1  # the last chunk of each sequence
    before = total - last

    def decays(e, keep):
        return torch.where(keep, e, -torch.inf).exp().float()

    c["lower"] = decays(b[..., :, None] - b[..., None, :], torch.ones(C, C, dtype=torch.bool, device=dev).tril())
    c["from_start"], c["to_end"] = b.exp().float()[..., None], (last[..., None] - b).exp().float()[..., None]
    # what chunk j's part is worth at the start of chunk i, and at the end of its sequence
    c["between"] = decays(before[..., :, None] - total[..., None, :], same & (order[None, :] < order[:, None]))
    c["at_end"] = decays(total[:, ends][..., :, None] - total[..., None, :], torch.arange(N, device=dev)[:, None] == seq[None, :])
    first = (ends - per + 1)[seq]
    c["h0_at_start"] = (before - before[:, first]).exp().float()
    c["h0_at_end"] = (total[:, ends] - before[:, ends - per + 1]).exp().float()
    return c


def _state_product(a, x):
    """[Hv, M, NC] x [Hv, NC, 128, 128] -> [Hv, M, 128, 128]"""
    return (a @ x.flatten(2)).unflatten(2, (DIM, DIM))


def _forward(c, h0):
    """Outputs [Hv, NC, C, 128], final states [N, Hv, 128, 128] and the states at the chunks' starts."""
    h0 = h0.transpose(0, 1)
    part = (c["v"] * c["to_end"]).mT @ c["k"]
    start = _state_product(c["between"], part) + c["h0_at_start"][..., None, None] * h0[:, c["seq"]]
    hT = _state_product(c["at_end"], part) + c["h0_at_end"][..., None, None] * h0
    o = ((c["q"] @ c["k"].mT) * c["lower"]) @ c["v"] + c["from_start"] * (c["q"] @ start.mT)
    return SCALE * o, hT.transpose(0, 1).contiguous(), start


def _tokens(x, c):
    """[Hv, NC, C, ...] -> [B, T, Hv, ...], the inverse of heads_first."""
    out = x.new_empty(c["Ttot"] + 1, *x.shape[:1], *x.shape[3:])
    out[c["tok"]] = x.movedim(0, 2)
    return out[:-1].reshape(*c["like"][:2], *out.shape[1:])


def _train(s):
    c = _chunks(s)
    o, hT, start = _forward(c, s["h0"])
    do, dhT = c["heads_first"](s["do"]), s["dhT"].transpose(0, 1)
    part = SCALE * (do * c["from_start"]).mT @ c["q"]
    # the adjoint of the state at each chunk's end, and of the initial state
    end = _state_product(c["between"].mT, part)
    end += (c["at_end"].gather(1, c["seq"].expand(c["hv"], 1, -1))[:, 0])[..., None, None] * dhT[:, c["seq"]]
    mine = (torch.arange(c["N"], device=do.device)[:, None] == c["seq"][None, :]).float()
    dh0 = _state_product(mine * c["h0_at_start"][:, None, :], part) + c["h0_at_end"][..., None, None] * dhT
    P, A = ((x @ y.mT) * c["lower"] * SCALE for x, y in ((c["q"], c["k"]), (do, c["v"])))
    dq = A @ c["k"] + SCALE * c["from_start"] * (do @ start)
    dk = A.mT @ c["q"] + c["to_end"] * (c["v"] @ end)
    dv = P.mT @ do + c["to_end"] * (c["k"] @ end.mT)
    out = dict(o=_tokens(o, c).to(torch.bfloat16), hT=hT, dv=_tokens(dv, c).to(torch.bfloat16), dh0=dh0.transpose(0, 1).contiguous())
    if s["gate"] == "token":  # a decay scales all that crosses its token: long sums that cancel, in 64 bits
        cross = (c["q"].double() * dq).sum(-1) - (c["k"].double() * dk).sum(-1)  # [Hv, NC, C]
        flat = cross.flatten(1)
        past = flat.flip(1).cumsum(1).flip(1).reshape(cross.shape)  # from here to the end of all sequences
        after = torch.cat([past[:, :, 0], past.new_zeros(c["hv"], 1)], dim=1)
        ends = torch.searchsorted(c["seq"], torch.arange(c["N"], device=do.device), right=True)
        whole = (hT.transpose(0, 1).double() * dhT).sum((-1, -2))  # [Hv, N]
        dg = past + (whole - after[:, ends])[:, c["seq"]][..., None]
        out["dg"] = _tokens(dg, c).to(torch.bfloat16)
    groups = (s["hqk"], s["hv"] // s["hqk"])
    out["dq"], out["dk"] = (_tokens(x.unflatten(0, groups).sum(1), c).to(torch.bfloat16) for x in (dq, dk))
    return out


# ---- the operators' definitions in 64 bits, token by token


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope_fwd":
        return tuple(_exact_rope(s, s[x].double(), s[x + "w"].double()) for x in ("q", "k"))
    if case["op"] == "rope_bwd":
        with torch.enable_grad():
            out = []
            for x, w, dy in ((s["q"], s["qw"], s["dq"]), (s["k"], s["kw"], s["dk"])):
                x, w = x.double().requires_grad_(), w.double().requires_grad_()
                out.append(torch.autograd.grad(_exact_rope(s, x, w), (x, w), dy.double()))
        return out[0][0], out[1][0], out[0][1], out[1][1]
    if case["op"] == "train":
        return _exact_train(s)
    idx = s["idx"].long()
    pool = s["pool"].double()
    o, S = _exact_scan(s, pool[idx])[:2]
    pool[idx] = S
    return o, pool


def _exact_rope(s, x, w):
    n = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w
    if s["inv_freq"] is None:
        return n
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), s["pos"].double()[:, :, None, None] * s["inv_freq"])
    R = s["rot"]
    if s["pairs"] == "half":
        z = torch.complex(n[..., :R // 2], n[..., R // 2:R]) * turn
        return torch.cat([z.real, z.imag, n[..., R:]], dim=-1)
    z = torch.view_as_complex(n[..., :R].unflatten(-1, (R // 2, 2)).contiguous()) * turn
    return torch.cat([torch.view_as_real(z).flatten(-2), n[..., R:]], dim=-1)


def _rows(s):
    """[N, longest] token of each sequence's place, and whether there is one."""
    B, T = s["v"].shape[:2]
    if "cu" in s:
        cu = s["cu"]
    else:
        cu = torch.arange(B + 1, device=s["v"].device) * T
    lens = cu[1:] - cu[:-1]
    at = torch.arange(int(lens.max()), device=cu.device)
    return (cu[:-1, None] + torch.minimum(at, lens[:, None] - 1)), at < lens[:, None]


def _by_step(s, name, tok, r=1):
    """[longest, N, Hv, 128] in 64 bits."""
    x = s[name].flatten(0, 1)
    return x[tok.t()].double().repeat_interleave(r, dim=2)


def _log_decays(s, tok):
    if s["gate"] == "token":
        return s["g"].flatten(0, 1)[tok.t()].double()
    return s["g"].double().expand(tok.shape[1], tok.shape[0], -1)


def _exact_scan(s, S, do=None):
    """o in the layout of v, the last state, and s S^T do for each step."""
    tok, there = _rows(s)
    r = s["hv"] // s["hqk"]
    q, k, v = _by_step(s, "q", tok, r), _by_step(s, "k", tok, r), _by_step(s, "v", tok)
    there = there.t()[..., None]
    g = torch.where(there, _log_decays(s, tok), 0.0).exp()
    v = torch.where(there[..., None], v, 0.0)
    o, dq = torch.zeros_like(v), None if do is None else torch.zeros_like(v)
    for t in range(len(q)):
        S = g[t][..., None, None] * S + v[t][..., :, None] * k[t][..., None, :]
        o[t] = SCALE * (S @ q[t][..., None])[..., 0]
        if do is not None:
            dq[t] = SCALE * (do[t][..., None, :] @ S)[..., 0, :]
    return _back(s, o, tok, there), S, dq


def _back(s, x, tok, there):
    out = x.new_zeros(s["v"].shape[0] * s["v"].shape[1], *x.shape[2:])
    keep = there[..., 0]
    out[tok.t()[keep]] = x[keep]
    return out.unflatten(0, s["v"].shape[:2])


def _exact_train(s):
    tok, there = _rows(s)
    there = there.t()[..., None]
    r = s["hv"] // s["hqk"]
    do = torch.where(there[..., None], _by_step(s, "do", tok), 0.0)
    o, hT, dq = _exact_scan(s, s["h0"].double(), do)
    q, k, v = _by_step(s, "q", tok, r), _by_step(s, "k", tok, r), _by_step(s, "v", tok)
    g = torch.where(there, _log_decays(s, tok), 0.0)
    G = s["dhT"].double()  # adjoint of the state after the step
    dk, dv = torch.zeros_like(v), torch.zeros_like(v)
    for t in range(len(q) - 1, -1, -1):
        G = G + SCALE * do[t][..., :, None] * q[t][..., None, :]
        dk[t] = (v[t][..., None, :] @ G)[..., 0, :]
        dv[t] = (G @ k[t][..., None])[..., 0]
        G = g[t].exp()[..., None, None] * G
    out = dict(o=o, hT=hT, dv=_back(s, dv, tok, there), dh0=G)
    if s["gate"] == "token":
        cross = torch.where(there, (q * dq - k * dk).sum(-1), 0.0)
        dg = cross.flip(0).cumsum(0).flip(0) + (hT * s["dhT"]).sum((-1, -2))
        out["dg"] = _back(s, dg, tok, there)
    for name, x in (("dq", dq), ("dk", dk)):
        out[name] = _back(s, x.unflatten(2, (s["hqk"], r)).sum(3), tok, there)
    return out
