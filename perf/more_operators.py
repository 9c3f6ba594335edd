"""Cases that measure the gated delta rule with a decay for each token and head, and layer norm with its
gradients: one pass through an operator of the package (``own`` true), or the same mathematics in
elementary torch operations (``own`` false).

Per value head h (it reads query/key head h // (Hv // Hqk)), with a value-first state S [128, 128]:

    S' = exp(g_t) S_{t-1},  u_t = v_t - S' k_t,  S_t = S' + beta_t u_t k_t^T,  o_t = s S_t q_t,  s = 1 / sqrt(128)

g (None: no decay) and beta are BF16 numbers of each token and head; queries and keys come normalised.
Layer norm: y = (x - mean) rstd w + b over the last dimension, rstd = 1 / sqrt(var + eps).
"""

import math
import random

import torch

own = False

DIM = 128
SCALE = 1.0 / math.sqrt(DIM)
CHUNK = 64  # tokens of one chunk in the plain form
EPS = 1e-5
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # the norm before a layer in one decode step of 16 requests
        dict(name="norm_step", op="norm_fwd", rows=16, width=4096, dtype="bf16", affine="both", wide=0),
        # the norm of a prompt batch of 8 x 1024 tokens, 12288 wide (96 heads of 128)
        dict(name="norm_prompts_12288", op="norm_fwd", rows=8192, width=12288, dtype="bf16", affine="both", wide=0),
        # its gradients in a training step of 4 x 2048 tokens, 4096 wide
        dict(name="norm_train_bwd", op="norm_bwd", rows=8192, width=4096, dtype="bf16", affine="both", wide=0),
        # gradients for a ragged batch of odd width in FP32, read from a wider buffer
        dict(name="norm_bwd_odd", op="norm_bwd", rows=1537, width=1001, dtype="fp32", affine="weight", wide=7),
        # the shortest prompt: one request of 64 tokens, two heads
        dict(name="prefill_64", op="prefill", lens="fixed", N=1, T=64, hqk=2, hv=2, gate="token", pool="fp32", spare=1),
        # 8 prompts of 1024 tokens, 96 heads, a BF16 state pool
        dict(name="prefill_8x1024_h96", op="prefill", lens="fixed", N=8, T=1024, hqk=96, hv=96, gate="token", pool="bf16", spare=4),
        # 24 prompts of 1 to 4000 tokens, 8 key heads for 64 value heads
        dict(name="prefill_24mixed_hqk8_hv64", op="prefill", lens="mixed", N=24, T=4000, hqk=8, hv=64, gate="token", pool="fp32",
             spare=4),
        # one long prompt of odd length: few rows, a long axis
        dict(name="prefill_32771_h32", op="prefill", lens="fixed", N=1, T=32771, hqk=16, hv=32, gate="token", pool="fp32", spare=1),
        # a training step (forward and gradients), 4 x 2048 tokens, 16 key heads for 32 value heads
        dict(name="train_4x2048_hqk16_hv32", op="train", lens="fixed", N=4, T=2048, hqk=16, hv=32, gate="token"),
        # a training step on packed sequences of 1 to 2000 tokens, 32 heads, the delta rule without decays
        dict(name="train_8mixed_h32", op="train", lens="mixed", N=8, T=2000, hqk=32, hv=32, gate="none"),
        # one token of one request, 32 heads
        dict(name="decode_1xh32", op="decode", N=1, hqk=32, hv=32, gate="token", pool="fp32", spare=3),
        # one token of 256 requests, 96 heads, a BF16 state pool
        dict(name="decode_256xh96", op="decode", N=256, hqk=96, hv=96, gate="token", pool="bf16", spare=8),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "prefill", "prefill", "train", "decode"])
    if op in ("norm_fwd", "norm_bwd"):
        width = _log_int(rng, 32, 16384)
        if rng.random() < 0.5:
            width = (width + 63) // 64 * 64
        rows = _log_int(rng, 1, min(40000, (8192 * 12288 if op == "norm_fwd" else 8192 * 4096) // width))
        return dict(op=op, rows=rows, width=width, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                    affine=rng.choice(["both", "both", "weight", "none"]), wide=rng.choice([0, 0, 64, 5]))
    hv = rng.choice([1, 2, 6, 16, 32, 48, 64, 96])
    hqk = rng.choice([d for d in (1, 2, 3, 8, 16, 32, 96) if hv % d == 0])
    gate = rng.choice(["token", "token", "token", "none"])
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
    if case["op"] in ("norm_fwd", "norm_bwd"):
        rows, width = case["rows"], case["width"]
        size = DTYPES[case["dtype"]].itemsize
        vectors = {"both": 2, "weight": 1, "none": 0}[case["affine"]]
        if case["op"] == "norm_fwd":  # reads x, writes y, mean, rstd
            return dict(bytes=2 * rows * width * size + 8 * rows + 4 * vectors * width, flops=8 * rows * width)
        # reads x, dy, mean, rstd and the weight; writes dx and the vectors' gradients
        return dict(bytes=3 * rows * width * size + 8 * rows + 4 * (vectors + (vectors > 0)) * width, flops=16 * rows * width)
    N, hqk, hv = case["N"], case["hqk"], case["hv"]
    Ttot = N if case["op"] == "decode" else sum(_lengths(case))
    gates = (4 if case["gate"] == "token" else 2) * Ttot * hv
    q, v, state = 2 * Ttot * hqk * DIM, 2 * Ttot * hv * DIM, N * hv * DIM * DIM
    step = 2 * Ttot * hv * DIM * DIM  # flops of one product of the state with a vector for each token
    if case["op"] == "train":  # reads q, k, v, g, beta, do, h0, dhT; writes o, hT, dq, dk, dv, dg, dbeta, dh0
        return dict(bytes=4 * q + 4 * v + 2 * gates + 4 * 4 * state, flops=9 * step)
    size = DTYPES[case["pool"]].itemsize
    return dict(bytes=2 * q + 2 * v + gates + 2 * size * state, flops=3 * step)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.bfloat16, by=1.0):
        return (by * torch.randn(shape, generator=gen, device="cuda")).to(dtype)

    def unit(*shape):
        x = torch.randn(shape, generator=gen, device="cuda")
        return (x / x.square().sum(-1, keepdim=True).sqrt()).bfloat16()

    s = dict(case)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        rows, width, dt = case["rows"], case["width"], DTYPES[case["dtype"]]
        shift = randn(rows, 1, dtype=torch.float32, by=0.3)
        s["x"] = (randn(rows, width + case["wide"], dtype=torch.float32) + shift).to(dt)[:, :width]
        s["w"] = None if case["affine"] == "none" else 1 + randn(width, dtype=torch.float32, by=0.1)
        s["b"] = randn(width, dtype=torch.float32, by=0.1) if case["affine"] == "both" else None
        if case["op"] == "norm_bwd":
            s["dy"] = randn(rows, width, dtype=dt)
            x = s["x"].double()  # what the forward of the step left
            mean = x.mean(-1)
            s["mean"] = mean.float()
            s["rstd"] = (x.square().mean(-1) - mean.square() + EPS).rsqrt().float()
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
    s["q"], s["k"], s["v"] = unit(B, T, hqk, DIM), unit(B, T, hqk, DIM), randn(B, T, hv, DIM)
    s["beta"] = torch.sigmoid(torch.randn((B, T, hv), generator=gen, device="cuda")).bfloat16()
    s["g"] = None
    if case["gate"] == "token":  # a step size for each token, a rate for each head
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
    if op == "norm_fwd":
        return lib.kda_layer_norm_fwd(s["x"], s["w"], s["b"], eps=EPS)
    if op == "norm_bwd":
        out = lib.kda_layer_norm_bwd(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], bias=s["b"] is not None)
        return [t for t in out if t is not None]
    if op == "decode":
        o = lib.kda_gated_delta_decode(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], s["idx"], state_indices_cpu=s["idx_cpu"])
        return o, s["pool"]
    if op == "prefill":
        o = lib.kda_gated_delta_prefill(s["q"], s["k"], s["v"], s["g"], s["beta"], s["pool"], s.get("cu"), s["idx"],
                                        cu_seqlens_cpu=s.get("cu_cpu"), state_indices_cpu=s["idx_cpu"])
        return o, s["pool"]
    # the context (workspace) is kept from step to step
    o, hT, s["ctx"] = lib.kda_gated_delta_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h0"], s.get("cu"),
                                              context_out=s.get("ctx"), cu_seqlens_cpu=s.get("cu_cpu"))
    dq, dk, dv, dg, dbeta, dh0 = lib.kda_gated_delta_bwd(s["ctx"], s["do"], s["dhT"])
    return dict(o=o, hT=hT, dq=dq, dk=dk, dv=dv, dbeta=dbeta, dh0=dh0, **({} if dg is None else {"dg": dg}))


# ---- the plain form


def _run_plain(s):
    op = s["op"]
    if op == "norm_fwd":
        x = s["x"].float()
        mean = x.mean(-1, keepdim=True)
        x = x - mean
        rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        y = x * rstd
        y = y if s["w"] is None else y * s["w"]
        y = y if s["b"] is None else y + s["b"]
        return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]
    if op == "norm_bwd":
        rstd = s["rstd"][:, None]
        n, dy = (s["x"].float() - s["mean"][:, None]) * rstd, s["dy"].float()
        t = dy if s["w"] is None else dy * s["w"]
        dx = rstd * (t - t.mean(-1, keepdim=True) - n * (t * n).mean(-1, keepdim=True))
        out = [dx.to(s["x"].dtype)]
        out += [] if s["w"] is None else [(dy * n).sum(0)]
        return out + ([] if s["b"] is None else [dy.sum(0)])
    if op == "decode":
        idx, r = s["idx"].long(), s["hv"] // s["hqk"]
        q, k = (s[x][:, 0].float().repeat_interleave(r, dim=1) for x in ("q", "k"))
        S = s["pool"][idx].float()
        if s["g"] is not None:
            S = S * s["g"][:, 0].float().exp()[..., None, None]
        u = s["v"][:, 0].float() - (S * k[..., None, :]).sum(-1)
        S = S + (s["beta"][:, 0].float()[..., None] * u)[..., :, None] * k[..., None, :]
        s["pool"][idx] = S.to(s["pool"].dtype)
        return (SCALE * (S * q[..., None, :]).sum(-1)).to(torch.bfloat16)[:, None], s["pool"]
    c = _chunks(s)
    if op == "prefill":
        idx = s["idx"].long()
        start, u, hT = _states(c, s["pool"][idx].float())
        s["pool"][idx] = hT.to(s["pool"].dtype)
        return _tokens(_outputs(c, start, u), c).to(torch.bfloat16), s["pool"]
    return _train(s, c)


def _chunks(s):
    """Every sequence's tokens in chunks, [NC, N, Hv, C, ...] (zeros where there is no token), and what a chunk has of its own."""
    N, hv, C = s["N"], s["hv"], CHUNK
    dev, Ttot = s["v"].device, s["v"].shape[0] * s["v"].shape[1]
    cu = s["cu"] if "cu" in s else torch.arange(N + 1, device=dev) * s["T"]
    longest = max(_lengths(s))
    NC = (longest + C - 1) // C
    at = torch.arange(NC * C, device=dev)
    tok = torch.where(at < (cu[1:] - cu[:-1])[:, None], cu[:-1, None] + at, Ttot).unflatten(1, (NC, C)).movedim(0, 1)  # [NC, N, C]

    def heads_first(x):
        x = x.reshape(Ttot, *x.shape[2:])
        x = torch.cat([x, x.new_zeros(1, *x.shape[1:])])[tok].float().movedim(3, 2)
        return x.repeat_interleave(hv // x.shape[2], dim=2)

    c = dict(tok=tok, Ttot=Ttot, N=N, NC=NC, like=s["v"].shape, heads_first=heads_first)
    c["q"], c["k"], c["v"] = (heads_first(s[x]) for x in ("q", "k", "v"))
    c["beta"] = heads_first(s["beta"])[..., None]
    g = torch.zeros_like(c["beta"][..., 0]) if s["g"] is None else heads_first(s["g"])
    b = g.double().cumsum(-1)
    lower = torch.ones(C, C, dtype=torch.bool, device=dev).tril()
    c["decay"] = torch.where(lower, b[..., :, None] - b[..., None, :], -torch.inf).exp().float()  # D_ij, j <= i
    c["from_start"], c["to_end"] = b.exp().float()[..., None], (b[..., -1:] - b).exp().float()[..., None]
    c["whole"] = b[..., -1].exp().float()[..., None, None]
    c["kk"] = (c["k"] @ c["k"].mT) * c["decay"] * ~torch.eye(C, dtype=torch.bool, device=dev)
    c["qk"] = SCALE * (c["q"] @ c["k"].mT) * c["decay"]
    # (1 + A)^-1 of the strictly lower A_ij = D_ij k_i . k_j beta_j, whose 64th power is zero
    A = -c["kk"] * c["beta"].mT
    A2 = A @ A
    A4 = A2 @ A2
    A8 = A4 @ A4
    A16 = A8 @ A8
    one = torch.eye(C, device=dev)
    c["solve"] = (one + A) @ (one + A2) @ (one + A4) @ (one + A8) @ (one + A16) @ (one + A16 @ A16)
    return c


def _states(c, S):
    """The states at the chunks' starts, u of every token, and the last states."""
    start, us = [], []
    for i in range(c["NC"]):
        start.append(S)
        k = c["k"][i]
        u = c["solve"][i] @ (c["v"][i] - c["from_start"][i] * (k @ S.mT))
        us.append(u)
        S = c["whole"][i] * S + (c["beta"][i] * c["to_end"][i] * u).mT @ k
    return torch.stack(start), torch.stack(us), S


def _outputs(c, start, u):
    return SCALE * c["from_start"] * (c["q"] @ start.mT) + c["qk"] @ (c["beta"] * u)


def _tokens(x, c):
    """[NC, N, Hv, C, ...] -> [B, T, Hv, ...], the inverse of heads_first."""
    out = x.new_empty(c["Ttot"] + 1, x.shape[2], *x.shape[4:])
    out[c["tok"]] = x.movedim(2, 3)
    return out[:-1].reshape(*c["like"][:2], *out.shape[1:])


def _train(s, c):
    start, u, hT = _states(c, s["h0"])
    o = _outputs(c, start, u)
    do, G = c["heads_first"](s["do"]), s["dhT"]
    end, rhos = [], []
    for i in reversed(range(c["NC"])):  # G: the adjoint of the state at the chunk's end
        end.append(G)
        direct = c["qk"][i].mT @ do[i] + c["to_end"][i] * (c["k"][i] @ G.mT)
        rho = c["solve"][i].mT @ (c["beta"][i] * direct)  # dv
        rhos.append(rho)
        G = c["whole"][i] * G + (SCALE * c["from_start"][i] * do[i]).mT @ c["q"][i] - (c["from_start"][i] * rho).mT @ c["k"][i]
    end, rho = torch.stack(end[::-1]), torch.stack(rhos[::-1])
    new = c["beta"] * u  # what enters the state with k
    A, R = SCALE * c["decay"] * (do @ new.mT), c["decay"].tril(-1) * (rho @ new.mT)
    dq = SCALE * c["from_start"] * (do @ start) + A @ c["k"]
    dk = A.mT @ c["q"] + c["to_end"] * (new @ end) - c["from_start"] * (rho @ start) - (R + R.mT) @ c["k"]
    dnew = c["qk"].mT @ do + c["to_end"] * (c["k"] @ end.mT) - c["kk"].mT @ rho
    bf16 = torch.bfloat16
    out = dict(o=_tokens(o, c).to(bf16), hT=hT, dv=_tokens(rho, c).to(bf16), dh0=G, dbeta=_tokens((dnew * u).sum(-1), c).to(bf16))
    if s["g"] is not None:  # a decay scales all that crosses its token: long sums that cancel, in 64 bits
        cross = ((do.double() * o).sum(-1) - (c["v"].double() * rho).sum(-1)).movedim(0, 2).flatten(2)  # [N, Hv, NC C]
        past = cross.flip(-1).cumsum(-1).flip(-1) + (hT.double() * s["dhT"]).sum((-1, -2))[..., None]
        out["dg"] = _tokens(past.unflatten(2, (c["NC"], CHUNK)).movedim(2, 0), c).to(bf16)
    groups = (s["hqk"], s["hv"] // s["hqk"])
    out["dq"], out["dk"] = (_tokens(x.unflatten(2, groups).sum(3), c).to(bf16) for x in (dq, dk))
    return out


# ---- the operators' definitions in 64 bits, token by token


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("norm_fwd", "norm_bwd"):
        return _exact_norm(s)
    if case["op"] == "train":
        return _exact_train(s)
    idx = s["idx"].long()
    pool = s["pool"].double()
    x = _by_step(s)
    S, o = pool[idx], torch.empty_like(x["v"])
    for t in range(len(o)):
        S, _, _ = _step(x, t, S)
        o[t] = SCALE * (S @ x["q"][t][..., None])[..., 0]
    pool[idx] = S
    return _back(s, x, o), pool


def _exact_norm(s):
    x = s["x"].double()
    centred = x - x.sum(-1, keepdim=True) / x.shape[-1]
    if s["op"] == "norm_fwd":
        rstd = 1 / ((centred * centred).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        y = centred * rstd * (1.0 if s["w"] is None else s["w"].double()) + (0.0 if s["b"] is None else s["b"].double())
        return y, (x - centred)[:, 0], rstd[:, 0]
    # through the row's mean and deviation, by automatic differentiation of the definition
    leaves = [x.requires_grad_()] + [t.double().requires_grad_() for t in (s["w"], s["b"]) if t is not None]
    with torch.enable_grad():
        c = x - x.sum(-1, keepdim=True) / x.shape[-1]
        y = c / ((c * c).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
        for i, t in enumerate(leaves[1:]):
            y = y * t if i == 0 else y + t
        return list(torch.autograd.grad(y, leaves, s["dy"].double()))


def _by_step(s):
    """Token tensors in 64 bits, [longest, N, Hv, ...]; where a sequence is over, beta, log decay and values are zero."""
    B, T = s["v"].shape[:2]
    cu = s["cu"] if "cu" in s else torch.arange(B + 1, device=s["v"].device) * T
    lens = cu[1:] - cu[:-1]
    at = torch.arange(int(lens.max()), device=cu.device)
    tok, there = (cu[:-1, None] + torch.minimum(at, lens[:, None] - 1)).t(), (at < lens[:, None]).t()[..., None]
    r = s["hv"] // s["hqk"]
    x = dict(tok=tok, there=there)
    for name in ("q", "k"):
        x[name] = s[name].flatten(0, 1)[tok].double().repeat_interleave(r, dim=2)
    for name in ("v", "do"):
        if name in s:
            x[name] = torch.where(there[..., None], s[name].flatten(0, 1)[tok].double(), 0.0)
    x["beta"] = torch.where(there, s["beta"].flatten(0, 1)[tok].double(), 0.0)
    x["g"] = torch.zeros_like(x["beta"]) if s["g"] is None else torch.where(there, s["g"].flatten(0, 1)[tok].double(), 0.0)
    return x


def _step(x, t, S):
    """The state after token t, the decayed one before it, and u."""
    D, k = x["g"][t].exp()[..., None, None] * S, x["k"][t]
    u = x["v"][t] - (D @ k[..., None])[..., 0]
    return D + (x["beta"][t][..., None] * u)[..., :, None] * k[..., None, :], D, u


def _back(s, x, y):
    out = y.new_zeros(s["v"].shape[0] * s["v"].shape[1], *y.shape[2:])
    keep = x["there"][..., 0]
    out[x["tok"][keep]] = y[keep]
    return out.unflatten(0, s["v"].shape[:2])


def _exact_train(s):
    x, every = _by_step(s), 64
    S, kept, L = s["h0"].double(), [], len(x["v"])
    o, dq, dk, dv = (torch.zeros_like(x["v"]) for _ in range(4))
    dg, dbeta = torch.zeros_like(x["g"]), torch.zeros_like(x["g"])
    for t in range(L):
        if t % every == 0:
            kept.append(S)
        S, _, _ = _step(x, t, S)
        o[t] = SCALE * (S @ x["q"][t][..., None])[..., 0]
    hT, G = S, s["dhT"].double()
    for first in range((L - 1) // every * every, -1, -every):
        steps, S = [], kept.pop()
        for t in range(first, min(first + every, L)):
            steps.append(_step(x, t, S))
            S = steps[-1][0]
        for t in range(min(first + every, L) - 1, first - 1, -1):
            S, D, u = steps.pop()
            k, do, beta = x["k"][t], x["do"][t], x["beta"][t]
            dq[t] = SCALE * (do[..., None, :] @ S)[..., 0, :]
            G = G + SCALE * do[..., :, None] * x["q"][t][..., None, :]
            Gk = (G @ k[..., None])[..., 0]
            dbeta[t] = (u * Gk).sum(-1)
            du = beta[..., None] * Gk
            dv[t] = du
            dk[t] = beta[..., None] * (u[..., None, :] @ G)[..., 0, :] - (du[..., None, :] @ D)[..., 0, :]
            G = G - du[..., :, None] * k[..., None, :]
            dg[t] = (G * D).sum((-1, -2))
            G = x["g"][t].exp()[..., None, None] * G
    out = dict(o=_back(s, x, o), hT=hT, dv=_back(s, x, dv), dbeta=_back(s, x, dbeta), dh0=G)
    if s["g"] is not None:
        out["dg"] = _back(s, x, dg)
    for name, y in (("dq", dq), ("dk", dk)):
        out[name] = _back(s, x, y.unflatten(2, (s["hqk"], s["hv"] // s["hqk"])).sum(3))
    return out
