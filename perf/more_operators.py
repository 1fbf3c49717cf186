"""The backward pass of a KDA layer: the gradients of the gated delta rule, of
the prompt's causal convolution and of the gated RMSNorm, and the activation
checkpoints in 8 bits that the latter two read. ``run`` computes them either
from elementary torch operations or through this package's calls (``own``), on
the same inputs.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one short sequence over 64 heads: latency
        dict(name="delta 64 tokens", op="delta", n=1, lo=64, hi=64, len_seed=1, H=64, Hk=64,
             K=128, V=128, dtype="bf16", gate="channel", rate="slow", cont=False),
        # the benchmark's batch as a training step sees it
        dict(name="delta 16x512", op="delta", n=16, lo=512, hi=512, len_seed=1, H=64, Hk=64,
             K=128, V=128, dtype="bf16", gate="channel", rate="slow", cont=False),
        # one long sequence that continues from a state and hands a gradient back to it,
        # channels of very different decay
        dict(name="delta 1x16384", op="delta", n=1, lo=16384, hi=16384, len_seed=1, H=32, Hk=32,
             K=128, V=128, dtype="bf16", gate="channel", rate="mixed", cont=True),
        # odd ragged sequences in full precision: key heads shared by two value heads, one
        # decay per head
        dict(name="delta ragged f32", op="delta", n=20, lo=1, hi=640, len_seed=3, H=8, Hk=4,
             K=64, V=64, dtype="f32", gate="head", rate="slow", cont=True),
        # one short sequence: latency
        dict(name="conv 64 tokens", op="conv", n=1, lo=64, hi=64, len_seed=1, H=64, d=128, W=4,
             dtype="bf16", cont=False, kept="whole"),
        # the benchmark's batch, its inputs kept in 8 bits
        dict(name="conv 16x512 8 bits", op="conv", n=16, lo=512, hi=512, len_seed=1, H=64, d=128,
             W=4, dtype="bf16", cont=False, kept="8 bits"),
        # odd ragged sequences that continue from a window, in full precision
        dict(name="conv ragged f32", op="conv", n=24, lo=1, hi=500, len_seed=5, H=9, d=64, W=3,
             dtype="f32", cont=True, kept="whole"),
        # the output norm of a short training step, forward with 8-bit checkpoints and backward
        # from them: latency
        dict(name="norm step 64 tokens", op="norm", rows=64, H=64, d=128, dtype="bf16",
             kept="8 bits"),
        # the same step of the benchmark's batch
        dict(name="norm step 16x512", op="norm", rows=8192, H=64, d=128, dtype="bf16",
             kept="8 bits"),
        # the norm's backward pass alone, from inputs in full precision, an odd number of rows
        dict(name="norm 999 f32", op="norm", rows=999, H=16, d=64, dtype="f32", kept="whole"),
        # the convolution's inputs of a short sequence put into 8 bits and read back: latency
        dict(name="checkpoint 64 tokens", op="checkpoint", rows=64, H=64, d=128, dtype="bf16"),
        # the same of the benchmark's batch
        dict(name="checkpoint 16x512", op="checkpoint", rows=8192, H=64, d=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["delta", "delta", "delta", "delta", "conv", "conv", "norm", "checkpoint"])
    seed = rng.randrange(1 << 20)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    kept = rng.choice(["whole", "8 bits"])
    if op in ("norm", "checkpoint"):
        case = dict(op=op, rows=_log(rng, 1, 4096), H=rng.randint(1, 64),
                    d=rng.choice([64, 128]), dtype=dtype)
        return dict(case, kept=kept) if op == "norm" else case
    if op == "conv":
        return dict(op=op, n=_log(rng, 1, 24), lo=1, hi=_log(rng, 2, 300), len_seed=seed,
                    H=rng.randint(1, 32), d=rng.choice([64, 128]), W=rng.choice([2, 3, 4]),
                    dtype=dtype, cont=rng.random() < 0.5, kept=kept)
    Hk = rng.choice([1, 2, 3, 4, 8, 16])
    n = _log(rng, 1, 16)
    hi = _log(rng, 16, 8192 // n)
    return dict(op=op, n=n, lo=rng.choice([1, hi]), hi=hi, len_seed=seed,
                cont=rng.random() < 0.5, H=Hk * rng.choice([1, 1, 2]), Hk=Hk,
                K=rng.choice([64, 128, 128]), V=rng.choice([32, 64, 96, 128, 128]), dtype=dtype,
                gate=rng.choice(["channel", "channel", "head"]),
                rate=rng.choice(["slow", "mixed"]))


def _lengths(case):
    r = random.Random(case["len_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]


# ----------------------------------------------------------------- the inputs

def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def _to_8_bits(x):
    """Codes and scale of every vector (last dimension): its largest magnitude is 127 steps."""
    x = x.double()
    scale = (x.abs().amax(-1) / 127.0).float()
    step = scale.double()[..., None]
    codes = torch.where(step > 0, torch.round(x / torch.where(step > 0, step, 1.0)), 0.0)
    return codes.to(torch.int8), scale


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)

    op, dt = case["op"], DTYPES[case["dtype"]]
    if op == "checkpoint":
        return dict(op=op, x=normal(case["rows"], 3, case["H"], case["d"]).to(dt))
    if op == "norm":
        shape = (case["rows"], case["H"], case["d"])
        return dict(op=op, kept=case["kept"], o=normal(*shape).mul_(0.3).to(dt),
                    z=normal(*shape).to(dt), dout=normal(*shape).to(dt),
                    norm_w=1.0 + 0.1 * normal(case["d"]), eps=1e-6)
    lens = _lengths(case)
    n, T, H = len(lens), sum(lens), case["H"]
    cu = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device=DEV)
    slots = n + 2
    slot = torch.randperm(slots, generator=gen, device=DEV)[:n].to(torch.int32)
    init = torch.full((n,), 1 if case["cont"] else 0, dtype=torch.int32, device=DEV)
    s = dict(op=op, lens=lens, cu=cu, slot=slot, init=init)
    if op == "conv":
        d, W = case["d"], case["W"]
        qkv = normal(T, 3, H, d).to(dt)
        s.update(kept=case["kept"], eps=1e-6, dtype=dt, dq=normal(T, H, d).to(dt),
                 dk=normal(T, H, d).to(dt), dv=normal(T, H, d).to(dt),
                 conv_w=torch.rand((3, W, H, d), generator=gen, device=DEV) - 0.5,
                 conv_state=normal(slots, 3, H, W - 1, d),
                 dconv_state=normal(slots, 3, H, W - 1, d))
        if case["kept"] == "whole":
            s["qkv"] = qkv
        else:  # as the forward pass has left them
            s["qkv"], s["qkv_scale"] = _to_8_bits(qkv)
        return s
    K, V, Hk = case["K"], case["V"], case["Hk"]
    gshape = (T, H, K) if case["gate"] == "channel" else (T, H)
    if case["rate"] == "slow":
        g = torch.nn.functional.logsigmoid(normal(*gshape) + 3.0)
    else:  # a rate of its own for every channel (or head), over a wide range
        lo, hi = math.log(0.004), math.log(3.0)
        rate = torch.exp(torch.rand(gshape[1:], generator=gen, device=DEV) * (hi - lo) + lo)
        g = -rate * torch.nn.functional.softplus(normal(*gshape))
    s.update(q=_unit(normal(T, Hk, K)).to(dt), k=_unit(normal(T, Hk, K)).to(dt),
             v=normal(T, H, V).to(dt), g=g, beta=torch.sigmoid(normal(T, H)),
             dout=normal(T, H, V).to(dt), state=0.05 * normal(slots, H, K, V),
             dstate=0.05 * normal(slots, H, K, V), scale=K ** -0.5)
    return s


# ------------------------------------------------------- the elementary forms

def _checkpoint_plain(s):
    codes, scale = _to_8_bits(s["x"])
    return (codes.float() * scale[..., None]).to(s["x"].dtype)


def _norm_plain(s):
    o, z, w, dt = s["o"].float(), s["z"].float(), s["norm_w"], s["o"].dtype
    dout, res = s["dout"].float(), {}
    if s["kept"] != "whole":  # the forward pass, and what it keeps
        r = 1.0 / torch.sqrt((o * o).mean(-1, keepdim=True) + s["eps"])
        res["out"] = (o * r * w / (1.0 + torch.exp(-z))).to(dt)
        (o, o_scale), (z, z_scale) = _to_8_bits(s["o"]), _to_8_bits(s["z"])
        o, z = o.float() * o_scale[..., None], z.float() * z_scale[..., None]
    r = 1.0 / torch.sqrt((o * o).mean(-1, keepdim=True) + s["eps"])
    n, sg = o * r, 1.0 / (1.0 + torch.exp(-z))
    dn = dout * w * sg
    do = r * (dn - n * (dn * n).mean(-1, keepdim=True))
    dz = dout * w * n * sg * (1.0 - sg)
    dw = (dout * n * sg).sum((0, 1))
    return dict(res, do=do.to(dt), dz=dz.to(dt), dnorm_w=dw)


def _positions(s):
    T = sum(s["lens"])
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return t, seq, t - s["cu"].long()[seq]


def _conv_plain(s):
    cw, eps, dt = s["conv_w"], s["eps"], s["dtype"]
    x = s["qkv"].float()
    if s["kept"] != "whole":
        x = x * s["qkv_scale"][..., None]
    W, n = cw.shape[1], len(s["lens"])
    t, seq, pos = _positions(s)
    start = s["cu"].long()[:-1]
    length = s["cu"].long()[1:] - start
    cont = (s["init"] != 0)[:, None, None, None, None]
    # the inputs before every request, oldest first: [n, W - 1, 3, H, d]
    hist = s["conv_state"][s["slot"].long()].permute(0, 3, 1, 2, 4) * cont
    dnew = s["dconv_state"][s["slot"].long()].permute(0, 3, 1, 2, 4)

    def at(place):  # the input at a place of the token's request, from the past where < 0
        new = x[(start[seq] + place).clamp(min=0, max=x.shape[0] - 1)]
        old = hist[seq, (W - 1 + place).clamp(min=0, max=W - 2)]
        return torch.where((place >= 0)[:, None, None, None], new, old)

    a = 0
    for w in range(W):
        a = a + cw[:, w] * at(pos - (W - 1) + w)
    sg = 1.0 / (1.0 + torch.exp(-a))
    y = a * sg
    dn = torch.stack([s["dq"], s["dk"], s["dv"]], 1).float()
    r = 1.0 / torch.sqrt((y[:, :2] * y[:, :2]).sum(-1, keepdim=True) + eps)
    u = y[:, :2] * r
    dy = torch.cat([r * (dn[:, :2] - u * (u * dn[:, :2]).sum(-1, keepdim=True)), dn[:, 2:]], 1)
    da = dy * sg * (1.0 + a * (1.0 - sg))
    dcw = torch.stack([(da * at(pos - (W - 1) + w)).sum(0) for w in range(W)], 1)

    def later(request, place):  # da at a place of a request, 0 outside it
        inside = (place >= 0) & (place < length[request])
        got = da[(start[request] + place).clamp(min=0, max=da.shape[0] - 1)]
        return torch.where(inside[:, None, None, None], got, 0.0)

    # a window's entry at a place: what the tokens behind it, and the window left behind, take
    def entry(request, place):
        total = 0
        for w in range(W):
            total = total + cw[:, w] * later(request, place + (W - 1) - w)
        kept = place - length[request] + W - 1
        last = dnew[request, kept.clamp(min=0, max=W - 2)]
        return total + torch.where((kept >= 0)[:, None, None, None], last, 0.0)

    dx = entry(seq, pos).to(dt)
    every = torch.arange(n, device=DEV)
    dold = torch.stack([entry(every, torch.full_like(every, m - (W - 1))) for m in range(W - 1)], 3)
    s["dconv_state"][s["slot"].long()] = dold * (s["init"] != 0)[:, None, None, None, None]
    return dict(dqkv=dx, dconv_w=dcw, dconv_state=s["dconv_state"])


def _delta_plain(s, C=16):
    H, group = s["v"].shape[1], s["v"].shape[1] // s["k"].shape[1]
    cu, dt = s["cu"].long(), s["q"].dtype
    n, longest = len(s["lens"]), -(-max(s["lens"]) // C) * C
    place = torch.arange(longest, device=DEV)
    inside = place[None] < (cu[1:] - cu[:-1])[:, None]
    idx = (cu[:-1, None] + place[None]).clamp(max=sum(s["lens"]) - 1)

    def take(x, group=1):  # [n, H, chunks, C, ...], zeros outside the requests
        x = x.float()[idx] * inside.reshape(inside.shape + (1,) * (x.dim() - 1))
        x = x.repeat_interleave(group, dim=2) if group > 1 else x
        return x.transpose(1, 2).unflatten(2, (longest // C, C))

    q, k = take(s["q"], group), take(s["k"], group)
    v, g, beta, do = (take(s[x]) for x in ("v", "g", "beta", "dout"))
    do = do * s["scale"]
    per_channel = g.dim() == 5
    if not per_channel:
        g = g[..., None].expand(k.shape)
    low, strict = torch.ones(C, C, device=DEV).tril(), torch.ones(C, C, device=DEV).tril(-1)
    eye = torch.eye(C, device=DEV)
    G = g.cumsum(3)
    # decay from token j to token i, per channel; nothing above the diagonal
    E = torch.exp((G[..., :, None, :] - G[..., None, :, :]).clamp(max=0.0)) * low[:, :, None]
    A = (k[..., :, None, :] * k[..., None, :, :] * E).sum(-1) * strict
    P = (q[..., :, None, :] * k[..., None, :, :] * E).sum(-1)
    L = A * beta[..., None, :]
    M, pw, m = eye - L, L, 2  # (I + L)^-1 = (I - L)(I + L^2)(I + L^4)...
    while m < C:
        pw, m = pw @ pw, 2 * m
        M = M + M @ pw
    eG, eR = torch.exp(G), torch.exp(G[..., -1:, :] - G)
    last = torch.exp(G[..., -1, :])[..., None]
    kG, kR, qG, b = k * eG, k * eR, q * eG, beta[..., None]
    kRt, qGt, kGt, Mt = (x.transpose(-1, -2).contiguous() for x in (kR, qG, kG, M))
    live = s["slot"].long()
    init = (s["init"] != 0)[:, None, None, None]

    S, Ss, Xs = s["state"][live] * init, [], []
    for c in range(longest // C):  # the states, forwards
        Ss.append(S)
        Xs.append(M[:, :, c] @ (v[:, :, c] - kG[:, :, c] @ S))
        S = last[:, :, c] * S + kRt[:, :, c] @ (b[:, :, c] * Xs[-1])
    S, X = torch.stack(Ss, 2), torch.stack(Xs, 2)
    U = b * X
    dU0 = P.transpose(-1, -2).contiguous() @ do
    dS, dSs, dUs, Ys = s["dstate"][live], [], [], []
    for c in reversed(range(longest // C)):  # their gradients, backwards
        dSs.append(dS)
        dUs.append(dU0[:, :, c] + kR[:, :, c] @ dS)
        Ys.append(Mt[:, :, c] @ (b[:, :, c] * dUs[-1]))
        dS = qGt[:, :, c] @ do[:, :, c] + last[:, :, c] * dS - kGt[:, :, c] @ Ys[-1]
    s["dstate"][live] = dS * init
    dS, dU, Y = (torch.stack(x[::-1], 2) for x in (dSs, dUs, Ys))

    Xt, St = X.transpose(-1, -2).contiguous(), S.transpose(-1, -2).contiguous()
    YX = (Y @ Xt) * strict
    dA, dP = -YX * beta[..., None, :], (do @ Xt) * beta[..., None, :] * low
    dbeta = (X * dU).sum(-1) - (A * YX).sum(-2)
    dq = (dP[..., None] * k[..., None, :, :] * E).sum(-2) + eG * (do @ St)
    rows = (dA[..., None] * k[..., None, :, :] * E).sum(-2) - eG * (Y @ St)
    ends = eR * (U @ dS.transpose(-1, -2).contiguous())
    cols = ((dA[..., None] * k[..., :, None, :] + dP[..., None] * q[..., :, None, :]) * E).sum(-3)
    dG = q * dq + k * (rows - cols - ends)
    dlast = (k * ends).sum(3) + last[..., 0] * (S * dS).sum(-1)
    dg = dG.flip(3).cumsum(3).flip(3) + dlast[..., None, :]

    def give(x, group=1):  # back to the packed rows
        x = x.flatten(2, 3).transpose(1, 2)  # [n, longest, H, ...]
        x = x.unflatten(2, (H // group, group)).sum(3) if group > 1 else x
        out = x.new_empty((sum(s["lens"]),) + x.shape[2:])
        out[idx[inside]] = x[inside]
        return out

    dg = give(dg)
    return dict(dq=give(dq, group).to(dt),
                dk=give(rows + cols + ends, group).to(dt), dv=give(Y).to(dt),
                dg=dg if per_channel else dg.sum(-1), dbeta=give(dbeta),
                dstate=s["dstate"])


# ------------------------------------------------------------------- one pass

def _run_own(s):
    import tril_solve_amd as kt
    op = s["op"]
    if op == "checkpoint":
        codes, scale = kt.checkpoint(s["x"])
        return kt.checkpoint_load(codes, scale, s["x"].dtype)
    if op == "norm":
        if s["kept"] == "whole":
            do, dz, dw = kt.gated_norm_backward(s["dout"], s["o"], s["z"], s["norm_w"],
                                                eps_norm=s["eps"])
            return dict(do=do, dz=dz, dnorm_w=dw)
        out, o, o_scale, z, z_scale = kt.gated_norm_checkpoint(s["o"], s["z"], s["norm_w"],
                                                               eps_norm=s["eps"])
        do, dz, dw = kt.gated_norm_backward(s["dout"], o, z, s["norm_w"], eps_norm=s["eps"],
                                            o_scale=o_scale, z_scale=z_scale)
        return dict(out=out, do=do, dz=dz, dnorm_w=dw)
    if op == "conv":
        dqkv, dw = kt.conv_prefill_backward(
            s["dq"], s["dk"], s["dv"], s["qkv"], s["conv_w"], s["cu"],
            conv_state=s["conv_state"], dconv_state=s["dconv_state"], slot=s["slot"],
            init=s["init"], eps_l2=s["eps"], qkv_scale=s.get("qkv_scale"))
        return dict(dqkv=dqkv, dconv_w=dw, dconv_state=s["dconv_state"])
    dq, dk, dv, dg, dbeta = kt.prefill_backward(
        s["dout"], s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"], state=s["state"],
        dstate=s["dstate"], slot=s["slot"], init=s["init"], scale=s["scale"])
    return dict(dq=dq, dk=dk, dv=dv, dg=dg, dbeta=dbeta, dstate=s["dstate"])


def run(s):
    if own:
        return _run_own(s)
    plain = {"checkpoint": _checkpoint_plain, "norm": _norm_plain, "conv": _conv_plain,
             "delta": _delta_plain}
    return plain[s["op"]](s)


# ---------------------------------------------------------- what it has to do

def work(case):
    op, e = case["op"], SIZE[case["dtype"]]
    if op == "checkpoint":
        vecs = 3 * case["rows"] * case["H"]
        n = vecs * case["d"]
        return {"bytes": n * (2 * e + 2) + 8 * vecs, "flops": 6 * n}
    if op == "norm":
        vecs = case["rows"] * case["H"]
        n = vecs * case["d"]
        back = 5 * n * e + 8 * case["d"]
        if case["kept"] == "whole":
            return {"bytes": back, "flops": 22 * n}
        # forward: o, z in, out and both checkpoints out; backward: checkpoints instead of o, z
        kept = 2 * n + 8 * vecs
        return {"bytes": 3 * n * e + kept + back - 2 * n * e + kept, "flops": 42 * n}
    lens = _lengths(case)
    T, H = sum(lens), case["H"]
    if op == "conv":
        n, W, d = T * 3 * H * case["d"], case["W"], case["d"]
        x = n * e if case["kept"] == "whole" else n + T * 3 * H * 4
        window = case["n"] * 3 * H * (W - 1) * d * 4
        return {"bytes": x + 2 * n * e + 6 * W * H * d * 4 + window * (3 if case["cont"] else 2),
                "flops": n * (6 * W + 20)}
    K, V, Hk = case["K"], case["V"], case["Hk"]
    g = 4 * (K if case["gate"] == "channel" else 1)
    row = 4 * Hk * K * e + 3 * H * V * e + 2 * H * (4 + g)
    state = case["n"] * H * K * V * 4 * (3 if case["cont"] else 2)
    # the least arithmetic: the states again (a product and a rank-1 update a token), then five
    # products and two rank-1 updates
    return {"bytes": T * row + state, "flops": T * H * 18 * K * V}


# ------------------------------------------------------ the definition, 64 bit

def _kept_in_8_bits(x):
    """The values that a checkpoint of x stands for."""
    big = x.double().abs().max(-1, keepdim=True).values
    step = (big / 127.0).float().double()
    return torch.where(big > 0, torch.round(x.double() / step) * step, 0.0)


def _exact_norm(s):
    o, z, w, dout = (s[x].double() for x in ("o", "z", "norm_w", "dout"))
    res = {}
    if s["kept"] != "whole":
        res["out"] = o * (o.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * w * z.sigmoid()
        o, z = _kept_in_8_bits(s["o"]), _kept_in_8_bits(s["z"])
    o, z, w = (x.detach().requires_grad_() for x in (o, z, w))
    out = o * (o.square().mean(-1, keepdim=True) + s["eps"]).rsqrt() * w * z.sigmoid()
    do, dz, dw = torch.autograd.grad(out, (o, z, w), dout)
    return dict(res, do=do, dz=dz, dnorm_w=dw)


def _exact_conv(s):
    """Request by request, differentiated."""
    x, cw = s["qkv"].double(), s["conv_w"].double().requires_grad_()
    if s["kept"] != "whole":
        x = x * s["qkv_scale"].double()[..., None]
    W, pool, b = cw.shape[1], s["dconv_state"].double(), 0
    dx, dcw = torch.empty_like(x), torch.zeros_like(cw)
    for r, n in enumerate(s["lens"]):
        slot, cont = int(s["slot"][r]), bool(s["init"][r] != 0)
        past = s["conv_state"][slot].double() * float(cont)
        line = torch.cat([past.permute(2, 0, 1, 3), x[b:b + n]]).requires_grad_()
        y = sum(cw[:, w] * line[w:w + n] for w in range(W))
        y = y * torch.sigmoid(y)
        unit = [y[:, p] / (y[:, p].square().sum(-1, keepdim=True) + s["eps"]).sqrt()
                for p in (0, 1)]
        left = line[n:].permute(1, 2, 0, 3)
        grads = [s[g][b:b + n].double() for g in ("dq", "dk", "dv")] + [pool[slot].clone()]
        dline, part = torch.autograd.grad(unit + [y[:, 2], left], (line, cw), grads)
        dx[b:b + n] = dline[W - 1:]
        dcw += part
        pool[slot] = dline[:W - 1].permute(1, 2, 0, 3) * float(cont)
        b += n
    return dict(dqkv=dx, dconv_w=dcw.detach(), dconv_state=pool)


def _exact_delta(s, stretch=64):
    """Token by token, all requests side by side: forwards, a state kept every `stretch` tokens,
    then backwards through the recurrence itself."""
    cu, lens = s["cu"].long(), torch.tensor(s["lens"], device=DEV)
    T, H, V = s["v"].shape
    K, group = s["k"].shape[-1], H // s["k"].shape[1]
    heads, longest = torch.arange(H, device=DEV) // group, max(s["lens"])
    live, cont = s["slot"].long(), (s["init"] != 0).double()[:, None, None, None]
    even = min(s["lens"]) == longest

    def token(t):
        row = (cu[:-1] + t).clamp(max=T - 1)
        on = (lens > t).double()[:, None]
        q, k, v, do = (s[x][row].double() for x in ("q", "k", "v", "dout"))
        q, k, g, beta = q[:, heads], k[:, heads], s["g"][row].double(), s["beta"][row].double()
        if not even:  # nothing happens behind a request's end
            q, k, do, g = q * on[..., None], k * on[..., None], do * on[..., None], \
                g * (on[..., None] if g.dim() == 3 else on)
            beta = beta * on
        a = torch.exp(g) if g.dim() == 3 else torch.exp(g)[..., None].expand(k.shape)
        return row, q, k, v, a, beta[..., None], do * s["scale"]

    def step(S, tok):
        _, q, k, v, a, beta, _ = tok
        mid = S * a[..., None]
        r = v - (k[:, :, None] @ mid)[:, :, 0]
        return mid, r, torch.addcmul(mid, k[..., None], (beta * r)[:, :, None])

    S, marks = s["state"].double()[live] * cont, []
    for t in range(longest):
        if t % stretch == 0:
            marks.append(S)
        S = step(S, token(t))[2]
    dS = s["dstate"].double()[live]
    out = {"dq": torch.zeros(T, H, K, dtype=torch.float64, device=DEV),
           "dv": torch.zeros(T, H, V, dtype=torch.float64, device=DEV),
           "dbeta": torch.zeros(T, H, dtype=torch.float64, device=DEV)}
    out["dk"], out["dg"] = torch.zeros_like(out["dq"]), torch.zeros_like(out["dq"])
    for m in reversed(range(len(marks))):
        S, kept = marks[m], []
        for t in range(m * stretch, min((m + 1) * stretch, longest)):
            tok = token(t)
            mid, r, S = step(S, tok)
            kept.append((t, tok, mid, r, S))
        while kept:
            t, (row, q, k, v, a, beta, do), mid, r, S = kept.pop()
            dq = (S @ do[..., None])[..., 0]
            dS = torch.addcmul(dS, q[..., None], do[:, :, None])
            u = beta * r
            du = (k[:, :, None] @ dS)[:, :, 0]
            dr = beta * du
            dk = (dS @ u[..., None] - mid @ dr[..., None])[..., 0]
            dS = torch.addcmul(dS, k[..., None], dr[:, :, None], value=-1.0)
            got = dict(dq=dq, dk=dk, dv=dr, dbeta=(du * r).sum(-1), dg=(dS * mid).sum(-1))
            dS = a[..., None] * dS
            on = slice(None) if even else lens > t
            for x in got:
                out[x][row[on]] = got[x][on]
    pool = s["dstate"].double()
    pool[live] = dS * cont
    if group > 1:
        for x in ("dq", "dk"):
            out[x] = out[x].unflatten(1, (H // group, group)).sum(2)
    if s["g"].dim() == 2:
        out["dg"] = out["dg"].sum(-1)
    return dict({x: out[x] for x in ("dq", "dk", "dv", "dg", "dbeta")}, dstate=pool)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "checkpoint":
        return _kept_in_8_bits(s["x"])
    if s["op"] == "norm":
        return _exact_norm(s)
    if s["op"] == "conv":
        return _exact_conv(s)
    return _exact_delta(s)
