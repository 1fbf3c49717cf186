"""The operators of a KDA layer around the chunk solver and the decode step:
chunk maps from request lengths, the prompt's causal convolution, the gated
delta rule (chunked for prompts, recurrent for a few tokens) and the gated
RMSNorm. ``run`` computes them either from elementary torch operations or
through this package's calls (``own``), on the same inputs.
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
        # a serving step's map: the prompts of one batch, for the 64-token solver
        dict(name="map 32 requests", op="map", n=32, lo=1, hi=2048, len_seed=1, chunk=64),
        # thousands of short requests, where a call without a map is slowest
        dict(name="map 4096 requests", op="map", n=4096, lo=0, hi=300, len_seed=2, chunk=32),
        # one short prompt of 64 tokens: latency
        dict(name="conv 64 tokens", op="conv", n=1, lo=64, hi=64, len_seed=1, H=64, d=128, W=4,
             dtype="bf16", cont=False),
        # 16 prompts of 512 tokens, the benchmark's batch
        dict(name="conv 16x512", op="conv", n=16, lo=512, hi=512, len_seed=1, H=64, d=128, W=4,
             dtype="bf16", cont=False),
        # one short prompt over 64 heads: latency
        dict(name="prefill 64 tokens", op="prefill", n=1, lo=64, hi=64, len_seed=1, H=64, Hk=64,
             K=128, V=128, dtype="bf16", gate="channel", rate="slow", cont=False),
        # the benchmark's batch through the whole delta rule
        dict(name="prefill 16x512", op="prefill", n=16, lo=512, hi=512, len_seed=1, H=64, Hk=64,
             K=128, V=128, dtype="bf16", gate="channel", rate="slow", cont=False),
        # one long prompt continued from a stored state, channels of very different decay
        dict(name="prefill 1x16384", op="prefill", n=1, lo=16384, hi=16384, len_seed=1, H=32,
             Hk=32, K=128, V=128, dtype="bf16", gate="channel", rate="mixed", cont=True),
        # odd ragged prompts in full precision: grouped key heads, one decay per head
        dict(name="prefill ragged f32", op="prefill", n=20, lo=1, hi=640, len_seed=3, H=8, Hk=4,
             K=64, V=64, dtype="f32", gate="head", rate="slow", cont=True),
        # single-token decoding of a batch
        dict(name="recurrent 32x1", op="recurrent", n=32, lo=1, hi=1, len_seed=1, H=32, Hk=32,
             K=128, V=128, dtype="bf16", gate="channel", rate="slow", cont=True, padding=0),
        # a few drafted tokens per request, some entries of the batch padding
        dict(name="recurrent 24x1-8", op="recurrent", n=24, lo=1, hi=8, len_seed=2, H=16, Hk=16,
             K=128, V=128, dtype="f16", gate="channel", rate="mixed", cont=True, padding=3),
        # the output norm of one short prompt: latency
        dict(name="norm 64 tokens", op="norm", rows=64, H=64, d=128, dtype="bf16"),
        # the output norm of the benchmark's batch
        dict(name="norm 16x512", op="norm", rows=8192, H=64, d=128, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["map", "conv", "prefill", "prefill", "prefill", "recurrent", "recurrent",
                     "norm"])
    seed = rng.randrange(1 << 20)
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "map":
        return dict(op=op, n=_log(rng, 1, 4096), lo=0, hi=_log(rng, 20, 300), len_seed=seed,
                    chunk=rng.choice([16, 32, 64]))
    if op == "norm":
        return dict(op=op, rows=_log(rng, 1, 4096), H=rng.randint(1, 64),
                    d=rng.choice([64, 128]), dtype=dtype)
    if op == "conv":
        return dict(op=op, n=_log(rng, 1, 24), lo=1, hi=_log(rng, 2, 300), len_seed=seed,
                    H=rng.randint(1, 32), d=rng.choice([64, 128]), W=rng.choice([2, 3, 4]),
                    dtype=dtype, cont=rng.random() < 0.5)
    Hk = rng.choice([1, 2, 3, 4, 8, 16])
    heads = dict(H=Hk * rng.choice([1, 1, 2]), Hk=Hk, K=rng.choice([64, 128, 128]),
                 V=rng.choice([64, 128, 128]), dtype=dtype,
                 gate=rng.choice(["channel", "channel", "head"]),
                 rate=rng.choice(["slow", "mixed"]))
    if op == "prefill":
        n = _log(rng, 1, 16)
        hi = _log(rng, 16, 8192 // n)
        return dict(op=op, n=n, lo=rng.choice([1, hi]), hi=hi, len_seed=seed,
                    cont=rng.random() < 0.5, **heads)
    n = _log(rng, 1, 64)
    return dict(op=op, n=n, lo=1, hi=rng.randint(1, 8), len_seed=seed, cont=rng.random() < 0.7,
                padding=rng.randint(0, n // 4), **heads)


def _lengths(case):
    r = random.Random(case["len_seed"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["n"])]


# ----------------------------------------------------------------- the inputs

def _unit(x):
    return x / x.norm(dim=-1, keepdim=True)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32)

    op = case["op"]
    if op == "norm":
        dt = DTYPES[case["dtype"]]
        shape = (case["rows"], case["H"], case["d"])
        return dict(op=op, o=normal(*shape).mul_(0.3).to(dt), z=normal(*shape).to(dt),
                    norm_w=1.0 + 0.1 * normal(case["d"]), eps=1e-6)
    if op == "map":
        # the lengths of a batch: those of the case, in another order for each seed
        lens = _lengths(case)
        lens = [lens[i] for i in torch.randperm(len(lens), generator=gen, device=DEV).tolist()]
        total = sum(lens)
        if total > 1:  # and a request cut off by another amount
            i = max(range(len(lens)), key=lens.__getitem__)
            lens[i] -= seed % min(lens[i], 13)
        return dict(op=op, lens=torch.tensor(lens, dtype=torch.int32, device=DEV), total=total,
                    chunk=case["chunk"])
    lens = _lengths(case)
    n, T, H = len(lens), sum(lens), case["H"]
    dt = DTYPES[case["dtype"]]
    cu = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device=DEV)
    slots = n + 2
    slot = torch.randperm(slots, generator=gen, device=DEV)[:n].to(torch.int32)
    init = torch.full((n,), 1 if case["cont"] else 0, dtype=torch.int32, device=DEV)
    s = dict(op=op, lens=lens, cu=cu, slot=slot, init=init)
    if op == "conv":
        d, W = case["d"], case["W"]
        s.update(qkv=normal(T, 3, H, d).to(dt), eps=1e-6,
                 conv_w=torch.rand((3, W, H, d), generator=gen, device=DEV) - 0.5,
                 conv_state=normal(slots, 3, H, W - 1, d))
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
             state=0.05 * normal(slots, H, K, V), scale=K ** -0.5)
    if case.get("padding"):
        s["slot"][:case["padding"]] = -1
    return s


# ------------------------------------------------------- the elementary forms

def _map_plain(s):
    lens, C = s["lens"].long(), s["chunk"]
    n = lens.numel()
    cu = torch.cat([lens.new_zeros(1), lens.cumsum(0)])
    chunks = (lens + C - 1) // C
    ends = chunks.cumsum(0)
    at = torch.arange(s["total"] // C + n, device=lens.device)
    req = torch.searchsorted(ends, at, right=True)
    inside = at < ends[-1]
    r = req.clamp(max=n - 1)
    pairs = torch.stack([r, at - (ends - chunks)[r]], 1)
    pairs = torch.where(inside[:, None], pairs, torch.full_like(pairs, -1))
    return dict(cu=cu.int(), map=pairs.int(), count=ends[-1:].int())


def _positions(s):
    T = sum(s["lens"])
    t = torch.arange(T, device=DEV)
    seq = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    return t, seq, t - s["cu"].long()[seq]


def _conv_plain(s):
    x, cw, eps = s["qkv"], s["conv_w"], s["eps"]
    W = cw.shape[1]
    t, seq, pos = _positions(s)
    # the previous inputs of every request, oldest first: [n, W - 1, 3, H, d]
    hist = s["conv_state"][s["slot"].long()].permute(0, 3, 1, 2, 4)
    hist = hist * (s["init"] != 0)[:, None, None, None, None]

    def at(place, request, start):  # the input at a place of a request, from the past where < 0
        new = x[(start + place).clamp(min=0, max=x.shape[0] - 1)].float()
        old = hist[request, (W - 1 + place).clamp(min=0, max=W - 2)]
        return torch.where((place >= 0)[:, None, None, None], new, old)

    start = s["cu"].long()[:-1]
    acc = 0
    for w in range(W):
        acc = acc + cw[:, w] * at(pos - (W - 1) + w, seq, start[seq])
    y = acc / (1.0 + torch.exp(-acc))
    n = torch.arange(len(s["lens"]), device=DEV)
    length = s["cu"].long()[1:] - start
    window = torch.stack([at(length - (W - 1) + j, n, start) for j in range(W - 1)], 3)
    s["conv_state"][s["slot"].long()] = window
    unit = y[:, :2] / torch.sqrt((y[:, :2] * y[:, :2]).sum(-1, keepdim=True) + eps)
    dt = x.dtype
    return dict(q=unit[:, 0].to(dt), k=unit[:, 1].to(dt), v=y[:, 2].to(dt),
                conv_state=s["conv_state"])


def _padded(s, step):
    """Indexes of the packed rows as [n, longest, up to a multiple of step]."""
    longest = -(-max(s["lens"]) // step) * step
    cu = s["cu"].long()
    place = torch.arange(longest, device=DEV)
    inside = place[None] < (cu[1:] - cu[:-1])[:, None]
    idx = (cu[:-1, None] + place[None]).clamp(max=sum(s["lens"]) - 1)
    return idx, inside


def _take(x, idx, inside, group=1):
    x = x.float()[idx] * inside.reshape(inside.shape + (1,) * (x.dim() - 1))
    x = x.repeat_interleave(group, dim=2) if group > 1 else x
    return x.transpose(1, 2)  # [n, H, longest, ...]


def _delta_plain(s, C):
    H, group = s["v"].shape[1], s["v"].shape[1] // s["k"].shape[1]
    idx, inside = _padded(s, C)
    q, k = (_take(s[x], idx, inside, group) for x in ("q", "k"))
    v, g, beta = (_take(s[x], idx, inside) for x in ("v", "g", "beta"))
    if g.dim() == 3:
        g = g[..., None].expand(k.shape)
    live = s["slot"] >= 0
    at = s["slot"].long().clamp(min=0)
    S = s["state"][at] * (s["init"] != 0)[:, None, None, None]
    eye = torch.eye(C, device=DEV)
    low, strict = torch.ones(C, C, device=DEV).tril(), torch.ones(C, C, device=DEV).tril(-1)
    outs = []
    for c in range(0, idx.shape[1], C):
        qc, kc, vc, bc = q[:, :, c:c + C], k[:, :, c:c + C], v[:, :, c:c + C], beta[:, :, c:c + C, None]
        G = g[:, :, c:c + C].cumsum(2)
        # decay from token j to token i, per channel; nothing above the diagonal
        E = torch.exp((G[:, :, :, None] - G[:, :, None]).clamp(max=0.0)) * low[:, :, None]
        P = (qc[:, :, :, None] * kc[:, :, None] * E).sum(-1)
        L = bc * (kc[:, :, :, None] * kc[:, :, None] * E).sum(-1) * strict
        X, pw, n = eye - L, L, 2  # (I + L)^-1 = (I - L)(I + L^2)(I + L^4)...
        while n < C:
            pw, n = pw @ pw, 2 * n
            X = X + X @ pw
        eG = torch.exp(G)
        U = X @ (bc * (vc - (kc * eG) @ S))
        outs.append((qc * eG) @ S + P @ U)
        last = G[:, :, -1:]
        S = torch.exp(last).transpose(2, 3) * S + (kc * torch.exp(last - G)).transpose(2, 3) @ U
    o = torch.cat(outs, 2) * s["scale"] * live[:, None, None, None]
    s["state"][at[live]] = S[live]
    out = torch.empty_like(s["v"])
    out[idx[inside]] = o.transpose(1, 2)[inside].to(out.dtype)
    return dict(out=out, state=s["state"])


def _norm_plain(s):
    o, z = s["o"].float(), s["z"].float()
    y = o / torch.sqrt((o * o).mean(-1, keepdim=True) + s["eps"]) * s["norm_w"]
    return (y / (1.0 + torch.exp(-z))).to(s["o"].dtype)


# ------------------------------------------------------------------- one pass

def _run_own(s):
    import tril_solve_amd as kt
    op = s["op"]
    if op == "map":
        cu, pairs, count = kt.chunk_map(s["lens"], s["total"], s["chunk"])
        return dict(cu=cu, map=pairs, count=count)
    if op == "conv":
        q, k, v = kt.conv_prefill(s["qkv"], s["conv_w"], s["cu"], conv_state=s["conv_state"],
                                  slot=s["slot"], init=s["init"], eps_l2=s["eps"])
        return dict(q=q, k=k, v=v, conv_state=s["conv_state"])
    if op == "norm":
        return kt.gated_norm(s["o"], s["z"], s["norm_w"], eps_norm=s["eps"])
    fn = kt.prefill if op == "prefill" else kt.recurrent
    out = fn(s["q"], s["k"], s["v"], s["g"], s["beta"], s["cu"], state=s["state"],
             slot=s["slot"], init=s["init"], scale=s["scale"])
    return dict(out=out, state=s["state"])


def run(s):
    if own:
        return _run_own(s)
    if s["op"] == "map":
        return _map_plain(s)
    if s["op"] == "conv":
        return _conv_plain(s)
    if s["op"] == "norm":
        return _norm_plain(s)
    return _delta_plain(s, 16 if s["op"] == "prefill" else max(s["lens"]))


# ---------------------------------------------------------- what it has to do

def work(case):
    op = case["op"]
    if op == "map":
        n, slots = case["n"], sum(_lengths(case)) // case["chunk"] + case["n"]
        return {"bytes": 4 * n + 4 * (n + 1) + 8 * slots + 4, "flops": 2 * n}
    e = SIZE[case["dtype"]]
    if op == "norm":
        n = case["rows"] * case["H"] * case["d"]
        return {"bytes": 3 * n * e + 4 * case["d"], "flops": 8 * n}
    lens = _lengths(case)
    T, H = sum(lens), case["H"]
    if op == "conv":
        n, W, d = T * 3 * H * case["d"], case["W"], case["d"]
        window = case["n"] * 3 * H * (W - 1) * d * 4
        return {"bytes": 2 * n * e + 3 * W * H * d * 4 + window * (2 if case["cont"] else 1),
                "flops": n * (2 * W + 8)}
    pad = case.get("padding", 0)
    live, seqs = sum(lens[pad:]), case["n"] - pad
    K, V = case["K"], case["V"]
    row = 2 * case["Hk"] * K * e + H * V * e + H * 4 + H * 4 * (K if case["gate"] == "channel" else 1)
    state = seqs * H * K * V * 4 * (2 if case["cont"] else 1)
    # the least arithmetic: two products with the state and one rank-1 update a token
    return {"bytes": live * row + T * H * V * e + state, "flops": live * H * 6 * K * V}


# ------------------------------------------------------ the definition, 64 bit

def _exact_map(s):
    lens, C = s["lens"].tolist(), s["chunk"]
    pairs = [(r, c) for r, n in enumerate(lens) for c in range(-(-n // C))]
    count = len(pairs)
    pairs += [(-1, -1)] * (s["total"] // C + len(lens) - count)
    return dict(cu=np.cumsum([0] + lens).astype(np.int32), map=np.asarray(pairs, np.int32),
                count=np.asarray([count], np.int32))


def _exact_conv(s):
    """Request by request: the inputs behind the window, convolved."""
    x, cw = s["qkv"].double(), s["conv_w"].double()
    W, pool = cw.shape[1], s["conv_state"].double()
    ys, b = [], 0
    for r, n in enumerate(s["lens"]):
        slot = int(s["slot"][r])
        past = pool[slot].permute(2, 0, 1, 3) * float(s["init"][r] != 0)  # [W - 1, 3, H, d]
        line = torch.cat([past, x[b:b + n]])
        ys.append(sum(cw[:, w] * line[w:w + n] for w in range(W)))
        pool[slot] = line[n:].permute(1, 2, 0, 3)
        b += n
    y = torch.cat(ys)
    y = y * torch.sigmoid(y)
    unit = [y[:, p] / (y[:, p].square().sum(-1, keepdim=True) + s["eps"]).sqrt() for p in (0, 1)]
    return dict(q=unit[0], k=unit[1], v=y[:, 2], conv_state=pool)


def _exact_delta(s):
    """Token by token, all requests side by side."""
    cu, lens = s["cu"].long(), torch.tensor(s["lens"], device=DEV)
    H, group = s["v"].shape[1], s["v"].shape[1] // s["k"].shape[1]
    live = s["slot"] >= 0
    at = s["slot"].long().clamp(min=0)
    S = s["state"].double()[at] * (s["init"] != 0)[:, None, None, None]
    out = torch.zeros(s["v"].shape, dtype=torch.float64, device=DEV)
    heads = torch.arange(H, device=DEV) // group
    per_channel = s["g"].dim() == 3
    longest = max(s["lens"])
    whole = min(s["lens"]) if bool(live.all()) else 0  # up to here every request has a token
    for t in range(longest):
        on = (lens > t) & live
        row = (cu[:-1] + t).clamp(max=out.shape[0] - 1)
        k, q = s["k"][row][:, heads].double(), s["q"][row][:, heads].double()
        a = torch.exp(s["g"][row].double())
        new = S * (a[..., None] if per_channel else a[..., None, None])
        u = s["beta"][row].double()[..., None] * (s["v"][row].double() - (k[:, :, None] @ new)[:, :, 0])
        new.addcmul_(k[..., None], u[:, :, None])
        o = s["scale"] * (q[:, :, None] @ new)[:, :, 0]
        if t < whole:
            S = new
            out[row] = o
        else:
            S = torch.where(on[:, None, None, None], new, S)
            out[row[on]] = o[on]
    pool = s["state"].double()
    pool[at[live]] = S[live]
    return dict(out=out, state=pool)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "map":
        return _exact_map(s)
    if s["op"] == "conv":
        return _exact_conv(s)
    if s["op"] == "norm":
        o, z = s["o"].double(), s["z"].double()
        rms = (o.square().mean(-1, keepdim=True) + s["eps"]).sqrt()
        return o / rms * s["norm_w"].double() * torch.sigmoid(z)
    return _exact_delta(s)
