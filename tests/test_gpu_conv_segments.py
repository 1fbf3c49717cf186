"""GPU tests of the convolution's gradients at every length of a wavefront's
segment (4 to 64 tokens, and more for long calls), where requests cross segments'
ends, rows are loaded ahead and the rings go round.

The reference is the definition in float64, differentiated by torch; elementwise
operations alone. Tolerances are those of test_gpu_backward: chains of at most 30
FP32 roundings of values up to ten times the root mean square, 2e-5 of the larger of
the value and that; dconv_w, a sum of T terms of random sign, is added over segments
of s tokens and then over r <= 512 rows of 4 s: 2^-24 sqrt((T s + r T) / 6 / T) <= 6e-7
of its norm for s <= 131, below the 2e-6 asked for."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module")
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tril_solve_amd
    return tril_solve_amd


def _segment(kt, tokens, H, d, W):
    """The segment of a call, from the rows of dconv_w that its workspace holds."""
    rows, left = divmod(kt.kda_conv_backward_workspace_size(tokens, 0, H, d, W),
                        3 * W * H * d * 4)
    assert left == 0
    fits = [s for s in range(4, 1024) if -(-tokens // (4 * s)) == rows]
    return [s for s in fits if s in (4, 8, 16, 32, 64) or tokens > 32768]


def _lengths(tokens, seed):
    """Requests of 0 to 5 tokens among ones of up to a sixth of the call."""
    gen = torch.Generator().manual_seed(seed)
    lens, left = [], tokens
    while left:
        top = tokens // 6 if torch.rand((), generator=gen) < 0.5 else 5
        n = min(left, int(torch.randint(0, top + 1, (), generator=gen)))
        lens.append(n)
        left -= n
    return lens


def _conv64(x, cw, window, eps):
    """Outputs [T, 3, H, d] of one request and the window that it leaves."""
    T, W = x.shape[0], cw.shape[1]
    line = torch.cat([window.permute(2, 0, 1, 3), x])
    a = sum(cw[:, w] * line[w:w + T] for w in range(W))
    y = a * torch.sigmoid(a)
    unit = y[:, :2] * torch.rsqrt((y[:, :2] ** 2).sum(-1, keepdim=True) + eps)
    return torch.cat([unit, y[:, 2:]], 1), line[T:].permute(1, 2, 0, 3)


def _close(got, want, name, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    err, size = (got - want).abs(), want.pow(2).mean().sqrt()
    half = 0.0 if name == "f32" else torch.finfo(TYPES[name]).eps / 2
    tiny = 2.0 ** -24 if name == "f16" else 0.0
    assert err.pow(2).mean().sqrt() <= (2e-6 + half) * size + tiny, what
    bound = 2e-5 * want.abs().clamp(min=float(size)) + half * want.abs() + tiny
    assert (err <= bound).all(), f"{what}: {float((err - bound).max()):.3g} past bound"


CASES = [
    # segment, tokens, H, d, W, type, from codes
    (4, 509, 3, 64, 4, "bf16", False),
    (4, 333, 5, 128, 2, "f32", True),
    (8, 1031, 16, 128, 4, "f16", False),
    (8, 2053, 16, 64, 3, "f32", True),
    (16, 2053, 16, 128, 4, "f32", False),
    (16, 2053, 16, 128, 3, "bf16", True),
    (16, 2053, 16, 128, 2, "f16", False),
    (32, 4099, 16, 128, 4, "f16", True),
    (32, 4111, 32, 64, 3, "f32", False),
    (32, 4111, 32, 64, 2, "bf16", False),
    (64, 8209, 16, 128, 4, "bf16", True),
    (64, 8209, 16, 128, 4, "f32", False),
    (64, 8209, 16, 128, 3, "f16", False),
    (64, 8209, 32, 64, 2, "f32", True),
    (79, 40007, 2, 64, 4, "f32", True),
    (79, 40007, 1, 128, 3, "bf16", False),
    (131, 66999, 1, 64, 4, "f16", False),
    (131, 66999, 1, 64, 2, "f32", False),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_segment(kt, case):
    seg, T, H, d, W, dtype, coded = case
    assert _segment(kt, T, H, d, W) == [seg] or \
        (T > 32768 and (T + 511) // 512 == seg and seg in _segment(kt, T, H, d, W))
    lens = _lengths(T, T + W)
    n, gen = len(lens), torch.Generator(device=DEV).manual_seed(T + W)
    new = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    dn = [new(T, H, d).to(TYPES[dtype]) for _ in range(3)]
    kw = {}
    if coded:
        x = torch.randint(-127, 128, (T, 3, H, d), generator=gen, device=DEV, dtype=torch.int8)
        kw["qkv_scale"] = torch.rand((T, 3, H), generator=gen, device=DEV) / 60
        x64 = x.double() * kw["qkv_scale"].double()[..., None]
    else:
        x = new(T, 3, H, d).to(TYPES[dtype])
        x64 = x.double()
    cw = torch.rand((3, W, H, d), generator=gen, device=DEV) - 0.5
    pool, dpool = new(n + 2, 3, H, W - 1, d), new(n + 2, 3, H, W - 1, d)
    slot = torch.randperm(n + 2, generator=gen, device=DEV)[:n].int()
    init = torch.randint(0, 2, (n,), generator=gen, device=DEV).int()
    cu = torch.tensor([0] + lens).cumsum(0).int().to(DEV)

    x64.requires_grad_()
    cw64, pool64 = cw.double().requires_grad_(), pool.double().requires_grad_()
    dnew, loss = dpool.double(), 0.0
    dn64 = torch.stack([g.double() for g in dn], 1)
    want_pool, at = dpool.double(), 0
    for i, (m, s, cont) in enumerate(zip(lens, slot.tolist(), init.tolist())):
        out, left = _conv64(x64[at:at + m], cw64, pool64[s] * float(cont), 1e-6)
        loss = loss + (out * dn64[at:at + m]).sum() + (left * dnew[s]).sum()
        at += m
    loss.backward()
    live = slot.long()
    want_pool[live] = pool64.grad[live]  # 0 where the request starts from zeros

    got = kt.conv_prefill_backward(*dn, x, cw, cu, conv_state=pool, dconv_state=dpool, slot=slot,
                                   init=init, **kw)
    _close(got[0], x64.grad, dtype, "dqkv")
    _close(got[1], cw64.grad, "f32", "dconv_w")
    _close(dpool, want_pool, "f32", "dconv_state")
