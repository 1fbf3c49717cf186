"""GPU tests of the forms that the KDA layer's calls take on large problems:
the delta rule with more workgroups than compute units (wavefronts that prepare
a chunk and walk it) and with up to that many of 32 columns to a wavefront
(wavefronts of either kind), and the convolution in segments of 8 and 16
tokens, against float64.

Tolerances: the state to 1e-6 of its norm (products to 2^-24 of a term, about
ten FP32 roundings of 1.7e-8 in the mean a chunk, up to four chunks, a factor of
3 for the inverse: 3.3e-7); outputs to 4e-6 of scale times the products' size N
(128 terms and four roundings a token in FP32, 2^-24 (sqrt(128) + 4 x 13) at the
steps of a chunk, which do not add up over tokens), plus the output's half step.
"""
import numpy as np
import pytest

from tests import gpu_helpers as gh
from tests import layer_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tril_solve_amd
    return tril_solve_amd


def _exact(c, lengths, slot, init, scale):
    """The recurrence in float64 on the GPU, all requests and heads a token at a
    time: (out, states, size as in layer_reference)."""
    d = lambda x: c[x].double()  # noqa: E731
    q, k, v, g, beta = d("q"), d("k"), d("v"), d("g"), d("beta")
    T, H, V = v.shape
    K, grp = k.shape[2], H // k.shape[1]
    q, k = q.repeat_interleave(grp, 1), k.repeat_interleave(grp, 1)
    if g.dim() == 2:
        g = g[:, :, None].expand(T, H, K)
    pool = d("state")
    out = torch.zeros((T, H, V), dtype=torch.float64, device=DEV)
    live = [n for n in range(len(lengths)) if 0 <= slot[n] < pool.shape[0]]
    at = torch.tensor([int(slot[n]) for n in live], device=DEV)
    keep = torch.tensor([float(init[n] != 0) for n in live], dtype=torch.float64, device=DEV)
    S = pool[at] * keep[:, None, None, None]
    first = np.concatenate([[0], np.cumsum(lengths)])
    size = S.square().sum(2).sqrt().max()
    for t in range(max(lengths)):
        on = [i for i, n in enumerate(live) if t < lengths[n]]
        if not on:
            break
        row = torch.tensor([int(first[live[i]]) + t for i in on], device=DEV)
        s = S[on] * torch.exp(g[row])[..., None]
        u = beta[row][..., None] * (v[row] - (s * k[row][..., None]).sum(2))
        s = s + k[row][..., None] * u[:, :, None]
        S[on] = s
        out[row] = scale * (s * q[row][..., None]).sum(2)
        size = torch.maximum(size, s.square().sum(2).sqrt().max() + v[row].abs().max())
    pool[at] = S
    return out, pool, float(size)


def _inputs(lengths, H, Hk, K, V, dtype, rate, gate, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    T, N, t = sum(lengths), len(lengths), gh.out_torch_dtype(dtype)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float64)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=DEV, dtype=torch.float64)

    c = {}
    for x in ("q", "k"):  # with a common direction, as a convolution leaves them
        y = torch.nn.functional.silu(normal(T, Hk, K) + normal(1, Hk, K))
        c[x] = (y / y.norm(dim=-1, keepdim=True)).to(t)
    c["v"] = normal(T, H, V).to(t)
    shape = (T, H, K) if gate == "channel" else (T, H)
    if rate == "slow":
        g = -0.05 * torch.nn.functional.softplus(normal(*shape))
    elif rate == "mixed":
        g = -torch.exp(uniform(*shape[1:]) * np.log(1000.0) + np.log(0.004)) * \
            torch.nn.functional.softplus(normal(*shape))
    else:  # far past e^{-64} over 16 tokens, and resets
        g = -torch.exp(uniform(*shape) * np.log(4000.0) + np.log(0.01))
        g[uniform(*shape) < 0.01] = -float("inf")
    c["g"] = g.float()
    c["beta"] = torch.sigmoid(normal(T, H) + 1).float()
    c["state"] = (0.2 * normal(N + 2, H, K, V)).float()
    return c


def _check(kt, lengths, H, Hk, K, V, dtype, out_dtype, rate, gate="channel", seed=0, cut=False):
    print(f"\n[forms] {lengths} H={H} Hk={Hk} K={K} V={V} {dtype}->{out_dtype} {rate} {gate}",
          flush=True)
    c = _inputs(lengths, H, Hk, K, V, dtype, rate, gate, seed)
    N, scale = len(lengths), K ** -0.5
    rng = np.random.default_rng(seed)
    slot = rng.permutation(N + 2)[:N].astype(np.int32)
    init = (np.arange(N) % 2).astype(np.int32)
    if N > 2:
        slot[1] = -1  # padding
    dev = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    cu = dev(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32))
    n = kt.kda_prefill_workspace_size(sum(lengths), N, H, K, V) if cut else 0
    assert bool(n) == cut
    S, out = c["state"].clone(), torch.full(c["v"].shape, 7.0, dtype=gh.out_torch_dtype(out_dtype),
                                            device=DEV)
    kt.kda_prefill(c["q"], c["k"], c["v"], c["g"], c["beta"], out, cu, state=S, slot=dev(slot),
                   init=dev(init),
                   workspace=torch.empty(n, dtype=torch.uint8, device=DEV) if n else None)
    want, pool, size = _exact(c, lengths, slot, init, scale)
    assert float((S.double() - pool).norm() / pool.norm()) <= 1e-6
    untouched = [s for s in range(N + 2) if s not in slot]
    assert torch.equal(S[untouched], c["state"][untouched])
    half = torch.finfo(out.dtype).eps / 2
    over = (out.double() - want).abs() - half * want.abs()
    assert float(over.max()) <= 4e-6 * scale * size, (float(over.max()), size)


LENS = [37, 64, 100, 1]


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"),
                                             ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("rate", ["slow", "mixed", "steep"])
@pytest.mark.parametrize("H", [30, 50, 70])  # 120, 200 and 280 walks of 128 columns
@pytest.mark.parametrize("K", [64, 128])
def test_prefill_forms(kt, K, H, rate, dtype, out_dtype):
    _check(kt, LENS, H, H, K, 128, dtype, out_dtype, rate, seed=H + K)


@pytest.mark.parametrize("rate", ["mixed", "steep"])
@pytest.mark.parametrize("gate", ["channel", "head"])
@pytest.mark.parametrize("H,Hk,V", [(40, 8, 96), (66, 33, 96), (30, 10, 256), (40, 40, 256),
                                    (80, 16, 64), (80, 20, 32), (50, 25, 160), (72, 9, 160)])
@pytest.mark.parametrize("K", [64, 128])
def test_prefill_forms_columns(kt, K, H, Hk, V, gate, rate):
    """Widths that do not fill a workgroup's columns, and shared key heads."""
    _check(kt, LENS, H, Hk, K, V, "bf16", "f16", rate, gate, seed=V + K)


@pytest.mark.parametrize("rate", ["slow", "mixed", "steep"])
@pytest.mark.parametrize("lengths,H,V", [([1100], 32, 128), ([1290], 33, 128), ([1300], 64, 128),
                                         ([1300, 1350], 16, 256), ([2000, 0, 1900], 20, 96)])
@pytest.mark.parametrize("K,dtype", [(128, "bf16"), (128, "f32"), (64, "f16")])
def test_prefill_forms_cut(kt, K, dtype, lengths, H, V, rate):
    """Prompts in segments whose outputs take 32 columns to a wavefront."""
    _check(kt, lengths, H, H, K, V, dtype, dtype, rate, seed=H, cut=True)


@pytest.mark.parametrize("K", [64, 128])
def test_prefill_forms_dense(kt, K):
    """[B, T, ...] in every form equals the packed call, bit for bit."""
    for B, H in ((3, 30), (3, 70), (3, 100)):
        c = _inputs([70] * B, H, H, K, 128, "bf16", "mixed", "channel", B)
        cu = torch.arange(0, 70 * B + 1, 70, dtype=torch.int32, device=DEV)
        S1, S2 = c["state"].clone(), c["state"].clone()
        a = [c[x] for x in ("q", "k", "v", "g", "beta")]
        packed = kt.prefill(*a, cu, state=S1)
        dense = kt.prefill(*[x.view((B, 70) + x.shape[1:]) for x in a], state=S2)
        assert torch.equal(dense.view(packed.shape), packed) and torch.equal(S1, S2)


# Convolution: segments of 8 tokens while three projections' wavefronts of 512
# channels leave the 256 compute units with fewer than eight each, else of 16.

@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,H,d", [(2900, 16, 128), (1500, 32, 64), (6000, 9, 128)])
def test_conv_segments(kt, T, H, d, dtype, W):
    """Ragged requests (some of no or few tokens) over segments of many blocks
    of rows: continued and new windows, padding, requests that begin and end
    anywhere in a segment."""
    rng = np.random.default_rng(T + W)
    lengths = []
    while sum(lengths) < T:
        lengths.append(int(rng.choice([0, 1, 2, 3, 5, 17, 40, 200, 700])))
    lengths[-1] -= sum(lengths) - T
    N = len(lengths)
    x = torch.from_numpy(rng.standard_normal((T, 3, H, d)).astype(np.float32)).to(
        gh.out_torch_dtype(dtype))
    cw = rng.uniform(-0.5, 0.5, (3, W, H, d)).astype(np.float32)
    pool = rng.standard_normal((N + 2, 3, H, W - 1, d)).astype(np.float32)
    slot = rng.permutation(N + 2)[:N].astype(np.int32)
    slot[rng.random(N) < 0.1] = -1
    init = rng.integers(0, 2, N).astype(np.int32)
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    cu = dev(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32))
    win = dev(pool)
    got = kt.conv_prefill(x.to(DEV), dev(cw), cu, conv_state=win, slot=dev(slot), init=dev(init))
    want, want_pool = ref.conv(x.double().numpy(), cw, lengths, pool, slot, init)
    half = torch.finfo(x.dtype).eps / 2
    for a, b in zip(got, want):
        # up to 24 FP32 roundings of values of at most 2 |x|
        assert (np.abs(gh.to_numpy_f64(a) - b) <= 2e-5 * (1 + np.abs(b)) + half * np.abs(b)).all()
    assert np.array_equal(win.cpu().numpy().astype(np.float64), want_pool)
    # in two pieces of every request, the same bits
    part = [n // 2 for n in lengths]
    first = np.concatenate([[0], np.cumsum(lengths)])[:-1]
    rows = [np.concatenate([np.arange(b, b + p) for b, p in zip(first, part)]).astype(np.int64),
            np.concatenate([np.arange(b + p, b + n) for b, p, n in zip(first, part, lengths)])]
    win = dev(pool)
    for i, count in enumerate((part, [n - p for n, p in zip(lengths, part)])):
        at = torch.from_numpy(rows[i])
        cu = dev(np.concatenate([[0], np.cumsum(count)]).astype(np.int32))
        start = dev(init) if i == 0 else None
        piece = kt.conv_prefill(x[at].contiguous().to(DEV), dev(cw), cu, conv_state=win,
                                slot=dev(slot), init=start)
        for a, b in zip(piece, got):
            assert torch.equal(a, b[at.to(DEV)])
    assert np.array_equal(win.cpu().numpy().astype(np.float64), want_pool)
