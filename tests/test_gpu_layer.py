"""GPU tests of the KDA layer's calls (chunk map, prompt convolution, gated
delta rule chunked and recurrent, gated RMSNorm) against float64 references.

Tolerances. A rounding to type t is off by at most eps_t / 2 relative.
  * conv, norm: a chain of at most 24 FP32 roundings of values bounded by the
    result's own magnitude (the convolution's by sum |tap x|, at most 2 here
    per unit input): 2e-5 (1 + |ref|), plus the output's half step.
  * delta rule, chunked: a product of two-part bfloat16 factors is off by at
    most 3 x 2^-18 of sum |a b| (two dropped residuals and lo lo), and
    sum |a b| <= |a| |b| <= N with unit keys, N the largest column norm of the
    state plus |v|. An output passes five such products in a row (k S, the
    chunk's L, its inverse, P U or q S, (k)^T U), an inverse of unit keys and
    beta < 1 amplifies by less than 3, and errors of earlier chunks decay with
    the state: 5 x 3 x 3 x 2^-18 N = 1.7e-4 N elementwise is never reached;
    half of it is asked for the state, and that times scale |q| for the
    output. The 2-norm of the error is held to 1e-5 of the result's norm, for
    roundings of random sign: sqrt(5) x 3 x 2^-18 / 3 = 8.5e-6.
  * recurrent: FP32 sums over 128 terms and one rounding per token and
    operation: 2^-24 x (sqrt(128) + 4 tokens) N, at most 4e-6 N here.
"""
import numpy as np
import pytest

import oracle
import synth
from tests import gpu_helpers as gh
from tests import layer_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module")
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tril_solve_amd
    return tril_solve_amd


def _t(name):
    return gh.out_torch_dtype(name)


def _round(x, name):
    """float32 array -> (device tensor of the type, its values in float64)."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(_t(name))
    return t.to(DEV), t.double().numpy()


def _dev(x, dtype=None):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _cu(lengths):
    return _dev(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32))


def _close(got, want, tol, name, what):
    err = np.abs(got - want)
    bound = tol + HALF[name] * np.abs(want)
    bad = ~(err <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} off, worst {np.nanmax(err - bound):.3g} past bound"


# ------------------------------------------------------------------ chunk map

MAPS = [([5], 64), ([0], 16), ([1, 0, 64, 65, 0, 127, 128, 0], 64), ([31, 32, 33, 1], 32),
        ("r5000", 16), ("r9001", 64), ([200000, 3, 0, 70000], 32), ([7, -3, 40], 16)]


def _lens(spec):
    if isinstance(spec, str):
        n = int(spec[1:])
        return np.random.default_rng(n).integers(0, 90, n).tolist()
    return spec


@pytest.mark.parametrize("spec,C", MAPS)
def test_chunk_map(kt, spec, C):
    lens = _lens(spec)
    total = sum(max(n, 0) for n in lens)
    cu, pairs, count = kt.chunk_map(_dev(np.asarray(lens, np.int32)), total, C)
    want = ref.chunk_map(lens, total, C, total // C + len(lens))
    assert np.array_equal(cu.cpu().numpy(), want[0])
    assert np.array_equal(pairs.cpu().numpy(), want[1])
    assert int(count) == want[2]


def test_chunk_map_bounds(kt):
    """Lengths past total_tokens stop there (also where their sum passes 2^31),
    a short map is cut, no map writes cu_seqlens alone, no request gives [0]."""
    lens = [100, 2 ** 31 - 1, 2 ** 31 - 1, 50]
    d = _dev(np.asarray(lens, np.int32))
    for rows in (0, 3, 9, 50):
        cu = torch.full((5,), 7, dtype=torch.int32, device=DEV)
        pairs = torch.full((rows + 1, 2), 7, dtype=torch.int32, device=DEV)
        count = torch.zeros(1, dtype=torch.int32, device=DEV)
        kt.kda_chunk_map(d, 500, 64, cu, pairs[:rows] if rows else None, count)
        want = ref.chunk_map(lens, 500, 64, rows)
        assert np.array_equal(cu.cpu().numpy(), want[0])
        assert np.array_equal(pairs[:rows].cpu().numpy(), want[1]) and int(count) == want[2]
        assert bool((pairs[rows] == 7).all())
    cu, pairs, count = kt.chunk_map(torch.empty(0, dtype=torch.int32, device=DEV), 0)
    assert cu.tolist() == [0] and pairs.shape == (0, 2) and int(count) == 0


@pytest.mark.parametrize("C", [16, 32, 64])
def test_chunk_map_feeds_the_solver(kt, C):
    """The solver and build-A on the map's entries, the (-1, -1) tail among
    them, equal their own scan of cu_seqlens bit for bit."""
    lens = [70, 0, 1, 64, 200, 16, 33]
    T, H = sum(lens), 3
    A = _dev(synth.delta_rule_A(lens, H, seed=5, upper="nan", chunk=C))
    cu, pairs, _ = kt.chunk_map(_dev(np.asarray(lens, np.int32)), T, C)
    X = kt.tril_inv(A, cu, chunk_indices=pairs, algo="fused")
    assert torch.equal(X, kt.tril_inv(A, cu, algo="fused"))
    if C == 64:
        k, g, beta = (_dev(x) for x in synth.delta_rule_inputs(lens, H, 6, K=128))
        Y = kt.kkt_tril_inv(k, g, beta, cu, chunk_indices=pairs)
        assert torch.equal(Y, kt.kkt_tril_inv(k, g, beta, cu))


def test_chunk_map_graph(kt):
    """Captured once, replayed on other lengths with eager work between."""
    lens = torch.zeros(40, dtype=torch.int32, device=DEV)
    cu = torch.empty(41, dtype=torch.int32, device=DEV)
    pairs = torch.empty((4000 // 32 + 40, 2), dtype=torch.int32, device=DEV)
    count = torch.empty(1, dtype=torch.int32, device=DEV)
    kt.kda_chunk_map(lens, 4000, 32, cu, pairs, count)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kt.kda_chunk_map(lens, 4000, 32, cu, pairs, count)
    rng = np.random.default_rng(1)
    for _ in range(4):
        now = rng.integers(0, 100, 40)
        lens.copy_(_dev(now.astype(np.int32)))
        pairs.fill_(9)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = ref.chunk_map(now, 4000, 32, pairs.shape[0])
        assert np.array_equal(cu.cpu().numpy(), want[0])
        assert np.array_equal(pairs.cpu().numpy(), want[1]) and int(count) == want[2]


# ----------------------------------------------------------------------- conv

def _conv_inputs(lengths, H, d, W, dtype, seed, slots=None):
    rng = np.random.default_rng(seed)
    T = sum(lengths)
    slots = slots or len(lengths) + 2
    x, x64 = _round(rng.standard_normal((T, 3, H, d)), dtype)
    return dict(x=x, x64=x64, cw=rng.uniform(-0.5, 0.5, (3, W, H, d)).astype(np.float32),
                pool=rng.standard_normal((slots, 3, H, W - 1, d)).astype(np.float32),
                slot=rng.permutation(slots)[:len(lengths)].astype(np.int32),
                init=rng.integers(0, 2, len(lengths)).astype(np.int32))


def _conv_check(kt, c, lengths, dtype, slot, init, pool=True, eps=1e-6):
    d_pool = _dev(c["pool"]) if pool else None
    got = kt.conv_prefill(c["x"], _dev(c["cw"]), _cu(lengths), conv_state=d_pool,
                          slot=None if slot is None else _dev(slot),
                          init=None if init is None else _dev(init), eps_l2=eps)
    want, want_pool = ref.conv(c["x64"], c["cw"], lengths, c["pool"] if pool else None, slot,
                               init, eps)
    for a, b, what in zip(got, want, "qkv"):
        a = gh.to_numpy_f64(a)
        _close(a, b, 2e-5 * (1 + np.abs(b)), dtype, what)
    if pool:
        assert np.array_equal(d_pool.cpu().numpy().astype(np.float64), want_pool)


CONV_LENS = [[1], [64], [0, 1, 2, 3, 0, 4, 15, 16, 17, 33, 0], [14, 1, 1, 1, 1, 40, 2], [130, 7]]


@pytest.mark.parametrize("lengths", CONV_LENS)
@pytest.mark.parametrize("W", [2, 3, 4])
def test_conv(kt, lengths, W):
    c = _conv_inputs(lengths, 3, 128, W, "f32", 10 + W)
    _conv_check(kt, c, lengths, "f32", c["slot"], c["init"])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("H,d", [(1, 64), (5, 64), (4, 128), (9, 128)])
def test_conv_types_and_heads(kt, H, d, dtype):
    lengths = [37, 0, 3, 80]
    c = _conv_inputs(lengths, H, d, 4, dtype, 20 + H)
    _conv_check(kt, c, lengths, dtype, c["slot"], c["init"])
    _conv_check(kt, c, lengths, dtype, None, None)          # request n continues slot n
    _conv_check(kt, c, lengths, dtype, None, None, pool=False)
    _conv_check(kt, c, lengths, dtype, c["slot"], None, eps=0.5)


def test_conv_padding_and_untouched_rows(kt):
    """Padding entries give zeros and touch nothing; rows behind the last
    request keep their bits; a dense batch equals the packed one."""
    lengths = [20, 30, 10]
    c = _conv_inputs(lengths, 2, 128, 4, "bf16", 30)
    slot = np.array([c["slot"][0], -1, 99], np.int32)
    _conv_check(kt, c, lengths, "bf16", slot, c["init"])
    q, k, v = (torch.full((60, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(3))
    cu = _dev(np.array([0, 20, 45], np.int32))
    kt.kda_conv_prefill(c["x"], _dev(c["cw"]), q, k, v, cu)
    assert bool((q[45:] == 7).all() and (k[45:] == 7).all() and (v[45:] == 7).all())
    assert not bool((v[:45] == 7).any())
    dense = kt.conv_prefill(c["x"].view(3, 20, 3, 2, 128), _dev(c["cw"]))
    packed = kt.conv_prefill(c["x"], _dev(c["cw"]), _cu([20, 20, 20]))
    for a, b in zip(dense, packed):
        assert torch.equal(a.view(b.shape), b)


def test_conv_of_no_tokens(kt):
    """Requests of no tokens: windows kept where they continue, zeroed where
    they start anew."""
    c = _conv_inputs([0, 0], 2, 64, 3, "f32", 31)
    c["init"][:] = [0, 1]
    _conv_check(kt, c, [0, 0], "f32", c["slot"], c["init"])


def test_conv_in_pieces(kt):
    """A prompt run in pieces on its window equals one piece, bit for bit."""
    c = _conv_inputs([100], 3, 128, 4, "bf16", 32)
    cw = _dev(c["cw"])
    pool = torch.zeros((1, 3, 3, 3, 128), device=DEV)
    whole = kt.conv_prefill(c["x"], cw, _cu([100]), conv_state=pool.clone())
    at = 0
    for n in (1, 2, 40, 17, 1, 39):
        part = kt.conv_prefill(c["x"][at:at + n].contiguous(), cw, _cu([n]), conv_state=pool)
        for a, b in zip(part, whole):
            assert torch.equal(a, b[at:at + n])
        at += n


# ----------------------------------------------------------------- delta rule

def _delta_inputs(lengths, H, Hk, K, V, dtype, seed, gate="channel", rate="slow", slots=None):
    rng = np.random.default_rng(seed)
    T, N = sum(lengths), len(lengths)
    slots = slots or N + 2

    def unit(*s):
        x = rng.standard_normal(s)
        return x / np.linalg.norm(x, axis=-1, keepdims=True)

    c = dict(H=H, K=K, V=V, dtype=dtype, lengths=lengths)
    c["q"], c["q64"] = _round(unit(T, Hk, K), dtype)
    c["k"], c["k64"] = _round(unit(T, Hk, K), dtype)
    c["v"], c["v64"] = _round(rng.standard_normal((T, H, V)), dtype)
    shape = (T, H, K) if gate == "channel" else (T, H)
    if rate == "slow":
        g = -np.logaddexp(0.0, -(rng.standard_normal(shape) + 3.0))
    elif rate == "mixed":
        r = np.exp(rng.uniform(np.log(0.004), np.log(4.0), shape[1:]))
        g = -r * np.logaddexp(0.0, rng.standard_normal(shape))
    else:  # steep: some channels far past what eight tokens of one factor can hold, some reset
        g = -np.exp(rng.uniform(np.log(0.01), np.log(40.0), shape))
        g[rng.random(shape) < 0.01] = -np.inf
    c["g"] = g.astype(np.float32)
    c["beta"] = (1 / (1 + np.exp(-rng.standard_normal((T, H))))).astype(np.float32)
    c["state"] = (0.2 * rng.standard_normal((slots, H, K, V))).astype(np.float32)
    c["slot"] = rng.permutation(slots)[:N].astype(np.int32)
    c["init"] = rng.integers(0, 2, N).astype(np.int32)
    return c


def _delta_run(kt, form, c, slot="own", init="own", pool=True, out_dtype=None, **kw):
    d = dict(state=_dev(c["state"]) if pool else None)
    for name, v in (("slot", slot), ("init", init)):
        v = c[name] if isinstance(v, str) else v
        d[name] = None if v is None else _dev(v)
    fn = kt.prefill if form == "prefill" else kt.recurrent
    out = fn(c["q"], c["k"], c["v"], _dev(c["g"]), _dev(c["beta"]), _cu(c["lengths"]),
             out_dtype=None if out_dtype is None else _t(out_dtype), **d, **kw)
    torch.cuda.synchronize()
    return out, d["state"]


def _delta_check(kt, form, c, slot="own", init="own", pool=True, out_dtype=None, scale=None):
    out, state = _delta_run(kt, form, c, slot, init, pool, out_dtype, scale=scale)
    scale = c["K"] ** -0.5 if scale is None else scale
    pick = lambda n, v: c[n] if isinstance(v, str) else v  # noqa: E731
    want, want_S, N = ref.delta_rule(c["q64"], c["k64"], c["v64"], c["g"], c["beta"],
                                     c["lengths"], c["state"] if pool else None,
                                     pick("slot", slot), pick("init", init), scale)
    unit = 8.5e-5 if form == "prefill" else 4e-6
    got = gh.to_numpy_f64(out)
    name = out_dtype or c["dtype"]
    _close(got, want, unit * N * scale * 1.01, name, "out")
    if pool:
        S = state.cpu().numpy().astype(np.float64)
        _close(S, want_S, unit * N, "f32", "state")
        norm = np.linalg.norm(want_S)
        assert norm == 0 or np.linalg.norm(S - want_S) <= 1e-5 * norm
    if name == "f32" and want.size:
        assert np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(want)


FORMS = ["prefill", "recurrent"]
DELTA_LENS = [[1], [32], [0, 1, 2, 7, 8, 9, 0], [15, 16, 17, 31, 33], [64, 65, 100], [257]]


@pytest.mark.parametrize("lengths", DELTA_LENS)
@pytest.mark.parametrize("form", FORMS)
def test_delta_lengths(kt, form, lengths):
    print(f"\n[delta] {form} lengths={lengths}", flush=True)
    _delta_check(kt, form, _delta_inputs(lengths, 2, 2, 128, 128, "f32", 40 + len(lengths)))


@pytest.mark.parametrize("H,Hk,K,V", [(1, 1, 64, 32), (2, 1, 64, 64), (6, 3, 128, 96),
                                      (3, 3, 128, 256), (4, 1, 64, 160), (2, 2, 128, 64)])
@pytest.mark.parametrize("gate", ["channel", "head"])
@pytest.mark.parametrize("form", FORMS)
def test_delta_heads(kt, form, gate, H, Hk, K, V):
    print(f"\n[delta] {form} H={H} Hk={Hk} K={K} V={V} gate={gate}", flush=True)
    _delta_check(kt, form, _delta_inputs([45, 3], H, Hk, K, V, "f32", 50 + V, gate=gate))


@pytest.mark.parametrize("out_dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("form", FORMS)
def test_delta_types(kt, form, dtype, out_dtype):
    for K in (64, 128):
        c = _delta_inputs([70, 9], 2, 2, K, 128, dtype, 60 + K)
        _delta_check(kt, form, c, out_dtype=out_dtype)


@pytest.mark.parametrize("rate", ["mixed", "steep"])
@pytest.mark.parametrize("gate", ["channel", "head"])
@pytest.mark.parametrize("form", FORMS)
def test_delta_decays(kt, form, gate, rate):
    """Slow and fast channels side by side, and decays past FP32's range with
    resets (-inf) among them."""
    for K in (64, 128):
        _delta_check(kt, form, _delta_inputs([100, 40, 5], 3, 3, K, 64, "f32", 70 + K, gate=gate,
                                             rate=rate))


@pytest.mark.parametrize("form", FORMS)
def test_delta_pools(kt, form):
    """No pool; slots of their own; padding entries; every init; a scale."""
    c = _delta_inputs([20, 33, 0, 12], 2, 2, 64, 64, "f32", 80)
    _delta_check(kt, form, c, pool=False)
    _delta_check(kt, form, c, slot=None, init=None)
    _delta_check(kt, form, c, init=np.zeros(4, np.int32), scale=0.7)
    _delta_check(kt, form, c, slot=np.array([3, -1, 1, 77], np.int32))


@pytest.mark.parametrize("form", FORMS)
def test_delta_of_no_tokens(kt, form):
    c = _delta_inputs([0, 0], 2, 2, 64, 64, "f32", 81)
    _delta_check(kt, form, c, init=np.array([0, 1], np.int32))


@pytest.mark.parametrize("form", FORMS)
def test_delta_rows_behind_the_last_request(kt, form):
    """Rows that belong to no request keep their bits, and what stands in them
    (NaN) reaches nothing, nor does what stands in a neighbouring request."""
    c = _delta_inputs([10, 40, 14], 2, 2, 128, 64, "f32", 82)
    cu = np.array([0, 10, 50], np.int32)
    for x in ("q", "k", "v"):
        c[x][50:] = float("nan")
        c[x][:10] = float("nan")
    for x in ("g", "beta"):
        c[x][50:] = np.nan
    out = torch.full(c["v"].shape, 7.0, device=DEV)
    fn = kt.kda_prefill if form == "prefill" else kt.kda_recurrent
    fn(c["q"], c["k"], c["v"], _dev(c["g"]), _dev(c["beta"]), out, _dev(cu))
    assert bool((out[50:] == 7).all())
    want, _, N = ref.delta_rule(c["q64"][10:50], c["k64"][10:50], c["v64"][10:50], c["g"][10:50],
                                c["beta"][10:50], [40], scale=128 ** -0.5)
    _close(gh.to_numpy_f64(out[10:50]), want, 8.5e-5 * N * 128 ** -0.5, "f32", "out")


@pytest.mark.parametrize("form", FORMS)
def test_delta_dense(kt, form):
    c = _delta_inputs([40, 40], 2, 1, 64, 64, "bf16", 83)
    fn = kt.prefill if form == "prefill" else kt.recurrent
    S1, S2 = _dev(c["state"]), _dev(c["state"])
    g, beta = _dev(c["g"]), _dev(c["beta"])
    packed = fn(c["q"], c["k"], c["v"], g, beta, _cu([40, 40]), state=S1)
    rows = lambda x: x.view((2, 40) + x.shape[1:])  # noqa: E731
    dense = fn(rows(c["q"]), rows(c["k"]), rows(c["v"]), rows(g), rows(beta), state=S2)
    assert torch.equal(dense.view(packed.shape), packed) and torch.equal(S1, S2)


@pytest.mark.parametrize("form", FORMS)
def test_delta_in_pieces(kt, form):
    """A prompt in pieces on its state agrees with the one-piece reference."""
    c = _delta_inputs([150], 2, 2, 128, 128, "f32", 84, slots=1)
    S = _dev(c["state"])
    g, beta = _dev(c["g"]), _dev(c["beta"])
    fn = kt.prefill if form == "prefill" else kt.recurrent
    outs, at = [], 0
    for n in (64, 1, 32, 50, 3):
        s = slice(at, at + n)
        outs.append(fn(c["q"][s], c["k"][s], c["v"][s], g[s], beta[s], _cu([n]), state=S))
        at += n
    want, want_S, N = ref.delta_rule(c["q64"], c["k64"], c["v64"], c["g"], c["beta"], [150],
                                     c["state"], scale=128 ** -0.5)
    _close(gh.to_numpy_f64(torch.cat(outs)), want, 8.5e-5 * N * 128 ** -0.5, "f32", "out")
    _close(S.cpu().numpy().astype(np.float64), want_S, 8.5e-5 * N, "f32", "state")


@pytest.mark.parametrize("form", FORMS)
def test_delta_repeats_and_streams(kt, form):
    """The same call gives the same bits, on the current stream, on another
    one, and replayed from a graph with eager work in between."""
    c = _delta_inputs([33, 70, 4], 4, 2, 128, 128, "bf16", 85)
    first, S0 = _delta_run(kt, form, c)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again, S1 = _delta_run(kt, form, c, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(first, again) and torch.equal(S0, S1)
    fn = kt.kda_prefill if form == "prefill" else kt.kda_recurrent
    S, out = _dev(c["state"]), torch.empty_like(first)
    a = dict(state=S, slot=_dev(c["slot"]), init=_dev(c["init"]))
    g, beta, cu = _dev(c["g"]), _dev(c["beta"]), _cu(c["lengths"])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fn(c["q"], c["k"], c["v"], g, beta, out, cu, **a)
    for _ in range(3):
        S.copy_(_dev(c["state"]))
        out.fill_(3.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(S, S0)
        _delta_run(kt, form, c)


@pytest.mark.parametrize("form", FORMS)
def test_delta_pool_past_4gib(kt, form):
    """Slots whose byte offsets need more than 32 bits; a slot that no request
    names keeps its bits."""
    c = _delta_inputs([40, 3], 32, 32, 128, 128, "bf16", 86, slots=2)
    pool = torch.zeros((2100, 32, 128, 128), device=DEV)
    pool[2000] = 7.0
    where = np.array([2099, 2050], np.int32)
    for i in range(2):
        pool[where[i]] = _dev(c["state"][i])
    fn = kt.prefill if form == "prefill" else kt.recurrent
    out = fn(c["q"], c["k"], c["v"], _dev(c["g"]), _dev(c["beta"]), _cu([40, 3]), state=pool,
             slot=_dev(where))
    same, S = _delta_run(kt, form, c, slot=None, init=None)
    assert torch.equal(out, same)
    assert torch.equal(pool[2099], S[0]) and torch.equal(pool[2050], S[1])
    assert bool((pool[2000] == 7.0).all()) and bool((pool[:2000] == 0).all())


# Prompts that are cut into segments (at least 16 chunks of 32 tokens a request,
# few heads): the same tolerances, since the products that carry a state over a
# segment are those that carry it over a chunk.

CUT_LENS = [[512], [513], [640, 600], [1100, 0, 31, 1, 1500], [1000, 1025, 63, 32]]


def _cut_size(kt, c):
    return kt.kda_prefill_workspace_size(sum(c["lengths"]), len(c["lengths"]), c["H"], c["K"],
                                         c["V"])


@pytest.mark.parametrize("lengths", CUT_LENS)
def test_prefill_cut_lengths(kt, lengths):
    c = _delta_inputs(lengths, 2, 2, 128, 128, "f32", 140 + len(lengths))
    assert _cut_size(kt, c) > 0
    _delta_check(kt, "prefill", c)


@pytest.mark.parametrize("H,Hk,K,V", [(1, 1, 64, 32), (6, 3, 128, 96), (2, 1, 128, 256),
                                      (4, 1, 64, 160), (64, 16, 64, 64)])
@pytest.mark.parametrize("gate", ["channel", "head"])
def test_prefill_cut_heads(kt, gate, H, Hk, K, V):
    c = _delta_inputs([700 if H <= 32 else 1300], H, Hk, K, V, "f32", 150 + V, gate=gate)
    assert _cut_size(kt, c) > 0
    _delta_check(kt, "prefill", c)


@pytest.mark.parametrize("dtype,out_dtype", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"),
                                             ("bf16", "f32"), ("f32", "f16")])
@pytest.mark.parametrize("rate", ["slow", "mixed", "steep"])
def test_prefill_cut_types_and_decays(kt, rate, dtype, out_dtype):
    """Also decays that leave nothing of a state within a segment (its map all
    but zero), and resets."""
    for K in (64, 128):
        c = _delta_inputs([900, 570], 2, 2, K, 64, dtype, 160 + K, rate=rate)
        assert _cut_size(kt, c) > 0
        _delta_check(kt, "prefill", c, out_dtype=out_dtype)


def test_prefill_cut_pools(kt):
    """No pool; slots of their own; padding entries; every init."""
    c = _delta_inputs([600, 33, 0, 1700], 2, 2, 64, 64, "f32", 170)
    assert _cut_size(kt, c) > 0
    _delta_check(kt, "prefill", c, pool=False)
    _delta_check(kt, "prefill", c, slot=None, init=None)
    _delta_check(kt, "prefill", c, init=np.zeros(4, np.int32), scale=0.7)
    _delta_check(kt, "prefill", c, slot=np.array([3, -1, 1, 77], np.int32))


def _with_workspace(kt, c, nbytes, fill=float("nan"), cu=None):
    """kda_prefill with a workspace of nbytes inside a larger filled buffer:
    out, state and the buffer before and after the workspace."""
    buf = torch.full((nbytes // 4 + 512,), fill, device=DEV)
    ws = buf[256:256 + nbytes // 4]
    S, out = _dev(c["state"]), torch.zeros_like(c["v"])
    kt.kda_prefill(c["q"], c["k"], c["v"], _dev(c["g"]), _dev(c["beta"]), out,
                   _cu(c["lengths"]) if cu is None else _dev(cu), state=S, slot=_dev(c["slot"]),
                   init=_dev(c["init"]), workspace=ws if nbytes else None)
    torch.cuda.synchronize()
    return out, S, torch.cat([buf[:256], buf[256 + nbytes // 4:]]), ws


def test_prefill_workspace_contents(kt):
    """What a workspace holds before does not matter, and nothing is written
    outside of it; with one that is too small, or none, requests run whole and
    it keeps its bits."""
    c = _delta_inputs([900, 0, 1300], 2, 2, 128, 128, "bf16", 171)
    n = _cut_size(kt, c)
    a = _with_workspace(kt, c, n)
    b = _with_workspace(kt, c, n, fill=5.0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert bool(a[2].isnan().all()) and bool((b[2] == 5.0).all())
    whole = _with_workspace(kt, c, 0)
    short = _with_workspace(kt, c, n - 16, fill=5.0)
    assert torch.equal(whole[0], short[0]) and torch.equal(whole[1], short[1])
    assert bool((short[3] == 5.0).all())
    big = _with_workspace(kt, c, n + 64)
    assert torch.equal(a[0], big[0]) and torch.equal(a[1], big[1])
    dense = _delta_inputs([800, 800], 2, 2, 128, 64, "bf16", 172)
    rows = lambda x: x.view((2, 800) + x.shape[1:])  # noqa: E731
    g, beta = _dev(dense["g"]), _dev(dense["beta"])
    S1, S2 = _dev(dense["state"]), _dev(dense["state"])
    packed = kt.prefill(dense["q"], dense["k"], dense["v"], g, beta, _cu([800, 800]), state=S1)
    got = kt.prefill(rows(dense["q"]), rows(dense["k"]), rows(dense["v"]), rows(g), rows(beta),
                     state=S2)
    assert torch.equal(got.view(packed.shape), packed) and torch.equal(S1, S2)


def test_prefill_cut_row_offsets_out_of_order(kt):
    """Offsets that go back or past the rows are clamped: more segments than the
    workspace holds are left out, and nothing outside of it is written."""
    c = _delta_inputs([1100, 0, 1100, 0], 2, 2, 64, 64, "bf16", 173)
    n = _cut_size(kt, c)
    assert n > 0
    for cu in ([0, 2200, 0, 2200, 2200], [0, 1100, 5000, -3, 2200], [2200, 0, 0, 0, 9]):
        out, S, around, _ = _with_workspace(kt, c, n, fill=5.0, cu=np.array(cu, np.int32))
        assert bool((around == 5.0).all())


def test_prefill_cut_streams_and_graphs(kt):
    """Two cut calls at once on streams and workspaces of their own, and a
    replayed one with eager calls in between, give the bits of a call alone."""
    c = _delta_inputs([1500, 600], 2, 2, 128, 128, "bf16", 174)
    first, S0 = _delta_run(kt, "prefill", c)
    g, beta, cu = _dev(c["g"]), _dev(c["beta"]), _cu(c["lengths"])
    rest = dict(slot=_dev(c["slot"]), init=_dev(c["init"]))
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for side in sides:
        S, out = _dev(c["state"]), torch.empty_like(first)
        ws = torch.empty(_cut_size(kt, c), dtype=torch.uint8, device=DEV)
        got.append((S, out, ws))
    torch.cuda.synchronize()
    for _ in range(3):
        for side, (S, out, ws) in zip(sides, got):
            with torch.cuda.stream(side):
                S.copy_(_dev(c["state"]))
            kt.kda_prefill(c["q"], c["k"], c["v"], g, beta, out, cu, state=S, workspace=ws,
                           stream=side, **rest)
    torch.cuda.synchronize()
    for S, out, _ in got:
        assert torch.equal(out, first) and torch.equal(S, S0)
    S, out, ws = got[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kt.kda_prefill(c["q"], c["k"], c["v"], g, beta, out, cu, state=S, workspace=ws, **rest)
    for _ in range(3):
        S.copy_(_dev(c["state"]))
        out.fill_(3.0)
        ws.fill_(77)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first) and torch.equal(S, S0)
        _delta_run(kt, "prefill", c)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("K", [64, 128])
def test_prefill_state_of_slow_and_steep_heads(kt, K, dtype):
    """One decay per head from 0.004 to 3.5 nats a token: a state that is large
    against what a chunk adds, and exponents of many powers of two. Each head's
    state to 2e-6 of its norm: products of parts kept to 2^-19 of a term (K =
    128 with an FP32 output; else 2^-24) leave 1e-6 of a slow head's state."""
    rates = np.array([0.004, 0.02, 0.1, 0.4, 1.0, 2.0, 3.5])
    for lengths in ([256], [640]):  # whole, and cut into segments
        c = _delta_inputs(lengths, 7, 7, K, 64, dtype, 180 + K, gate="head")
        rng = np.random.default_rng(181)
        c["g"] = (-rates * np.logaddexp(0.0, rng.standard_normal(c["g"].shape))).astype(np.float32)
        _, S = _delta_run(kt, "prefill", c, slot=None, init=None)
        _, want, _ = ref.delta_rule(c["q64"], c["k64"], c["v64"], c["g"], c["beta"], lengths,
                                    c["state"], None, None, K ** -0.5)
        off = S.cpu().numpy().astype(np.float64)[0] - want[0]
        for h in range(7):
            assert np.linalg.norm(off[h]) <= 2e-6 * np.linalg.norm(want[0, h]), (lengths, h)


@pytest.mark.parametrize("requests,H", [(1, 257), (3, 100), (200, 2)])
def test_prefill_many_workgroups(kt, requests, H):
    """More workgroups than compute units: wavefronts that prepare and walk."""
    c = _delta_inputs([37] * requests, H, H, 64, 32, "bf16", 175)
    assert _cut_size(kt, c) == 0
    _delta_check(kt, "prefill", c)
    c = _delta_inputs([37] * requests, H, H, 128, 32, "f32", 176, rate="mixed")
    _delta_check(kt, "prefill", c)


# ----------------------------------------------------------------------- norm

@pytest.mark.parametrize("out_dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shape", [(1, 1, 64), (7, 3, 128), (2, 5, 9, 64), (130, 2, 128)])
def test_norm(kt, shape, dtype, out_dtype):
    rng = np.random.default_rng(sum(shape))
    o, o64 = _round(0.3 * rng.standard_normal(shape), dtype)
    z, z64 = _round(3 * rng.standard_normal(shape), dtype)
    w = (1 + 0.1 * rng.standard_normal(shape[-1])).astype(np.float32)
    for eps in (1e-6, 0.5):
        got = gh.to_numpy_f64(kt.gated_norm(o, z, _dev(w), eps, out_dtype=_t(out_dtype)))
        want = ref.gated_norm(o64, z64, w, eps)
        _close(got, want, 2e-5 * (1 + np.abs(want)), out_dtype, "norm")
    if dtype == out_dtype:
        want = kt.gated_norm(o, z, _dev(w))
        kt.kda_gated_norm(o, z, _dev(w), o)  # in place
        assert torch.equal(o, want)


# ------------------------------------------------------------------- together

@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layer_as_served(kt, form, dtype):
    """A batch of prompts through the chunk map, the convolution, the delta
    rule and the norm, then decode steps on the pools they left: every output
    agrees with the decode step's oracle run token by token."""
    lengths, H, d, W, steps = [37, 5, 64], 3, 128, 4, 2
    N, T = len(lengths), sum(lengths)
    base = synth.decode_inputs(N, H, W=W, seed=90)
    rng = np.random.default_rng(91)
    cw, nw = base["conv_w"], base["norm_w"]
    x, x64 = _round(rng.standard_normal((T, 3, H, d)), dtype)
    z, z64 = _round(rng.standard_normal((T, H, d)), dtype)
    g = -np.logaddexp(0.0, -(rng.standard_normal((T, H, d)) + 3.0)).astype(np.float32)
    beta = (1 / (1 + np.exp(-rng.standard_normal((T, H))))).astype(np.float32)
    S, win = _dev(base["state"]), _dev(base["conv_state"])
    slot, init = _dev(base["slot"]), torch.zeros(N, dtype=torch.int32, device=DEV)
    cu, pairs, _ = kt.chunk_map(_dev(np.asarray(lengths, np.int32)), T)
    assert torch.equal(cu, _cu(lengths))
    pool = dict(slot=slot, init=init)
    q, k, v = kt.conv_prefill(x, _dev(cw), cu, conv_state=win, **pool)
    fn = kt.prefill if form == "prefill" else kt.recurrent
    o = fn(q, k, v, _dev(g), _dev(beta), cu, state=S, out_dtype=torch.float32, **pool)
    y = gh.to_numpy_f64(kt.gated_norm(o, z.float(), _dev(nw)))
    # the oracle: one decode step per token, from zeros
    S64 = np.zeros(base["state"].shape)
    w64 = np.zeros(base["conv_state"].shape)
    S64_out = np.zeros((T, H, d))
    bits = (lambda a: synth.to_bf16_bits(a)) if dtype == "bf16" else (lambda a: a)
    for n, m in enumerate(lengths):
        b = sum(lengths[:n])
        one = base["slot"][n:n + 1]
        for t in range(b, b + m):
            r, S64, w64 = oracle.kda_decode(
                bits(x64[t:t + 1].astype(np.float32)), g[t:t + 1], beta[t:t + 1],
                bits(z64[t:t + 1].astype(np.float32)), nw, cw, one, S64, w64, dtype, 1e-6, 1e-6)
            S64_out[t] = r[0]
    # q, k and v were rounded to the tensors' type in between: half a step each, and the norm
    # divides by an rms of about 0.1 of its largest entries
    tol = 2e-4 if dtype == "f32" else 60 * 2.0 ** -8
    assert np.abs(y - S64_out).max() <= tol
    rel = np.linalg.norm(y - S64_out) / np.linalg.norm(S64_out)
    assert rel <= (2e-5 if dtype == "f32" else 3 * 2.0 ** -8)
    idx = base["slot"]
    got = S[torch.from_numpy(idx.astype(np.int64)).to(DEV)].cpu().numpy()
    rel = np.linalg.norm(got - S64[idx]) / np.linalg.norm(S64[idx])
    assert rel <= (2e-5 if dtype == "f32" else 3 * 2.0 ** -8)
    # decoding goes on from there
    S64[idx] = got
    w64 = win.cpu().numpy().astype(np.float64)
    S64_full = S.cpu().numpy().astype(np.float64)
    for step in range(steps):
        nxt = synth.decode_inputs(N, H, W=W, seed=95 + step)
        out = torch.empty((N, H, d), device=DEV)
        kt.kda_decode_step(_dev(nxt["qkv"]), _dev(nxt["z"]), _dev(nxt["g"]), _dev(nxt["beta"]),
                           _dev(nw), _dev(cw), slot, S, win, out)
        r, S64_full, w64 = oracle.kda_decode(nxt["qkv"], nxt["g"], nxt["beta"], nxt["z"], nw, cw,
                                             idx, S64_full, w64, "f32", 1e-6, 1e-6)
        assert gh.excess(gh.to_numpy_f64(out), r, "f32") <= 0
