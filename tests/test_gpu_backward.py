"""GPU tests of the KDA layer's backward pass and of the 8-bit checkpoints against
float64 references.

Tolerances. A rounding to type t is off by at most eps_t / 2 relative.
  * delta rule: a gradient passes at most ten chained sums (forwards k S, the
    chunk's matrices, their inverse, U, S; backwards dU, Y, dS, the products with
    both states, the pairs) of FP32 products, 128 terms or fewer each, whose
    roundings of random sign add as the root of their number: 2^-24 sqrt(10) of
    the terms, times 3 for the inverse of unit keys and beta < 1 (and its
    transpose), times 2 for terms that are larger than their sums: 1.1e-6 of the
    2-norm. 2e-6 is asked for it, and 40 times that elementwise of the larger of
    the value and the root mean square; outputs of 16 bits add their half step.
  * convolution, norm: chains of at most 30 FP32 roundings (and of the 1-ulp
    reciprocals and exponentials) of values bounded by the terms: 2e-5 of the
    larger of the value and the root mean square; dconv_w and dnorm_w are sums of
    random sign over the tokens, 2^-24 sqrt(tokens) of their largest partial sums:
    2e-6 of the 2-norm.
  * checkpoints: codes and scales are exact.
"""
import numpy as np
import pytest

from tests import backward_reference as bref
from tests import layer_reference as ref
from tests.test_gpu_layer import HALF, _cu, _dev, _round, _t

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tril_solve_amd
    return tril_solve_amd


def _np(t):
    return t.double().cpu().numpy()


def _check(got, want, name, what, norm=2e-6, each=8e-5):
    """2-norm and elementwise bounds of a gradient of type `name`."""
    got, want = _np(got), np.asarray(want)
    assert got.shape == want.shape, what
    if not want.size:
        return
    assert np.isfinite(got).all(), what
    err, size = np.abs(got - want), np.sqrt((want ** 2).mean())
    tiny = 2.0 ** -24 if name == "f16" else 0.0  # half the smallest binary16
    assert np.sqrt((err ** 2).mean()) <= (norm + (0 if name == "f32" else HALF[name])) * size + tiny, \
        f"{what}: {np.sqrt((err ** 2).mean()) / size:.3g} of the norm"
    bound = each * np.maximum(size, np.abs(want)) + tiny
    if name != "f32":
        bound += HALF[name] * np.abs(want)
    assert (err <= bound).all(), f"{what}: {(err - bound).max():.3g} past bound"


# ------------------------------------------------------------------ delta rule

def _delta(lens, H, Hk, K, V, dtype="f32", odt="f32", gate="channel", rate="slow", slots=0, seed=0,
           tail=0):
    """Inputs on the device and their values in float64. slots 0: no pools."""
    rng = np.random.default_rng(seed)
    T = sum(lens) + tail
    unit = lambda x: x / np.sqrt((x ** 2).sum(-1, keepdims=True))  # noqa: E731
    d, h = {}, {}
    for name, x, t in (("q", unit(rng.normal(size=(T, Hk, K))), dtype),
                       ("k", unit(rng.normal(size=(T, Hk, K))), dtype),
                       ("v", rng.normal(size=(T, H, V)), dtype),
                       ("dout", rng.normal(size=(T, H, V)), odt)):
        d[name], h[name] = _round(x, t)
    shape = (T, H, K) if gate == "channel" else (T, H)
    if rate == "slow":
        g = -np.log1p(np.exp(-rng.normal(size=shape) - 3.0))
    elif rate == "mixed":
        g = -np.exp(rng.uniform(np.log(0.004), np.log(3.0), shape[1:])) * rng.random(shape) * 2
    else:  # steep: also resets, falls of hundreds, and none at all
        g = -rng.choice([0.0, 0.01, 1.0, 6.0, 40.0, 300.0, np.inf], size=shape,
                        p=[.2, .3, .2, .1, .1, .05, .05])
    h["g"] = g.astype(np.float32)
    h["beta"] = rng.random((T, H)).astype(np.float32)
    d["g"], d["beta"] = _dev(h["g"]), _dev(h["beta"])
    if slots:
        n = len(lens)
        h["state"] = rng.normal(size=(slots, H, K, V)).astype(np.float32)
        h["dstate"] = rng.normal(size=(slots, H, K, V)).astype(np.float32)
        h["slot"] = rng.permutation(slots)[:n].astype(np.int32)
        h["init"] = rng.integers(0, 2, n).astype(np.int32)
        for x in ("state", "dstate", "slot", "init"):
            d[x] = _dev(h[x])
    d["cu"] = _cu(lens)
    return d, h


def _run_delta(kt, d, scale=0.1, **kw):
    grads = kt.prefill_backward(d["dout"], d["q"], d["k"], d["v"], d["g"], d["beta"], d["cu"],
                                state=d.get("state"), dstate=d.get("dstate"), slot=d.get("slot"),
                                init=d.get("init"), scale=scale, **kw)
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta"), grads))


def _want_delta(h, lens, scale=0.1):
    T = sum(lens)
    return bref.delta_rule_grad(*(h[x][:T] for x in ("dout", "q", "k", "v", "g", "beta")), lens,
                                h.get("state"), h.get("dstate"), h.get("slot"), h.get("init"),
                                scale)


def _compare_delta(got, want, dtype, rows, what=""):
    for x in got:
        t = dtype if x in ("dq", "dk", "dv") else "f32"
        _check(got[x][:rows], want[x], t, f"{what} {x}")


CASES = [
    # lengths, H, Hk, K, V, inputs, dout, gate, rate, slots
    ([1], 1, 1, 64, 32, "f32", "f32", "channel", "slow", 0),
    ([64], 2, 2, 128, 128, "f32", "f32", "channel", "slow", 0),
    ([65, 1, 0, 63, 128], 2, 1, 64, 96, "f32", "f32", "head", "mixed", 7),
    ([16, 17, 15, 33, 2], 4, 2, 128, 64, "bf16", "bf16", "channel", "mixed", 5),
    ([200, 0, 3], 3, 3, 64, 256, "f16", "f32", "channel", "slow", 4),
    ([129], 2, 2, 128, 160, "bf16", "f16", "head", "slow", 2),
    ([130, 5], 6, 2, 128, 224, "f32", "bf16", "channel", "mixed", 3),
    ([40, 90], 2, 2, 64, 64, "f16", "f16", "head", "mixed", 2),
    ([70, 2, 64], 2, 2, 128, 32, "f32", "f32", "channel", "steep", 3),
    ([100, 31], 3, 1, 64, 128, "f32", "f32", "head", "steep", 2),
    ([500], 1, 1, 128, 128, "f32", "f32", "channel", "mixed", 1),
    ([100, 64], 4, 2, 64, 64, "bf16", "bf16", "channel", "mixed", 3),
    ([70, 9], 2, 1, 64, 64, "f32", "f32", "channel", "steep", 2),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[3]}-{c[4]}-{c[5]}-{c[8]}")
def test_delta(kt, case):
    lens, H, Hk, K, V, dtype, odt, gate, rate, slots = case
    d, h = _delta(lens, H, Hk, K, V, dtype, odt, gate, rate, slots, seed=len(lens) + K + V)
    got = _run_delta(kt, d)
    want, pool = _want_delta(h, lens)
    _compare_delta(got, want, dtype, sum(lens))
    if slots:
        live = np.zeros(slots, bool)
        live[h["slot"]] = True
        new = _np(d["dstate"])
        assert np.array_equal(new[~live], h["dstate"][~live])
        _check(d["dstate"], pool, "f32", "dstate")
        cold = h["slot"][h["init"] == 0]
        assert (new[cold] == 0).all()
        assert torch.equal(d["state"], _dev(h["state"]))  # only read


def test_delta_reset_has_no_gradient(kt):
    """A gate of -inf: nothing in front of it reaches what is behind, and its
    own gradient is 0."""
    d, h = _delta([150], 2, 2, 64, 64, seed=3)
    for t in (5, 64, 100, 127):
        d["g"][t] = -np.inf
    h["g"] = d["g"].cpu().numpy()
    got = _run_delta(kt, d)
    want, _ = _want_delta(h, [150])
    _compare_delta(got, want, "f32", 150)
    for t in (5, 64, 100, 127):
        assert (got["dg"][t] == 0).all()
    d["dout"][100:] = 0.0
    got = _run_delta(kt, d)
    for x in ("dq", "dv", "dg", "dbeta"):
        assert (got[x][100:] == 0).all(), x


def test_delta_without_writes(kt):
    """beta of 0 (the inverse of a column by division would fail) and of 1, and
    keys of 0."""
    d, h = _delta([90, 70], 2, 2, 64, 64, seed=4)
    d["beta"][10:40] = 0.0
    d["beta"][40:60] = 1.0
    d["k"][70:75] = 0.0
    h["beta"], h["k"] = d["beta"].cpu().numpy(), d["k"].cpu().numpy()
    want, _ = _want_delta(h, [90, 70])
    _compare_delta(_run_delta(kt, d), want, "f32", 160)


@pytest.mark.parametrize("pools", ["state", "dstate", "neither"])
def test_delta_one_pool(kt, pools):
    lens = [70, 20]
    d, h = _delta(lens, 2, 2, 64, 64, slots=3, seed=5)
    for x in ("state", "dstate"):
        if x != pools:
            d.pop(x), h.pop(x)
    if pools == "neither":  # slot and init are ignored
        h.pop("slot"), h.pop("init")
    got = _run_delta(kt, d)
    want, pool = _want_delta(h, lens)
    _compare_delta(got, want, "f32", 90)
    if pool is not None:
        _check(d["dstate"], pool, "f32", "dstate")


def test_delta_padding_and_rows_behind(kt):
    """Padding entries: zeros, no pool touched; rows of no request stay as they
    were."""
    lens = [66, 10, 40]
    d, h = _delta(lens, 2, 1, 64, 64, slots=4, seed=6, tail=9)
    h["slot"] = np.asarray([2, -1, 4], np.int32)
    d["slot"] = _dev(h["slot"])
    T = sum(lens)
    grads = [torch.full_like(d[x], 7.0) for x in ("q", "k", "v", "g", "beta")]
    n = kt.kda_prefill_backward_workspace_size(T + 9, 3, 2, 1, 64, 64)
    ws = torch.full((n // 4,), float("nan"), device=DEV)  # what is there does not matter
    kt.kda_prefill_backward(d["dout"], d["q"], d["k"], d["v"], d["g"], d["beta"], *grads, ws,
                            d["cu"], d["state"], d["dstate"], d["slot"], d["init"], 0.1)
    got = dict(zip(("dq", "dk", "dv", "dg", "dbeta"), grads))
    want, pool = _want_delta(h, lens)
    _compare_delta(got, want, "f32", T)
    _check(d["dstate"], pool, "f32", "dstate")
    for x in got:
        assert (got[x][66:T] == 0).all() and (got[x][T:] == 7).all(), x


def test_delta_dense_is_packed(kt):
    B, T = 3, 77
    d, _ = _delta([T] * B, 4, 2, 128, 64, slots=3, seed=7)
    d["slot"] = d["init"] = None
    keep = d["dstate"].clone()
    packed = _run_delta(kt, d)
    after, d["dstate"] = d["dstate"], keep
    dense = {x: (t.reshape((B, T) + t.shape[1:]) if x not in ("cu", "state", "dstate") and
                 t is not None else t) for x, t in d.items()}
    dense["cu"] = None
    got = _run_delta(kt, dense)
    for x in got:
        assert torch.equal(got[x].flatten(0, 1), packed[x]), x
    assert torch.equal(dense["dstate"], after)


def test_delta_in_parts(kt):
    """A long sequence in two parts, forwards through one pool and backwards
    through the other, against the whole."""
    T, at = 200, 75
    d, h = _delta([T], 2, 2, 64, 64, slots=1, seed=8)
    d["slot"], d["init"] = None, None
    h["slot"] = h["init"] = None
    want, pool = _want_delta(h, [T])
    state = d["state"].clone()
    parts = []
    for a, b in ((0, at), (at, T)):
        p = {x: d[x][a:b] for x in ("q", "k", "v", "g", "beta", "dout")}
        p.update(cu=_cu([b - a]), state=state.clone(), dstate=d["dstate"])
        kt.prefill(p["q"], p["k"], p["v"], p["g"], p["beta"], p["cu"], state=state, scale=0.1)
        parts.append(p)
    back = [_run_delta(kt, p) for p in reversed(parts)]
    got = {x: torch.cat([back[1][x], back[0][x]]) for x in back[0]}
    _compare_delta(got, want, "f32", T)
    _check(d["dstate"], pool, "f32", "dstate")


def test_delta_same_bits_streams_and_graph(kt):
    lens = [100, 64, 30]
    d, _ = _delta(lens, 4, 2, 128, 128, "bf16", "bf16", slots=3, seed=9)
    keep = d["dstate"].clone()
    first = _run_delta(kt, d)
    left = d["dstate"].clone()

    def same(got):
        for x in got:
            assert torch.equal(got[x], first[x]), x
        assert torch.equal(d["dstate"], left)

    d["dstate"].copy_(keep)
    same(_run_delta(kt, d))
    side = torch.cuda.Stream()
    d["dstate"].copy_(keep)
    side.wait_stream(torch.cuda.current_stream())
    got = _run_delta(kt, d, stream=side)
    side.synchronize()
    same(got)
    # captured with its own workspace, replayed on new inputs with eager work between
    grads = [torch.empty_like(d[x]) for x in ("q", "k", "v", "g", "beta")]
    ws = torch.empty(kt.kda_prefill_backward_workspace_size(194, 3, 4, 2, 128, 128),
                     dtype=torch.uint8, device=DEV)

    def call():
        kt.kda_prefill_backward(d["dout"], d["q"], d["k"], d["v"], d["g"], d["beta"], *grads, ws,
                                d["cu"], d["state"], d["dstate"], d["slot"], d["init"], 0.1)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for i in range(3):
        d["v"].normal_()
        d["dstate"].copy_(keep)
        graph.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in grads] + [d["dstate"].clone()]
        d["dstate"].copy_(keep)
        eager = _run_delta(kt, d)
        for a, b in zip(mine, list(eager.values()) + [d["dstate"]]):
            assert torch.equal(a, b), i


def test_delta_nonfinite_stays_in_its_request(kt):
    lens = [80, 70]
    d, h = _delta(lens, 4, 2, 64, 64, slots=2, seed=10)
    d["slot"] = _dev(np.asarray([0, 1], np.int32))
    clean = _run_delta(kt, {**d, "dstate": d["dstate"].clone()})
    for name, where in (("v", (20, 1, 3)), ("g", (30, 1, 5)), ("k", (64, 0, 2)), ("dout", (79, 1, 9)),
                        ("beta", (5, 1))):
        x = {**d, name: d[name].clone(), "dstate": d["dstate"].clone()}
        x[name][where] = float("nan")
        got = _run_delta(kt, x)
        bad = False
        for y in got:
            assert torch.equal(got[y][80:], clean[y][80:]), (name, y)  # the other request
            if y in ("dv", "dg", "dbeta"):  # heads of the other key head
                assert torch.equal(got[y][:80, 2:], clean[y][:80, 2:]), (name, y)
            bad |= bool(got[y][:80].isnan().any())
        assert bad, name


def test_delta_no_tokens(kt):
    """Requests of no tokens hand their gradient on, or zeros; a call of none."""
    d, h = _delta([0, 5, 0], 2, 2, 64, 32, slots=3, seed=11)
    h["init"] = np.asarray([1, 1, 0], np.int32)
    d["init"] = _dev(h["init"])
    _run_delta(kt, d)
    s = h["slot"]
    new = d["dstate"].cpu().numpy()
    assert np.array_equal(new[s[0]], h["dstate"][s[0]]) and (new[s[2]] == 0).all()
    d, h = _delta([0, 0], 2, 2, 64, 32, slots=2, seed=12)
    d["init"].fill_(0)
    _run_delta(kt, d)
    assert (d["dstate"] == 0).all()
    assert _run_delta(kt, {**d, "cu": torch.zeros(1, dtype=torch.int32, device=DEV), "slot": None,
                           "init": None})["dq"].numel() == 0


def test_delta_many_requests(kt):
    """More requests than a wavefront has lanes, most of them of a few tokens."""
    lens = np.random.default_rng(13).integers(0, 9, 300).tolist()
    d, h = _delta(lens, 1, 1, 64, 32, slots=300, seed=14)
    got = _run_delta(kt, d)
    want, pool = _want_delta(h, lens)
    _compare_delta(got, want, "f32", sum(lens))
    _check(d["dstate"], pool, "f32", "dstate")


@pytest.mark.parametrize("V", [32, 128])
def test_delta_many_walks(kt, V):
    """The walks of 32 columns to a workgroup (many requests and heads) give what
    those of 16 columns (single requests) do."""
    n, H = 70, 16
    lens = [65 if i % 7 else 1 for i in range(n)]
    if V == 32:
        n, lens = 64, lens[:64]
    d, h = _delta(lens, H, H, 64, V, "bf16", "bf16", slots=n, seed=15)
    got = _run_delta(kt, {**d, "dstate": d["dstate"].clone()})
    cu = np.concatenate([[0], np.cumsum(lens)])
    for i in (0, 1, 37, n - 1):
        a, b = int(cu[i]), int(cu[i + 1])
        one = {x: d[x][a:b] for x in ("q", "k", "v", "g", "beta", "dout")}
        one.update(cu=_cu([b - a]), state=d["state"], dstate=d["dstate"].clone(),
                   slot=d["slot"][i:i + 1], init=d["init"][i:i + 1])
        alone = _run_delta(kt, one)
        for x in got:
            assert torch.equal(got[x][a:b], alone[x]), (i, x)


def test_delta_long_workspace(kt):
    """Requests whose part of the workspace lies past 2^33 bytes give what they do
    alone."""
    n, H = 600, 64
    d, _ = _delta([1] * n, H, H, 128, 128, "bf16", "bf16", seed=16)
    assert kt.kda_prefill_backward_workspace_size(n, n, H, H, 128, 128) > 2 ** 33
    got = _run_delta(kt, d)
    for i in (0, 399, 405, n - 1):
        one = {x: d[x][i:i + 1] for x in ("q", "k", "v", "g", "beta", "dout")}
        alone = _run_delta(kt, {**one, "cu": _cu([1])})
        for x in got:
            assert torch.equal(got[x][i:i + 1], alone[x]), (i, x)


# ----------------------------------------------------------------- convolution

def _conv(lens, H, d, W, dtype, slots=0, seed=0, tail=0, coded=False):
    rng = np.random.default_rng(seed)
    T = sum(lens) + tail
    t, h = {}, {}
    for x in ("dq", "dk", "dv"):
        t[x], h[x] = _round(rng.normal(size=(T, H, d)), dtype)
    if coded:
        h["codes"] = rng.integers(-127, 128, (T, 3, H, d)).astype(np.int8)
        h["scale"] = (rng.random((T, 3, H)) / 60).astype(np.float32)
        t["qkv"], t["qkv_scale"] = _dev(h["codes"]), _dev(h["scale"])
        h["qkv"] = h["codes"].astype(np.float64) * h["scale"][..., None]
    else:
        t["qkv"], h["qkv"] = _round(rng.normal(size=(T, 3, H, d)), dtype)
    h["conv_w"] = (rng.random((3, W, H, d)) - 0.5).astype(np.float32)
    t["conv_w"] = _dev(h["conv_w"])
    if slots:
        shape = (slots, 3, H, W - 1, d)
        h["conv_state"] = rng.normal(size=shape).astype(np.float32)
        h["dconv_state"] = rng.normal(size=shape).astype(np.float32)
        h["slot"] = rng.permutation(slots)[:len(lens)].astype(np.int32)
        h["init"] = rng.integers(0, 2, len(lens)).astype(np.int32)
        for x in ("conv_state", "dconv_state", "slot", "init"):
            t[x] = _dev(h[x])
    t["cu"] = _cu(lens)
    return t, h


def _run_conv(kt, t, **kw):
    return kt.conv_prefill_backward(t["dq"], t["dk"], t["dv"], t["qkv"], t["conv_w"], t["cu"],
                                    conv_state=t.get("conv_state"),
                                    dconv_state=t.get("dconv_state"), slot=t.get("slot"),
                                    init=t.get("init"), qkv_scale=t.get("qkv_scale"), **kw)


def _want_conv(h, lens):
    T = sum(lens)
    return bref.conv_grad(h["dq"][:T], h["dk"][:T], h["dv"][:T], h["qkv"][:T], h["conv_w"], lens,
                          h.get("conv_state"), h.get("dconv_state"), h.get("slot"), h.get("init"))


CONVS = [
    ([1], 1, 64, 4, "f32", 0, False),
    ([64], 2, 128, 4, "bf16", 0, False),
    ([1, 2, 0, 3, 5, 4, 70], 3, 64, 4, "f32", 9, False),
    ([3, 1, 0, 129], 5, 128, 3, "f16", 4, True),
    ([33, 2, 1, 1], 2, 64, 2, "bf16", 4, True),
    ([700], 1, 128, 4, "f32", 1, True),
]


@pytest.mark.parametrize("case", CONVS, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-{c[4]}-{c[6]}")
def test_conv(kt, case):
    lens, H, d, W, dtype, slots, coded = case
    t, h = _conv(lens, H, d, W, dtype, slots, seed=len(lens) + d, tail=3, coded=coded)
    T = sum(lens)
    dx, dw = torch.full((T + 3, 3, H, d), 7.0, dtype=_t(dtype), device=DEV), \
        torch.full((3, W, H, d), 7.0, device=DEV)
    n = kt.kda_conv_backward_workspace_size(T + 3, len(lens), H, d, W)
    ws = torch.full((n // 4,), float("nan"), device=DEV)
    kt.kda_conv_backward(t["dq"], t["dk"], t["dv"], t["qkv"], t["conv_w"], dx, dw, ws, t["cu"],
                         t.get("conv_state"), t.get("dconv_state"), t.get("slot"), t.get("init"),
                         qkv_scale=t.get("qkv_scale"))
    want = _want_conv(h, lens)
    _check(dx[:T], want[0], dtype, "dqkv", norm=2e-6, each=2e-5)
    assert (dx[T:] == 7).all()
    _check(dw, want[1], "f32", "dconv_w", norm=2e-6, each=2e-5)
    if slots:
        _check(t["dconv_state"], want[2], "f32", "dconv_state", norm=2e-6, each=2e-5)
        rest = np.setdiff1d(np.arange(slots), h["slot"])
        assert np.array_equal(t["dconv_state"].cpu().numpy()[rest], h["dconv_state"][rest])
        assert torch.equal(t["conv_state"], _dev(h["conv_state"]))


def test_conv_segments(kt):
    """Every length of segments (4 to 64 tokens, and more), requests across their
    ends."""
    for lens, H in (([90, 300], 4), ([700, 2000, 50], 4), ([5000, 4000], 8)):
        t, h = _conv(lens, H, 64, 4, "f32", 3, seed=H)
        got = _run_conv(kt, t)
        want = _want_conv(h, lens)
        for g, w, x in zip(got + (t["dconv_state"],), want, ("dqkv", "dconv_w", "dconv_state")):
            _check(g, w, "f32", x, norm=2e-6, each=2e-5)


def test_conv_padding_dense_and_bits(kt):
    t, h = _conv([20, 9, 30], 2, 64, 4, "f32", 4, seed=3)
    h["slot"] = np.asarray([1, 7, -1], np.int32)
    t["slot"] = _dev(h["slot"])
    keep = t["dconv_state"].clone()
    got = _run_conv(kt, t)
    want = _want_conv(h, [20, 9, 30])
    _check(got[0], want[0], "f32", "dqkv", each=2e-5)
    _check(got[1], want[1], "f32", "dconv_w", each=2e-5)
    _check(t["dconv_state"], want[2], "f32", "dconv_state", each=2e-5)
    assert (got[0][20:] == 0).all()
    t["dconv_state"].copy_(keep)
    again = _run_conv(kt, t)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    # dense
    t, _ = _conv([31] * 3, 2, 128, 3, "bf16", 3, seed=4)
    t["slot"] = t["init"] = None
    keep = t["dconv_state"].clone()
    packed = _run_conv(kt, t)
    after = t["dconv_state"].clone()
    for x in ("dq", "dk", "dv", "qkv"):
        t[x] = t[x].reshape((3, 31) + t[x].shape[1:])
    t["cu"], t["dconv_state"] = None, keep
    dense = _run_conv(kt, t)
    assert torch.equal(dense[0].flatten(0, 1), packed[0]) and torch.equal(dense[1], packed[1])
    assert torch.equal(keep, after)


def test_conv_no_tokens(kt):
    t, h = _conv([0, 0], 2, 64, 4, "f32", 2, seed=5)
    t["init"] = _dev(np.asarray([1, 0], np.int32))
    dx, dw = _run_conv(kt, t)
    assert dx.numel() == 0 and (dw == 0).all()
    new, s = t["dconv_state"].cpu().numpy(), h["slot"]
    assert np.array_equal(new[s[0]], h["dconv_state"][s[0]]) and (new[s[1]] == 0).all()


def test_conv_large_values(kt):
    """Sums of the taps far out on both sides: slopes of 1 and 0, no NaN."""
    t, h = _conv([40], 1, 64, 4, "f32", seed=6)
    t["qkv"] *= 300.0
    h["qkv"] = _np(t["qkv"])
    with np.errstate(over="ignore"):
        want = _want_conv(h, [40])
    got = _run_conv(kt, t)
    _check(got[0], want[0], "f32", "dqkv", norm=2e-5, each=2e-4)
    _check(got[1], want[1], "f32", "dconv_w", norm=2e-5, each=2e-4)


# -------------------------------------------------------------------- the norm

@pytest.mark.parametrize("rows,H,d,dtype", [(1, 1, 64, "f32"), (7, 3, 128, "f32"),
                                            (33, 5, 64, "bf16"), (400, 16, 128, "f16"),
                                            (3000, 16, 128, "bf16")])
@pytest.mark.parametrize("coded", [False, True])
def test_norm(kt, rows, H, d, dtype, coded):
    rng = np.random.default_rng(rows + d)
    shape = (rows, H, d)
    dout, hd = _round(rng.normal(size=shape), dtype)
    o, ho = _round(rng.normal(size=shape) * 0.3, dtype)
    z, hz = _round(rng.normal(size=shape) * 2, dtype)
    w, hw = _round(1 + 0.1 * rng.normal(size=d), "f32")
    kw = {}
    if coded:
        (co, so), (cz, sz) = bref.checkpoint(ho), bref.checkpoint(hz)
        ho, hz = co * so.astype(np.float64)[..., None], cz * sz.astype(np.float64)[..., None]
        o, z, kw = _dev(co), _dev(cz), dict(o_scale=_dev(so), z_scale=_dev(sz))
    do, dz, dw = kt.gated_norm_backward(dout, o, z, w, **kw)
    want = bref.gated_norm_grad(hd, ho, hz, hw)
    _check(do, want[0], dtype, "do", each=2e-5)
    _check(dz, want[1], dtype, "dz", each=2e-5)
    _check(dw, want[2], "f32", "dnorm_w", each=2e-5)
    again = kt.gated_norm_backward(dout, o, z, w, **kw)
    for a, b in zip((do, dz, dw), again):
        assert torch.equal(a, b)


def test_norm_edges(kt):
    """Gates far out (exp overflows), vectors of zeros, no rows."""
    z = torch.tensor([-200.0, -90.0, -30.0, 0.0, 30.0, 200.0], device=DEV)
    z = z[:, None, None].expand(6, 1, 64).contiguous()
    gen = torch.Generator(device=DEV).manual_seed(1)
    o = torch.randn(z.shape, generator=gen, device=DEV)
    o[3] = 0.0
    dout = torch.randn(z.shape, generator=gen, device=DEV)
    w = torch.ones(64, device=DEV)
    got = kt.gated_norm_backward(dout, o, z, w)
    with np.errstate(over="ignore"):
        want = bref.gated_norm_grad(_np(dout), _np(o), _np(z), _np(w))
    for a, b in zip(got, want):
        assert torch.isfinite(a).all()
        for r in range(a.shape[0] if a.dim() == 3 else 0):  # every row by itself: they differ by 1e80
            size = np.abs(b[r]).max()
            assert np.abs(_np(a[r]) - b[r]).max() <= 2e-5 * size + 1e-37
    empty = torch.empty((0, 2, 64), device=DEV)
    do, dz, dw = kt.gated_norm_backward(empty, empty, empty, w)
    assert do.numel() == 0 and (dw == 0).all()


# ----------------------------------------------------------------- checkpoints

@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
def test_checkpoint_exact(kt, dtype, d):
    rng = np.random.default_rng(d)
    x = rng.normal(size=(50, 3, 5, d))
    x[0] = 0.0
    # steps that are powers of two, and values halfway between them
    half = rng.integers(-254, 255, (10, 3, 5, d)) / 2
    half[..., 0] = 127.0
    x[1:11] = half * 2.0 ** rng.integers(-3, 4, (10, 1, 1, 1))
    x[11] *= 2.0 ** -9
    t, h = _round(x, dtype)
    codes, scale = kt.checkpoint(t)
    want, step = bref.checkpoint(h)
    assert np.array_equal(scale.cpu().numpy(), step)
    assert np.array_equal(codes.cpu().numpy(), want)
    back = kt.checkpoint_load(codes, scale, torch.float32)
    values = want.astype(np.float32) * step[..., None]
    assert np.array_equal(back.cpu().numpy(), values)
    for name in ("bf16", "f16"):
        got = kt.checkpoint_load(codes, scale, _t(name))
        assert torch.equal(got, torch.from_numpy(values).to(_t(name)).to(DEV))


def test_checkpoint_halfway_of_uneven_steps(kt):
    """x next to (c + 1/2) steps for steps that are not powers of two, one place of
    FP32 to either side."""
    rng = np.random.default_rng(7)
    top = rng.uniform(0.1, 10, 400).astype(np.float32)
    step = (top.astype(np.float64) / 127).astype(np.float32).astype(np.float64)
    x = ((rng.integers(0, 127, (400, 64)) + 0.5) * step[:, None]).astype(np.float32)
    x = np.where(rng.random(x.shape) < 0.5, x, np.nextafter(x, np.float32(np.inf)))
    x = np.minimum(x, top[:, None]) * rng.choice([-1, 1], x.shape).astype(np.float32)
    x[:, 0] = top
    codes, scale = kt.checkpoint(_dev(x[:, None]))
    want, sc = bref.checkpoint(x[:, None])
    assert np.array_equal(scale.cpu().numpy(), sc) and np.array_equal(codes.cpu().numpy(), want)


def test_checkpoint_edges(kt):
    x = torch.ones((6, 1, 64), device=DEV)
    x[0] *= 2.0 ** -111
    x[1] *= 2.0 ** -110
    x[2] *= 3e38
    x[3, 0, 5] = float("nan")
    x[4, 0, 5] = float("inf")
    x[5, 0, 5] = -float("inf")
    codes, scale = kt.checkpoint(x)
    assert (codes[0] == 0).all() and scale[0] == 0
    assert (codes[1:3] == 127).all()
    back = kt.checkpoint_load(codes, scale, torch.float32)
    assert back[3:].isnan().all() and torch.isfinite(back[:3]).all()
    assert torch.allclose(back[1:3], x[1:3], rtol=1e-6, atol=0)
    c, s = kt.checkpoint(torch.empty((0, 2, 128), device=DEV))
    assert c.numel() == 0 and kt.checkpoint_load(c, s).numel() == 0


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "bf16"), ("f16", "f32")])
def test_norm_checkpoint_is_both(kt, dtype, out):
    rng = np.random.default_rng(3)
    o, _ = _round(rng.normal(size=(77, 3, 128)), dtype)
    z, _ = _round(rng.normal(size=(77, 3, 128)), dtype)
    w = _dev((1 + 0.1 * rng.normal(size=128)).astype(np.float32))
    got = kt.gated_norm_checkpoint(o, z, w, out_dtype=_t(out))
    assert torch.equal(got[0], kt.gated_norm(o, z, w, out_dtype=_t(out)))
    for a, b in zip(got[1:], kt.checkpoint(o) + kt.checkpoint(z)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------- the layer

@pytest.mark.parametrize("coded", [False, True])
def test_layer(kt, coded):
    """A training step of the layer: convolution, delta rule, norm, and back,
    its inputs kept whole or in 8 bits, against the references in a chain."""
    lens, H, d, W = [70, 3, 130], 2, 64, 4
    T, scale = sum(lens), d ** -0.5
    rng = np.random.default_rng(1)
    f32 = lambda *s: rng.normal(size=s).astype(np.float32)  # noqa: E731
    qkv, cw, z, w = f32(T, 3, H, d), f32(3, W, H, d) * 0.5, f32(T, H, d), 1 + 0.1 * f32(d)
    g, beta, dout = -rng.random((T, H, d)).astype(np.float32) * 0.3, \
        rng.random((T, H)).astype(np.float32), f32(T, H, d)
    t = {k: _dev(v) for k, v in dict(qkv=qkv, cw=cw, z=z, w=w, g=g, beta=beta, dout=dout).items()}
    cu = _cu(lens)
    # forwards
    q, k, v = kt.conv_prefill(t["qkv"], t["cw"], cu)
    o = kt.prefill(q, k, v, t["g"], t["beta"], cu, scale=scale)
    if coded:
        x8, xs = kt.checkpoint(t["qkv"])
        out, o8, os, z8, zs = kt.gated_norm_checkpoint(o, t["z"], t["w"])
        do, dz, dw = kt.gated_norm_backward(t["dout"], o8, z8, t["w"], o_scale=os, z_scale=zs)
    else:
        out = kt.gated_norm(o, t["z"], t["w"])
        do, dz, dw = kt.gated_norm_backward(t["dout"], o, t["z"], t["w"])
    # backwards
    dq, dk, dv, dg, dbeta = kt.prefill_backward(do, q, k, v, t["g"], t["beta"], cu, scale=scale)
    dx, dcw = kt.conv_prefill_backward(dq, dk, dv, x8 if coded else t["qkv"], t["cw"], cu,
                                       qkv_scale=xs if coded else None)
    # the references: from the float64 forward pass, and from what was kept of it
    (rq, rk, rv), _ = ref.conv(qkv, cw, lens)
    ro, _, _ = ref.delta_rule(rq, rk, rv, g, beta, lens, scale=scale)
    kept = lambda a: (lambda c, s: c * s.astype(np.float64)[..., None])(*bref.checkpoint(a))  # noqa: E731
    # (codes of o from the kernel's own o: a value near a half may fall the other way)
    no, nz, nx = (kept(_np(o)), kept(z), kept(qkv)) if coded else (ro, z, qkv)
    wo, wz, ww = bref.gated_norm_grad(dout, no, nz, w)
    want, _ = bref.delta_rule_grad(wo, rq, rk, rv, g, beta, lens, scale=scale)
    wx, wcw, _ = bref.conv_grad(want["dq"], want["dk"], want["dv"], nx, cw, lens)
    # (three operators in a row, each to its own tolerance)
    for got, right, name in ((out, ref.gated_norm(ro, z, w), "out"), (do, wo, "do"), (dz, wz, "dz"),
                             (dw, ww, "dnorm_w"), (dg, want["dg"], "dg"),
                             (dbeta, want["dbeta"], "dbeta"), (dx, wx, "dqkv"),
                             (dcw, wcw, "dconv_w")):
        _check(got, right, "f32", name, norm=6e-6, each=2.4e-4)


def test_step_in_a_graph(kt):
    """Checkpoints and all gradients of a step, captured, on pools that the step
    changes: the eager step's bits on every replay, whatever ran between."""
    lens, H, d, W, slots = [70, 3, 0, 130], 2, 128, 4, 6
    T = sum(lens)
    gen = torch.Generator(device=DEV).manual_seed(4)
    new = lambda *s, dt=torch.bfloat16: torch.randn(s, generator=gen, device=DEV).to(dt)  # noqa: E731
    f32 = torch.float32
    qkv, z, dout, do = new(T, 3, H, d), new(T, H, d), new(T, H, d), new(T, H, d)
    o, cw, w = new(T, H, d), new(3, W, H, d, dt=f32) * 0.5, 1 + 0.1 * new(d, dt=f32)
    g, beta = -torch.rand(T, H, d, device=DEV) * 0.3, torch.rand(T, H, device=DEV)
    q, k, v = (torch.nn.functional.normalize(new(T, H, d).float(), dim=-1).bfloat16()
               for _ in range(3))
    state, conv_state = new(slots, H, d, d, dt=f32), new(slots, 3, H, W - 1, d, dt=f32)
    pools0 = (new(slots, H, d, d, dt=f32), new(slots, 3, H, W - 1, d, dt=f32))
    slot = torch.tensor([4, 0, 2, -1], dtype=torch.int32, device=DEV)
    init = torch.tensor([1, 0, 1, 1], dtype=torch.int32, device=DEV)
    cu = _cu(lens)

    def step(dstate, dconv_state):
        x8, xs = kt.checkpoint(qkv)
        out, o8, os, z8, zs = kt.gated_norm_checkpoint(o, z, w)
        dn, dz, dw = kt.gated_norm_backward(dout, o8, z8, w, o_scale=os, z_scale=zs)
        dq, dk, dv, dg, dbeta = kt.prefill_backward(dn, q, k, v, g, beta, cu, state, dstate, slot,
                                                    init)
        dx, dcw = kt.conv_prefill_backward(dq, dk, dv, x8, cw, cu, conv_state, dconv_state, slot,
                                           init, qkv_scale=xs)
        back = kt.checkpoint_load(x8, xs)
        return [x8, xs, out, o8, os, z8, zs, dn, dz, dw, dq, dk, dv, dg, dbeta, dx, dcw, back]

    pools = [p.clone() for p in pools0]
    want = step(*pools) + [p.clone() for p in pools]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*pools)
    for i in range(3):
        for p, p0 in zip(pools, pools0):
            p.copy_(p0)
        for x in got:
            x.zero_()
        graph.replay()
        for n, (a, b) in enumerate(zip(got + pools, want)):
            assert torch.equal(a, b), (i, n)
        step(*[p.clone() for p in pools0])
        torch.cuda.synchronize()
