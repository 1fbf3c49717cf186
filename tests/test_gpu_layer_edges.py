"""GPU tests of the KDA layer's calls at the edges of what they allow."""
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


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _behind(first, rest):
    """An int32 vector that lies right behind the entry `first`."""
    return _dev(np.array([first] + list(rest), np.int32))[1:]


@pytest.mark.parametrize("B", [1, 3, 70])
def test_dense_conv_of_no_tokens(kt, B):
    """[B, 0, ...]: windows kept where they continue, zeroed where they start
    anew, and no entry before the first one looked at: it names a live slot with
    init 0 here, whose window would be zeroed."""
    rng = np.random.default_rng(B)
    H, d, W = 2, 64, 4
    pool = rng.standard_normal((B + 2, 3, H, W - 1, d)).astype(np.float32)
    order = rng.permutation(B + 2).astype(np.int32)
    slot, init = _behind(order[B], order[:B]), _behind(0, [1] + [0] * (B - 1))
    win = _dev(pool)
    x = torch.empty((B, 0, 3, H, d), device=DEV)
    q, k, v = kt.conv_prefill(x, torch.ones((3, W, H, d), device=DEV), conv_state=win, slot=slot,
                              init=init)
    assert q.shape == k.shape == v.shape == (B, 0, H, d)
    pool[order[1:B]] = 0.0
    assert np.array_equal(win.cpu().numpy(), pool)
    kt.conv_prefill(x, torch.ones((3, W, H, d), device=DEV), conv_state=win)  # request n, slot n
    assert np.array_equal(win.cpu().numpy(), pool)


@pytest.mark.parametrize("form", ["prefill", "recurrent"])
def test_dense_delta_rule_of_no_tokens(kt, form):
    B, H, K, V = 3, 2, 64, 64
    rng = np.random.default_rng(7)
    pool = rng.standard_normal((B + 2, H, K, V)).astype(np.float32)
    order = rng.permutation(B + 2).astype(np.int32)
    S = _dev(pool)
    qk, x = torch.empty((B, 0, H, K), device=DEV), torch.empty((B, 0, H, V), device=DEV)
    fn = kt.prefill if form == "prefill" else kt.recurrent
    out = fn(qk, qk, x, torch.empty((B, 0, H, K), device=DEV), torch.empty((B, 0, H), device=DEV),
             state=S, slot=_behind(order[B], order[:B]), init=_behind(0, [1, 0, 0]))
    assert out.shape == (B, 0, H, V)
    pool[order[1:B]] = 0.0
    assert np.array_equal(S.cpu().numpy(), pool)


# A value that is not finite reaches the outputs of its own token and of later
# ones of its request and head (from v: of its column), and nothing else. The
# outputs before it are the exact ones to 4e-6 of the largest products' size: 128
# terms and a few roundings a token in FP32, 2^-24 (sqrt(128) + 4 x 40).

_FORMS = {"recurrent": dict(requests=1, H=2), "narrow": dict(requests=1, H=2),
          "roles": dict(requests=4, H=48), "whole": dict(requests=6, H=48),
          "cut": dict(requests=1, H=2, cut=True)}


def _problem(requests, H, K, V, dtype, T, seed):
    rng = np.random.default_rng(seed)
    n = requests * T
    unit = lambda: (lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True))(  # noqa: E731
        rng.standard_normal((n, H, K)))
    t = gh.out_torch_dtype(dtype)
    low = lambda x: torch.from_numpy(x).to(t).double().numpy()  # noqa: E731
    return dict(q=low(unit()), k=low(unit()), v=low(rng.standard_normal((n, H, V))),
                g=(-0.1 * rng.random((n, H, K))).astype(np.float32).astype(np.float64),
                beta=rng.uniform(0.2, 0.9, (n, H)).astype(np.float32).astype(np.float64),
                state=0.2 * rng.standard_normal((requests, H, K, V)))


def _delta(kt, form, c, requests, T, dtype, cut=False, **_):
    t = gh.out_torch_dtype(dtype)
    q, k, v = (torch.from_numpy(c[x]).to(t).to(DEV) for x in "qkv")
    g, beta, S = (_dev(c[x].astype(np.float32)) for x in ("g", "beta", "state"))
    cu = _dev((T * np.arange(requests + 1)).astype(np.int32))
    out = torch.empty_like(v)
    if form == "recurrent":
        kt.kda_recurrent(q, k, v, g, beta, out, cu, state=S)
    else:
        n = kt.kda_prefill_workspace_size(v.shape[0], requests, v.shape[1], k.shape[2],
                                          v.shape[2]) if cut else 0
        assert bool(n) == cut
        ws = torch.empty(n, dtype=torch.uint8, device=DEV) if cut else None
        kt.kda_prefill(q, k, v, g, beta, out, cu, state=S, workspace=ws)
    return gh.to_numpy_f64(out), S.cpu().numpy()


@pytest.mark.parametrize("what,value", [("v", np.nan), ("v", np.inf), ("v", -np.inf),
                                        ("k", np.nan), ("k", np.inf), ("k", -np.inf),
                                        ("beta", np.nan), ("beta", np.inf), ("beta", -np.inf),
                                        ("g", np.nan), ("g", np.inf), ("q", np.nan)])
@pytest.mark.parametrize("K,dtype", [(128, "bf16"), (64, "f32")])
@pytest.mark.parametrize("form", list(_FORMS))
def test_values_that_are_not_finite(kt, form, K, dtype, what, value):
    f = _FORMS[form]
    T, V, h = 530 if f.get("cut") else 70, 128, 1
    r = f["requests"] - 1  # the last request
    for at in ((40, 500, 517) if f.get("cut") else (0, 5, 21, 40)):
        print(f"\n[not finite] {form} {what} {value} token {at}", flush=True)
        c = _problem(f["requests"], f["H"], K, V, dtype, T, 50 + K)
        clean, S_clean = _delta(kt, form, c, T=T, dtype=dtype, **f)
        row = r * T + at
        if what == "beta":
            c[what][row, h] = value
        else:
            c[what][row, h, 3] = value
        out, S = _delta(kt, form, c, T=T, dtype=dtype, **f)
        hit = np.zeros(out.shape, bool)  # what has to be not finite
        last = row + 1 if what == "q" else (r + 1) * T
        hit[row:last, h, 3 if what == "v" else slice(None)] = True
        assert not np.isfinite(out[hit]).any()
        hit_S = np.zeros(S.shape, bool)
        if what != "q":
            hit_S[r, h, :, 3 if what == "v" else slice(None)] = True
        assert not np.isfinite(S[hit_S]).any()
        # all else: the same bits, but for the request and head whose decays,
        # keys or write strengths changed, to the exact outputs
        own = np.zeros(out.shape, bool)
        own[r * T:(r + 1) * T, h] = what in ("k", "beta", "g")
        assert np.array_equal(out[~hit & ~own], clean[~hit & ~own])
        assert np.array_equal(S[~hit_S], S_clean[~hit_S])
        if what in ("k", "beta", "g") and at > 0:
            s = slice(r * T, row)
            part = lambda x: c[x][s, h:h + 1]  # noqa: E731
            want, _, N = ref.delta_rule(part("q"), part("k"), part("v"), part("g"), part("beta"),
                                        [at], c["state"][r:r + 1, h:h + 1], None, None, K ** -0.5)
            half = torch.finfo(gh.out_torch_dtype(dtype)).eps / 2
            assert (np.abs(out[s, h:h + 1] - want) <= 4e-6 * N + half * np.abs(want)).all()


def test_pools_without_slots_are_refused(kt):
    """They have no address in torch, and would pass for no pool at all: the
    requests' new state would be lost. No request needs none."""
    q, x = torch.ones((4, 2, 64), device=DEV), torch.ones((4, 2), device=DEV)
    cu = _dev(np.array([0, 4], np.int32))
    none = _dev(np.array([0], np.int32))
    S, win = torch.empty((0, 2, 64, 64), device=DEV), torch.empty((0, 3, 2, 3, 64), device=DEV)
    for fn in (kt.prefill, kt.recurrent):
        with pytest.raises(ValueError, match="slots"):
            fn(q, q, q, q, x, cu, state=S)
        assert fn(q[:0], q[:0], q[:0], q[:0], x[:0], none, state=S).shape == (0, 2, 64)
    qkv, cw = torch.ones((4, 3, 2, 64), device=DEV), torch.ones((3, 4, 2, 64), device=DEV)
    with pytest.raises(ValueError, match="slots"):
        kt.conv_prefill(qkv, cw, cu, conv_state=win)
    assert kt.conv_prefill(qkv[:0], cw, none, conv_state=win)[0].shape == (0, 2, 64)


@pytest.mark.parametrize("steep", [False, True])
@pytest.mark.parametrize("form", list(_FORMS))
def test_several_values_that_are_not_finite(kt, form, steep):
    """Two values in one chunk, a key between and after them, decays that reset
    channels beside: each column is left exact up to its first one."""
    f = _FORMS[form]
    T, K, V, h, dtype = 530 if f.get("cut") else 70, 64, 96, 0, "f32"
    c = _problem(f["requests"], f["H"], K, V, dtype, T, 9)
    if steep:
        c["g"] *= 100.0
        c["g"][::7, :, ::5] = -np.inf
    b = T - 40 if f.get("cut") else 32  # first token of a chunk (cut: somewhere in the last)
    c["v"][b + 9, h, 7], c["v"][b + 20, h, 3], c["v"][b + 1, h, 95] = np.inf, np.nan, -np.inf
    c["k"][b + 14, h, 0], c["k"][b + 25, h, 5] = np.nan, np.inf
    out, S = _delta(kt, form, c, T=T, dtype=dtype, **f)
    stop = np.full(V, b + 14)
    stop[7], stop[95] = b + 9, b + 1
    part = lambda x: c[x][:b + 14, h:h + 1]  # noqa: E731
    clean = np.where(np.isfinite(part("v")), part("v"), 0.0)
    want, _, N = ref.delta_rule(part("q"), part("k"), clean, part("g"), part("beta"), [b + 14],
                                c["state"][:1, h:h + 1], None, None, K ** -0.5)
    for col in range(V):
        n = stop[col]
        assert not np.isfinite(out[n:T, h, col]).any()
        assert (np.abs(out[:n, h, col] - want[:n, 0, col]) <= 4e-6 * N).all()
    assert not np.isfinite(S[0, h]).any() and np.isfinite(S[0, 1:]).all()
