"""Host-side refusals of the backward pass and the checkpoints (CPU only: every
call here returns before any launch), and the float64 gradients against
differences of the forward references.

A central difference of step h in float64 is off by h^2 / 6 times the third
derivative and by the values' rounding over h: with h = 1e-5 and values of about
one, 1e-10 and 1e-11, so 1e-7 relative to the largest gradient leaves room for
third derivatives up to 1e3.
"""
import ctypes

import numpy as np
import pytest

from tests import backward_reference as bref
from tests import layer_reference as ref


@pytest.fixture(scope="module")
def kt():
    import tril_solve_amd
    return tril_solve_amd


P = ctypes.c_void_p
G = 1 << 30  # tensors a GiB apart


def _delta(kt, dense=False, do=1 * G, od=0, q=2 * G, k=3 * G, v=4 * G, d=0, g=5 * G, b=6 * G,
           dq=7 * G, dk=8 * G, dv=9 * G, dg=10 * G, db=11 * G, cu=12 * G, n=2, T=64, H=4, Hk=2,
           K=128, V=128, gate=128, S=13 * G, dS=14 * G, slot=15 * G, init=16 * G, slots=2,
           scale=1.0, ws=17 * G, wsb=G):
    fn = getattr(kt._lib, f"kda_prefill_backward_{'dense' if dense else 'packed'}")
    req = (n, T) if dense else (P(cu), n, T)
    return fn(P(do), od, P(q), P(k), P(v), d, P(g), P(b), P(dq), P(dk), P(dv), P(dg), P(db), *req,
              H, Hk, K, V, gate, P(S), P(dS), P(slot), P(init), slots, scale, P(ws), wsb, None)


def test_delta_refusals(kt):
    E, U = kt.KDA_ERR_INVALID_ARG, kt.KDA_ERR_UNSUPPORTED
    for kw in [dict(d=3), dict(od=-1), dict(H=0), dict(Hk=0), dict(H=4, Hk=3), dict(K=0),
               dict(V=0), dict(gate=2), dict(gate=64), dict(scale=float("nan")),
               dict(scale=float("inf")), dict(n=-1), dict(T=-1), dict(cu=None),
               dict(cu=12 * G + 2), dict(slots=-1), dict(slots=0), dict(slot=None, slots=1),
               dict(S=13 * G + 4), dict(dS=14 * G + 8), dict(b=6 * G + 2), dict(db=None),
               dict(b=None), dict(ws=17 * G + 8), dict(ws=None)]:
        assert _delta(kt, **kw) == E, kw
    names = ["do", "q", "k", "v", "g", "dq", "dk", "dv", "dg"]
    for x in names:
        assert _delta(kt, **{x: None}) == E, x
        assert _delta(kt, **{x: 40 * G + 8}) == E, x
    for x in ["dq", "dk", "dv", "dg", "db", "dS", "ws"]:  # what is written overlaps nothing
        for at in range(1, 18):
            kw = {x: at * G}
            own = dict(dq=7, dk=8, dv=9, dg=10, db=11, dS=14, ws=17)[x]
            if at != own:
                assert _delta(kt, **kw) == E, kw
    for kw in [dict(K=96, gate=96), dict(V=48), dict(V=288), dict(H=8192), dict(T=2 ** 31),
               dict(n=2 ** 31), dict(n=2 ** 21, H=8), dict(T=2 ** 30), dict(slots=2 ** 31),
               dict(n=2 ** 20, H=4, V=256, slots=2 ** 21), dict(T=2 ** 27, H=4)]:
        assert _delta(kt, **kw) == U, kw
    need = kt.kda_prefill_backward_workspace_size(64, 2, 4, 2, 128, 128)
    assert 0 < need < G
    assert _delta(kt, wsb=need - 1) == kt.KDA_ERR_WORKSPACE
    assert _delta(kt, ws=None, wsb=0) == kt.KDA_ERR_WORKSPACE
    assert _delta(kt, dense=True, n=2 ** 20, T=2 ** 20) == U
    assert _delta(kt, dense=True, n=-1) == E
    # nothing to do
    assert _delta(kt, n=0, cu=None) == kt.KDA_OK
    assert _delta(kt, T=0, dS=None, **{x: None for x in names + ["b", "db", "ws"]},
                  wsb=0) == kt.KDA_OK


def test_workspace_queries(kt):
    size = kt.kda_prefill_backward_workspace_size
    for args in [(-1, 1, 4, 4, 128, 128), (1, -1, 4, 4, 128, 128), (1, 1, 0, 1, 128, 128),
                 (1, 1, 4, 3, 128, 128)]:
        with pytest.raises(kt.KdaError) as e:
            size(*args)
        assert e.value.status == kt.KDA_ERR_INVALID_ARG
    for args in [(1, 1, 4, 4, 96, 128), (1, 1, 4, 4, 128, 48), (2 ** 31, 1, 4, 4, 128, 128),
                 (2 ** 30, 1, 64, 64, 128, 128)]:
        with pytest.raises(kt.KdaError) as e:
            size(*args)
        assert e.value.status == kt.KDA_ERR_UNSUPPORTED
    assert size(0, 5, 4, 4, 128, 128) == 0
    # a chunk slot for every 64 tokens and request; shared key heads take FP32 gradients more
    one = size(64, 0, 1, 1, 128, 128)
    assert size(640, 3, 4, 4, 128, 128) == 13 * 4 * one and one <= 400_000
    assert size(640, 3, 4, 2, 128, 128) == 13 * 4 * one + 2 * 640 * 4 * 128 * 4
    size = kt.kda_conv_backward_workspace_size
    for args in [(-1, 1, 4, 128, 4), (1, -1, 4, 128, 4), (1, 1, 0, 128, 4), (1, 1, 4, 128, 0)]:
        with pytest.raises(kt.KdaError) as e:
            size(*args)
        assert e.value.status == kt.KDA_ERR_INVALID_ARG
    for args in [(1, 1, 4, 96, 4), (1, 1, 4, 128, 5), (2 ** 31, 1, 4, 128, 4)]:
        with pytest.raises(kt.KdaError) as e:
            size(*args)
        assert e.value.status == kt.KDA_ERR_UNSUPPORTED
    assert size(0, 2, 4, 128, 4) == 2 * 3 * 4 * 3 * 128 * 4
    # the rows of dconv_w stay few however long the call
    assert size(2 ** 31 - 100, 1, 4, 128, 4) <= 130 * 3 * 4 * 4 * 128 * 4
    assert kt.kda_gated_norm_backward_workspace_size(0, 4, 128) == 0
    assert kt.kda_gated_norm_backward_workspace_size(1 << 20, 64, 128) == 2048 * 128 * 4


def _conv(kt, dense=False, dq=1 * G, dk=2 * G, dv=3 * G, d=0, x=4 * G, sc=None, cw=5 * G,
          dx=6 * G, dcw=7 * G, cu=8 * G, n=2, T=64, H=4, hd=128, W=4, S=9 * G, dS=10 * G,
          slot=11 * G, init=12 * G, slots=2, eps=1e-6, ws=13 * G, wsb=G):
    fn = getattr(kt._lib, f"kda_conv_backward_{'dense' if dense else 'packed'}")
    req = (n, T) if dense else (P(cu), n, T)
    return fn(P(dq), P(dk), P(dv), d, P(x), P(sc), P(cw), P(dx), P(dcw), *req, H, hd, W, P(S),
              P(dS), P(slot), P(init), slots, eps, P(ws), wsb, None)


def test_conv_refusals(kt):
    E, U = kt.KDA_ERR_INVALID_ARG, kt.KDA_ERR_UNSUPPORTED
    for kw in [dict(d=5), dict(H=0), dict(hd=0), dict(W=0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(n=-1), dict(T=-3), dict(cu=None), dict(dq=None),
               dict(dk=None), dict(dv=None), dict(x=None), dict(cw=None), dict(dx=None),
               dict(dcw=None), dict(x=4 * G + 8), dict(x=4 * G + 4, sc=14 * G),
               dict(sc=14 * G + 2), dict(S=9 * G + 4), dict(slots=0), dict(slot=None, slots=1),
               dict(ws=13 * G + 4), dict(dx=1 * G), dict(dx=4 * G), dict(dx=7 * G),
               dict(dcw=5 * G), dict(dS=9 * G), dict(dS=11 * G), dict(ws=6 * G), dict(ws=12 * G)]:
        assert _conv(kt, **kw) == E, kw
    for kw in [dict(hd=96), dict(W=1), dict(W=5), dict(H=5000), dict(T=2 ** 31),
               dict(n=2 ** 24, slots=2 ** 25), dict(n=2 ** 22, slots=2 ** 25)]:
        assert _conv(kt, **kw) == U, kw
    need = kt.kda_conv_backward_workspace_size(64, 2, 4, 128, 4)
    assert _conv(kt, wsb=need - 1) == kt.KDA_ERR_WORKSPACE
    assert _conv(kt, dense=True, n=2 ** 20, T=2 ** 20) == U


def test_norm_and_checkpoint_refusals(kt):
    E, U = kt.KDA_ERR_INVALID_ARG, kt.KDA_ERR_UNSUPPORTED

    def norm(do=1 * G, o=2 * G, z=3 * G, d=0, so=None, sz=None, w=4 * G, d_o=5 * G, dz=6 * G,
             dw=7 * G, rows=4, H=2, hd=128, eps=1e-6, ws=8 * G, wsb=G):
        return kt._lib.kda_gated_norm_backward(P(do), P(o), P(z), d, P(so), P(sz), P(w), P(d_o),
                                               P(dz), P(dw), rows, H, hd, eps, P(ws), wsb, None)

    for kw in [dict(d=4), dict(rows=-1), dict(H=0), dict(hd=0), dict(eps=-1.0), dict(do=None),
               dict(o=None), dict(z=None), dict(w=None), dict(d_o=None), dict(dz=None),
               dict(dw=None), dict(so=9 * G), dict(sz=9 * G), dict(o=2 * G + 8),
               dict(o=2 * G + 4, so=9 * G, sz=10 * G), dict(so=9 * G + 1, sz=10 * G),
               dict(d_o=2 * G), dict(d_o=1 * G), dict(dz=5 * G), dict(dw=4 * G), dict(ws=7 * G),
               dict(ws=8 * G + 4), dict(ws=None)]:
        assert norm(**kw) == E, kw
    for kw in [dict(hd=96), dict(H=5000), dict(rows=2 ** 31), dict(rows=2 ** 28)]:
        assert norm(**kw) == U, kw
    assert norm(wsb=511) == kt.KDA_ERR_WORKSPACE

    def save(x=1 * G, d=0, c=2 * G, s=3 * G, rows=4, H=2, hd=128):
        return kt._lib.kda_checkpoint(P(x), d, P(c), P(s), rows, H, hd, None)

    def load(c=1 * G, s=2 * G, o=3 * G, d=0, rows=4, H=2, hd=128):
        return kt._lib.kda_checkpoint_load(P(c), P(s), P(o), d, rows, H, hd, None)

    def both(o=1 * G, z=2 * G, d=0, w=3 * G, out=4 * G, od=0, oc=5 * G, os=6 * G, zc=7 * G,
             zs=8 * G, rows=4, H=2, hd=128, eps=1e-6):
        return kt._lib.kda_gated_norm_checkpoint(P(o), P(z), d, P(w), P(out), od, P(oc), P(os),
                                                 P(zc), P(zs), rows, H, hd, eps, None)

    for fn, bad in [(save, [dict(d=3), dict(x=None), dict(c=None), dict(s=None), dict(x=G + 8),
                            dict(c=2 * G + 4), dict(s=3 * G + 2), dict(c=G + 64), dict(s=2 * G)]),
                    (load, [dict(d=-1), dict(c=None), dict(s=None), dict(o=None), dict(c=G + 4),
                            dict(o=3 * G + 8), dict(o=1 * G), dict(o=2 * G)]),
                    (both, [dict(d=3), dict(od=3), dict(eps=-1.0), dict(oc=None), dict(zs=None),
                            dict(out=1 * G), dict(oc=2 * G), dict(zc=5 * G), dict(os=8 * G),
                            dict(zc=7 * G + 4), dict(out=4 * G + 8)])]:
        for kw in bad + [dict(rows=-1), dict(H=0), dict(hd=0)]:
            assert fn(**kw) == E, (fn.__name__, kw)
        for kw in [dict(hd=96), dict(H=5000), dict(rows=2 ** 28)]:
            assert fn(**kw) == U, (fn.__name__, kw)
        assert fn(rows=0) == kt.KDA_OK


def test_binding_refuses(kt):
    import torch
    q, g, b = torch.zeros(4, 1, 64), torch.zeros(4, 1, 64), torch.zeros(4, 1)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    ws = torch.empty(16, dtype=torch.uint8)
    with pytest.raises(ValueError):  # host tensors
        kt.kda_prefill_backward(q, q, q, q, g, b, q, q, q, g, b, ws, cu)
    with pytest.raises(ValueError):
        kt.kda_gated_norm_backward(q, q, q, torch.ones(64), q, q, torch.ones(64), ws)
    with pytest.raises(ValueError):
        kt.checkpoint(q)
    with pytest.raises(ValueError):
        kt.checkpoint_load(q.to(torch.int8), b)
    with pytest.raises(ValueError):
        kt.conv_prefill_backward(q, q, q, torch.zeros(4, 3, 64), torch.zeros(3, 4, 1, 64), cu)


def _differences(loss, x, picks, h=1e-5):
    out = []
    for i in picks:
        keep = x[i]
        x[i] = keep + h
        hi = loss()
        x[i] = keep - h
        lo = loss()
        x[i] = keep
        out.append((hi - lo) / (2 * h))
    return np.asarray(out)


def _picks(rng, x, n=12):
    return [tuple(rng.integers(0, s) for s in x.shape) for _ in range(n)]


def test_delta_gradients_against_differences():
    rng = np.random.default_rng(1)
    lens, H, Hk, K, V = [3, 0, 5, 1], 4, 2, 6, 5
    T = sum(lens)
    slot, init = np.asarray([2, 4, 0, 1]), np.asarray([1, 1, 0, 1])
    x = dict(q=rng.normal(size=(T, Hk, K)), k=rng.normal(size=(T, Hk, K)) / np.sqrt(K),
             v=rng.normal(size=(T, H, V)), g=-rng.random((T, H, K)), beta=rng.random((T, H)),
             state=rng.normal(size=(5, H, K, V)))
    do, dS = rng.normal(size=(T, H, V)), rng.normal(size=(5, H, K, V))
    used = np.zeros((5, 1, 1, 1))
    used[slot] = 1.0

    def loss():
        out, pool, _ = ref.delta_rule(x["q"], x["k"], x["v"], x["g"], x["beta"], lens, x["state"],
                                      slot, init, scale=0.3)
        return (out * do).sum() + (pool * dS * used).sum()

    for per_head in (False, True):
        if per_head:
            x["g"] = -rng.random((T, H))
        got, dpool = bref.delta_rule_grad(do, x["q"], x["k"], x["v"], x["g"], x["beta"], lens,
                                          x["state"], dS, slot, init, scale=0.3)
        got["dstate"] = dpool * used
        for name in ("q", "k", "v", "g", "beta", "state"):
            picks = _picks(rng, x[name])
            want = _differences(loss, x[name], picks)
            have = np.asarray([got["d" + name][i] for i in picks])
            assert np.abs(have - want).max() <= 1e-7 * max(1.0, np.abs(want).max()), name


def test_conv_and_norm_gradients_against_differences():
    rng = np.random.default_rng(2)
    lens, H, d, W = [4, 1, 0, 2], 2, 5, 4
    T = sum(lens)
    slot, init = np.asarray([1, 3, 0, 2]), np.asarray([1, 1, 1, 0])
    x = dict(qkv=rng.normal(size=(T, 3, H, d)), conv_w=rng.normal(size=(3, W, H, d)),
             conv_state=rng.normal(size=(4, 3, H, W - 1, d)))
    dn = [rng.normal(size=(T, H, d)) for _ in range(3)]
    dwin = rng.normal(size=(4, 3, H, W - 1, d))

    def loss():
        out, pool = ref.conv(x["qkv"], x["conv_w"], lens, x["conv_state"], slot, init, eps=1e-3)
        return sum((a * b).sum() for a, b in zip(out, dn)) + (pool * dwin).sum()

    dx, dcw, dpool = bref.conv_grad(*dn, x["qkv"], x["conv_w"], lens, x["conv_state"], dwin, slot,
                                    init, eps=1e-3)
    for name, got in (("qkv", dx), ("conv_w", dcw), ("conv_state", dpool)):
        picks = _picks(rng, x[name], 30)
        want = _differences(loss, x[name], picks)
        have = np.asarray([got[i] for i in picks])
        assert np.abs(have - want).max() <= 1e-7 * max(1.0, np.abs(want).max()), name

    y = dict(o=rng.normal(size=(3, 2, 8)), z=rng.normal(size=(3, 2, 8)), w=rng.normal(size=8))
    do = rng.normal(size=(3, 2, 8))
    grads = bref.gated_norm_grad(do, y["o"], y["z"], y["w"], 1e-3)
    for name, got in zip("ozw", grads):
        picks = _picks(rng, y[name])
        want = _differences(lambda: (ref.gated_norm(y["o"], y["z"], y["w"], 1e-3) * do).sum(),
                            y[name], picks)
        have = np.asarray([got[i] for i in picks])
        assert np.abs(have - want).max() <= 1e-7 * max(1.0, np.abs(want).max()), name
