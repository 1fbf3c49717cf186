"""Host-side refusals of the KDA layer's calls (CPU only: every call here
returns before any launch), and the references of the GPU tests against each
other."""
import ctypes

import numpy as np
import pytest

from tests import layer_reference as ref


@pytest.fixture(scope="module")
def kt():
    import tril_solve_amd
    return tril_solve_amd


P = ctypes.c_void_p
G = 1 << 30  # tensors a GiB apart


def _delta(kt, form="prefill", dense=False, q=1 * G, k=2 * G, v=3 * G, d=0, g=4 * G, b=5 * G,
           o=6 * G, od=0, cu=7 * G, n=2, T=64, H=4, Hk=2, K=128, V=128, gate=128, S=8 * G,
           slot=9 * G, init=10 * G, slots=2, scale=1.0, ws=None, wsb=0):
    fn = getattr(kt._lib, f"kda_{form}_{'dense' if dense else 'packed'}")
    tail = (P(ws), wsb, None) if form == "prefill" else (None,)
    req = (n, T) if dense else (P(cu), n, T)
    return fn(P(q), P(k), P(v), d, P(g), P(b), P(o), od, *req, H, Hk, K, V, gate, P(S), P(slot),
              P(init), slots, scale, *tail)


@pytest.mark.parametrize("form", ["prefill", "recurrent"])
def test_delta_refusals(kt, form):
    E, U = kt.KDA_ERR_INVALID_ARG, kt.KDA_ERR_UNSUPPORTED
    bad = [dict(d=3), dict(od=-1), dict(H=0), dict(Hk=0), dict(H=4, Hk=3), dict(K=0), dict(V=0),
           dict(gate=2), dict(gate=64), dict(scale=float("nan")), dict(scale=float("inf")),
           dict(n=-1), dict(T=-1), dict(cu=None), dict(cu=7 * G + 2), dict(q=None), dict(k=None),
           dict(v=None), dict(g=None), dict(b=None), dict(o=None), dict(q=G + 8), dict(o=6 * G + 4),
           dict(g=4 * G + 4), dict(S=8 * G + 4), dict(slot=9 * G + 1), dict(slots=-1),
           dict(slots=0), dict(slot=None, slots=1), dict(o=1 * G), dict(o=3 * G + 64),
           dict(o=8 * G), dict(S=4 * G), dict(o=9 * G)]
    if form == "prefill":
        bad.append(dict(ws=11 * G + 8, wsb=64))
        bad.append(dict(wsb=64))
        # prompts that are cut: the workspace is used, and may not overlap
        n = kt.kda_prefill_workspace_size(2048, 2, 4, 128, 128)
        assert 0 < n < G
        for at in (1, 2, 3, 4, 5, 6, 8):
            bad.append(dict(T=2048, ws=at * G, wsb=n))
        bad += [dict(T=2048, ws=7 * G + 16 - n, wsb=n), dict(T=2048, ws=9 * G, wsb=n),
                dict(T=2048, ws=10 * G, wsb=n)]
    for kw in bad:
        assert _delta(kt, form, **kw) == E, kw
    for kw in [dict(K=96, gate=96), dict(K=256, gate=256), dict(V=48), dict(V=288), dict(H=8192),
               dict(T=2 ** 31), dict(n=2 ** 31), dict(n=2 ** 21), dict(slots=2 ** 31)]:
        assert _delta(kt, form, **kw) == U, kw
    assert _delta(kt, form, dense=True, n=2 ** 20, T=2 ** 20) == U
    assert _delta(kt, form, dense=True, n=-1) == E
    # nothing to do
    assert _delta(kt, form, n=0, cu=None) == kt.KDA_OK
    assert _delta(kt, form, T=0, S=None, q=None, k=None, v=None, g=None, b=None, o=None) == kt.KDA_OK


def test_prefill_workspace_query(kt):
    for args in [(-1, 1, 4, 128, 128), (1, -1, 4, 128, 128), (1, 1, 0, 128, 128)]:
        with pytest.raises(kt.KdaError) as e:
            kt.kda_prefill_workspace_size(*args)
        assert e.value.status == kt.KDA_ERR_INVALID_ARG
    for args in [(1, 1, 4, 96, 128), (1, 1, 4, 128, 48), (2 ** 31, 1, 4, 128, 128)]:
        with pytest.raises(kt.KdaError) as e:
            kt.kda_prefill_workspace_size(*args)
        assert e.value.status == kt.KDA_ERR_UNSUPPORTED
    size = kt.kda_prefill_workspace_size
    assert size(0, 0, 4, 128, 128) == 0
    # no cut: short prompts, many heads or requests
    assert size(511, 1, 4, 128, 128) == 0 and size(1023, 2, 4, 128, 128) == 0
    assert size(1279, 1, 64, 128, 128) == 0 and size(1280, 1, 64, 128, 128) > 0
    assert size(65536, 1, 65, 128, 128) == 0 and size(65536, 1, 33, 128, 256) == 0
    assert size(1 << 20, 65, 1, 128, 128) == 0 and size(0, 1, 1, 64, 32) == 0
    # segments of whole chunks: [segments, H, K, V + K] and [requests, H, K, V]
    for T, n, H, K, V in [(512, 1, 1, 128, 128), (16384, 1, 32, 128, 128), (5000, 7, 3, 64, 96),
                          (2 ** 31 - 100, 1, 1, 128, 256), (2 ** 31 - 100, 64, 1, 64, 32)]:
        words = size(T, n, H, K, V) // 4 - n * H * K * V
        segments = words // (H * K * (V + K))
        assert words == segments * H * K * (V + K) and 2 <= segments - n <= 256 * n


def _conv(kt, dense=False, x=1 * G, d=0, cw=2 * G, q=3 * G, k=4 * G, v=5 * G, cu=6 * G, n=2, T=64,
          H=4, hd=128, W=4, S=7 * G, slot=8 * G, init=9 * G, slots=2, eps=1e-6):
    fn = kt._lib.kda_conv_prefill_dense if dense else kt._lib.kda_conv_prefill_packed
    req = (n, T) if dense else (P(cu), n, T)
    return fn(P(x), d, P(cw), P(q), P(k), P(v), *req, H, hd, W, P(S), P(slot), P(init), slots, eps,
              None)


def test_conv_refusals(kt):
    E, U = kt.KDA_ERR_INVALID_ARG, kt.KDA_ERR_UNSUPPORTED
    for kw in [dict(d=5), dict(H=0), dict(hd=0), dict(W=0), dict(eps=-1.0),
               dict(eps=float("nan")), dict(n=-1), dict(T=-3), dict(cu=None), dict(x=None),
               dict(cw=None), dict(q=None), dict(k=None), dict(v=None), dict(x=G + 2),
               dict(cw=2 * G + 4), dict(S=7 * G + 4), dict(slots=0), dict(slot=None, slots=1),
               dict(q=1 * G), dict(q=4 * G), dict(v=7 * G), dict(S=2 * G)]:
        assert _conv(kt, **kw) == E, kw
    for kw in [dict(hd=96), dict(hd=256), dict(W=1), dict(W=5), dict(H=5000), dict(T=2 ** 31)]:
        assert _conv(kt, **kw) == U, kw
    assert _conv(kt, dense=True, n=2 ** 20, T=2 ** 20) == U
    assert _conv(kt, n=0) == kt.KDA_OK
    assert _conv(kt, T=0, S=None) == kt.KDA_OK


def test_map_and_norm_refusals(kt):
    E, U = kt.KDA_ERR_INVALID_ARG, kt.KDA_ERR_UNSUPPORTED

    def chunk_map(lens=1 * G, n=2, T=64, C=64, cu=2 * G, m=3 * G, rows=3, cnt=4 * G):
        return kt._lib.kda_chunk_map(P(lens), n, T, C, P(cu), P(m), rows, P(cnt), None)

    for kw in [dict(n=-1), dict(T=-1), dict(rows=-1), dict(C=48), dict(m=None), dict(rows=0),
               dict(cu=None), dict(lens=None), dict(lens=G + 2), dict(m=3 * G + 4),
               dict(cu=1 * G), dict(m=2 * G), dict(cnt=3 * G)]:
        assert chunk_map(**kw) == E, kw
    for kw in [dict(n=2 ** 31), dict(T=2 ** 31), dict(rows=2 ** 31)]:
        assert chunk_map(**kw) == U, kw

    def norm(o=1 * G, z=2 * G, d=0, w=3 * G, out=4 * G, od=0, rows=4, H=2, hd=128, eps=1e-6):
        return kt._lib.kda_gated_norm(P(o), P(z), d, P(w), P(out), od, rows, H, hd, eps, None)

    for kw in [dict(d=4), dict(od=4), dict(rows=-1), dict(H=0), dict(hd=0), dict(eps=-1.0),
               dict(o=None), dict(z=None), dict(w=None), dict(out=None), dict(o=G + 8),
               dict(out=4 * G + 2), dict(w=3 * G + 2), dict(out=2 * G), dict(out=G + 64),
               dict(out=1 * G, od=1)]:
        assert norm(**kw) == E, kw
    for kw in [dict(hd=96), dict(H=5000), dict(rows=2 ** 31), dict(rows=2 ** 28)]:
        assert norm(**kw) == U, kw
    assert norm(rows=0) == kt.KDA_OK


def test_binding_refuses_host_tensors(kt):
    import torch
    q = torch.zeros(4, 1, 64)
    with pytest.raises(ValueError):
        kt.kda_prefill(q, q, q, torch.zeros(4, 1, 64), torch.zeros(4, 1), torch.zeros(4, 1, 64),
                       torch.tensor([0, 4], dtype=torch.int32))
    with pytest.raises(ValueError):
        kt.kda_gated_norm(q, q, torch.ones(64), torch.empty_like(q))
    with pytest.raises(ValueError):
        kt.chunk_map(torch.tensor([4], dtype=torch.int32), 4, 48)


def test_reference_against_the_decode_oracle():
    """The tests' token-by-token reference against the decode step's oracle
    (another implementation) over five tokens."""
    import oracle
    import synth
    H, d, W = 2, 128, 3
    base = synth.decode_inputs(1, H, W=W, seed=3)
    S, win = base["state"].astype(np.float64), base["conv_state"].astype(np.float64)
    toks = [synth.decode_inputs(1, H, W=W, seed=10 + t) for t in range(5)]
    cat = lambda n: np.concatenate([t[n] for t in toks])  # noqa: E731
    (q, k, v), want_win = ref.conv(cat("qkv"), base["conv_w"], [5], win, base["slot"])
    o, want_S, _ = ref.delta_rule(q, k, v, cat("g"), cat("beta"), [5], S, base["slot"],
                                  scale=d ** -0.5)
    y = ref.gated_norm(o, cat("z"), base["norm_w"])
    for t in range(5):
        r, S, win = oracle.kda_decode(toks[t]["qkv"], toks[t]["g"], toks[t]["beta"],
                                      toks[t]["z"], base["norm_w"], base["conv_w"], base["slot"],
                                      S, win, "f32", 1e-6, 1e-6)
        assert np.abs(r[0] - y[t]).max() < 1e-12
    assert np.abs(S - want_S).max() < 1e-12 and np.abs(win - want_win).max() < 1e-12
