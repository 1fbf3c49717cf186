"""GPU tests of the backward pass: values that are not finite stay where they belong,
and FP32 gradients of long sequences, over whose chunks roundings could add up.

Tolerance of the long sequences. A chunk adds to the state, and to the gradient that
walks the other way, roundings of at most three of 2^-24 of it (products of 64 terms,
their sum, the decay); they are of random sign and, without decays and with keys of
unit length, fade over some 2 K tokens, so at most sqrt(4,224 / 64) = 8.1 times that
is there at once: 1.5e-6 of the state's norm for each of the two, 2.1e-6 for both, on
top of the 2e-6 of one chunk (test_gpu_backward): 4.1e-6 of a gradient's norm."""
import numpy as np
import pytest

from tests import backward_reference as bref
from tests.test_gpu_backward import (DEV, _check, _conv, _delta, _run_conv, _run_delta,  # noqa: F401
                                     _want_delta, kt)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def _is_nan(got, want_nan, clean, what):
    """NaN (or infinities) only where want_nan, the clean call's bits elsewhere."""
    assert torch.equal(got[~want_nan], clean[~want_nan]), what


@pytest.mark.parametrize("W", [2, 4])
@pytest.mark.parametrize("coded", [False, True])
def test_conv_nonfinite_stays(kt, W, coded):
    """Within W - 1 tokens, its request, projection and head."""
    lens, H, d = [150, 1, 90], 3, 64
    t, h = _conv(lens, H, d, W, "f32", 4, seed=W, coded=coded)
    t["init"] = torch.ones_like(t["init"])
    run = lambda x: _run_conv(kt, x) + (x["dconv_state"],)  # noqa: E731
    copy = lambda: {k: v.clone() for k, v in t.items()}  # noqa: E731
    clean = run(copy())
    slot = int(t["slot"][2])
    first, behind = 151, sum(lens)
    # name, index, projection, head, rows of dqkv that it may reach
    cases = [("dq", (20, 1, 5), 0, 1, range(20 - W + 1, 21)),
             ("dv", (149, 2, 7), 2, 2, range(149 - W + 1, 150)),
             ("dk", (150, 0, 0), 1, 0, range(150, 151)),
             ("conv_state", (slot, 1, 2, W - 2, 9), 1, 2, range(first, first + W - 1)),
             ("dconv_state", (slot, 0, 0, 0, 3), 0, 0, range(behind - W + 1, behind)),
             ("qkv_scale" if coded else "qkv", (64, 0, 2) if coded else (64, 0, 2, 1), 0, 2,
              range(64 - W + 1, 64 + W))]
    for bad in (float("nan"), float("inf")):
        for name, where, p, head, rows in cases:
            x = copy()
            x[name][where] = bad
            got = run(x)
            dx, dw, pool = (torch.zeros(g.shape, dtype=torch.bool, device=DEV) for g in got)
            dx[rows.start:rows.stop, p, head] = True
            dw[p, :, head] = True
            n = 0 if rows.stop <= 150 else 1 if rows.stop <= 151 else 2
            pool[int(t["slot"][n]), p, head] = n > 0 and name != "dconv_state"
            for a, b, m in zip(got, clean, (dx, dw, pool)):
                _is_nan(a, m, b, (name, bad))
            assert not all(torch.isfinite(g).all() for g in got), (name, bad)


def test_norm_nonfinite_stays(kt):
    """Its own vector, and the weights' gradient."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    new = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    ins = dict(dout=new(300, 3, 128), o=new(300, 3, 128), z=new(300, 3, 128), w=new(128))
    clean = kt.gated_norm_backward(*ins.values())
    for name in ("dout", "o", "z"):
        x = {k: v.clone() for k, v in ins.items()}
        x[name][77, 1, 5] = float("nan")
        got = kt.gated_norm_backward(*x.values())
        mask = torch.zeros((300, 3, 128), dtype=torch.bool, device=DEV)
        mask[77, 1] = True
        for a, b in zip(got[:2], clean):
            _is_nan(a, mask, b, name)
            assert a[77, 1].isnan().any(), name
        assert got[2].isnan().any() and got[2].isnan().sum() <= 128, name


LONG = [  # K, V, H, Hk, gate, decays
    (64, 64, 2, 1, "head", "none"),
    (128, 128, 1, 1, "channel", "none"),
    (128, 64, 2, 2, "channel", "mixed"),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(map(str, c)))
def test_delta_long_f32(kt, case):
    K, V, H, Hk, gate, rate = case
    T = 4200
    d, h = _delta([T], H, Hk, K, V, "f32", "f32", gate, "mixed", 1, seed=K + V)
    if rate == "none":
        d["g"].zero_()
        h["g"] = np.zeros_like(h["g"])
    d["init"].fill_(1)
    h["init"][:] = 1
    got = _run_delta(kt, d)
    want, pool = _want_delta(h, [T])
    for x in got:
        _check(got[x], want[x], "f32", x, norm=4.1e-6, each=40 * 4.1e-6)
    _check(d["dstate"], pool, "f32", "dstate", norm=4.1e-6, each=40 * 4.1e-6)
