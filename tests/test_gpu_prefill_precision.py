"""GPU tests of what the chunked delta rule keeps of exact arithmetic, on keys
as a convolution leaves them (a common direction in them) and decays so slow
that the state is large against what a chunk adds, against float64.

Tolerance of the state, 1e-6 of its norm. Every product that it is summed from
is kept to about 2^-24 of each term (three dropped products of parts of at most
2^-26 each), and an FP32 sum rounds by 2^-25 at most, 2^-25 / sqrt(3) = 1.7e-8
in the mean. A chunk takes the state through about ten such roundings (two
factors, six products of the update and, through U, those of k S and of the
inverse): sqrt(10) x 1.7e-8 = 5.5e-8 of its norm; 16 chunks without decay,
roundings of random sign, 4 x 5.5e-8 = 2.2e-7; keys with a common direction make
the inverse of I + L larger than that of unrelated ones by up to 3, which enters
what a chunk adds. Together below 7e-7. FP32 outputs are summed
from the state and U likewise.

Tolerance of 16-bit outputs against the exact ones rounded once: an error e
moves a value over a rounding's border with probability at most 2 |e| / step,
and then by a step of at most eps |x| (bf16: eps = 2^-7, f16: 2^-10). With e of
norm 5e-7 (half of the FP32 outputs' bound; without the decays' extremes) the
difference has a norm of at most sqrt(2 x 5e-7 x eps): 8.9e-5 and 3.2e-5.
"""
import numpy as np
import pytest

from tests import gpu_helpers as gh
from tests import layer_reference as ref

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
STATE = 1e-6


@pytest.fixture(scope="module")
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tril_solve_amd
    return tril_solve_amd


def _dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def _keys(rng, T, H, K, kind):
    x = rng.standard_normal((T, H, K))
    mean = rng.standard_normal((1, H, K))
    if kind == "silu":
        x = x / (1 + np.exp(-x))
    elif kind == "channel means":  # silu of inputs whose channels have means
        x = x + 2 * mean
        x = x / (1 + np.exp(-x))
    elif kind == "common":
        x = 0.44 * x + 0.9 * mean
    return x / np.linalg.norm(x, axis=-1, keepdims=True)


def _inputs(lengths, H, K, V, dtype, keys, rate, seed):
    rng = np.random.default_rng(seed)
    T = sum(lengths)
    c = dict(lengths=lengths, H=H, K=K, V=V)
    for name, x in (("q", _keys(rng, T, H, K, keys)), ("k", _keys(rng, T, H, K, keys)),
                    ("v", rng.standard_normal((T, H, V)))):
        t = torch.from_numpy(x.astype(np.float32)).to(gh.out_torch_dtype(dtype))
        c[name], c[name + "64"] = t.to(DEV), t.double().numpy()
    r = np.exp(rng.uniform(np.log(0.004), np.log(4.0), (H, K))) if rate == "mixed" else rate
    c["g"] = (-r * np.logaddexp(0.0, rng.standard_normal((T, H, K)))).astype(np.float32)
    c["beta"] = (1 / (1 + np.exp(-rng.standard_normal((T, H)) - 2))).astype(np.float32)
    c["state"] = (0.2 * rng.standard_normal((len(lengths), H, K, V))).astype(np.float32)
    return c


def _run(kt, c, out_dtype, cut):
    """(out, state) on the GPU, in segments (cut) or not."""
    out = torch.empty(c["v"].shape, dtype=gh.out_torch_dtype(out_dtype), device=DEV)
    S, ws = _dev(c["state"]), None
    if cut:
        n = kt.kda_prefill_workspace_size(sum(c["lengths"]), len(c["lengths"]), c["H"], c["K"],
                                          c["V"])
        assert n > 0
        ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    cu = _dev(np.concatenate([[0], np.cumsum(c["lengths"])]).astype(np.int32))
    kt.kda_prefill(c["q"], c["k"], c["v"], _dev(c["g"]), _dev(c["beta"]), out, cu, state=S,
                   workspace=ws)
    torch.cuda.synchronize()
    return out, S


def _exact(c):
    return ref.delta_rule(c["q64"], c["k64"], c["v64"], c["g"], c["beta"], c["lengths"],
                          c["state"], None, None, c["K"] ** -0.5)


def _off(got, want):
    return np.linalg.norm(gh.to_numpy_f64(got) - want) / np.linalg.norm(want)


@pytest.mark.parametrize("keys,rate", [("isotropic", 0.004), ("silu", 0.004),
                                       ("channel means", 0.004), ("channel means", 0.05),
                                       ("channel means", "mixed"), ("common", 0.05)])
@pytest.mark.parametrize("K,dtype,out_dtype", [(128, "bf16", "bf16"), (128, "f16", "f16"),
                                               (64, "bf16", "bf16"), (64, "f32", "f32")])
def test_state_of_alike_keys(kt, K, dtype, out_dtype, keys, rate):
    c = _inputs([512], 2, K, 128, dtype, keys, rate, 200 + K)
    _, want, _ = _exact(c)
    for cut in (False, True):
        _, S = _run(kt, c, out_dtype, cut)
        assert _off(S, want) <= STATE, (cut, _off(S, want))


@pytest.mark.parametrize("keys,rate", [("isotropic", 0.004), ("silu", 0.05),
                                       ("channel means", 0.004), ("common", "mixed")])
@pytest.mark.parametrize("K,dtype", [(128, "f32"), (128, "bf16"), (64, "f32"), (64, "f16")])
def test_fp32_outputs_of_alike_keys(kt, K, dtype, keys, rate):
    """An FP32 output is summed from the state and from the chunk's U in the
    same products: state and output to the same share of their norms."""
    c = _inputs([512], 2, K, 128, dtype, keys, rate, 210 + K)
    want_out, want, _ = _exact(c)
    for cut in (False, True):
        out, S = _run(kt, c, "f32", cut)
        assert _off(S, want) <= STATE, (cut, _off(S, want))
        assert _off(out, want_out) <= STATE, (cut, _off(out, want_out))


@pytest.mark.parametrize("keys,rate", [("isotropic", 0.05), ("silu", 0.004),
                                       ("channel means", 0.05), ("common", "mixed")])
@pytest.mark.parametrize("lengths,H", [([512], 2), ([40] * 5, 64)])
@pytest.mark.parametrize("K,dtype", [(128, "bf16"), (128, "f16"), (64, "bf16"), (64, "f16")])
def test_16_bit_outputs_are_rounded_once(kt, K, dtype, lengths, H, keys, rate):
    """One request, and more walks than compute units."""
    c = _inputs(lengths, H, K, 128, dtype, keys, rate, 220 + K)
    want = torch.from_numpy(_exact(c)[0]).to(gh.out_torch_dtype(dtype)).double().numpy()
    out, _ = _run(kt, c, dtype, False)
    eps = torch.finfo(gh.out_torch_dtype(dtype)).eps
    assert _off(out, want) <= np.sqrt(2 * 5e-7 * eps), _off(out, want)
