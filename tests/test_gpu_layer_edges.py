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
