"""Host-side refusals of the KDA layer's calls on requests of no tokens (CPU
only: every call here returns before any launch)."""
import ctypes

import pytest

P = ctypes.c_void_p
G = 1 << 30  # tensors a GiB apart


@pytest.fixture(scope="module")
def kt():
    import tril_solve_amd
    return tril_solve_amd


@pytest.mark.parametrize("form", ["prefill", "recurrent"])
def test_delta_pools_over_lists(kt, form):
    """A pool that lies over the offsets or the slots is refused also where
    there is no token to read."""
    fn = getattr(kt._lib, f"kda_{form}_packed")
    tail = (P(None), 0, None) if form == "prefill" else (None,)
    for state in (1 * G, 2 * G, 3 * G, 3 * G - 16):
        assert fn(None, None, None, 0, None, None, None, 0, P(G), 2, 0, 4, 2, 128, 128, 128,
                  P(state), P(2 * G), P(3 * G), 2, 1.0, *tail) == kt.KDA_ERR_INVALID_ARG, state


def test_conv_pools_over_lists(kt):
    for pool in (1 * G, 2 * G, 3 * G, 4 * G, 4 * G - 16):
        assert kt._lib.kda_conv_prefill_packed(
            None, 0, P(4 * G), None, None, None, P(G), 2, 0, 4, 128, 4, P(pool), P(2 * G),
            P(3 * G), 2, 1e-6, None) == kt.KDA_ERR_INVALID_ARG, pool
