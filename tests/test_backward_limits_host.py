"""The largest sizes that the backward pass, the checkpoints and the gated norm take
(CPU only: every call here returns before any launch; one that passes the limits ends
at its missing workspace or pointers)."""
import pytest

from tests.test_backward_host import G, P, _conv, kt  # noqa: F401


def _window_blocks(H, d, W):
    return -(-3 * (W - 1) * H * d // 1024)


def _tap_blocks(H, d, W):
    return -(-3 * W * H * d // 1024)


@pytest.mark.parametrize("H", [1, 3639, 3640, 4096])
@pytest.mark.parametrize("d,W", [(64, 2), (128, 4)])
def test_conv_takes_all_heads(kt, H, d, W):
    """One request passes with and without the windows' gradients."""
    for dS in (10 * G, None):
        assert _conv(kt, n=1, T=1, H=H, hd=d, W=W, dS=dS, wsb=0) == kt.KDA_ERR_WORKSPACE
    assert kt.kda_conv_backward_workspace_size(1, 1, H, d, W) > 0


@pytest.mark.parametrize("H,d,W", [(1, 64, 2), (64, 128, 4), (3639, 128, 4), (4096, 128, 4),
                                   (5, 64, 3)])
def test_conv_requests_up_to_the_launch(kt, H, d, W):
    """The sum kernel's workgroups of 256 threads stay below 2^32 threads in all: the
    last number of requests that does so passes, the next one does not."""
    most = (2 ** 24 - 1 - _tap_blocks(H, d, W)) // _window_blocks(H, d, W)
    slots = dict(slot=1 << 50, init=1 << 51, slots=1, S=None, cu=1 << 52, dS=1 << 53)
    assert _conv(kt, n=most, H=H, hd=d, W=W, wsb=0, **slots) == kt.KDA_ERR_WORKSPACE
    assert _conv(kt, n=most + 1, H=H, hd=d, W=W, wsb=0, **slots) == kt.KDA_ERR_UNSUPPORTED
    # without the windows' gradients that launch has the taps alone
    slots["dS"] = None
    assert _conv(kt, n=most + 1, H=H, hd=d, W=W, wsb=0, **slots) == kt.KDA_ERR_WORKSPACE
    assert _conv(kt, n=2 ** 24 - 1, H=H, hd=d, W=W, wsb=0, **slots) == kt.KDA_ERR_WORKSPACE
    assert _conv(kt, n=2 ** 24, H=H, hd=d, W=W, wsb=0, **slots) == kt.KDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("H", [1, 2, 3, 5, 16, 4096])
@pytest.mark.parametrize("d", [64, 128])
def test_vectors_up_to_the_launch(kt, H, d):
    """rows x H < 2^28, and no launch of 2^32 threads: workgroups of 256, d / 8 lanes
    to a vector."""
    L, far = kt._lib, [P(i << 50) for i in range(1, 9)]

    def norm(rows):
        return L.kda_gated_norm_backward(*far[:3], 0, None, None, *far[3:7], rows, H, d, 1e-6,
                                         None, 0, None)

    def save(rows):
        return L.kda_checkpoint(None, 0, *far[:2], rows, H, d, None)

    def load(rows):
        return L.kda_checkpoint_load(None, *far[:2], 0, rows, H, d, None)

    def both(rows):
        return L.kda_gated_norm_checkpoint(None, *far[:1], 0, *far[1:3], 0, *far[3:7], rows, H, d,
                                           1e-6, None)

    def forward(rows):
        return L.kda_gated_norm(None, *far[:1], 0, *far[1:3], 0, rows, H, d, 1e-6, None)

    most = (2 ** 28 - 1) // H
    assert norm(most) == kt.KDA_ERR_WORKSPACE and norm(most + 1) == kt.KDA_ERR_UNSUPPORTED
    if d == 128:
        most = (2 ** 28 - 16) // H
    assert -(-most * H * (d // 8) // 256) * 256 < 2 ** 32
    for call in (save, load, both, forward):
        assert call(most) == kt.KDA_ERR_INVALID_ARG  # past the sizes, at the null pointer
        assert call(most + 1) == kt.KDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("H", [1, 3, 64, 4096])
@pytest.mark.parametrize("K,V", [(64, 32), (128, 256)])
def test_delta_up_to_the_launch(kt, H, K, V):
    """(total_tokens / 64 + num_seqs) x H < 2^23, and num_seqs x H x V / 32 < 2^24 - 64
    (the query's sizes are the call's)."""
    def takes(tokens, n):
        try:
            return kt.kda_prefill_backward_workspace_size(tokens, n, H, H, K, V) > 0
        except kt.KdaError as e:
            assert e.status == kt.KDA_ERR_UNSUPPORTED
            return False

    slots = (2 ** 23 - 1) // H
    assert takes(64 * (slots - 1) + 63, 1) and not takes(64 * slots, 1)
    walks = min((2 ** 24 - 65) // (H * (V // 32)), slots)
    assert takes(63, walks)
    assert not takes(63, 2 ** 21 // H + 1 if V == 256 else slots + 1)
