"""GPU tests of the backward pass at its largest head counts and of values at the
ends of FP32, tolerances as in test_gpu_backward."""
import numpy as np
import pytest

from tests.test_gpu_backward import DEV, _check, _conv, _run_conv, _want_conv, kt  # noqa: F401

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,lens", [(3640, [1, 2]), (4096, [3, 0, 1])])
def test_conv_windows_of_all_heads(kt, H, lens):
    """Gradients of windows of 128 channels, four taps and up to 4,096 heads."""
    t, h = _conv(lens, H, 128, 4, "f32", 4, seed=H)
    got = _run_conv(kt, t)
    want = _want_conv(h, lens)
    for g, w, x in zip(got + (t["dconv_state"],), want, ("dqkv", "dconv_w", "dconv_state")):
        _check(g, w, "f32", x, each=2e-5)
