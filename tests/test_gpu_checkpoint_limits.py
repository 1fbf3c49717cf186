"""GPU tests of 8-bit checkpoints of the largest floats: 127 steps of what is kept
must not overflow, so every finite vector reads back finite, within half a step of
what it was, and so do the gradients that read its codes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
MAX = np.finfo(np.float32).max


@pytest.fixture(scope="module")
def kt():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import tril_solve_amd
    return tril_solve_amd


def _vectors(d):
    """Largest magnitudes from the largest float downwards, of both signs, other
    values below them."""
    rng = np.random.default_rng(d)
    tops = [MAX]
    for _ in range(40):
        tops.append(np.nextafter(tops[-1], np.float32(0)))
    tops = np.asarray(tops + [MAX * np.float32(0.75), np.float32(2.0 ** 127)], np.float32)
    x = (rng.uniform(-1, 1, (len(tops), 1, d)) * tops[:, None, None]).astype(np.float32)
    x[:, 0, 3] = tops * rng.choice([-1, 1], len(tops))
    x[0, 0, 3], x[0, 0, 9], x[1, 0, 3] = MAX, -MAX, -tops[1]
    return x


def _expect(x):
    """Codes and scale: max / 127 rounded to FP32, the float below it where 127 of
    those pass FP32's largest; codes exact."""
    top = np.abs(x).max(-1)
    scale = top / np.float32(127)
    with np.errstate(over="ignore"):
        scale = np.where(np.isinf(scale * np.float32(127)), np.nextafter(scale, np.float32(0)),
                         scale).astype(np.float32)
    return np.rint(x.astype(np.float64) / scale[..., None].astype(np.float64)), scale


@pytest.mark.parametrize("d", [64, 128])
def test_largest_floats(kt, d):
    x = _vectors(d)
    t = torch.from_numpy(x).to(DEV)
    codes, scale = kt.checkpoint(t)
    want, step = _expect(x)
    assert np.array_equal(scale.cpu().numpy(), step)
    assert np.array_equal(codes.cpu().numpy(), want)
    back = kt.checkpoint_load(codes, scale, torch.float32).double().cpu().numpy()
    assert np.isfinite(back).all()
    # half a step, the rounding of the scale (half a place, or one and a half where
    # it is the float below) on 127 of it, and that of the product
    half = step[..., None].astype(np.float64) * (0.5 + 127 * 2.0 ** -22)
    assert (np.abs(back - x) <= half).all()
    out = kt.gated_norm_checkpoint(t, t, torch.ones(d, device=DEV))
    assert torch.equal(out[1], codes) and torch.equal(out[2], scale)
    assert torch.equal(out[3], codes) and torch.equal(out[4], scale)
    # the norm's gradients of them: the mean square passes FP32 and the vector's own
    # gradient is 0, as from the tensor itself, where an infinity would leave NaN
    small, w = torch.ones_like(t), torch.ones(d, device=DEV)
    c1, s1 = kt.checkpoint(small)
    grads = kt.gated_norm_backward(small, codes, c1, w, o_scale=scale, z_scale=s1)
    for g in grads + kt.gated_norm_backward(small, t, small, w):
        assert torch.isfinite(g).all()
