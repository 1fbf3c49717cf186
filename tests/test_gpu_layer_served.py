"""GPU tests of the KDA layer's calls as a serving loop makes them: prompts, then
several drafted tokens per request on the pools left behind, then decode steps;
and marshalled calls issued again and again."""
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


def test_drafted_tokens_between_prompts_and_decode_steps(kt):
    """Two rounds of 1 to 5 drafted tokens through the convolution, the recurrent
    form and the norm, on the windows and states of the prompts; the decode step
    goes on from them. Against the operators in float64 over each request's tokens
    in one piece, FP32 throughout: as far as in the layer's other tests (2e-4 of a
    norm's outputs, 2e-5 of their norm)."""
    H, d, W, prompts = 3, 128, 4, [37, 5, 64]
    N, rng = len(prompts), np.random.default_rng(5)
    rounds = [prompts, [3, 1, 5], [2, 4, 1], [1, 1, 1]]
    total = [sum(r[n] for r in rounds) for n in range(N)]
    x = [rng.standard_normal((t, 3, H, d)).astype(np.float32) for t in total]
    z = [rng.standard_normal((t, H, d)).astype(np.float32) for t in total]
    g = [-np.logaddexp(0.0, -(rng.standard_normal((t, H, d)) + 3.0)).astype(np.float32)
         for t in total]
    beta = [(1 / (1 + np.exp(-rng.standard_normal((t, H))))).astype(np.float32) for t in total]
    cw = rng.uniform(-0.5, 0.5, (3, W, H, d)).astype(np.float32)
    nw = (1 + 0.1 * rng.standard_normal(d)).astype(np.float32)
    slots = N + 2
    S = _dev(rng.standard_normal((slots, H, d, d)).astype(np.float32))
    win = _dev(rng.standard_normal((slots, 3, H, W - 1, d)).astype(np.float32))
    slot = rng.permutation(slots)[:N].astype(np.int32)
    pool = dict(slot=_dev(slot))
    got = [[] for _ in range(N)]
    at = [0] * N
    for i, lens in enumerate(rounds):
        part = lambda a: np.concatenate([a[n][at[n]:at[n] + lens[n]]  # noqa: E731,B023
                                         for n in range(N)])
        if i == 3:
            y = torch.empty((N, H, d), device=DEV)
            kt.kda_decode_step(_dev(part(x)), _dev(part(z)), _dev(part(g)), _dev(part(beta)),
                               _dev(nw), _dev(cw), pool["slot"], S, win, y)
        else:
            cu, _, _ = kt.chunk_map(_dev(np.asarray(lens, np.int32)), sum(lens))
            init = torch.zeros(N, dtype=torch.int32, device=DEV) if i == 0 else None
            q, k, v = kt.conv_prefill(_dev(part(x)), _dev(cw), cu, conv_state=win, init=init,
                                      **pool)
            fn = kt.prefill if i == 0 else kt.recurrent
            o = fn(q, k, v, _dev(part(g)), _dev(part(beta)), cu, state=S, init=init, **pool)
            y = kt.gated_norm(o, _dev(part(z)), _dev(nw))
        y, b = gh.to_numpy_f64(y), 0
        for n in range(N):
            got[n].append(y[b:b + lens[n]])
            b += lens[n]
            at[n] += lens[n]
    (q, k, v), _ = ref.conv(np.concatenate(x), cw, total)
    want, states, _ = ref.delta_rule(q, k, v, np.concatenate(g), np.concatenate(beta), total,
                                     np.zeros((N, H, d, d)), scale=d ** -0.5)
    want = ref.gated_norm(want, np.concatenate(z), nw)
    have = np.concatenate([np.concatenate(p) for p in got])
    assert np.abs(have - want).max() <= 2e-4
    assert np.linalg.norm(have - want) <= 2e-5 * np.linalg.norm(want)
    left = S.cpu().numpy().astype(np.float64)[slot]
    assert np.linalg.norm(left - states) <= 2e-5 * np.linalg.norm(states)


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("form", ["prefill", "recurrent"])
def test_prepared_calls(kt, form, dense):
    """A marshalled call, issued three times on fresh states, also on a stream of
    its own, gives the bits of the call itself."""
    rng = np.random.default_rng(6)
    B, T, H, K, V = 2, 600, 2, 64, 96
    lead = (B, T) if dense else (B * T,)
    q, k = (torch.nn.functional.normalize(_dev(rng.standard_normal(lead + (H, K))), dim=-1).float()
            for _ in range(2))
    v = _dev(rng.standard_normal(lead + (H, V)).astype(np.float32))
    g, beta = -0.1 * torch.rand(lead + (H, K), device=DEV), torch.rand(lead + (H,), device=DEV)
    cu = None if dense else _dev(np.array([0, 500, B * T], np.int32))
    start = _dev(rng.standard_normal((3, H, K, V)).astype(np.float32))
    slot, init = _dev(np.array([2, 0], np.int32)), _dev(np.array([1, 0], np.int32))
    S, out, more = start.clone(), torch.empty_like(v), {}
    if form == "prefill":
        n = kt.kda_prefill_workspace_size(B * T, B, H, K, V)
        assert n > 0
        more = dict(workspace=torch.empty(n, dtype=torch.uint8, device=DEV))
    direct, prepare = ((kt.kda_prefill, kt.prepare_prefill) if form == "prefill" else
                       (kt.kda_recurrent, kt.prepare_recurrent))
    args = (q, k, v, g, beta, out, cu, S, slot, init, 0.3)
    direct(*args, **more)
    want, want_S = out.clone(), S.clone()
    side = torch.cuda.Stream()
    for stream in (None, side):
        call = prepare(*args, stream=stream, **more)
        for _ in range(3):
            S.copy_(start)
            out.fill_(5.0)
            torch.cuda.synchronize()
            call()
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(S, want_S)
    with pytest.raises(ValueError):
        prepare(q, k, v, g, beta, out[..., :64], cu, S, **more)
