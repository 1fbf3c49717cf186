"""Python binding of the KDA layer's backward pass and of its 8-bit activation
checkpoints (see include/kda_tril.h). Argument marshalling only; the functions
named like the C entry points write into given tensors, the short names allocate
their outputs and the workspace.
"""
from __future__ import annotations

import ctypes
from functools import lru_cache

import torch

from . import _alloc_stream, _check, _i32, _i64, _lib, _p, _sz
from .layer import (_DENSE, _PACKED, _addr, _bad, _code, _empty_as, _f, _float32, _int, _int32,
                    _place, _requests, _workspace_args)

_POOLS = [_p, _p, _p, _p, _i64]                 # state dstate slot init num_slots
_DELTA = [_p, _int, _p, _p, _p, _int] + [_p] * 7  # dout dtype q k v dtype g beta dq dk dv dg dbeta
_CONV = [_p, _p, _p, _int] + [_p] * 5           # dq dk dv dtype qkv scale conv_w dqkv dconv_w
_WS = [_p, _sz, _p]
_ARGS = {
    "kda_prefill_backward_workspace_size": [_i64, _i64] + [_i32] * 4 + [ctypes.POINTER(_sz)],
    "kda_prefill_backward_packed": _DELTA + _PACKED + [_i32] * 5 + _POOLS + [_f] + _WS,
    "kda_prefill_backward_dense": _DELTA + _DENSE + [_i32] * 5 + _POOLS + [_f] + _WS,
    "kda_conv_backward_workspace_size": [_i64, _i64] + [_i32] * 3 + [ctypes.POINTER(_sz)],
    "kda_conv_backward_packed": _CONV + _PACKED + [_i32] * 3 + _POOLS + [_f] + _WS,
    "kda_conv_backward_dense": _CONV + _DENSE + [_i32] * 3 + _POOLS + [_f] + _WS,
    "kda_gated_norm_backward_workspace_size": [_i64, _i32, _i32, ctypes.POINTER(_sz)],
    "kda_gated_norm_backward": [_p, _p, _p, _int] + [_p] * 6 + [_i64, _i32, _i32, _f] + _WS,
    "kda_checkpoint": [_p, _int, _p, _p, _i64, _i32, _i32, _p],
    "kda_checkpoint_load": [_p, _p, _p, _int, _i64, _i32, _i32, _p],
    "kda_gated_norm_checkpoint": [_p, _p, _int, _p, _p, _int] + [_p] * 4 +
                                 [_i64, _i32, _i32, _f, _p],
}
EXPORTED = tuple(_ARGS)
for _n, _a in _ARGS.items():
    getattr(_lib, _n).restype = _int
    getattr(_lib, _n).argtypes = _a


# (the queries depend on the sizes alone; asked once for each of them, a call spends 2 us
# less on them)
@lru_cache(maxsize=256)
def _size(name, *args) -> int:
    b = _sz(0)
    _check(getattr(_lib, name)(*args, ctypes.byref(b)))
    return int(b.value)


def _bytes(nbytes, like, stream):
    """A workspace that belongs to the stream of the call."""
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    with _alloc_stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device)


def _new_as(t, shape, dtype, stream):
    if stream is None:
        return t.new_empty(shape, dtype=dtype)
    with _alloc_stream(stream):
        return t.new_empty(shape, dtype=dtype)


def _pools(n, state, dstate, slot, init, shape, names):
    """(C arguments) of the two pools of a backward call."""
    _float32(names[0], state)
    _float32(names[1], dstate)
    _int32(n, "slot", slot)
    _int32(n, "init", init)
    slots = 0
    for name, t in zip(names, (state, dstate)):
        if t is not None:
            if t.shape[1:] != shape:
                _bad(f"{name} must be [slots, {', '.join(map(str, shape))}]")
            slots = t.shape[0]
            if slots == 0 and n > 0:  # (torch gives it no address: it would pass for no pool)
                _bad(f"{name} has no slots")
    if state is not None and dstate is not None and state.shape[0] != dstate.shape[0]:
        _bad(f"{names[0]} and {names[1]} must have the same slots")
    return _addr(state), _addr(dstate), _addr(slot), _addr(init), slots


def _vectors(t):
    """(rows, H, d) of vectors [.., H, d]."""
    if t.dim() < 2:
        _bad("vectors are [.., H, d]")
    H, d = t.shape[-2:]
    return (t.numel() // (H * d) if H and d else 0), H, d


def _codes(name, t, shape):
    if t.dtype != torch.int8 or t.shape != shape:
        _bad(f"{name} must be int8 {list(shape)}")


# ---- the gated delta rule ---------------------------------------------------

def kda_prefill_backward_workspace_size(total_tokens: int, num_seqs: int, H: int, Hk: int, K: int,
                                        V: int) -> int:
    """Workspace bytes of kda_prefill_backward. Host only."""
    return _size("kda_prefill_backward_workspace_size", total_tokens, num_seqs, H, Hk, K, V)


def kda_prefill_backward(dout, q, k, v, g, beta, dq, dk, dv, dg, dbeta, workspace,
                         cu_seqlens=None, state=None, dstate=None, slot=None, init=None,
                         scale=None, stream=None) -> None:
    """Gradients of kda_prefill from its inputs and its output's gradient
    ``dout``, written into dq, dk, dv, dg, dbeta. ``state``: the pool as the
    forward call found it; ``dstate`` (in place): the gradient of the new states,
    then of the old ones."""
    s = _place(stream, (dout, q, k, v, g, beta, dq, dk, dv, dg, dbeta, cu_seqlens, state, dstate,
                        slot, init, workspace))
    qs, vs, gs = q.shape, v.shape, g.shape
    n, req = _requests(qs, 3, cu_seqlens)
    rows, (Hk, K), (H, V) = vs[:-1], qs[-2:], vs[-2:]
    if k.shape != qs or vs[:-2] != qs[:-2] or dout.shape != vs or beta.shape != rows:
        _bad("shapes: q, k [.., Hk, K], v, dout [.., H, V], beta [.., H]")
    if dq.shape != qs or dk.shape != qs or dv.shape != vs or dg.shape != gs or dbeta.shape != rows:
        _bad("gradients must have the shapes of q, k, v, g, beta")
    if not q.dtype == k.dtype == v.dtype == dq.dtype == dk.dtype == dv.dtype:
        _bad("q, k, v, dq, dk and dv must have one dtype")
    gate = K if len(gs) == len(vs) else 1
    if gs != (rows + (K,) if gate == K else rows):
        _bad("g must be [.., H, K] or [.., H]")
    for name, t in (("g", g), ("beta", beta), ("dg", dg), ("dbeta", dbeta)):
        _float32(name, t)
    pools = _pools(n, state, dstate, slot, init, (H, K, V), ("state", "dstate"))
    fn = _lib.kda_prefill_backward_dense if cu_seqlens is None else _lib.kda_prefill_backward_packed
    _check(fn(dout.data_ptr(), _code(dout), q.data_ptr(), k.data_ptr(), v.data_ptr(), _code(q),
              g.data_ptr(), beta.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(),
              dg.data_ptr(), dbeta.data_ptr(), *req, H, Hk, K, V, gate, *pools,
              K ** -0.5 if scale is None else scale, *_workspace_args(workspace), s))


def prefill_backward(dout, q, k, v, g, beta, cu_seqlens=None, state=None, dstate=None, slot=None,
                     init=None, scale=None, stream=None):
    """Convenience form of kda_prefill_backward: returns (dq, dk, dv, dg, dbeta)
    and allocates the workspace with torch."""
    grads = [_empty_as(t, None, stream) for t in (q, k, v, g, beta)]
    n, (H, V) = v.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1, v.shape[-2:]
    Hk, K = q.shape[-2:]
    nbytes = kda_prefill_backward_workspace_size(v.numel() // max(H * V, 1), n, H, Hk, K, V)
    kda_prefill_backward(dout, q, k, v, g, beta, *grads, _bytes(nbytes, v, stream), cu_seqlens,
                         state, dstate, slot, init, scale, stream)
    return tuple(grads)


# ---- the prompt's causal convolution ------------------------------------------

def kda_conv_backward_workspace_size(total_tokens: int, num_seqs: int, H: int, head_dim: int,
                                     conv_width: int) -> int:
    """Workspace bytes of kda_conv_backward. Host only."""
    return _size("kda_conv_backward_workspace_size", total_tokens, num_seqs, H, head_dim,
                 conv_width)


def kda_conv_backward(dq, dk, dv, qkv, conv_w, dqkv, dconv_w, workspace, cu_seqlens=None,
                      conv_state=None, dconv_state=None, slot=None, init=None, eps_l2=1e-6,
                      qkv_scale=None, stream=None) -> None:
    """Gradients of kda_conv_prefill from its inputs and the gradients dq, dk, dv
    [.., H, d] of its outputs, written into dqkv [.., 3, H, d] and dconv_w. With
    ``qkv_scale`` [.., 3, H], qkv holds a checkpoint's codes. ``conv_state``: the
    pool as the forward call found it; ``dconv_state`` (in place): the gradient of
    the new windows, then of the old ones."""
    s = _place(stream, (dq, dk, dv, qkv, conv_w, dqkv, dconv_w, workspace, cu_seqlens, conv_state,
                        dconv_state, slot, init, qkv_scale))
    shape, taps = qkv.shape, conv_w.shape
    n, req = _requests(shape, 4, cu_seqlens)
    W, (H, d) = taps[1] if len(taps) == 4 else 0, shape[-2:]
    if shape[-3] != 3 or taps != (3, W, H, d) or dconv_w.shape != taps or dqkv.shape != shape:
        _bad("shapes: qkv, dqkv [.., 3, H, d], conv_w, dconv_w [3, W, H, d]")
    rows = shape[:-3] + (H, d)
    if dq.shape != rows or dk.shape != rows or dv.shape != rows:
        _bad("dq, dk, dv must be [.., H, d]")
    if not dq.dtype == dk.dtype == dv.dtype == dqkv.dtype:
        _bad("dq, dk, dv, dqkv must have one dtype")
    if qkv_scale is not None:
        _codes("qkv", qkv, shape)
        _float32("qkv_scale", qkv_scale)
        if qkv_scale.shape != shape[:-1]:
            _bad("qkv_scale must be [.., 3, H]")
    elif qkv.dtype != dqkv.dtype:
        _bad("qkv must have dqkv's dtype")
    _float32("conv_w", conv_w)
    _float32("dconv_w", dconv_w)
    pools = _pools(n, conv_state, dconv_state, slot, init, (3, H, W - 1, d),
                   ("conv_state", "dconv_state"))
    fn = _lib.kda_conv_backward_dense if cu_seqlens is None else _lib.kda_conv_backward_packed
    _check(fn(dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _code(dqkv), qkv.data_ptr(),
              _addr(qkv_scale), conv_w.data_ptr(), dqkv.data_ptr(), dconv_w.data_ptr(), *req, H, d,
              W, *pools, eps_l2, *_workspace_args(workspace), s))


def conv_prefill_backward(dq, dk, dv, qkv, conv_w, cu_seqlens=None, conv_state=None,
                          dconv_state=None, slot=None, init=None, eps_l2=1e-6, qkv_scale=None,
                          stream=None):
    """Convenience form of kda_conv_backward: returns (dqkv, dconv_w) and
    allocates the workspace with torch."""
    if qkv.dim() < 4 or conv_w.dim() != 4:
        _bad("shapes: qkv [.., 3, H, d], conv_w [3, W, H, d]")
    dqkv, dconv_w = _empty_as(qkv, dq.dtype, stream), _empty_as(conv_w, None, stream)
    n = qkv.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1
    H, d = qkv.shape[-2:]
    nbytes = kda_conv_backward_workspace_size(qkv.numel() // max(3 * H * d, 1), n, H, d,
                                              conv_w.shape[1])
    kda_conv_backward(dq, dk, dv, qkv, conv_w, dqkv, dconv_w, _bytes(nbytes, qkv, stream),
                      cu_seqlens, conv_state, dconv_state, slot, init, eps_l2, qkv_scale, stream)
    return dqkv, dconv_w


# ---- the gated RMSNorm --------------------------------------------------------

def kda_gated_norm_backward_workspace_size(rows: int, H: int, head_dim: int) -> int:
    """Workspace bytes of kda_gated_norm_backward. Host only."""
    return _size("kda_gated_norm_backward_workspace_size", rows, H, head_dim)


def kda_gated_norm_backward(dout, o, z, norm_w, do, dz, dnorm_w, workspace, eps_norm=1e-6,
                            o_scale=None, z_scale=None, stream=None) -> None:
    """Gradients of kda_gated_norm over the last dimension of dout, o, z, do, dz
    [.., H, d], and dnorm_w [d]. With ``o_scale`` and ``z_scale`` [.., H], o and z
    hold checkpoints' codes."""
    s = _place(stream, (dout, o, z, norm_w, do, dz, dnorm_w, workspace, o_scale, z_scale))
    rows, H, d = _vectors(dout)
    shape = dout.shape
    if o.shape != shape or z.shape != shape or do.shape != shape or dz.shape != shape or \
            norm_w.shape != (d,) or dnorm_w.shape != (d,):
        _bad("shapes: dout, o, z, do, dz [.., H, d], norm_w, dnorm_w [d]")
    if not dout.dtype == do.dtype == dz.dtype:
        _bad("dout, do and dz must have one dtype")
    if (o_scale is None) != (z_scale is None):
        _bad("o_scale and z_scale go together")
    if o_scale is not None:
        for name, t, sc in (("o", o, o_scale), ("z", z, z_scale)):
            _codes(name, t, shape)
            _float32(f"{name}_scale", sc)
            if sc.shape != shape[:-1]:
                _bad(f"{name}_scale must be [.., H]")
    elif not o.dtype == z.dtype == dout.dtype:
        _bad("o and z must have dout's dtype")
    _float32("norm_w", norm_w)
    _float32("dnorm_w", dnorm_w)
    _check(_lib.kda_gated_norm_backward(
        dout.data_ptr(), o.data_ptr(), z.data_ptr(), _code(dout), _addr(o_scale), _addr(z_scale),
        norm_w.data_ptr(), do.data_ptr(), dz.data_ptr(), dnorm_w.data_ptr(), rows, H, d, eps_norm,
        *_workspace_args(workspace), s))


def gated_norm_backward(dout, o, z, norm_w, eps_norm=1e-6, o_scale=None, z_scale=None,
                        stream=None):
    """Convenience form of kda_gated_norm_backward: returns (do, dz, dnorm_w) and
    allocates the workspace with torch."""
    do, dz = _empty_as(dout, None, stream), _empty_as(dout, None, stream)
    dnorm_w = _empty_as(norm_w, None, stream)
    ws = _bytes(kda_gated_norm_backward_workspace_size(*_vectors(dout)), dout, stream)
    kda_gated_norm_backward(dout, o, z, norm_w, do, dz, dnorm_w, ws, eps_norm, o_scale, z_scale,
                            stream)
    return do, dz, dnorm_w


# ---- activation checkpoints -----------------------------------------------------

def kda_checkpoint(x, codes, scale, stream=None) -> None:
    """The vectors x [.., H, d] as int8 codes [.., H, d] and scales [.., H]."""
    s = _place(stream, (x, codes, scale))
    rows, H, d = _vectors(x)
    _codes("codes", codes, x.shape)
    _float32("scale", scale)
    if scale.shape != x.shape[:-1]:
        _bad("scale must be [.., H]")
    _check(_lib.kda_checkpoint(x.data_ptr(), _code(x), codes.data_ptr(), scale.data_ptr(), rows, H,
                               d, s))


def checkpoint(x, stream=None):
    """Convenience form of kda_checkpoint: returns (codes, scale)."""
    codes = _empty_as(x, torch.int8, stream)
    scale = _new_as(x, x.shape[:-1], torch.float32, stream)
    kda_checkpoint(x, codes, scale, stream)
    return codes, scale


def kda_checkpoint_load(codes, scale, out, stream=None) -> None:
    """out [.., H, d] = codes x scale, the values of a checkpoint."""
    s = _place(stream, (codes, scale, out))
    rows, H, d = _vectors(out)
    _codes("codes", codes, out.shape)
    _float32("scale", scale)
    if scale.shape != out.shape[:-1]:
        _bad("scale must be [.., H]")
    _check(_lib.kda_checkpoint_load(codes.data_ptr(), scale.data_ptr(), out.data_ptr(), _code(out),
                                    rows, H, d, s))


def checkpoint_load(codes, scale, dtype=torch.bfloat16, stream=None):
    """Convenience form of kda_checkpoint_load: returns the values in ``dtype``."""
    out = _empty_as(codes, dtype, stream)
    kda_checkpoint_load(codes, scale, out, stream)
    return out


def kda_gated_norm_checkpoint(o, z, norm_w, out, o_codes, o_scale, z_codes, z_scale,
                              eps_norm=1e-6, stream=None) -> None:
    """kda_gated_norm that also writes the checkpoints of o and z (out must not be o)."""
    s = _place(stream, (o, z, norm_w, out, o_codes, o_scale, z_codes, z_scale))
    rows, H, d = _vectors(o)
    shape = o.shape
    if z.shape != shape or out.shape != shape or norm_w.shape != (d,):
        _bad("shapes: o, z, out [.., H, d], norm_w [d]")
    if z.dtype != o.dtype:
        _bad("z must have o's dtype")
    _float32("norm_w", norm_w)
    for name, codes, scale in (("o", o_codes, o_scale), ("z", z_codes, z_scale)):
        _codes(f"{name}_codes", codes, shape)
        _float32(f"{name}_scale", scale)
        if scale.shape != shape[:-1]:
            _bad(f"{name}_scale must be [.., H]")
    _check(_lib.kda_gated_norm_checkpoint(
        o.data_ptr(), z.data_ptr(), _code(o), norm_w.data_ptr(), out.data_ptr(), _code(out),
        o_codes.data_ptr(), o_scale.data_ptr(), z_codes.data_ptr(), z_scale.data_ptr(), rows, H, d,
        eps_norm, s))


def gated_norm_checkpoint(o, z, norm_w, eps_norm=1e-6, out_dtype=None, stream=None):
    """Convenience form of kda_gated_norm_checkpoint: returns (out, o_codes,
    o_scale, z_codes, z_scale)."""
    out = _empty_as(o, out_dtype, stream)
    o_codes, z_codes = _empty_as(o, torch.int8, stream), _empty_as(o, torch.int8, stream)
    o_scale = _new_as(o, o.shape[:-1], torch.float32, stream)
    z_scale = _new_as(o, o.shape[:-1], torch.float32, stream)
    kda_gated_norm_checkpoint(o, z, norm_w, out, o_codes, o_scale, z_codes, z_scale, eps_norm,
                              stream)
    return out, o_codes, o_scale, z_codes, z_scale
