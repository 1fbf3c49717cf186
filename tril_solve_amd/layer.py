"""Python binding of the KDA layer's calls around the solver and the decode
step (see include/kda_tril.h): chunk maps, the prompt's causal convolution, the
gated delta rule (chunked ``prefill`` and token-by-token ``recurrent``) and the
gated RMSNorm. Argument marshalling only; the functions named like the C entry
points write into given tensors, the short names allocate their outputs.
"""
from __future__ import annotations

import ctypes

import torch

from . import (CHUNK_SIZES, _alloc_stream, _check, _i32, _i64, _lib, _p, _prepared, _sz)

_int, _f = ctypes.c_int, ctypes.c_float
_DELTA = [_p, _p, _p, _int, _p, _p, _p, _int]            # q k v dtype g beta out dtype
_HEADS = [_i32] * 5 + [_p, _p, _p, _i64, _f]             # H Hk K V gate_dim; pool; scale
_PACKED, _DENSE = [_p, _i64, _i64], [_i64, _i64]
_ARGS = {
    "kda_chunk_map": [_p, _i64, _i64, _i32, _p, _p, _i64, _p, _p],
    "kda_conv_prefill_packed": [_p, _int, _p, _p, _p, _p] + _PACKED + [_i32] * 3 +
                               [_p, _p, _p, _i64, _f, _p],
    "kda_conv_prefill_dense": [_p, _int, _p, _p, _p, _p] + _DENSE + [_i32] * 3 +
                              [_p, _p, _p, _i64, _f, _p],
    "kda_prefill_workspace_size": [_i64, _i64, _i32, _i32, _i32, ctypes.POINTER(_sz)],
    "kda_prefill_packed": _DELTA + _PACKED + _HEADS + [_p, _sz, _p],
    "kda_prefill_dense": _DELTA + _DENSE + _HEADS + [_p, _sz, _p],
    "kda_recurrent_packed": _DELTA + _PACKED + _HEADS + [_p],
    "kda_recurrent_dense": _DELTA + _DENSE + _HEADS + [_p],
    "kda_gated_norm": [_p, _p, _int, _p, _p, _int, _i64, _i32, _i32, _f, _p],
}
EXPORTED = tuple(_ARGS)
for _n, _a in _ARGS.items():
    getattr(_lib, _n).restype = _int
    getattr(_lib, _n).argtypes = _a

_CODES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _code(t) -> int:
    c = _CODES.get(t.dtype)
    if c is None:
        raise TypeError(f"unsupported dtype {t.dtype} (float32, bfloat16 or float16)")
    return c


_current_device = torch._C._cuda_getDevice
_current_stream = torch._C._cuda_getCurrentRawStream


def _bad(what: str):
    raise ValueError(what)


# The checks below run on every call, ahead of a launch of a few microseconds:
# conditions are tested in place and messages built only for a refusal.

def _place(stream, tensors):
    """Stream handle of a call. Every tensor has to be a contiguous cuda
    tensor of the current device: the launch goes to a stream of that device."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None:
            if t.get_device() != dev or dev < 0:
                _bad(f"expected cuda tensors of one device, got "
                     f"{[str(x.device) for x in tensors if x is not None]}")
            if not t.is_contiguous():
                _bad("inputs must be contiguous")
    if dev != _current_device():
        _bad(f"tensors are on cuda:{dev}, which is not the current device")
    if stream is None:
        return _current_stream(dev)
    if stream.device.index != dev:
        _bad(f"tensors on cuda:{dev}, stream on {stream.device}")
    return stream.cuda_stream


def _addr(t):
    return None if t is None else t.data_ptr()


def _int32(n, name, t):
    """An int32 vector of n entries (or None)."""
    if t is not None and (t.dtype != torch.int32 or t.dim() != 1 or t.numel() != n):
        _bad(f"{name} must be int32 [{n}]")


def _float32(name, t):
    if t is not None and t.dtype != torch.float32:
        _bad(f"{name} must be float32")


def _requests(shape, lead, cu_seqlens):
    """(number of requests, their C arguments) of token tensors of this shape,
    the token dimension followed by `lead` - 1 others."""
    if cu_seqlens is None:
        if len(shape) != lead + 1:
            _bad("dense inputs are [B, T, ...]")
        return shape[0], (shape[0], shape[1])
    if len(shape) != lead:
        _bad("packed inputs are [T, ...]")
    n = cu_seqlens.numel() - 1
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or n < 0:
        _bad("cu_seqlens must be int32 [requests + 1]")
    return n, (cu_seqlens.data_ptr(), n, shape[0])


# ---- chunk maps ------------------------------------------------------------

def kda_chunk_map(seq_lens, total_tokens, chunk_size, cu_seqlens, chunk_indices=None,
                  num_chunks=None, stream=None) -> None:
    """cu_seqlens [N + 1] and chunk_indices [M, 2] (rows past the last chunk
    are -1) from int32 request lengths [N]; num_chunks [1] is optional."""
    s = _place(stream, (seq_lens, cu_seqlens, chunk_indices, num_chunks))
    n = seq_lens.numel()
    _int32(n, "seq_lens", seq_lens)
    _int32(n + 1, "cu_seqlens", cu_seqlens)
    _int32(1, "num_chunks", num_chunks)
    most = 0
    if chunk_indices is not None:
        if chunk_indices.dtype != torch.int32 or chunk_indices.dim() != 2 or \
                chunk_indices.shape[1] != 2:
            _bad("chunk_indices must be int32 [M, 2]")
        most = chunk_indices.shape[0]
    _check(_lib.kda_chunk_map(seq_lens.data_ptr(), n, total_tokens, chunk_size,
                              cu_seqlens.data_ptr(), _addr(chunk_indices) if most else None, most,
                              _addr(num_chunks), s))


def chunk_map(seq_lens, total_tokens: int, chunk_size: int = 64, stream=None):
    """(cu_seqlens [N + 1], chunk_indices [floor(T / C) + N, 2], num_chunks [1])
    of requests with int32 lengths ``seq_lens`` [N] (on the GPU) that together
    take ``total_tokens`` rows. Entries past the last chunk are (-1, -1), which
    every call that takes ``chunk_indices`` skips."""
    if chunk_size not in CHUNK_SIZES:
        _bad(f"chunk size {chunk_size} (16, 32 or 64)")
    n = seq_lens.numel()
    _int32(n, "seq_lens", seq_lens)
    with _alloc_stream(stream):
        cu = seq_lens.new_empty(n + 1)
        pairs = seq_lens.new_empty((total_tokens // chunk_size + n, 2))
        count = seq_lens.new_empty(1)
    kda_chunk_map(seq_lens, total_tokens, chunk_size, cu, pairs, count, stream)
    return cu, pairs, count


# ---- the prompt's causal convolution ----------------------------------------

def kda_conv_prefill(qkv, conv_w, q, k, v, cu_seqlens=None, conv_state=None, slot=None, init=None,
                     eps_l2=1e-6, stream=None) -> None:
    """Causal convolution, silu and L2 norms of packed [T, 3, H, d] (with
    ``cu_seqlens``) or dense [B, T, 3, H, d] inputs into q, k, v [.., H, d];
    ``conv_state`` [slots, 3, H, W - 1, d] is updated in place."""
    s = _place(stream, (qkv, conv_w, q, k, v, cu_seqlens, conv_state, slot, init))
    shape, taps = qkv.shape, conv_w.shape
    n, req = _requests(shape, 4, cu_seqlens)
    W, (H, d) = taps[1] if len(taps) == 4 else 0, shape[-2:]
    if shape[-3] != 3 or taps != (3, W, H, d):
        _bad("shapes: qkv [.., 3, H, d], conv_w [3, W, H, d]")
    rows = shape[:-3] + (H, d)
    if q.shape != rows or k.shape != rows or v.shape != rows:
        _bad("q, k, v must be [.., H, d]")
    if not q.dtype == k.dtype == v.dtype == qkv.dtype:
        _bad("q, k, v must have qkv's dtype")
    _float32("conv_w", conv_w)
    _float32("conv_state", conv_state)
    _int32(n, "slot", slot)
    _int32(n, "init", init)
    slots = 0
    if conv_state is not None:
        windows = conv_state.shape
        if windows[1:] != (3, H, W - 1, d):
            _bad("conv_state must be [slots, 3, H, W - 1, d]")
        slots = windows[0]
        if slots == 0 and n > 0:  # (torch gives it no address: it would pass for no pool)
            _bad("conv_state has no slots")
    fn = _lib.kda_conv_prefill_dense if cu_seqlens is None else _lib.kda_conv_prefill_packed
    _check(fn(qkv.data_ptr(), _code(qkv), conv_w.data_ptr(), q.data_ptr(), k.data_ptr(),
              v.data_ptr(), *req, H, d, W, _addr(conv_state), _addr(slot), _addr(init), slots,
              eps_l2, s))


def conv_prefill(qkv, conv_w, cu_seqlens=None, conv_state=None, slot=None, init=None, eps_l2=1e-6,
                 stream=None):
    """Convenience form of kda_conv_prefill: returns (q, k, v)."""
    shape = qkv.shape[:-3] + qkv.shape[-2:]
    with _alloc_stream(stream):
        q = qkv.new_empty(shape)
        k, v = torch.empty_like(q), torch.empty_like(q)
    kda_conv_prefill(qkv, conv_w, q, k, v, cu_seqlens, conv_state, slot, init, eps_l2, stream)
    return q, k, v


# ---- the gated delta rule ---------------------------------------------------

def _delta_args(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale, stream, workspace):
    s = _place(stream, (q, k, v, g, beta, out, cu_seqlens, state, slot, init, workspace))
    qs, vs = q.shape, v.shape
    n, req = _requests(qs, 3, cu_seqlens)
    rows, (Hk, K), (H, V) = vs[:-1], qs[-2:], vs[-2:]
    if k.shape != qs or vs[:-2] != qs[:-2] or out.shape != vs or beta.shape != rows:
        _bad("shapes: q, k [.., Hk, K], v, out [.., H, V], beta [.., H]")
    if not q.dtype == k.dtype == v.dtype:
        _bad("q, k and v must have one dtype")
    gs = g.shape
    gate = K if len(gs) == len(vs) else 1
    if gs != (rows + (K,) if gate == K else rows):
        _bad("g must be [.., H, K] or [.., H]")
    _float32("g", g)
    _float32("beta", beta)
    _float32("state", state)
    _int32(n, "slot", slot)
    _int32(n, "init", init)
    slots = 0
    if state is not None:
        states = state.shape
        if states[1:] != (H, K, V):
            _bad("state must be [slots, H, K, V]")
        slots = states[0]
        if slots == 0 and n > 0:
            _bad("state has no slots")
    if scale is None:
        scale = K ** -0.5
    return ((q.data_ptr(), k.data_ptr(), v.data_ptr(), _code(q), g.data_ptr(), beta.data_ptr(),
             out.data_ptr(), _code(out)) + req +
            (H, Hk, K, V, gate, _addr(state), _addr(slot), _addr(init), slots, scale), s)


def _empty_as(t, dtype, stream):
    """An output shaped like t, allocated for the stream of the call."""
    if stream is None:
        return torch.empty_like(t, dtype=dtype)
    with _alloc_stream(stream):
        return torch.empty_like(t, dtype=dtype)


def _workspace_args(workspace):
    return (None, 0) if workspace is None else (workspace.data_ptr(),
                                                workspace.numel() * workspace.element_size())


def kda_prefill_workspace_size(total_tokens: int, num_seqs: int, H: int, K: int, V: int) -> int:
    """Workspace bytes with which kda_prefill may cut long requests into
    segments (0: it would not). Host only."""
    b = _sz(0)
    _check(_lib.kda_prefill_workspace_size(total_tokens, num_seqs, H, K, V, ctypes.byref(b)))
    return int(b.value)


def _prefill_call(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale, workspace, stream):
    args, s = _delta_args(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale, stream,
                          workspace)
    fn = _lib.kda_prefill_dense if cu_seqlens is None else _lib.kda_prefill_packed
    return fn, args + _workspace_args(workspace) + (s,)


def kda_prefill(q, k, v, g, beta, out, cu_seqlens=None, state=None, slot=None, init=None,
                scale=None, workspace=None, stream=None) -> None:
    """The gated delta rule over prompts, in chunks: q, k [T, Hk, K], v, out
    [T, H, V], g [T, H, K] or [T, H], beta [T, H] (packed with ``cu_seqlens``,
    else [B, T, ...]); ``state`` [slots, H, K, V] is updated in place. ``scale``
    defaults to K ** -0.5."""
    fn, args = _prefill_call(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale,
                             workspace, stream)
    _check(fn(*args))


def prepare_prefill(q, k, v, g, beta, out, cu_seqlens=None, state=None, slot=None, init=None,
                    scale=None, workspace=None, stream=None):
    """Marshalled form of one kda_prefill call."""
    return _prepared(*_prefill_call(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale,
                                    workspace, stream))


def prefill(q, k, v, g, beta, cu_seqlens=None, state=None, slot=None, init=None, scale=None,
            out_dtype=None, stream=None):
    """Convenience form of kda_prefill: returns out (``out_dtype``, default v's
    dtype) and allocates the workspace with torch."""
    out = _empty_as(v, out_dtype, stream)
    n, (H, V) = v.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1, v.shape[-2:]
    tokens, ws = v.numel() // max(H * V, 1), None
    if tokens >= 512 * n:  # else no workspace is wanted
        nbytes = kda_prefill_workspace_size(tokens, n, H, q.shape[-1], V)
        if nbytes:
            with _alloc_stream(stream):
                ws = torch.empty(nbytes, dtype=torch.uint8, device=v.device)
    kda_prefill(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale, ws, stream)
    return out


def _recurrent_call(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale, stream):
    args, s = _delta_args(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale, stream,
                          None)
    fn = _lib.kda_recurrent_dense if cu_seqlens is None else _lib.kda_recurrent_packed
    return fn, args + (s,)


def kda_recurrent(q, k, v, g, beta, out, cu_seqlens=None, state=None, slot=None, init=None,
                  scale=None, stream=None) -> None:
    """kda_prefill's recurrence token by token, for a few tokens per request
    (same arguments, no workspace)."""
    fn, args = _recurrent_call(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale, stream)
    _check(fn(*args))


def prepare_recurrent(q, k, v, g, beta, out, cu_seqlens=None, state=None, slot=None, init=None,
                      scale=None, stream=None):
    """Marshalled form of one kda_recurrent call."""
    return _prepared(*_recurrent_call(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale,
                                      stream))


def recurrent(q, k, v, g, beta, cu_seqlens=None, state=None, slot=None, init=None, scale=None,
              out_dtype=None, stream=None):
    """Convenience form of kda_recurrent: returns out (``out_dtype``, default
    v's dtype)."""
    out = _empty_as(v, out_dtype, stream)
    kda_recurrent(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale, stream)
    return out


# ---- the gated RMSNorm --------------------------------------------------------

def kda_gated_norm(o, z, norm_w, out, eps_norm=1e-6, stream=None) -> None:
    """out = o / sqrt(mean(o^2) + eps) * norm_w * sigmoid(z) over the last
    dimension of o, z, out [.., H, d]; out may be o."""
    s = _place(stream, (o, z, norm_w, out))
    shape = o.shape
    if len(shape) < 2 or z.shape != shape or out.shape != shape or norm_w.shape != shape[-1:]:
        _bad("shapes: o, z, out [.., H, d], norm_w [d]")
    if z.dtype != o.dtype:
        _bad("z must have o's dtype")
    _float32("norm_w", norm_w)
    H, d = shape[-2:]
    rows = o.numel() // (H * d) if H and d else 0
    _check(_lib.kda_gated_norm(o.data_ptr(), z.data_ptr(), _code(o), norm_w.data_ptr(),
                               out.data_ptr(), _code(out), rows, H, d, eps_norm, s))


def gated_norm(o, z, norm_w, eps_norm=1e-6, out_dtype=None, stream=None):
    """Convenience form of kda_gated_norm: returns out (``out_dtype``, default
    o's dtype)."""
    out = _empty_as(o, out_dtype, stream)
    kda_gated_norm(o, z, norm_w, out, eps_norm, stream)
    return out
