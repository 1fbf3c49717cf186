"""Python binding of the KDA layer's calls around the solver and the decode
step (see include/kda_tril.h): chunk maps, the prompt's causal convolution, the
gated delta rule (chunked ``prefill`` and token-by-token ``recurrent``) and the
gated RMSNorm. Argument marshalling only; the functions named like the C entry
points write into given tensors, the short names allocate their outputs.
"""
from __future__ import annotations

import ctypes

import torch

from . import (CHUNK_SIZES, _alloc_stream, _check, _i32, _i64, _lib, _p, _prepared,
               _require, _sz)

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


def _place(first, stream, *tensors):
    """Stream handle of a call. Every tensor has to be a contiguous cuda
    tensor of the current device: the launch goes to a stream of that device."""
    dev = first.device
    _require(dev.type == "cuda", f"expected cuda tensors, got one on {dev}")
    _require(dev.index == torch.cuda.current_device(),
             f"tensors are on {dev}, which is not the current device")
    for t in (first, *tensors):
        if t is not None:
            _require(t.device == dev, f"tensors on {dev} and {t.device}")
            _require(t.is_contiguous(), "inputs must be contiguous")
    if stream is None:
        return torch.cuda.current_stream(dev).cuda_stream
    _require(stream.device == dev, f"tensors on {dev}, stream on {stream.device}")
    return stream.cuda_stream


def _addr(t):
    return None if t is None else t.data_ptr()


def _int32(n, **tensors):
    """int32 vectors of n entries (None: not given)."""
    for name, t in tensors.items():
        if t is not None:
            _require(t.dtype == torch.int32 and t.dim() == 1 and t.numel() == n,
                     f"{name} must be int32 [{n}]")


def _float32(**tensors):
    for name, t in tensors.items():
        if t is not None:
            _require(t.dtype == torch.float32, f"{name} must be float32")


def _requests(x, lead, cu_seqlens):
    """(number of requests, their C arguments) of a token tensor whose token
    dimension is followed by `lead` - 1 others."""
    if cu_seqlens is None:
        _require(x.dim() == lead + 1, "dense inputs are [B, T, ...]")
        return x.shape[0], (x.shape[0], x.shape[1])
    _require(x.dim() == lead, "packed inputs are [T, ...]")
    _require(cu_seqlens.dtype == torch.int32 and cu_seqlens.dim() == 1 and
             cu_seqlens.numel() >= 1, "cu_seqlens must be int32 [requests + 1]")
    n = cu_seqlens.numel() - 1
    return n, (cu_seqlens.data_ptr(), n, x.shape[0])


# ---- chunk maps ------------------------------------------------------------

def kda_chunk_map(seq_lens, total_tokens, chunk_size, cu_seqlens, chunk_indices=None,
                  num_chunks=None, stream=None) -> None:
    """cu_seqlens [N + 1] and chunk_indices [M, 2] (rows past the last chunk
    are -1) from int32 request lengths [N]; num_chunks [1] is optional."""
    s = _place(seq_lens, stream, cu_seqlens, chunk_indices, num_chunks)
    n = seq_lens.numel()
    _int32(n, seq_lens=seq_lens)
    _int32(n + 1, cu_seqlens=cu_seqlens)
    _int32(1, num_chunks=num_chunks)
    most = 0
    if chunk_indices is not None:
        _require(chunk_indices.dtype == torch.int32 and chunk_indices.dim() == 2 and
                 chunk_indices.shape[1] == 2, "chunk_indices must be int32 [M, 2]")
        most = chunk_indices.shape[0]
    _check(_lib.kda_chunk_map(seq_lens.data_ptr(), n, total_tokens, chunk_size,
                              cu_seqlens.data_ptr(), _addr(chunk_indices) if most else None, most,
                              _addr(num_chunks), s))


def chunk_map(seq_lens, total_tokens: int, chunk_size: int = 64, stream=None):
    """(cu_seqlens [N + 1], chunk_indices [floor(T / C) + N, 2], num_chunks [1])
    of requests with int32 lengths ``seq_lens`` [N] (on the GPU) that together
    take ``total_tokens`` rows. Entries past the last chunk are (-1, -1), which
    every call that takes ``chunk_indices`` skips."""
    _require(chunk_size in CHUNK_SIZES, f"chunk size {chunk_size} (16, 32 or 64)")
    n = seq_lens.numel()
    with _alloc_stream(stream):
        cu = torch.empty(n + 1, dtype=torch.int32, device=seq_lens.device)
        pairs = torch.empty((total_tokens // chunk_size + n, 2), dtype=torch.int32,
                            device=seq_lens.device)
        count = torch.empty(1, dtype=torch.int32, device=seq_lens.device)
    kda_chunk_map(seq_lens, total_tokens, chunk_size, cu, pairs, count, stream)
    return cu, pairs, count


# ---- the prompt's causal convolution ----------------------------------------

def kda_conv_prefill(qkv, conv_w, q, k, v, cu_seqlens=None, conv_state=None, slot=None, init=None,
                     eps_l2=1e-6, stream=None) -> None:
    """Causal convolution, silu and L2 norms of packed [T, 3, H, d] (with
    ``cu_seqlens``) or dense [B, T, 3, H, d] inputs into q, k, v [.., H, d];
    ``conv_state`` [slots, 3, H, W - 1, d] is updated in place."""
    s = _place(qkv, stream, conv_w, q, k, v, cu_seqlens, conv_state, slot, init)
    n, req = _requests(qkv, 4, cu_seqlens)
    H, d = qkv.shape[-2:]
    W = conv_w.shape[1] if conv_w.dim() == 4 else 0
    _require(qkv.shape[-3] == 3 and conv_w.shape == (3, W, H, d),
             "shapes: qkv [.., 3, H, d], conv_w [3, W, H, d]")
    rows = qkv.shape[:-3] + (H, d)
    _require(q.shape == rows and k.shape == rows and v.shape == rows, "q, k, v must be [.., H, d]")
    _require(q.dtype == qkv.dtype and k.dtype == qkv.dtype and v.dtype == qkv.dtype,
             "q, k, v must have qkv's dtype")
    _float32(conv_w=conv_w, conv_state=conv_state)
    _int32(n, slot=slot, init=init)
    slots = 0
    if conv_state is not None:
        slots = conv_state.shape[0]
        _require(conv_state.shape == (slots, 3, H, W - 1, d),
                 "conv_state must be [slots, 3, H, W - 1, d]")
    fn = _lib.kda_conv_prefill_dense if cu_seqlens is None else _lib.kda_conv_prefill_packed
    _check(fn(qkv.data_ptr(), _code(qkv), conv_w.data_ptr(), q.data_ptr(), k.data_ptr(),
              v.data_ptr(), *req, H, d, W, _addr(conv_state), _addr(slot), _addr(init), slots,
              eps_l2, s))


def conv_prefill(qkv, conv_w, cu_seqlens=None, conv_state=None, slot=None, init=None, eps_l2=1e-6,
                 stream=None):
    """Convenience form of kda_conv_prefill: returns (q, k, v)."""
    shape = qkv.shape[:-3] + qkv.shape[-2:]
    with _alloc_stream(stream):
        q = torch.empty(shape, dtype=qkv.dtype, device=qkv.device)
        k, v = torch.empty_like(q), torch.empty_like(q)
    kda_conv_prefill(qkv, conv_w, q, k, v, cu_seqlens, conv_state, slot, init, eps_l2, stream)
    return q, k, v


# ---- the gated delta rule ---------------------------------------------------

def _delta_args(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale, stream, workspace):
    s = _place(q, stream, k, v, g, beta, out, cu_seqlens, state, slot, init, workspace)
    n, req = _requests(q, 3, cu_seqlens)
    lead, (Hk, K) = q.shape[:-2], q.shape[-2:]
    H, V = v.shape[-2:]
    _require(k.shape == q.shape and v.shape[:-2] == lead and out.shape == v.shape and
             beta.shape == lead + (H,), "shapes: q, k [.., Hk, K], v, out [.., H, V], beta [.., H]")
    _require(k.dtype == q.dtype and v.dtype == q.dtype, "q, k and v must have one dtype")
    if g.dim() == v.dim():
        _require(g.shape == lead + (H, K), "g must be [.., H, K] or [.., H]")
        gate = K
    else:
        _require(g.shape == beta.shape, "g must be [.., H, K] or [.., H]")
        gate = 1
    _float32(g=g, beta=beta, state=state)
    _int32(n, slot=slot, init=init)
    slots = 0
    if state is not None:
        slots = state.shape[0]
        _require(state.shape == (slots, H, K, V), "state must be [slots, H, K, V]")
    if scale is None:
        scale = K ** -0.5
    return ((q.data_ptr(), k.data_ptr(), v.data_ptr(), _code(q), g.data_ptr(), beta.data_ptr(),
             out.data_ptr(), _code(out)) + req +
            (H, Hk, K, V, gate, _addr(state), _addr(slot), _addr(init), slots, scale), s)


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
    with _alloc_stream(stream):
        out = torch.empty(v.shape, dtype=out_dtype or v.dtype, device=v.device)
        n = v.shape[0] if cu_seqlens is None else cu_seqlens.numel() - 1
        tokens = v.shape[0] * v.shape[1] if cu_seqlens is None else v.shape[0]
        nbytes = kda_prefill_workspace_size(tokens, n, v.shape[-2], q.shape[-1], v.shape[-1])
        ws = torch.empty(nbytes, dtype=torch.uint8, device=v.device) if nbytes else None
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
    with _alloc_stream(stream):
        out = torch.empty(v.shape, dtype=out_dtype or v.dtype, device=v.device)
    kda_recurrent(q, k, v, g, beta, out, cu_seqlens, state, slot, init, scale, stream)
    return out


# ---- the gated RMSNorm --------------------------------------------------------

def kda_gated_norm(o, z, norm_w, out, eps_norm=1e-6, stream=None) -> None:
    """out = o / sqrt(mean(o^2) + eps) * norm_w * sigmoid(z) over the last
    dimension of o, z, out [.., H, d]; out may be o."""
    s = _place(o, stream, z, norm_w, out)
    _require(o.dim() >= 2 and z.shape == o.shape and out.shape == o.shape and
             norm_w.shape == o.shape[-1:], "shapes: o, z, out [.., H, d], norm_w [d]")
    _require(z.dtype == o.dtype, "z must have o's dtype")
    _float32(norm_w=norm_w)
    H, d = o.shape[-2:]
    rows = o.numel() // (H * d) if H * d else 0
    _check(_lib.kda_gated_norm(o.data_ptr(), z.data_ptr(), _code(o), norm_w.data_ptr(),
                               out.data_ptr(), _code(out), rows, H, d, eps_norm, s))


def gated_norm(o, z, norm_w, eps_norm=1e-6, out_dtype=None, stream=None):
    """Convenience form of kda_gated_norm: returns out (``out_dtype``, default
    o's dtype)."""
    with _alloc_stream(stream):
        out = torch.empty(o.shape, dtype=out_dtype or o.dtype, device=o.device)
    kda_gated_norm(o, z, norm_w, out, eps_norm, stream)
    return out
