"""Binding of linear attention with a per-head decay and of the 8-bit state
cache (include/kata.h): argument checks and marshalling, as in ``_abi``.

Token tensors are [T, H, width] with the last two dimensions dense; the
stride between tokens is free (a multiple of 16 bytes), so the parts of a
fused projection go in as they are.  Every tensor of a call is on one device,
which need not be the current one.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from ._abi import _check, _dtype_code, _stream_ptr, lib


def _tensor(t, name, dtype, shape, device):
    """Pointer of a contiguous CUDA tensor of this type and shape (None in `shape`: any size)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, the call's tensors are on %s" % (name, t.device, device))
    if t.dim() != len(shape) or any(w is not None and w != s for w, s in zip(shape, t.shape)):
        raise ValueError("%s must have the shape %s, got %s" % (
            name, tuple("*" if w is None else w for w in shape), tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr()


def _opt(t, name, dtype, shape, device):
    return None if t is None else _tensor(t, name, dtype, shape, device)


def _rows(t, name, dtype, shape, device):
    """(pointer, elements from one row to the next) of a [rows, H, width] tensor, dense within a row."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, the call's tensors are on %s" % (name, t.device, device))
    if t.dim() != 3 or tuple(t.shape) != tuple(shape):
        raise ValueError("%s must have the shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    n, H, w = shape
    if t.numel() and ((w > 1 and t.stride(2) != 1) or (H > 1 and t.stride(1) != w)):
        raise ValueError("%s must be dense within a token (its last two dimensions contiguous)" % name)
    return t.data_ptr(), (t.stride(0) if n > 1 else H * w)


def _lead(q, v, what):
    for t, name in ((q, "q"), (v, "v")):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError("%s must be a CUDA tensor" % name)
        if t.dim() != 3:
            raise ValueError("%s must be [%s, H, width], got %s" % (name, what, tuple(t.shape)))
    return q.shape[0], q.shape[1], q.shape[2], v.shape[2], q.device


def _workspace(ws, need, device, stream):
    """The caller's workspace, or one that the allocator keeps until `stream` is past the call."""
    if ws is None:
        if need == 0:
            return None, 0
        ws = torch.empty(need, dtype=torch.uint8, device=device)
        if stream is not None:
            ws.record_stream(stream)
    elif not ws.is_cuda or ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor on %s" % device)
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _sequences(cu_seqlens, device):
    if cu_seqlens is None:
        return None, 1
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [N + 1]")
    return _tensor(cu_seqlens, "cu_seqlens", torch.int32, (None,), device), cu_seqlens.numel() - 1


def kata_fwd_linear_decay_workspace_size(T, H, d, dv, N) -> int:
    return int(lib().kata_fwd_linear_decay_workspace_size(T, H, d, dv, N))


def kata_bwd_linear_decay_workspace_size(T, H, d, dv, N) -> int:
    return int(lib().kata_bwd_linear_decay_workspace_size(T, H, d, dv, N))


def kata_fwd_linear_decay(q, k, v, log_decay, cu_seqlens=None, scale=1.0, S0=None, S_out=None, slots=None,
                          resume=None, return_state=False, zero_outside=None, o=None, workspace=None, stream=None):
    """Linear attention with a per-head decay over packed prompts:
    S_t = exp(log_decay) S_{t-1} + k_t v_t^T, o_t = scale * q_t^T S_t.

    q,k [T,H,d], v [T,H,dv] (bf16, d and dv 64 or 128), log_decay [H] fp32
    (<= 0), cu_seqlens [N+1] int32 (None: one sequence).  S0 and S_out are
    pools of states [n_slots,H,d,dv] fp32 (may be the same tensor); slots [N]
    int32 names each sequence's row (None: row n; negative: from zero, not
    kept) and resume [N] uint8 those that start from S0 (None: all).  Returns
    o, or (o, S_out) with return_state=True, which allocates S_out [N,H,d,dv]
    where none is given.  Rows of o outside every sequence are zeroed when
    zero_outside is true (None: when o is allocated here).
    """
    T, H, d, dv, dev = _lead(q, v, "T")
    code = _dtype_code(q)
    qp, qs = _rows(q, "q", q.dtype, (T, H, d), dev)
    kp, ks = _rows(k, "k", q.dtype, (T, H, d), dev)
    vp, vs = _rows(v, "v", q.dtype, (T, H, dv), dev)
    cu, N = _sequences(cu_seqlens, dev)
    if return_state and S_out is None:
        if slots is not None:
            raise ValueError("with slots, give the pool S_out that the final states go to")
        S_out = torch.empty((N, H, d, dv), dtype=torch.float32, device=dev)
    pool = S0 if S0 is not None else S_out
    n_slots = 0 if pool is None else pool.shape[0]
    state = (n_slots, H, d, dv)
    if zero_outside is None:
        zero_outside = o is None
    if o is None:
        o = torch.empty((T, H, dv), dtype=q.dtype, device=dev)
    op, os_ = _rows(o, "o", q.dtype, (T, H, dv), dev)
    with torch.cuda.device(dev):
        ws, ws_bytes = _workspace(workspace, kata_fwd_linear_decay_workspace_size(T, H, d, dv, N), dev, stream)
        _check("kata_fwd_linear_decay", lib().kata_fwd_linear_decay(
            qp, kp, vp, op, T, H, d, dv, qs, ks, vs, os_, _tensor(log_decay, "log_decay", torch.float32, (H,), dev),
            float(scale), cu, N, _opt(S0, "S0", torch.float32, state, dev),
            _opt(S_out, "S_out", torch.float32, state, dev), _opt(slots, "slots", torch.int32, (N,), dev), n_slots,
            _opt(resume, "resume", torch.uint8, (N,), dev), int(bool(zero_outside)), code, ws, ws_bytes,
            _stream_ptr(stream)))
    return (o, S_out) if return_state else o


def kata_bwd_linear_decay(q, k, v, dO, log_decay, cu_seqlens=None, scale=1.0, S0=None, dS_out=None,
                          return_dS0=False, workspace=None, stream=None):
    """Gradients (dq, dk, dv), or (dq, dk, dv, dS0) with return_dS0=True, of
    kata_fwd_linear_decay for dO [T,H,dv] and the gradient dS_out of the final
    states; S0, dS_out, dS0 are [N,H,d,dv] fp32.  Rows outside every sequence
    get zeros; the decays get no gradient."""
    T, H, d, dvw, dev = _lead(q, v, "T")
    code = _dtype_code(q)
    qp, qs = _rows(q, "q", q.dtype, (T, H, d), dev)
    kp, ks = _rows(k, "k", q.dtype, (T, H, d), dev)
    vp, vs = _rows(v, "v", q.dtype, (T, H, dvw), dev)
    dop = _tensor(dO, "dO", q.dtype, (T, H, dvw), dev)
    cu, N = _sequences(cu_seqlens, dev)
    state = (N, H, d, dvw)
    dq = torch.empty((T, H, d), dtype=q.dtype, device=dev)
    dk = torch.empty((T, H, d), dtype=q.dtype, device=dev)
    dv = torch.empty((T, H, dvw), dtype=q.dtype, device=dev)
    dS0 = torch.empty(state, dtype=torch.float32, device=dev) if return_dS0 else None
    with torch.cuda.device(dev):
        ws, ws_bytes = _workspace(workspace, kata_bwd_linear_decay_workspace_size(T, H, d, dvw, N), dev, stream)
        _check("kata_bwd_linear_decay", lib().kata_bwd_linear_decay(
            qp, kp, vp, dop, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), T, H, d, dvw, qs, ks, vs,
            _tensor(log_decay, "log_decay", torch.float32, (H,), dev), float(scale), cu, N,
            _opt(S0, "S0", torch.float32, state, dev), _opt(dS_out, "dS_out", torch.float32, state, dev),
            None if dS0 is None else dS0.data_ptr(), code, ws, ws_bytes, _stream_ptr(stream)))
    return (dq, dk, dv, dS0) if return_dS0 else (dq, dk, dv)


class KataAttentionLinearDecay(torch.autograd.Function):
    """Autograd wrapper of kata_fwd_linear_decay and kata_bwd_linear_decay (marshalling only)."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, cu_seqlens, scale, S0, return_state):
        o, S = kata_fwd_linear_decay(q, k, v, log_decay, cu_seqlens, scale, S0=S0, return_state=True) \
            if return_state else (kata_fwd_linear_decay(q, k, v, log_decay, cu_seqlens, scale, S0=S0), None)
        ctx.scale = float(scale)
        ctx.save_for_backward(q, k, v, log_decay, cu_seqlens, S0)
        ctx.set_materialize_grads(False)
        return (o, S) if return_state else o

    @staticmethod
    @once_differentiable
    def backward(ctx, dO, dS=None):
        q, k, v, log_decay, cu_seqlens, S0 = ctx.saved_tensors
        dO = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if dO is None else dO.contiguous()
        want = S0 is not None and ctx.needs_input_grad[6]
        g = kata_bwd_linear_decay(q, k, v, dO, log_decay, cu_seqlens, ctx.scale, S0=S0,
                                  dS_out=None if dS is None else dS.contiguous(), return_dS0=want)
        return g[0], g[1], g[2], None, None, None, (g[3] if want else None), None


def kata_attention_linear_decay(q, k, v, log_decay, cu_seqlens=None, scale=1.0, S0=None, return_state=False):
    """Differentiable linear attention with a per-head decay over packed
    sequences, q,k [T,H,d], v [T,H,dv] (bf16); S0 [N,H,d,dv] fp32.  Returns o,
    or (o, S_out) with return_state=True; gradients reach q, k, v and S0."""
    if isinstance(log_decay, torch.Tensor) and log_decay.requires_grad:
        raise ValueError("log_decay gets no gradient: pass log_decay.detach()")
    return KataAttentionLinearDecay.apply(q, k, v, log_decay, cu_seqlens, scale, S0, return_state)


def kata_decode_step_linear_decay(q, k, v, S, log_decay, slots=None, scale=1.0, o=None, stream=None):
    """One token for each of n streams: S <- exp(log_decay) S + k v^T and
    o = scale * q^T S, in place on the pool S [n_slots,H,d,dv] fp32.  q,k
    [n,H,d], v [n,H,dv] (bf16 or fp32); slots [n] int32 names each stream's
    row (None: row i; negative: padding, whose row of o is zero)."""
    n, H, d, dv, dev = _lead(q, v, "n")
    code = _dtype_code(q)
    qp, qs = _rows(q, "q", q.dtype, (n, H, d), dev)
    kp, ks = _rows(k, "k", q.dtype, (n, H, d), dev)
    vp, vs = _rows(v, "v", q.dtype, (n, H, dv), dev)
    if o is None:
        o = torch.empty((n, H, dv), dtype=q.dtype, device=dev)
    op, os_ = _rows(o, "o", q.dtype, (n, H, dv), dev)
    with torch.cuda.device(dev):
        _check("kata_decode_step_linear_decay", lib().kata_decode_step_linear_decay(
            qp, kp, vp, op, _tensor(S, "S", torch.float32, (None, H, d, dv), dev), n, H, d, dv, qs, ks, vs, os_,
            _tensor(log_decay, "log_decay", torch.float32, (H,), dev), float(scale),
            _opt(slots, "slots", torch.int32, (n,), dev), S.shape[0], code, _stream_ptr(stream)))
    return o


def _pools(S, cache, scale, slots, entries, z, z_cache):
    if not isinstance(S, torch.Tensor) or not S.is_cuda:
        raise TypeError("S must be a CUDA tensor")
    if S.dim() != 4:
        raise ValueError("S must be [n_slots, H, rows, dv], got %s" % (tuple(S.shape),))
    dev = S.device
    n_slots, H, rows, dv = S.shape
    if not isinstance(cache, torch.Tensor) or cache.dim() != 4:
        raise ValueError("cache must be an int8 tensor [n_entries, H, rows, dv]")
    n_entries = cache.shape[0]
    if (z is None) != (z_cache is None):
        raise ValueError("z and z_cache: both or neither")
    counts = [t.numel() for t in (slots, entries) if t is not None]
    n = counts[0] if counts else min(n_slots, n_entries)
    return dict(
        S=_tensor(S, "S", torch.float32, (n_slots, H, rows, dv), dev),
        cache=_tensor(cache, "cache", torch.int8, (n_entries, H, rows, dv), dev),
        scale=_tensor(scale, "scale", torch.float32, (n_entries, H, rows), dev),
        z=_opt(z, "z", torch.float32, (n_slots, H, rows), dev),
        z_cache=_opt(z_cache, "z_cache", torch.float32, (n_entries, H, rows), dev),
        slots=_opt(slots, "slots", torch.int32, (n,), dev), entries=_opt(entries, "entries", torch.int32, (n,), dev),
        n_slots=n_slots, n_entries=n_entries, n=n, H=H, rows=rows, dv=dv, dev=dev)


def kata_state_store_q8(S, cache, scale, slots=None, entries=None, z=None, z_cache=None, stream=None):
    """Write states to the 8-bit cache: slot slots[i] of S [n_slots,H,rows,dv]
    fp32 to entry entries[i] of cache [n_entries,H,rows,dv] int8 and scale
    [n_entries,H,rows] fp32, each row as round(x / scale) with scale =
    max|x| / 127; z [n_slots,H,rows] is copied to z_cache.  slots and entries
    are int32 (None: 0, 1, ...); a negative index skips its pair."""
    a = _pools(S, cache, scale, slots, entries, z, z_cache)
    with torch.cuda.device(a["dev"]):
        _check("kata_state_store_q8", lib().kata_state_store_q8(
            a["S"], a["z"], a["n_slots"], a["cache"], a["scale"], a["z_cache"], a["n_entries"], a["slots"],
            a["entries"], a["n"], a["H"], a["rows"], a["dv"], _stream_ptr(stream)))


def kata_state_load_q8(cache, scale, S, entries=None, slots=None, z=None, z_cache=None, stream=None):
    """Read states back from the 8-bit cache: entry entries[i] to slot
    slots[i] of S (and z).  Several slots may be loaded from one entry."""
    a = _pools(S, cache, scale, slots, entries, z, z_cache)
    with torch.cuda.device(a["dev"]):
        _check("kata_state_load_q8", lib().kata_state_load_q8(
            a["cache"], a["scale"], a["z_cache"], a["n_entries"], a["S"], a["z"], a["n_slots"], a["entries"],
            a["slots"], a["n"], a["H"], a["rows"], a["dv"], _stream_ptr(stream)))
