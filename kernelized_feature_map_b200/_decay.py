"""Linear attention with a per-head decay and the 8-bit state cache: the
functions a user calls.  Argument checks and marshalling to the C ABI
(include/kata.h) are compiled, in csrc/binding.cpp.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from ._abi import KataError, _upstream, lib

_native = None


def _load():
    """The compiled binding (raises if it has not been built)."""
    global _native
    lib()
    try:
        from . import _binding
    except ImportError as e:
        raise RuntimeError("the binding is not built or does not fit this torch (run: python -m "
                           "kernelized_feature_map_b200.build --force); there is no fallback path: %s" % e) from e
    _binding.set_error(KataError)
    _native = _binding
    return _native


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
    zero_outside is true (None: when o is allocated here).  The last two
    dimensions of q, k, v and o are dense; the stride between tokens is free (a
    multiple of 16 bytes), so the parts of a fused projection go in as they
    are.  All tensors are on one device, which need not be the current one.
    With stream (a torch.cuda.Stream) the call runs there instead of on the
    current stream, and what it allocates belongs to that stream; the caller
    keeps its own tensors until the call has run there (record_stream).
    S_out and o, where given, are written in place, which autograd learns.
    """
    return (_native or _load()).fwd(q, k, v, log_decay, cu_seqlens, scale, S0, S_out, slots, resume, return_state,
                                    zero_outside, o, workspace, stream)


def kata_bwd_linear_decay(q, k, v, dO, log_decay, cu_seqlens=None, scale=1.0, S0=None, dS_out=None,
                          return_dS0=False, workspace=None, stream=None):
    """Gradients (dq, dk, dv), or (dq, dk, dv, dS0) with return_dS0=True, of
    kata_fwd_linear_decay for dO [T,H,dv] and the gradient dS_out of the final
    states; S0, dS_out, dS0 are [N,H,d,dv] fp32.  Rows outside every sequence
    get zeros; the decays get no gradient."""
    return (_native or _load()).bwd(q, k, v, dO, log_decay, cu_seqlens, scale, S0, dS_out, return_dS0, workspace,
                                    stream)


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
        dO = torch.zeros(v.shape, dtype=v.dtype, device=v.device) if dO is None else _upstream(dO)
        want = S0 is not None and ctx.needs_input_grad[6]
        g = kata_bwd_linear_decay(q, k, v, dO, log_decay, cu_seqlens, ctx.scale, S0=S0,
                                  dS_out=_upstream(dS), return_dS0=want)
        return g[0], g[1], g[2], None, None, None, (g[3] if want else None), None


def kata_attention_linear_decay(q, k, v, log_decay, cu_seqlens=None, scale=1.0, S0=None, return_state=False):
    """Differentiable linear attention with a per-head decay over packed
    sequences, q,k [T,H,d], v [T,H,dv] (bf16); S0 [N,H,d,dv] fp32.  Returns o,
    or (o, S_out) with return_state=True; gradients reach q, k, v and S0.  To
    capture the backward pass into a CUDA graph, release eager autograd graphs
    of the same leaves first: torch ties a leaf's accumulation to the stream of
    the first graph that is alive, and refuses the capture otherwise."""
    if isinstance(log_decay, torch.Tensor) and log_decay.requires_grad:
        raise ValueError("log_decay gets no gradient: pass log_decay.detach()")
    if S0 is not None and S0.shape[0] != (1 if cu_seqlens is None else cu_seqlens.shape[0] - 1):
        raise ValueError("S0 must have one state for each sequence")
    return KataAttentionLinearDecay.apply(q, k, v, log_decay, cu_seqlens, scale, S0, return_state)


def kata_decode_step_linear_decay(q, k, v, S, log_decay, slots=None, scale=1.0, o=None, stream=None):
    """One token for each of n streams: S <- exp(log_decay) S + k v^T and
    o = scale * q^T S, in place on the pool S [n_slots,H,d,dv] fp32.  q,k
    [n,H,d], v [n,H,dv] (bf16 or fp32); slots [n] int32 names each stream's
    row (None: row i; negative: padding, whose row of o is zero)."""
    return (_native or _load()).step(q, k, v, S, log_decay, slots, scale, o, stream)


def kata_state_store_q8(S, cache, scale, slots=None, entries=None, z=None, z_cache=None, stream=None):
    """Write states to the 8-bit cache: slot slots[i] of S [n_slots,H,rows,dv]
    fp32 to entry entries[i] of cache [n_entries,H,rows,dv] int8 and scale
    [n_entries,H,rows] fp32, each row as round(x / scale) with scale =
    max|x| / 127; z [n_slots,H,rows] is copied to z_cache.  slots and entries
    are int32 (None: 0, 1, ...); a negative index skips its pair."""
    (_native or _load()).store(S, cache, scale, slots, entries, z, z_cache, stream)


def kata_state_load_q8(cache, scale, S, entries=None, slots=None, z=None, z_cache=None, stream=None):
    """Read states back from the 8-bit cache: entry entries[i] to slot
    slots[i] of S (and z).  Several slots may be loaded from one entry."""
    (_native or _load()).load(cache, scale, S, entries, slots, z, z_cache, stream)
