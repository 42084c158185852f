"""Calls of linear attention with a per-head decay that their documentation
allows, or that are to be refused, at the C ABI and without a GPU: every call
here is refused before anything is launched, and the status says by which
check."""
import ctypes

import pytest

from kernelized_feature_map_b200 import _abi, build

INVALID, UNSUPPORTED, MISALIGNED = 1, 2, 3
BASE = 1 << 32  # never dereferenced
P = ctypes.c_void_p(BASE)


@pytest.fixture(scope="module")
def L():
    build.build()
    return _abi.lib()


def _fwd(L, N=3, S0=None, S_out=None, slots=None, n_slots=0, H=2, d=64, dv=128, T=100, ks=132):
    """A forward whose keys' stride is misaligned unless it is given: the check behind those of the sizes and states."""
    return L.kata_fwd_linear_decay(P, P, P, P, T, H, d, dv, H * d, ks, H * dv, H * dv, P, 1.0, P, N, S0, S_out, slots,
                                   n_slots, None, 0, 1, None, 0, None)


@pytest.mark.parametrize("rows", [3, 8])
def test_states_of_one_call_may_lie_next_to_each_other(L, rows):
    """Without slots a call touches the first N rows of a pool: a fresh pool of N = 3 states `rows` states below S0
    does not overlap it, although S0 has nine."""
    state = 2 * 64 * 128 * 4
    S0, fresh = ctypes.c_void_p(BASE + rows * state), ctypes.c_void_p(BASE)
    assert _fwd(L, S0=S0, S_out=fresh, n_slots=9) == MISALIGNED
    assert _fwd(L, S0=fresh, S_out=S0, n_slots=9) == MISALIGNED
    # two states away the third row is shared; and with slots any of the nine may be
    assert _fwd(L, S0=ctypes.c_void_p(BASE + 2 * state), S_out=fresh, n_slots=9) == INVALID
    assert _fwd(L, S0=S0, S_out=fresh, n_slots=9, slots=P) == INVALID


def test_calls_whose_search_would_hold_the_gpu_are_refused(L):
    """The time of a call grows with the square of its sequences or streams; a call of a million would take minutes."""
    assert _fwd(L, N=1 << 15, H=16, ks=16 * 64 + 4) == MISALIGNED  # half of the bound
    assert _fwd(L, N=1 << 16, H=16, ks=16 * 64 + 4) == UNSUPPORTED
    assert _fwd(L, N=1 << 20, H=1, ks=68) == UNSUPPORTED

    def bwd(N, H):
        return L.kata_bwd_linear_decay(P, P, P, P, P, P, P, 100, H, 64, 64, H * 64, H * 64 + 4, H * 64, P, 1.0, P, N,
                                       None, None, None, 1, None, 0, None)

    assert bwd(1 << 14, 16) == MISALIGNED and bwd(1 << 15, 16) == UNSUPPORTED

    def step(n, H, dv, slots):
        return L.kata_decode_step_linear_decay(P, P, P, P, P, n, H, 64, dv, H * 64, H * 64 + 2, H * dv, H * dv, P, 1.0,
                                               slots, n, 1, None)

    assert step(1 << 16, 16, 128, P) == MISALIGNED and step(1 << 20, 16, 128, P) == UNSUPPORTED
    assert step(1 << 20, 16, 128, None) == MISALIGNED
    assert step(1 << 20, 1, 64, P) == MISALIGNED
    # what is refused needs no workspace, and a long call of one sequence is not refused
    assert L.kata_fwd_linear_decay_workspace_size(1 << 22, 16, 64, 64, 1 << 16) == 0
    assert L.kata_fwd_linear_decay_workspace_size(1 << 22, 16, 64, 64, 1) > 0
