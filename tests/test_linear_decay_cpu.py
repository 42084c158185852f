"""Linear attention with a per-head decay and the 8-bit state cache, without a
GPU: the oracle's two forms agree, its gradients are the derivatives, and the
entry points refuse bad arguments before anything is launched."""
import ctypes

import numpy as np
import pytest
import torch

import kernelized_feature_map_b200 as K
from kernelized_feature_map_b200 import _abi, build
from oracle import linear_decay as od

CU = [0, 0, 5, 6, 13]
G = np.array([0.0, -0.01, -0.7, -np.inf])


def _inputs(seed, d=3, dv=4, T=15, H=4):
    r = np.random.default_rng(seed)
    return (r.standard_normal((T, H, d)), r.standard_normal((T, H, d)), r.standard_normal((T, H, dv)),
            r.standard_normal((len(CU) - 1, H, d, dv)))


@pytest.mark.parametrize("state", [False, True])
def test_oracle_forms_agree(state):
    q, k, v, S0 = _inputs(0)
    S0 = S0 if state else None
    a, b = od.forward(q, k, v, G, CU, 0.3, S0), od.recurrent(q, k, v, G, CU, 0.3, S0)
    np.testing.assert_allclose(a[0], b[0], rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(a[1], b[1], rtol=1e-12, atol=1e-13)
    assert (a[0][13:] == 0).all()


def test_oracle_gradients_are_the_derivatives():
    q, k, v, S0 = _inputs(1)
    r = np.random.default_rng(2)
    dO, dS = r.standard_normal(v.shape), r.standard_normal(S0.shape)
    dO[13:] = 0

    def loss(q, k, v, S0):
        o, S = od.recurrent(q, k, v, G, CU, 0.3, S0)
        return (o * dO).sum() + (S * dS).sum()

    grads = od.backward(q, k, v, dO, G, CU, 0.3, S0, dS)
    args = [q, k, v, S0]
    for i, g in enumerate(grads):
        u = r.standard_normal(g.shape)
        up, dn = list(args), list(args)
        up[i], dn[i] = args[i] + 1e-4 * u, args[i] - 1e-4 * u
        # the loss is linear in each argument, so the difference is exact up to rounding
        assert (loss(*up) - loss(*dn)) / 2e-4 == pytest.approx((g * u).sum(), rel=1e-8, abs=1e-8)


def test_oracle_q8_rows():
    x = np.zeros((6, 4), np.float32)
    x[0] = [127, -63.5, 0.5, 1.5]       # scale 1: ties to even
    x[1] = [2.0 ** -127, 0, 0, 0]       # too small for a scale: held as zero
    x[2] = [np.inf, 1, 1, 1]
    x[3] = [np.nan, 1, 1, 1]
    x[4] = [3e38, -3e38, 1, 0]
    c, s = od.store_q8(x)
    assert c[0].tolist() == [127, -64, 0, 2] and s[0] == 1
    assert s[1] == 0 and np.isnan(s[2:4]).all() and (c[1:4] == 0).all()
    assert c[4].tolist() == [127, -127, 0, 0] and s[5] == 0
    back = od.load_q8(c, s)
    assert np.isnan(back[2:4]).all() and (back[1] == 0).all()
    assert np.abs(back[4] - x[4]).max() <= s[4] / 2


@pytest.fixture(scope="module")
def L():
    build.build()
    return _abi.lib()


P = ctypes.c_void_p(4096)    # never dereferenced: every call here is refused
ODD = ctypes.c_void_p(4104)


def _fwd(L, q=P, k=P, v=P, o=P, T=100, H=2, d=64, dv=128, qs=128, ks=128, vs=256, os=256, g=P, cu=P, N=3, S0=None,
         S_out=None, slots=None, n_slots=0, dt=1, ws=None, wsb=0):
    return L.kata_fwd_linear_decay(q, k, v, o, T, H, d, dv, qs, ks, vs, os, g, 1.0, cu, N, S0, S_out, slots, n_slots,
                                   None, 0, dt, ws, wsb, None)


@pytest.mark.parametrize("args,status", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(N=-1), 1), (dict(dt=7), 1), (dict(g=None), 1), (dict(q=None), 1),
    (dict(o=None), 1), (dict(cu=None), 1), (dict(n_slots=-1), 1), (dict(S0=P, n_slots=2), 1),
    (dict(S0=P, S_out=ctypes.c_void_p(4096 + 64), n_slots=3), 1), (dict(qs=127), 1), (dict(vs=128), 1),
    (dict(d=32), 2), (dict(dv=96), 2), (dict(d=256), 2), (dict(dt=0), 2), (dict(T=(1 << 30) + 1), 2),
    (dict(N=(1 << 20) + 1), 2), (dict(H=4097, qs=1 << 20, ks=1 << 20, vs=1 << 20, os=1 << 20), 2),
    (dict(ks=1 << 37), 2), (dict(q=ODD), 3), (dict(o=ODD), 3), (dict(ks=132), 3), (dict(os=257), 3),
    (dict(cu=ctypes.c_void_p(4098)), 3), (dict(S0=ODD, n_slots=3), 3),
])
def test_forward_refuses(L, args, status):
    assert _fwd(L, **args) == status


def test_empty_forward_is_a_no_op(L):
    assert _fwd(L, T=0) == 0 and _fwd(L, N=0) == 0 and _fwd(L, T=0, N=0) == 0


def _bwd(L, q=P, dO=P, dq=P, dv=P, T=100, H=2, d=64, w=128, qs=128, ks=128, vs=256, g=P, cu=P, N=3, S0=None, dS=None,
         dS0=None, dt=1):
    return L.kata_bwd_linear_decay(q, P, P, dO, dq, P, dv, T, H, d, w, qs, ks, vs, g, 1.0, cu, N, S0, dS, dS0, dt,
                                   None, 0, None)


@pytest.mark.parametrize("args,status", [
    (dict(T=-1), 1), (dict(H=0), 1), (dict(g=None), 1), (dict(dO=None), 1), (dict(dv=None), 1), (dict(cu=None), 1),
    (dict(qs=120), 1), (dict(dS=P, dS0=P), 1), (dict(S0=P, dS0=P), 1), (dict(d=16), 2), (dict(w=80), 2),
    (dict(dt=0), 2), (dict(dq=ODD), 3), (dict(vs=260), 3), (dict(dS0=ODD), 3),
])
def test_backward_refuses(L, args, status):
    assert _bwd(L, **args) == status


def _step(L, q=P, o=P, S=P, n=3, H=2, d=64, dv=128, qs=128, ks=128, vs=256, os=256, g=P, slots=None, n_slots=3, dt=1):
    return L.kata_decode_step_linear_decay(q, P, P, o, S, n, H, d, dv, qs, ks, vs, os, g, 1.0, slots, n_slots, dt,
                                           None)


@pytest.mark.parametrize("args,status", [
    (dict(n=-1), 1), (dict(H=0), 1), (dict(dt=3), 1), (dict(S=None), 1), (dict(g=None), 1), (dict(n_slots=2), 1),
    (dict(n_slots=-1, slots=P), 1), (dict(qs=64), 1), (dict(d=32), 2), (dict(dv=16), 2), (dict(S=ODD), 3),
    (dict(qs=132), 3), (dict(o=ODD), 3), (dict(slots=ctypes.c_void_p(4097)), 3), (dict(os=258, dt=0), 3),
])
def test_step_refuses(L, args, status):
    assert _step(L, **args) == status


def test_empty_step_is_a_no_op(L):
    assert _step(L, n=0) == 0


def _q8(L, load, S=P, z=None, n_slots=4, cache=P, scale=P, zc=None, n_entries=4, slots=P, entries=P, n=3, H=2, rows=64,
        dv=64):
    if load:
        return L.kata_state_load_q8(cache, scale, zc, n_entries, S, z, n_slots, entries, slots, n, H, rows, dv, None)
    return L.kata_state_store_q8(S, z, n_slots, cache, scale, zc, n_entries, slots, entries, n, H, rows, dv, None)


@pytest.mark.parametrize("load", [False, True])
@pytest.mark.parametrize("args,status", [
    (dict(n=-1), 1), (dict(H=0), 1), (dict(rows=0), 1), (dict(n_slots=-1), 1), (dict(z=P), 1), (dict(zc=P), 1),
    (dict(S=None), 1), (dict(cache=None), 1), (dict(scale=None), 1), (dict(slots=None, n=5), 1),
    (dict(entries=None, n=5), 1), (dict(dv=32), 2), (dict(dv=256), 2), (dict(n=65536), 2),
    (dict(H=1 << 16, rows=1 << 16), 2), (dict(S=ODD), 3), (dict(cache=ctypes.c_void_p(4098)), 3),
])
def test_q8_refuses(L, load, args, status):
    assert _q8(L, load, **args) == status


def test_empty_q8_is_a_no_op(L):
    assert _q8(L, False, n=0) == 0 and _q8(L, True, n=0) == 0


def test_workspace_queries(L):
    for f in (_abi.lib().kata_fwd_linear_decay_workspace_size, _abi.lib().kata_bwd_linear_decay_workspace_size):
        assert f(0, 2, 64, 64, 1) == 0 and f(100, 2, 64, 64, 0) == 0
        assert f(100, 2, 32, 64, 1) == 0 and f(-5, 2, 64, 64, 1) == 0
        assert f(100, 2, 64, 64, 1) == 0  # one short sequence needs no records


def test_binding_requires_cuda_tensors():
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    g = torch.zeros(2)
    with pytest.raises(TypeError):
        K.kata_fwd_linear_decay(x, x, x, g)
    with pytest.raises(TypeError):
        K.kata_bwd_linear_decay(x, x, x, x, g)
    with pytest.raises(TypeError):
        K.kata_decode_step_linear_decay(x, x, x, torch.zeros(4, 2, 64, 64), g)
    with pytest.raises(TypeError):
        K.kata_state_store_q8(torch.zeros(1, 1, 64, 64), torch.zeros(1, 1, 64, 64, dtype=torch.int8),
                              torch.zeros(1, 1, 64))
    with pytest.raises(ValueError):
        K.kata_attention_linear_decay(x, x, x, g.requires_grad_())


def test_plan_of_segments(L):
    """Through the workspace: short and many even sequences are not cut, long ones with few heads are; the records of
    a cut call are [segments, H, d, dv] fp32 for each walk."""
    size = L.kata_fwd_linear_decay_workspace_size
    assert size(75, 16, 64, 64, 1) == 0 and size(1337, 8, 64, 128, 5) == 0 and size(256, 1, 128, 128, 1) == 0
    one = size(131072, 16, 128, 128, 1)
    assert one > 0 and one % (16 * 128 * 128 * 4) == 0 and one // (16 * 128 * 128 * 4) <= 16
    assert size(9000, 1, 64, 64, 1) // (64 * 64 * 4) > 16  # enough segments for the scan
    assert L.kata_bwd_linear_decay_workspace_size(9000, 1, 64, 64, 1) >= 3 * 64 * 64 * 4
    assert size(-1, 1, 64, 64, 1) == 0 and size(100, 1, 32, 64, 1) == 0


def test_binding_refuses_host_tensors():
    build.build()
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    g, S = torch.zeros(2), torch.zeros(1, 2, 64, 64)
    for call in (lambda: K.kata_fwd_linear_decay(x, x, x, g), lambda: K.kata_bwd_linear_decay(x, x, x, x, g),
                 lambda: K.kata_decode_step_linear_decay(x, x, x, S, g),
                 lambda: K.kata_state_store_q8(S, S, S), lambda: K.kata_state_load_q8(S, S, S),
                 lambda: K.kata_fwd_linear_decay(None, x, x, g)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        K.kata_attention_linear_decay(x, x, x, g.requires_grad_())


def test_attention_needs_a_state_for_each_sequence():
    import kernelized_feature_map_b200 as K
    x = torch.zeros(8, 1, 64, dtype=torch.bfloat16)
    cu = torch.tensor([0, 5, 8], dtype=torch.int32)
    for states, edges in ((3, cu), (1, cu), (2, None)):
        with pytest.raises(ValueError, match="one state for each sequence"):
            K.kata_attention_linear_decay(x, x, x, torch.zeros(1), edges, S0=torch.zeros(states, 1, 64, 64))
