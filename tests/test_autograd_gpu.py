"""What the calls on tensors write in place (states, outputs that are given) is
known to autograd: torch's version counter of it rises, and of nothing else.  And
the differentiable functions take a gradient from anywhere in memory."""
import pytest
import torch

import kernelized_feature_map_b200 as K

pytestmark = pytest.mark.gpu


def _x(*shape):
    return torch.randn(shape, device="cuda").to(torch.bfloat16)


def _calls():
    B, H, T, p, dv = 1, 2, 70, 16, 64
    q, k, v, o = _x(B, H, T, p), _x(B, H, T, p), _x(B, H, T, dv), torch.zeros(B, H, T, dv, device="cuda", dtype=torch.bfloat16)
    S, z = torch.zeros(B, H, p * p, dv, device="cuda"), torch.ones(B, H, p * p, device="cuda")
    D = torch.zeros(B, H, T, device="cuda")
    q1, k1, v1 = _x(B, H, p), _x(B, H, p), _x(B, H, dv)
    yield "quadratic", lambda: K.kata_fwd_quadratic(q, k, v, o=o), [q, k, v], [o]
    yield "train", lambda: K.kata_fwd_quadratic_train(q, k, v, o=o, D=D), [q, k, v], [o, D]
    yield "chunked", lambda: K.kata_fwd_chunked(q, k, v, S_out=S, z_out=z, return_state=True, o=o), [q, k, v], [S, z, o]
    yield "chunked from a state", lambda: K.kata_fwd_chunked(q, k, v, S0=S, z0=z, o=o), [q, S, z], [o]
    yield "decode", lambda: K.kata_decode_step(q1, k1, v1, S, z), [q1, k1, v1], [S, z]
    d, g = 32, 2
    qm, km = _x(B, H, d), _x(B, H, d)
    Sm, zm = torch.zeros(B, H, g * p * p, dv, device="cuda"), torch.ones(B, H, g * p * p, device="cuda")
    yield "decode mg", lambda: K.kata_decode_step_mg(qm, km, v1, Sm, zm, g), [qm, km, v1], [Sm, zm]
    yield "decode sg", lambda: K.kata_decode_step_sg(qm, km, v1, S, z, g), [qm, km, v1], [S, z]


def test_written_tensors_have_a_new_version():
    for name, call, read, wrote in _calls():
        before = [[t._version for t in ts] for ts in (read, wrote)]
        call()
        assert [t._version for t in read] == before[0], name
        assert all(t._version > v for t, v in zip(wrote, before[1])), name


def test_a_state_decoded_on_after_it_was_saved_is_an_error():
    q, k, v = _x(1, 2, 16), _x(1, 2, 16), _x(1, 2, 64)
    S, z = torch.zeros(1, 2, 256, 64, device="cuda"), torch.ones(1, 2, 256, device="cuda")
    w = torch.ones(1, 2, 256, 64, device="cuda", requires_grad=True)
    y = (w * S).sum()
    K.kata_decode_step(q, k, v, S, z)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_inference_tensors_have_no_version():
    q, k, v = _x(1, 2, 16), _x(1, 2, 16), _x(1, 2, 64)
    with torch.inference_mode():
        S, z = torch.zeros(1, 2, 256, 64, device="cuda"), torch.ones(1, 2, 256, device="cuda")
        K.kata_decode_step(q, k, v, S, z)
    K.kata_decode_step(q, k, v, S, z)
    assert S.any()


@pytest.mark.parametrize("path", ["flash", "chunked", "mg", "sg"])
def test_gradients_that_start_anywhere_in_memory(path):
    """The output behind a concatenation of flat tensors: its gradient is dense, but starts on 2 bytes."""
    B, H, T, dv = 1, 2, 150, 64
    d = 16 if path in ("flash", "chunked") else 32
    q, k, v = _x(B, H, T, d).requires_grad_(), _x(B, H, T, d).requires_grad_(), _x(B, H, T, dv).requires_grad_()
    o = {"flash": lambda: K.kata_attention(q, k, v), "chunked": lambda: K.kata_attention_chunked(q, k, v),
         "mg": lambda: K.kata_attention_mg(q, k, v, 2), "sg": lambda: K.kata_attention_sg(q, k, v, 2)}[path]()
    dO, pad = _x(B, H, T, dv), torch.zeros(3, dtype=torch.bfloat16, device="cuda")
    want = torch.autograd.grad(o, (q, k, v), dO, retain_graph=True)
    got = torch.autograd.grad(torch.cat([pad, o.flatten()]), (q, k, v), torch.cat([pad, dO.flatten()]))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
