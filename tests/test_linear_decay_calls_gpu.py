"""Linear attention with a per-head decay and the 8-bit state cache: calls that
the documentation allows and that the other tests leave out."""
import numpy as np
import pytest
import torch

import kernelized_feature_map_b200 as K
from kernelized_feature_map_b200 import _abi
from oracle import linear_decay as od

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    from kernelized_feature_map_b200 import build
    build.build()
    torch.cuda.synchronize()
    K.kata_get_status()
    yield
    torch.cuda.synchronize()
    assert K.kata_get_status() == _abi.KATA_OK


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def bf(g, *shape):
    return torch.randn(shape, device="cuda", generator=g).to(torch.bfloat16)


def edges(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("lens", [[30, 170], [5000, 200]])
def test_a_fresh_state_for_each_sequence_from_a_larger_pool(lens):
    """S0 has more states than the call has sequences, and what the call allocates for S_out can lie right below it
    (where the allocator cuts both from the start of a free block)."""
    r, H, d, N = gen(0), 16, 128, len(lens)
    T, g, cu = sum(lens), torch.linspace(-0.5, 0, H, device="cuda"), edges(lens)
    q, k, v = (bf(r, T, H, d) for _ in range(3))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    block = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    del block
    below = torch.empty(N, H, d, d, device="cuda")
    S0 = torch.randn(N + 29, H, d, d, device="cuda", generator=r)
    few = S0[:N].clone()
    del below
    o, S = K.kata_fwd_linear_decay(q, k, v, g, cu, 0.1, S0=S0, return_state=True)
    assert S.shape == (N, H, d, d)
    want_o, want = K.kata_fwd_linear_decay(q, k, v, g, cu, 0.1, S0=few, return_state=True)
    assert torch.equal(S, want) and torch.equal(o, want_o)


def test_q8_rows_at_the_smallest_scales_are_exact():
    """Scales in [2^-126, 2^-125) with an odd significand, whose half is no fp32 value, and values on or next to the
    borders between two integers."""
    r = np.random.default_rng(3)
    rows, dv = 4096, 64
    x = np.zeros((rows, dv), np.float32)
    unit = 2.0 ** -149  # every value and scale here is a multiple of it
    for i in range(rows):
        s = (1 << 23) + 2 * int(r.integers(0, 1 << 22)) + 1
        k = r.integers(-126, 126, dv)
        y = ((2 * k + 1) * s) // 2 + r.integers(-1, 3, dv)  # (k + 1/2) s is an integer and a half
        x[i] = (y * unit).astype(np.float32)
        x[i, 0] = np.float32(127 * s * unit)
    c, s = od.store_q8(x)
    assert ((s >= 2.0 ** -126) & (s < 2.0 ** -125)).all() and (np.round(s / unit) % 2 == 1).mean() > 0.3
    cache = torch.empty((1, 1, rows, dv), dtype=torch.int8, device="cuda")
    scale = torch.empty((1, 1, rows), device="cuda")
    K.kata_state_store_q8(torch.from_numpy(x).cuda().view(1, 1, rows, dv), cache, scale)
    assert np.array_equal(scale.cpu().numpy()[0, 0], s)
    wrong = np.argwhere(cache.cpu().numpy()[0, 0] != c)
    assert not len(wrong), (len(wrong), wrong[:3])


def test_no_tokens_at_the_largest_number_of_heads():
    H, d = 4096, 128
    empty = [torch.empty(0, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    S0 = torch.randn(1, H, d, d, device="cuda", generator=gen(1))
    g = torch.zeros(H, device="cuda")
    _, S = K.kata_fwd_linear_decay(*empty[:3], g, S0=S0, return_state=True)
    assert torch.equal(S, S0)
    dS0 = K.kata_bwd_linear_decay(*empty, g, dS_out=S0, return_dS0=True)[3]
    assert torch.equal(dS0, S0)
    _, S = K.kata_fwd_linear_decay(*empty[:3], g, return_state=True)
    assert not S.any()


def test_what_a_call_writes_is_known_to_autograd():
    """A state saved for a backward pass and written since is an error there, as with torch's own operations, and not
    a wrong gradient; what is only read keeps its version."""
    r, H, d = gen(2), 2, 64
    x, g = bf(r, 5, H, d), torch.full((H,), -0.1, device="cuda")
    S = torch.randn(3, H, d, d, device="cuda", generator=r)
    z, zc, sc = (torch.zeros(3, H, d, device="cuda") for _ in range(3))
    cache, o = torch.zeros(3, H, d, d, dtype=torch.int8, device="cuda"), torch.zeros_like(x)
    calls = [
        (lambda: K.kata_fwd_linear_decay(x, x, x, g, S0=S, return_state=True), []),
        (lambda: K.kata_fwd_linear_decay(x, x, x, g, S0=S, S_out=S, o=o), [S, o]),
        (lambda: K.kata_decode_step_linear_decay(x[:3], x[:3], x[:3], S, g), [S]),
        (lambda: K.kata_decode_step_linear_decay(x[:3], x[:3], x[:3], S, g, o=o[:3]), [S, o]),
        (lambda: K.kata_state_store_q8(S, cache, sc, z=z, z_cache=zc), [cache, sc, zc]),
        (lambda: K.kata_state_load_q8(cache, sc, S, z=z, z_cache=zc), [S, z]),
        (lambda: K.kata_bwd_linear_decay(x, x, x, x, g, S0=S[:1], dS_out=S[:1]), []),
    ]
    every = [x, g, S, z, zc, sc, cache, o]
    for call, wrote in calls:
        before = [t._version for t in every]
        call()
        for t, v in zip(every, before):
            assert (t._version > v) == any(t is w for w in wrote)
    q, k, v = (bf(r, 5, H, d).requires_grad_() for _ in range(3))
    S0 = torch.randn(1, H, d, d, device="cuda", generator=r)
    y = K.kata_attention_linear_decay(q, k, v, g, S0=S0)
    K.kata_decode_step_linear_decay(x[:1], x[:1], x[:1], S0, g)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():
        T = torch.zeros(3, H, d, d, device="cuda")
    K.kata_decode_step_linear_decay(x[:3], x[:3], x[:3], T, g)  # inference tensors have no version
    with torch.inference_mode():
        K.kata_decode_step_linear_decay(x[:3], x[:3], x[:3], T, g)
    assert T.any()


def test_gradients_that_start_anywhere_in_memory():
    """The outputs behind a concatenation of flat tensors: their gradients are dense, but start on 2 or 4 bytes."""
    r, H, d, cu = gen(4), 2, 64, edges([20, 30])
    q, k, v = (bf(r, 50, H, d).requires_grad_() for _ in range(3))
    S0 = torch.randn(2, H, d, d, device="cuda", generator=r).requires_grad_()
    g, leaves = torch.full((H,), -0.1, device="cuda"), (q, k, v, S0)
    o, S = K.kata_attention_linear_decay(q, k, v, g, cu, 0.1, S0=S0, return_state=True)
    dO, dS = bf(r, 50, H, d), torch.randn(2, H, d, d, device="cuda", generator=r)
    want = torch.autograd.grad((o, S), leaves, (dO, dS), retain_graph=True)
    flat = [torch.cat([torch.zeros(3, dtype=t.dtype, device="cuda"), t.flatten()]) for t in (o, S)]
    up = [torch.cat([torch.zeros(3, dtype=t.dtype, device="cuda"), t.flatten()]) for t in (dO, dS)]
    got = torch.autograd.grad(flat, leaves, up)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_states_behind_two_to_the_31_elements():
    """The last slots of a pool, and entries of a cache, of more elements than 32 bits count."""
    n, H, d = 140000, 1, 128
    r, last = gen(6), n - 1
    pool = torch.empty(n, H, d, d, device="cuda")
    cache, scale = torch.empty(n, H, d, d, dtype=torch.int8, device="cuda"), torch.empty(n, H, d, device="cuda")
    z, zc = torch.empty(n, H, d, device="cuda"), torch.empty(n, H, d, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    first = torch.randn(1, H, d, d, device="cuda", generator=r)
    pool[last - 1], z[last - 1] = first[0], first[0, :, :, 0]
    K.kata_state_store_q8(pool, cache, scale, slots=i32(last - 1), entries=i32(last), z=z, z_cache=zc)
    K.kata_state_load_q8(cache, scale, pool, entries=i32(last), slots=i32(last), z=z, z_cache=zc)
    small = [torch.empty_like(t[:1]) for t in (cache, scale, pool)]
    K.kata_state_store_q8(first, small[0], small[1])
    K.kata_state_load_q8(small[0], small[1], small[2])
    assert torch.equal(cache[last], small[0][0]) and torch.equal(pool[last], small[2][0])
    assert torch.equal(z[last], first[0, :, :, 0])
    g, S = torch.tensor([-0.1], device="cuda"), small[2].clone()
    x = [bf(r, 1, H, d) for _ in range(3)]
    o = K.kata_decode_step_linear_decay(*x, pool, g, slots=i32(last))
    assert torch.equal(o, K.kata_decode_step_linear_decay(*x, S, g)) and torch.equal(pool[last], S[0])
    for T in (50, 5000):  # whole, and cut
        x = [bf(r, T, H, d) for _ in range(3)]
        o = K.kata_fwd_linear_decay(*x, g, scale=0.1, S0=pool, S_out=pool, slots=i32(last))
        want, S = K.kata_fwd_linear_decay(*x, g, scale=0.1, S0=S, return_state=True)
        assert torch.equal(o, want) and torch.equal(pool[last], S[0])


def test_tokens_behind_two_to_the_31_elements():
    """Parts of a projection so wide that the last tokens lie behind 2^31 elements, and an output likewise."""
    T, H, d, wide = 3001, 1, 64, 1 << 20
    r, cu = gen(7), edges([2900, 1, 100])
    rows = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")
    parts = [rows[:, 64 * i:64 * i + 64].view(T, H, d) for i in (0, 1, 16000, 5)]
    dense = [bf(r, T, H, d) for _ in range(3)]
    for t, x in zip(parts, dense):
        t.copy_(x)
    g = torch.tensor([-0.01], device="cuda")
    o = K.kata_fwd_linear_decay(*parts[:3], g, cu, 0.1, o=parts[3])
    assert torch.equal(o, K.kata_fwd_linear_decay(*dense, g, cu, 0.1))
    assert all(torch.equal(t, x) for t, x in zip(parts, dense))
    dO = bf(r, T, H, d)
    got = K.kata_bwd_linear_decay(*parts[:3], dO, g, cu, 0.1)
    assert all(torch.equal(a, b) for a, b in zip(got, K.kata_bwd_linear_decay(*dense, dO, g, cu, 0.1)))
    o1 = K.kata_decode_step_linear_decay(*parts[:3], torch.zeros(T, H, d, d, device="cuda"), g)
    assert torch.equal(o1, K.kata_decode_step_linear_decay(*dense, torch.zeros(T, H, d, d, device="cuda"), g))
