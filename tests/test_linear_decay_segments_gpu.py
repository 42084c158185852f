"""Linear attention with a per-head decay where sequences are cut into segments,
at the widths and calls that the small cases leave out, against the formulas in
64 bits.

The plan cuts sequences longer than an even share of the work.  With few
segments each walk sums the records before its own; with many (one head, 9000
tokens: 35 segments) a scan does.  Tolerances as for the small cases: u = 2^-8
of the value and 1.02 u of the terms' magnitudes for a bf16 output, u relative
in the 2-norm; 2^-15 of the terms' magnitudes and 1e-5 in the 2-norm for a
state.
"""
import numpy as np
import pytest
import torch

import kernelized_feature_map_b200 as K
from kernelized_feature_map_b200 import _abi

pytestmark = pytest.mark.gpu

U = 2.0 ** -8


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


def bf(g, *shape, std=1.0):
    return (torch.randn(shape, device="cuda", generator=g) * std).to(torch.bfloat16)


def decays(H):
    ks = [np.log1p(-2.0 ** -5), -0.5, np.log1p(-2.0 ** -12), 0.0, -30.0]
    return torch.tensor([ks[h % 5] for h in range(H)], dtype=torch.float32, device="cuda")


def attend(q, k, v, g, scale, S0):
    """(o, S, |.| of the terms of o, of S) of one sequence in fp64; [x, H, *] in, S0 [H, d, dv]."""
    out = []
    for f in (lambda t: t.double(), lambda t: t.double().abs()):
        Q, Kk, V, S = f(q).transpose(0, 1), f(k).transpose(0, 1), f(v).transpose(0, 1), f(S0)
        x = q.shape[0]
        t = torch.arange(x, device="cuda", dtype=torch.float64)
        gg = g.double()[:, None]
        o = torch.exp(gg * (t + 1))[..., None] * (Q @ S)
        step = max(64, int(2e7 // max(1, x * q.shape[1])))
        for a in range(0, x, step):
            b = min(x, a + step)
            away = t[a:b, None] - t[None, :b]
            w = torch.exp(gg[..., None] * away.clamp(min=0)) * (away >= 0)
            o[:, a:b] += (Q[:, a:b] @ Kk[:, :b].transpose(1, 2) * w) @ V[:, :b]
        S1 = torch.exp(gg * x)[..., None] * S + (Kk * torch.exp(gg * (x - 1 - t))[..., None]).transpose(1, 2) @ V
        out += [abs(scale) * o.transpose(0, 1) if len(out) else scale * o.transpose(0, 1), S1]
    return out


def close_bf16(got, want, mag):
    got = got.double()
    assert torch.isfinite(got).all()
    bad = (got - want).abs() > U * want.abs() + 1.02 * U * mag + 1e-30
    assert not bad.any(), (bad.nonzero()[:3], got[bad][:3], want[bad][:3])
    if want.numel() > 1000:
        assert torch.linalg.norm(got - want) <= U * torch.linalg.norm(want)


def close_state(got, want, mag):
    got = got.double()
    assert torch.isfinite(got).all()
    assert ((got - want).abs() <= 2.0 ** -15 * mag + 1e-30).all()
    assert torch.linalg.norm(got - want) <= 1e-5 * torch.linalg.norm(want) + 1e-30


def edges(lens, before=0):
    return torch.tensor(np.concatenate([[before], before + np.cumsum(lens)]), dtype=torch.int32, device="cuda")


# one head and a long sequence: scanned; more heads, or several sequences: each walk sums the records before its own
CUT = [(1, 128, 128, [9000]), (8, 128, 128, [3001]), (3, 128, 64, [2500, 0, 700, 4097, 1]), (16, 64, 128, [4000, 30] * 3),
       (2, 64, 64, [64] * 40 + [6000] + [1] * 40 + [5000])]


@pytest.mark.parametrize("H,d,dv,lens", CUT)
@pytest.mark.parametrize("in_place", [True, False])
def test_prompt_cut(H, d, dv, lens, in_place):
    """States go in and out of a pool larger than the call, some sequences fresh, one without a slot; rows of padding
    before and behind hold NaN and keep what o held."""
    r, N = gen(H + d), len(lens)
    T = sum(lens) + 9
    q, k, v = bf(r, T, H, d), bf(r, T, H, d), bf(r, T, H, dv)
    for t in (q, k, v):
        t[:4] = t[T - 5:] = float("nan")
    pool = torch.randn(N + 3, H, d, dv, device="cuda", generator=r) * 3
    out = pool if in_place else torch.full_like(pool, 9.0)
    before = pool.clone()
    perm = np.random.default_rng(N).permutation(N + 3)[:N].tolist()
    resume = [n % 3 != 1 for n in range(N)]
    if N > 3:
        perm[2] = -1
    o = torch.full((T, H, dv), 5.0, dtype=torch.bfloat16, device="cuda")
    g = decays(H)
    K.kata_fwd_linear_decay(q, k, v, g, edges(lens, 4), 0.125, S0=pool, S_out=out,
                            slots=torch.tensor(perm, dtype=torch.int32, device="cuda"),
                            resume=torch.tensor(resume, dtype=torch.uint8, device="cuda"), o=o)
    a = 4
    for n, x in enumerate(lens):
        s = perm[n]
        S0 = before[s] if s >= 0 and resume[n] else torch.zeros_like(before[0])
        want, S1, mag, Sm = attend(q[a:a + x], k[a:a + x], v[a:a + x], g, 0.125, S0)
        close_bf16(o[a:a + x], want, mag)
        if s >= 0:
            close_state(out[s], S1, Sm)
        a += x
    assert (o[:4] == 5).all() and (o[T - 5:] == 5).all()
    for s in set(range(N + 3)) - set(perm):
        assert torch.equal(out[s], before[s]) if in_place else (out[s] == 9).all()


@pytest.mark.parametrize("H,d,dv,lens", [(1, 128, 128, [4500]), (4, 128, 64, [1500, 0, 900, 3]), (2, 64, 128, [5000, 5])])
def test_gradients_cut(H, d, dv, lens):
    r, N, T = gen(7 * H + d), len(lens), sum(lens) + 3
    q, k, v, dO = bf(r, T, H, d), bf(r, T, H, d), bf(r, T, H, dv), bf(r, T, H, dv)
    for t in (q, k, v, dO):
        t[T - 3:] = float("nan")
    S0, dS = (torch.randn(N, H, d, dv, device="cuda", generator=r) for _ in range(2))
    g = decays(H)
    got = K.kata_bwd_linear_decay(q, k, v, dO, g, edges(lens), 0.3, S0=S0, dS_out=dS, return_dS0=True)
    assert all((x[T - 3:] == 0).all() for x in got[:3])
    a = 0
    for n, x in enumerate(lens):
        part = slice(a, a + x)
        a += x
        Q, Kk, V, D = (t[part] for t in (q, k, v, dO))
        # dq: the walk of (dO, v, k) from S0^T; dk and dv backwards from dS / a, which joins unscaled
        tr = lambda S: S.transpose(1, 2).contiguous()  # noqa: E731
        want, _, mag, _ = attend(D, V, Kk, g, 0.3, tr(S0[n]))
        close_bf16(got[0][part], want, mag)
        flip = lambda t: t.flip(0)  # noqa: E731
        R = dS[n].double() / torch.exp(g.double())[:, None, None] / 0.3
        live = torch.isfinite(R).all() and (g > -20).all()
        if not live:  # a^-1 overflows what the reference can hold: those heads without it
            keep = g > -20
            Q, Kk, V, D, R, gg = Q[:, keep], Kk[:, keep], V[:, keep], D[:, keep], R[keep], g[keep]
        else:
            keep, gg = torch.ones_like(g, dtype=torch.bool), g
        want, _, mag, _ = attend(flip(V), flip(D), flip(Q), gg, 0.3, tr(R))
        close_bf16(got[1][part][:, keep], flip(want), flip(mag))
        want, R1, mag, Rm = attend(flip(Kk), flip(Q), flip(D), gg, 0.3, R)
        close_bf16(got[2][part][:, keep], flip(want), flip(mag))
        a1 = 0.3 * torch.exp(gg.double())[:, None, None]
        close_state(got[3][n][keep], a1 * R1, a1 * Rm)


def test_states_and_out_on_sixteen_bytes():
    """Pools and outputs that start on 16 bytes, but on no larger boundary."""
    H, d, dv, lens = 2, 64, 128, [200, 128, 5]
    r, T = gen(3), 333
    q, k, v, g = bf(r, T, H, d), bf(r, T, H, d), bf(r, T, H, dv), decays(H)
    S0 = torch.randn(3, H, d, dv, device="cuda", generator=r)
    flat = torch.zeros(S0.numel() + 4, device="cuda")
    odd = flat[4:].view_as(S0).copy_(S0)
    wide = torch.zeros(T * H * dv + 8, dtype=torch.bfloat16, device="cuda")
    o1, S1 = K.kata_fwd_linear_decay(q, k, v, g, edges(lens), 0.2, S0=S0, return_state=True)
    o2 = K.kata_fwd_linear_decay(q, k, v, g, edges(lens), 0.2, S0=odd, S_out=odd, o=wide[8:].view(T, H, dv))
    assert torch.equal(o1, o2) and torch.equal(S1, odd) and (flat[:4] == 0).all() and (wide[:8] == 0).all()


@pytest.mark.parametrize("scale", [0.0, -0.5])
def test_scale(scale):
    r = gen(4)
    q, k, v, dO = (bf(r, 150, 2, 64) for _ in range(4))
    g = decays(2)
    o = K.kata_fwd_linear_decay(q, k, v, g, None, scale)
    grads = K.kata_bwd_linear_decay(q, k, v, dO, g, None, scale)
    one = K.kata_fwd_linear_decay(q, k, v, g, None, 1.0)
    # the scale enters before a rounding or after one: u for each of the two outputs
    assert ((o.double() - scale * one.double()).abs() <= 2 * U * abs(scale) * one.double().abs()
            + 2.04 * U * abs(scale) * attend(q, k, v, g, 1.0, torch.zeros(2, 64, 64, device="cuda"))[2]).all()
    if scale == 0:
        assert (o == 0).all() and all((x == 0).all() for x in grads)


def test_what_masked_tokens_hold_does_not_matter():
    """Infinities, NaN and the type's extremes in the next sequence, in the same tile, at the largest and smallest
    lengths of a tail."""
    g = decays(2)
    for x in (1, 63, 64, 127, 129, 255):
        r = gen(x)
        q, k, v, dO = (bf(r, x + 140, 2, 128) for _ in range(4))
        clean = [K.kata_fwd_linear_decay(q, k, v, g, edges([x, 140]), 0.1)[:x]]
        clean += [t[:x] for t in K.kata_bwd_linear_decay(q, k, v, dO, g, edges([x, 140]), 0.1)]
        for bad in (float("inf"), float("nan"), torch.finfo(torch.bfloat16).min):
            for t in (q, k, v, dO):
                t[x:] = bad
            got = [K.kata_fwd_linear_decay(q, k, v, g, edges([x, 140]), 0.1)[:x]]
            got += [t[:x] for t in K.kata_bwd_linear_decay(q, k, v, dO, g, edges([x, 140]), 0.1)]
            assert all(torch.equal(a, b) for a, b in zip(clean, got))


@pytest.mark.parametrize("lens", [[300, 20], [9000]])
def test_short_wait_limit_reports_timeout_then_recovers(lens):
    """A wait that runs out ends its CTA's work, and the next call is whole again (one launch; sums and walks)."""
    r, T = gen(5), sum(lens)
    q, k, v, dO = (bf(r, T, 1, 128) for _ in range(4))
    g = decays(1)
    run = lambda: (K.kata_fwd_linear_decay(q, k, v, g, edges(lens), 0.1),  # noqa: E731
                   *K.kata_bwd_linear_decay(q, k, v, dO, g, edges(lens), 0.1))
    want = run()
    torch.cuda.synchronize()
    assert K.kata_get_status() == _abi.KATA_OK
    try:
        K.kata_set_wait_limit(0)
        K.kata_fwd_linear_decay(q, k, v, g, edges(lens), 0.1)
        assert K.kata_get_status() == _abi.KATA_ERR_TIMEOUT
        K.kata_bwd_linear_decay(q, k, v, dO, g, edges(lens), 0.1)
        assert K.kata_get_status() == _abi.KATA_ERR_TIMEOUT
    finally:
        K.kata_set_wait_limit(-1)
    assert all(torch.equal(a, b) for a, b in zip(want, run()))
    assert K.kata_get_status() == _abi.KATA_OK


def test_backward_captured():
    """The gradients captured into a CUDA graph (eager autograd graphs of the leaves released before, as torch asks)
    and replayed with new inputs."""
    r = gen(6)
    q, k, v = (bf(r, 300, 2, 64).requires_grad_() for _ in range(3))
    g, cu = decays(2), edges([100, 200])
    dO = bf(r, 300, 2, 64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm-up on the capture's kind of stream
        torch.autograd.grad(K.kata_attention_linear_decay(q, k, v, g, cu, 0.1), (q, k, v), dO)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = K.kata_attention_linear_decay(q, k, v, g, cu, 0.1)
        grads = torch.autograd.grad(o, (q, k, v), dO)
    with torch.no_grad():
        q.copy_(bf(gen(8), 300, 2, 64))
    graph.replay()
    torch.cuda.synchronize()
    want = K.kata_bwd_linear_decay(q.detach(), k.detach(), v.detach(), dO, g, cu, 0.1)
    assert all(torch.equal(a, b) for a, b in zip(grads, want))
    assert torch.equal(o.detach(), K.kata_fwd_linear_decay(q.detach(), k.detach(), v.detach(), g, cu, 0.1))


def test_calls_on_two_streams_at_once():
    """Calls with workspaces of their own do not meet, whatever runs beside them."""
    r, H, lens = gen(9), 2, [6000, 10, 900]
    T, g, cu = sum(lens), decays(2), edges(lens)
    sets = [tuple(bf(r, T, H, 64) for _ in range(3)) for _ in range(2)]
    want = [K.kata_fwd_linear_decay(*s, g, cu, 0.1, return_state=True) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i].append(K.kata_fwd_linear_decay(*sets[i], g, cu, 0.1, return_state=True))
    torch.cuda.synchronize()
    for i in range(2):
        for o, S in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(S, want[i][1])


def test_chain_of_launches_that_overlap():
    """Each call's kernels may start before the call before them ends: they must still see its results."""
    H, d, dv, n = 16, 128, 128, 8
    r, g = gen(10), decays(16)
    pool = torch.zeros(n, H, d, dv, device="cuda")
    cache = torch.zeros(n, H, d, dv, dtype=torch.int8, device="cuda")
    sc = torch.zeros(n, H, d, device="cuda")
    x = [bf(r, n, H, w) for w in (d, d, dv)]
    prompts = [bf(r, 40 * n, H, w) for w in (d, d, dv)]
    idx = torch.arange(n, dtype=torch.int32, device="cuda")
    cu = edges([40] * n)

    def run(sync):
        pool.zero_()
        outs = []
        for _ in range(6):
            for f in (lambda: K.kata_fwd_linear_decay(*prompts, g, cu, 0.1, S0=pool, S_out=pool, slots=idx),
                      lambda: K.kata_decode_step_linear_decay(*x, pool, g, slots=idx, scale=0.1),
                      lambda: K.kata_state_store_q8(pool, cache, sc, idx, idx),
                      lambda: K.kata_state_load_q8(cache, sc, pool, idx, idx)):
                y = f()
                if y is not None:
                    outs.append(y)
                if sync:
                    torch.cuda.synchronize()
        return outs + [pool.clone(), cache.clone(), sc.clone()]

    want = run(True)
    for _ in range(3):
        got = run(False)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("call", ["prompt", "gradients", "step"])
def test_what_a_given_stream_writes_is_its_own(call):
    """A call on another stream than the current one gets no memory that work
    queued on the current one still reads (a block let go there may be handed
    out again there at once, but not elsewhere)."""
    r, T, H, d = gen(31), 512, 16, 128
    q, k, v, dO = (bf(r, T, H, d) for _ in range(4))
    g, S = decays(H), torch.zeros(2, T, H, d, d, device="cuda") if call == "step" else None
    other = torch.cuda.Stream()
    torch.cuda.synchronize()

    def run(pool, **kw):
        if call == "prompt":
            return K.kata_fwd_linear_decay(q, k, v, g, scale=0.1, return_state=True, **kw)
        if call == "gradients":
            return K.kata_bwd_linear_decay(q, k, v, dO, g, scale=0.1, return_dS0=True, **kw)
        return (K.kata_decode_step_linear_decay(q, k, v, S[pool], g, scale=0.1, **kw),)

    want = run(0)
    blocks = [torch.full_like(t, 3.0) for t in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    copies = [b.clone() for b in blocks]
    del blocks
    got = run(1, stream=other)
    torch.cuda.synchronize()
    assert all(bool((c == 3.0).all()) for c in copies)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
