"""Linear attention with a per-head decay on packed sequences (prompts,
gradients, single tokens) and the 8-bit cache of its states, against the fp64
oracle.

Tolerances, u = 2^-8 being half a bf16 step relative to the value:
* a bf16 output: u for its own rounding, and u of the terms' magnitudes for
  each of the rounded factors (the weights inside a chunk, the copy of the
  state that the query meets, of which a term meets one): elementwise
  u |o| + 1.02 u M with M the sum of the terms' magnitudes.  Relative to the
  2-norm the roundings are independent and at most u / sqrt(3) each: u.
* an fp32 state: k times its decay is held as two bf16 values, off by at most
  u^2 = 2^-16 relative, 2^-16 / 3 in the mean square; with the fp32 sums
  elementwise 2^-15 M and 1e-5 relative to the 2-norm.  (Three values where the
  state that leaves holds a 16th or more of them: test_linear_decay_exact_gpu.py
  has the closer bound.)
* one token in fp32: a few roundings of 2^-24; the sums over up to 128 terms
  (in the state, over the steps walked) 2^-24 each: 128 * 2^-24 M.
"""
import numpy as np
import pytest
import torch

import kernelized_feature_map_b200 as K
from kernelized_feature_map_b200 import _abi
from oracle import linear_decay as od

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
DIMS = [(64, 64), (64, 128), (128, 64), (128, 128)]
# lengths of the packed sequences; the third number in each is what stands before and behind them
PACKS = {
    "one": ([1], 0, 0),
    "two": ([2], 0, 3),
    "tile-1": ([127], 0, 0),
    "tile": ([128], 0, 1),
    "tile+1": ([129], 2, 0),
    "empties": ([0, 1, 0, 0, 130, 0], 0, 5),
    "ragged": ([5, 128, 257, 1, 300, 64], 7, 9),
    "many": ([3] * 70 + [0] * 5 + [140], 0, 0),
}


@pytest.fixture(scope="module", autouse=True)
def library():
    from kernelized_feature_map_b200 import build
    build.build()
    assert torch.cuda.is_available()
    torch.cuda.synchronize()
    K.kata_get_status()
    yield
    torch.cuda.synchronize()
    assert K.kata_get_status() == _abi.KATA_OK


def bf(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda().to(torch.bfloat16)


def f32(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).cuda()


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def npy(t):
    return t.detach().double().cpu().numpy()


def decays(kind, H):
    if kind == "none":
        return np.zeros(H, np.float32)
    if kind == "strong":
        return np.array([[-np.inf, -30.0, -1.0, -3.0][h % 4] for h in range(H)], np.float32)
    return np.array([[np.log1p(-2.0 ** -5), -0.5, np.log1p(-2.0 ** -12), 0.0][h % 4] for h in range(H)], np.float32)


class Problem:
    def __init__(self, lens, before, behind, H, d, dv, seed=0, decay="mixed"):
        r = np.random.default_rng(seed)
        self.cu = np.concatenate([[0], np.cumsum(lens)]) + before
        self.T, self.N, self.H, self.d, self.dv = int(self.cu[-1]) + behind, len(lens), H, d, dv
        self.inside = np.zeros(self.T, bool)
        self.inside[self.cu[0]:self.cu[-1]] = True
        draw = lambda w: npy(bf(r.standard_normal((self.T, H, w))))  # noqa: E731  bf16 values
        self.q, self.k, self.v, self.dO = draw(d), draw(d), draw(dv), draw(dv)
        self.S0 = r.standard_normal((self.N, H, d, dv)).astype(np.float32) * 2
        self.dS = r.standard_normal((self.N, H, d, dv)).astype(np.float32)
        self.g, self.scale = decays(decay, H), d ** -0.5

    def dev(self, x):
        """On the device, with NaN in the rows outside every sequence."""
        t = bf(x)
        t[torch.from_numpy(~self.inside).cuda()] = float("nan")
        return t

    def inputs(self):
        return self.dev(self.q), self.dev(self.k), self.dev(self.v), f32(self.g), i32(self.cu)


def close_bf16(got, want, mag, inside, scale=1.0):
    got, want, mag = npy(got)[inside], want[inside], mag[inside]
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > scale * (U * np.abs(want) + 1.02 * U * mag) + 1e-30
    assert not bad.any(), (np.argwhere(bad)[:3], got[bad][:3], want[bad][:3])
    if want.size > 1000:
        assert np.linalg.norm(got - want) <= U * np.linalg.norm(want)


def close_state(got, want, mag):
    got = npy(got)
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= 2.0 ** -15 * mag + 1e-30).all(), np.abs(got - want).max()
    if want.size:
        assert np.linalg.norm(got - want) <= 1e-5 * np.linalg.norm(want) + 1e-30


# --------------------------------------------------------------------------
# prompts
# --------------------------------------------------------------------------
@pytest.mark.parametrize("pack", list(PACKS))
@pytest.mark.parametrize("d,dv", DIMS)
def test_prompt(pack, d, dv):
    p = Problem(*PACKS[pack], H=3, d=d, dv=dv)
    q, k, v, g, cu = p.inputs()
    o, S = K.kata_fwd_linear_decay(q, k, v, g, cu, p.scale, S0=f32(p.S0), return_state=True)
    want, Sw = od.forward(p.q, p.k, p.v, p.g, p.cu, p.scale, p.S0)
    mag, Sm = od.magnitude(p.q, p.k, p.v, p.g, p.cu, p.scale, p.S0)
    close_bf16(o, want, mag, p.inside)
    close_state(S, Sw, Sm)
    assert (npy(o)[~p.inside] == 0).all()


@pytest.mark.parametrize("decay", ["none", "strong", "mixed"])
@pytest.mark.parametrize("T", [65, 400])
def test_prompt_decays(decay, T):
    p = Problem([T], 0, 0, H=4, d=64, dv=64, decay=decay)
    q, k, v, g, _ = p.inputs()
    o, S = K.kata_fwd_linear_decay(q, k, v, g, None, p.scale, return_state=True)
    want, Sw = od.forward(p.q, p.k, p.v, p.g, p.cu, p.scale)
    mag, Sm = od.magnitude(p.q, p.k, p.v, p.g, p.cu, p.scale)
    close_bf16(o, want, mag, p.inside)
    close_state(S, Sw, Sm)


def test_prompt_pool_slots_and_resume():
    """A pool larger than the call: named slots, fresh and resumed sequences, one without a slot; the rest untouched."""
    p = Problem([40, 200, 0, 0, 3, 150], 0, 4, H=2, d=128, dv=64)
    q, k, v, g, cu = p.inputs()
    pool = f32(np.random.default_rng(5).standard_normal((9, 2, 128, 64)))
    before = pool.clone()
    slots, resume = [7, 2, 0, 4, -1, 5], [1, 0, 1, 0, 1, 1]
    S0 = np.stack([npy(before)[s] if s >= 0 and r else np.zeros((2, 128, 64)) for s, r in zip(slots, resume)])
    o = torch.full((p.T, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    K.kata_fwd_linear_decay(q, k, v, g, cu, p.scale, S0=pool, S_out=pool, slots=i32(slots),
                            resume=torch.tensor(resume, dtype=torch.uint8, device="cuda"), o=o)
    want, Sw = od.forward(p.q, p.k, p.v, p.g, p.cu, p.scale, S0)
    mag, Sm = od.magnitude(p.q, p.k, p.v, p.g, p.cu, p.scale, S0)
    close_bf16(o, want, mag, p.inside)
    assert (npy(o)[~p.inside] == 7).all()  # the caller's rows behind the last sequence stay as they were
    for n, s in enumerate(slots):
        if s >= 0:
            close_state(pool[s], Sw[n], Sm[n])
    for s in set(range(9)) - set(slots):
        assert torch.equal(pool[s], before[s])


def test_prompt_strided_inputs():
    """The parts of one fused projection, and an output inside a wider buffer."""
    p = Problem([130, 70], 0, 0, H=2, d=64, dv=128)
    fused = torch.full((p.T, 8 + 2 * 64 * 2 + 2 * 128 + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    q, k = fused[:, 8:136].view(p.T, 2, 64), fused[:, 136:264].view(p.T, 2, 64)
    v = fused[:, 264:520].view(p.T, 2, 128)
    for t, x in ((q, p.q), (k, p.k), (v, p.v)):
        t.copy_(bf(x))
    wide = torch.full((p.T, 320), 3.0, dtype=torch.bfloat16, device="cuda")
    o = K.kata_fwd_linear_decay(q, k, v, f32(p.g), i32(p.cu), p.scale, o=wide[:, 32:288].view(p.T, 2, 128))
    want, _ = od.forward(p.q, p.k, p.v, p.g, p.cu, p.scale)
    mag, _ = od.magnitude(p.q, p.k, p.v, p.g, p.cu, p.scale)
    close_bf16(o, want, mag, p.inside)
    assert (wide[:, :32] == 3).all() and (wide[:, 288:] == 3).all()
    dense = K.kata_fwd_linear_decay(bf(p.q), bf(p.k), bf(p.v), f32(p.g), i32(p.cu), p.scale)
    assert torch.equal(dense, o)


@pytest.mark.parametrize("H,lens", [(1, [9000]), (2, [6000, 10, 0, 5000]), (5, [4097, 8192])])
def test_prompt_long(H, lens):
    """Lengths that are cut into segments, with states in and out."""
    p = Problem(lens, 0, 0, H=H, d=64, dv=64)
    q, k, v, g, cu = p.inputs()
    pool = f32(p.S0)
    o = K.kata_fwd_linear_decay(q, k, v, g, cu, p.scale, S0=pool, S_out=pool)
    t = lambda x: torch.from_numpy(np.asarray(x, np.float64)).cuda()  # noqa: E731
    want, Sw, mag, Sm = [], [], [], []
    for n, (a, b) in enumerate(zip(p.cu[:-1], p.cu[1:])):
        for out, st, ab in ((want, Sw, False), (mag, Sm, True)):
            f = (lambda x: t(x).abs()) if ab else t
            x, y, z, S = f(p.q[a:b]).transpose(0, 1), f(p.k[a:b]).transpose(0, 1), f(p.v[a:b]).transpose(0, 1), f(p.S0[n])
            L, gg = int(b - a), t(p.g)[:, None]
            i = torch.arange(L, device="cuda", dtype=torch.float64)
            W = torch.exp(gg[..., None] * (i[:, None] - i[None, :]).clamp(min=0)).tril()
            out.append((p.scale * ((x @ y.transpose(1, 2) * W) @ z + torch.exp(gg * (i + 1))[..., None] * (x @ S))).transpose(0, 1))
            st.append(torch.exp(gg * L)[..., None] * S + (y * torch.exp(gg * (L - 1 - i))[..., None]).transpose(1, 2) @ z)
    close_bf16(o, npy(torch.cat(want)), npy(torch.cat(mag)), p.inside)
    close_state(pool, npy(torch.stack(Sw)), npy(torch.stack(Sm)))


def test_prompt_without_tokens_or_sequences():
    g = f32(decays("mixed", 2))
    e = lambda w: torch.empty(0, 2, w, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    S0 = f32(np.random.default_rng(0).standard_normal((3, 2, 64, 128)))
    o, S = K.kata_fwd_linear_decay(e(64), e(64), e(128), g, i32([0, 0, 0, 0]), S0=S0, return_state=True)
    assert o.shape == (0, 2, 128) and torch.equal(S, S0)
    _, S = K.kata_fwd_linear_decay(e(64), e(64), e(128), g, i32([0, 0, 0, 0]), return_state=True)
    assert (S == 0).all()
    x = torch.randn(5, 2, 64, device="cuda").to(torch.bfloat16)
    o = K.kata_fwd_linear_decay(x, x, x, g, i32([0]))
    assert (o == 0).all()
    dq, dk, dv = K.kata_bwd_linear_decay(x, x, x, x, g, i32([5]))
    assert not (dq.any() or dk.any() or dv.any())


# --------------------------------------------------------------------------
# gradients
# --------------------------------------------------------------------------
def grad_check(p, state):
    q, k, v, g, cu = p.inputs()
    S0, dS = (f32(p.S0), f32(p.dS)) if state else (None, None)
    got = K.kata_bwd_linear_decay(q, k, v, p.dev(p.dO), g, cu, p.scale, S0=S0, dS_out=dS, return_dS0=True)
    s0, ds = (p.S0, p.dS) if state else (None, None)
    want = od.backward(p.q, p.k, p.v, p.dO, p.g, p.cu, p.scale, s0, ds)
    ab = lambda x: None if x is None else np.abs(x)  # noqa: E731
    mag = od.backward(ab(p.q), ab(p.k), ab(p.v), ab(p.dO), p.g, p.cu, p.scale, ab(s0), ab(ds))
    for x, w, m in zip(got[:3], want, mag):
        close_bf16(x, w, m, p.inside)
        assert (npy(x)[~p.inside] == 0).all()
    close_state(got[3], want[3], mag[3])


@pytest.mark.parametrize("pack", list(PACKS))
@pytest.mark.parametrize("d,dv", DIMS)
def test_gradients(pack, d, dv):
    grad_check(Problem(*PACKS[pack], H=2, d=d, dv=dv, seed=3), state=True)


@pytest.mark.parametrize("decay", ["none", "strong", "mixed"])
def test_gradients_decays(decay):
    grad_check(Problem([300, 20], 0, 0, H=4, d=64, dv=64, seed=4, decay=decay), state=False)


def test_gradients_long():
    grad_check(Problem([4500, 300], 0, 2, H=1, d=64, dv=64, seed=5), state=True)


def test_autograd():
    p = Problem([100, 0, 157], 0, 3, H=2, d=64, dv=64, seed=6)
    q, k, v, g, cu = p.inputs()
    S0 = f32(p.S0)
    for t in (q, k, v, S0):
        t.requires_grad_()
    o, S = K.kata_attention_linear_decay(q, k, v, g, cu, p.scale, S0=S0, return_state=True)
    assert (npy(o)[~p.inside] == 0).all()
    dO, dS = bf(p.dO * p.inside[:, None, None]), f32(p.dS)
    # a gradient that arrives transposed in memory
    dOt = dO.transpose(0, 1).contiguous().transpose(0, 1)
    got = torch.autograd.grad((o, S), (q, k, v, S0), (dOt, dS))
    direct = K.kata_bwd_linear_decay(q.detach(), k.detach(), v.detach(), dO, g, cu, p.scale, S0=S0.detach(),
                                     dS_out=dS, return_dS0=True)
    for a, b in zip(got, direct):
        assert torch.equal(a, b)
    # only the state, only the output, and no state at all
    o, S = K.kata_attention_linear_decay(q, k, v, g, cu, p.scale, S0=S0, return_state=True)
    got = torch.autograd.grad(S, (k, v, S0), dS)
    want = od.backward(p.q, p.k, p.v, 0 * p.dO, p.g, p.cu, p.scale, p.S0, p.dS)
    mag = od.backward(np.abs(p.q), np.abs(p.k), np.abs(p.v), 0 * p.dO, p.g, p.cu, p.scale, np.abs(p.S0), np.abs(p.dS))
    close_bf16(got[0], want[1], mag[1], p.inside)
    close_bf16(got[1], want[2], mag[2], p.inside)
    close_state(got[2], want[3], mag[3])
    o = K.kata_attention_linear_decay(q, k, v, g, cu, p.scale)
    got = torch.autograd.grad(o, (q, k, v), dO)
    want = K.kata_bwd_linear_decay(q.detach(), k.detach(), v.detach(), dO, g, cu, p.scale)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_by_differences():
    """The forward is linear in each input: (f(x + h u) - f(x - h u)) / 2h is the derivative along u, up to the
    roundings of o (u |o| each, the upstream gradient weighing them)."""
    p = Problem([90, 140], 0, 0, H=2, d=64, dv=64, seed=7)
    q, k, v, g, cu = p.inputs()
    dO = bf(p.dO)
    grads = K.kata_bwd_linear_decay(q, k, v, dO, g, cu, p.scale)
    for i in range(3):
        w = torch.randn(grads[i].shape, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).to(torch.bfloat16)
        args = [q, k, v]
        args[i] = w  # linear: the derivative along w is f with w in x's place
        o = npy(K.kata_fwd_linear_decay(*args, g, cu, p.scale))
        mag, _ = od.magnitude(*[npy(a) for a in args], p.g, p.cu, p.scale)
        gm = od.backward(np.abs(p.q), np.abs(p.k), np.abs(p.v), np.abs(p.dO), p.g, p.cu, p.scale)[i]
        left, right = (o * npy(dO)).sum(), (npy(grads[i]) * npy(w)).sum()
        # roundings on either side are independent: their sum grows as the root of the sum of squares
        noise = np.sqrt(((3 * U * mag * npy(dO)) ** 2).sum() + ((3 * U * gm * npy(w)) ** 2).sum())
        assert abs(left - right) <= noise


# --------------------------------------------------------------------------
# single tokens
# --------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,dv", DIMS)
@pytest.mark.parametrize("n", [1, 5, 40])
def test_step(dtype, d, dv, n):
    r = np.random.default_rng(n)
    H, slots = 3, n + 4
    conv = bf if dtype == "bf16" else f32
    q, k, v = (conv(r.standard_normal((n, H, w))) for w in (d, d, dv))
    S = f32(r.standard_normal((slots, H, d, dv)))
    before = S.clone()
    idx = r.permutation(slots)[:n]
    idx[n // 2:n // 2 + n // 5] = -1
    g = decays("mixed", H)
    o = K.kata_decode_step_linear_decay(q, k, v, S, f32(g), slots=i32(idx), scale=0.25)
    a = np.exp(g.astype(np.float64))[:, None, None]
    for i, s in enumerate(idx):
        if s < 0:
            assert (o[i] == 0).all()
            continue
        old, x, y, z = npy(before[s]), npy(q[i]), npy(k[i]), npy(v[i])
        new = a * old + y[:, :, None] * z[:, None, :]
        mag = a * np.abs(old) + np.abs(y)[:, :, None] * np.abs(z)[:, None, :]
        assert (np.abs(npy(S[s]) - new) <= 4 * 2.0 ** -24 * mag).all()
        want = 0.25 * np.einsum("hd,hde->he", x, new)
        m = 0.25 * np.einsum("hd,hde->he", np.abs(x), mag)
        assert (np.abs(npy(o[i]) - want) <= 132 * 2.0 ** -24 * m + (U * np.abs(want) if dtype == "bf16" else 0)).all()
    for s in set(range(slots)) - set(int(x) for x in idx):
        assert torch.equal(S[s], before[s])


def test_step_strided_rows_and_whole_pool():
    n, H, d, dv = 6, 2, 64, 64
    r = np.random.default_rng(0)
    fused = bf(r.standard_normal((n, 3 * H * 64 + 8)))
    q, k, v = (fused[:, i * 128:(i + 1) * 128].view(n, H, 64) for i in range(3))
    S = f32(r.standard_normal((n + 2, H, d, dv)))
    S2, tail, g = S.clone(), S[n:].clone(), f32(decays("mixed", H))
    o = K.kata_decode_step_linear_decay(q, k, v, S, g)
    o2 = K.kata_decode_step_linear_decay(q.contiguous(), k.contiguous(), v.contiguous(), S2, g, slots=i32(range(n)))
    assert torch.equal(o, o2) and torch.equal(S, S2) and torch.equal(S[n:], tail)


# --------------------------------------------------------------------------
# the 8-bit cache
# --------------------------------------------------------------------------
@pytest.mark.parametrize("rows,dv", [(64, 64), (128, 128), (256, 16), (1, 16), (3, 64), (37, 128), (1024, 64)])
@pytest.mark.parametrize("with_z", [False, True])
def test_q8_is_exact(rows, dv, with_z):
    r = np.random.default_rng(rows)
    H, slots, entries = 2, 7, 5
    x = (r.standard_normal((slots, H, rows, dv)) * np.exp(3 * r.standard_normal((slots, H, rows, 1)))).astype(np.float32)
    z = r.standard_normal((slots, H, rows)).astype(np.float32) if with_z else None
    S, zd = f32(x), None if z is None else f32(z)
    cache = torch.full((entries, H, rows, dv), 99, dtype=torch.int8, device="cuda")
    scale = torch.full((entries, H, rows), 9.0, device="cuda")
    zc = None if z is None else torch.full((entries, H, rows), 9.0, device="cuda")
    src, dst = [3, -1, 6, 0], [4, 2, 1, -1]
    K.kata_state_store_q8(S, cache, scale, i32(src), i32(dst), z=zd, z_cache=zc)
    c, s = od.store_q8(x)
    for a, b in ((3, 4), (6, 1)):
        assert np.array_equal(cache[b].cpu().numpy(), c[a]) and np.array_equal(scale[b].cpu().numpy(), s[a])
        if with_z:
            assert np.array_equal(zc[b].cpu().numpy(), z[a])
    for b in (0, 2, 3):
        assert (cache[b] == 99).all() and (scale[b] == 9).all()
    # back: one entry to two slots, the others untouched
    out = torch.full_like(S, 5.0)
    zo = None if z is None else torch.full_like(zd, 5.0)
    K.kata_state_load_q8(cache, scale, out, i32([4, 1, 4, -1]), i32([0, 2, 6, 3]), z=zo, z_cache=zc)
    for a, b in ((3, 0), (6, 2), (3, 6)):
        assert np.array_equal(out[b].cpu().numpy(), od.load_q8(c[a], s[a]))
        assert (np.abs(out[b].cpu().numpy().astype(np.float64) - x[a]) <= s[a][..., None] * (0.5 + 2.0 ** -16)).all()
        if with_z:
            assert np.array_equal(zo[b].cpu().numpy(), z[a])
    for b in (1, 3, 4, 5):
        assert (out[b] == 5).all()


def test_q8_special_rows():
    """Ties, tiny rows, subnormals, the largest finite values, infinities and NaN; values next to borders."""
    r = np.random.default_rng(1)
    x = r.standard_normal((1, 1, 64, 64)).astype(np.float32)
    x[0, 0, 0] = 0
    x[0, 0, 1, :4] = [127, -63.5, 0.5, 1.5]
    x[0, 0, 1, 4:] = np.arange(60, dtype=np.float32) + 0.5
    x[0, 0, 2] = np.float32(2.0 ** -140)
    x[0, 0, 3] *= np.float32(2.0 ** -118)  # scales near the smallest that is held
    x[0, 0, 4, 5] = np.inf
    x[0, 0, 5, 6] = -np.inf
    x[0, 0, 6, 63] = np.nan
    x[0, 0, 7, 0] = np.finfo(np.float32).max
    for i in range(8, 64):  # next to (k + 1/2) scale, from either side
        m = np.float32(r.uniform(0.1, 10))
        s = np.float32(np.float64(m) / 127)
        y = ((np.arange(64) + 0.5) * np.float64(s)).astype(np.float32)
        x[0, 0, i] = np.nextafter(y, np.where(r.random(64) < 0.5, -np.inf, np.inf).astype(np.float32))
        x[0, 0, i, 0] = -m
    cache = torch.empty((1, 1, 64, 64), dtype=torch.int8, device="cuda")
    scale = torch.empty((1, 1, 64), device="cuda")
    S = f32(x)
    K.kata_state_store_q8(S, cache, scale)
    c, s = od.store_q8(x)
    assert np.array_equal(cache.cpu().numpy(), c)
    assert np.array_equal(scale.cpu().numpy(), s, equal_nan=True)
    K.kata_state_load_q8(cache, scale, S)
    assert np.array_equal(S.cpu().numpy(), od.load_q8(c, s), equal_nan=True)


# --------------------------------------------------------------------------
# together, and what is refused
# --------------------------------------------------------------------------
def test_serving_run():
    """Prompts into a pool, decoding, parking in the 8-bit cache, a fork, more decoding: each step against the oracle
    going on from the states that the pool really holds."""
    H, d, dv, scale = 2, 64, 128, 0.125
    p = Problem([50, 200], 0, 0, H=H, d=d, dv=dv, seed=8)
    q, k, v, g, cu = p.inputs()
    pool = torch.zeros(5, H, d, dv, device="cuda")
    K.kata_fwd_linear_decay(q, k, v, g, cu, scale, S0=pool, S_out=pool, slots=i32([3, 1]),
                            resume=torch.zeros(2, dtype=torch.uint8, device="cuda"))
    r = np.random.default_rng(9)
    a = np.exp(p.g.astype(np.float64))[:, None, None]

    def decode(slots):
        x, y, z = (bf(r.standard_normal((len(slots), H, w))) for w in (d, d, dv))
        held = npy(pool)
        o = K.kata_decode_step_linear_decay(x, y, z, pool, g, slots=i32(slots), scale=scale)
        for i, s in enumerate(slots):
            S = a * held[s] + npy(y[i])[:, :, None] * npy(z[i])[:, None, :]
            m = a * np.abs(held[s]) + np.abs(npy(y[i]))[:, :, None] * np.abs(npy(z[i]))[:, None, :]
            want, mag = (scale * np.einsum("hd,hde->he", f(npy(x[i])), T) for f, T in ((np.asarray, S), (np.abs, m)))
            assert (np.abs(npy(o[i]) - want) <= U * np.abs(want) + 132 * 2.0 ** -24 * mag).all()

    for _ in range(3):
        decode([1, 3])
    cache = torch.zeros(2, H, d, dv, dtype=torch.int8, device="cuda")
    sc = torch.zeros(2, H, d, device="cuda")
    K.kata_state_store_q8(pool, cache, sc, slots=i32([3]), entries=i32([1]))
    K.kata_state_load_q8(cache, sc, pool, entries=i32([1, 1]), slots=i32([0, 4]))
    assert torch.equal(pool[0], pool[4])
    rows = pool[3].abs().amax(-1, keepdim=True)
    assert ((pool[0] - pool[3]).abs() <= rows / 127 * (0.5 + 2.0 ** -16)).all()
    decode([1, 0, 4])
    # the same continuation as one more prompt from the pool
    held = npy(pool)
    p2 = Problem([20, 9], 0, 0, H=H, d=d, dv=dv, seed=10)
    q, k, v, g, cu = p2.inputs()
    o = K.kata_fwd_linear_decay(q, k, v, g, cu, scale, S0=pool, S_out=pool, slots=i32([4, 1]))
    want, Sw = od.forward(p2.q, p2.k, p2.v, p2.g, p2.cu, scale, held[[4, 1]])
    mag, Sm = od.magnitude(p2.q, p2.k, p2.v, p2.g, p2.cu, scale, held[[4, 1]])
    close_bf16(o, want, mag, p2.inside)
    close_state(pool[[4, 1]], Sw, Sm)


def test_kata_states_in_the_cache():
    """The squared-feature state of the chunked path, parked and read back, goes on decoding."""
    B, H, T, p, dv = 2, 2, 70, 16, 64
    gen = torch.Generator("cuda").manual_seed(0)
    x = lambda *s: torch.randn(s, device="cuda", generator=gen).to(torch.bfloat16)  # noqa: E731
    _, S, z = K.kata_fwd_chunked(x(B, H, T, p), x(B, H, T, p), x(B, H, T, dv), return_state=True)
    cache = torch.zeros(4, H, p * p, dv, dtype=torch.int8, device="cuda")
    sc, zc = torch.zeros(4, H, p * p, device="cuda"), torch.zeros(4, H, p * p, device="cuda")
    K.kata_state_store_q8(S, cache, sc, entries=i32([3, 0]), z=z, z_cache=zc)
    S2, z2 = torch.zeros_like(S), torch.zeros_like(z)
    K.kata_state_load_q8(cache, sc, S2, entries=i32([3, 0]), z=z2, z_cache=zc)
    assert torch.equal(z, z2)
    q, k, v = x(B, H, p), x(B, H, p), x(B, H, dv)
    # o = N / D is off by the rows' half steps, weighed by the squared scores of the features
    w = (q.float()[..., :, None] * q.float()[..., None, :]).reshape(B, H, p * p)
    step = S.abs().amax(-1) / 127 * (0.5 + 2.0 ** -16)
    den = (w * (z + (k.float()[..., :, None] * k.float()[..., None, :]).reshape(B, H, p * p))).sum(-1)
    bound = ((w.abs() * step).sum(-1) / den)[..., None]
    a = K.kata_decode_step(q, k, v, S, z).float()
    b = K.kata_decode_step(q, k, v, S2, z2).float()
    assert ((a - b).abs() <= bound + U * (a.abs() + b.abs()) + 1e-4 * bound).all()


def expect_invalid(call):
    torch.cuda.synchronize()
    assert K.kata_get_status() == _abi.KATA_OK
    out = call()
    assert K.kata_get_status() == _abi.KATA_ERR_INVALID_ARG
    assert K.kata_get_status() == _abi.KATA_OK
    return out


def test_bad_device_indices_are_reported_and_bounded():
    H, d = 2, 64
    x = torch.randn(20, H, d, device="cuda").to(torch.bfloat16)
    g = f32(decays("mixed", H))
    for cu in ([0, 15, 10, 20], [0, 30], [-4, 20], [0, 21, 20], [5, 0]):
        o = expect_invalid(lambda: K.kata_fwd_linear_decay(x, x, x, g, i32(cu)))
        assert torch.isfinite(o).all()
        expect_invalid(lambda: K.kata_bwd_linear_decay(x, x, x, x, g, i32(cu)))
    pool = torch.randn(3, H, d, d, device="cuda")
    before = pool.clone()
    # out of range, and the same slot twice: the first keeps it
    expect_invalid(lambda: K.kata_fwd_linear_decay(x, x, x, g, i32([0, 10, 20]), S0=pool, S_out=pool, slots=i32([3, 1])))
    assert torch.equal(pool[[0, 2]], before[[0, 2]]) and not torch.equal(pool[1], before[1])
    pool.copy_(before)
    expect_invalid(lambda: K.kata_fwd_linear_decay(x, x, x, g, i32([0, 10, 20]), S0=pool, S_out=pool, slots=i32([1, 1])))
    want = before.clone()
    K.kata_fwd_linear_decay(x[:10], x[:10], x[:10], g, S0=want, S_out=want, slots=i32([1]))
    assert torch.equal(pool, want)
    # without states to write, a shared prefix is no error
    K.kata_fwd_linear_decay(x, x, x, g, i32([0, 10, 20]), S0=pool, slots=i32([1, 1]))
    assert K.kata_get_status() == _abi.KATA_OK
    y = x[:4].contiguous()
    for slots in ([0, 3, -1, 1], [2, 0, 2, 1]):
        pool.copy_(before)
        o = expect_invalid(lambda: K.kata_decode_step_linear_decay(y, y, y, pool, g, slots=i32(slots)))
        want = before.clone()
        ok = [s if s < 3 and s not in slots[:i] else -1 for i, s in enumerate(slots)]
        assert torch.equal(o, K.kata_decode_step_linear_decay(y, y, y, want, g, slots=i32(ok)))
        assert torch.equal(pool, want)
    cache = torch.zeros(2, H, d, d, dtype=torch.int8, device="cuda")
    sc = torch.zeros(2, H, d, device="cuda")
    for slots, entries in (([0, 1], [2, 0]), ([3, 1], [1, 0]), ([1, 0], [0, 0])):
        cache.zero_()
        expect_invalid(lambda: K.kata_state_store_q8(pool, cache, sc, slots=i32(slots), entries=i32(entries)))
        c, _ = od.store_q8(pool[1].cpu().numpy())
        assert np.array_equal(cache[0].cpu().numpy(), c) and not cache[1].any()
    pool.copy_(before)
    expect_invalid(lambda: K.kata_state_load_q8(cache, sc, pool, slots=i32([2, 2]), entries=i32([0, 1])))
    expect_invalid(lambda: K.kata_state_load_q8(cache, sc, pool, slots=i32([7, 1]), entries=i32([0, 5])))
    assert torch.equal(pool[:2], before[:2])
    # a decay above 1, and one that is not a number, count as none
    for bad in (0.5, float("nan")):
        h = torch.tensor([bad, -0.1], device="cuda")
        o = expect_invalid(lambda: K.kata_fwd_linear_decay(x, x, x, h))
        assert torch.equal(o, K.kata_fwd_linear_decay(x, x, x, torch.tensor([0.0, -0.1], device="cuda")))


def test_binding_refuses():
    H = 2
    x = torch.zeros(8, H, 64, dtype=torch.bfloat16, device="cuda")
    g, S = torch.zeros(H, device="cuda"), torch.zeros(1, H, 64, 64, device="cuda")
    fwd = K.kata_fwd_linear_decay
    with pytest.raises(ValueError):
        fwd(x, x[:7], x, g)
    with pytest.raises(TypeError):
        fwd(x, x.float(), x, g)
    with pytest.raises(TypeError):
        fwd(x.half(), x.half(), x.half(), g)
    with pytest.raises(K.KataError):
        fwd(x.float(), x.float(), x.float(), g)
    with pytest.raises(ValueError):
        fwd(x.transpose(1, 2), x, x, g)
    with pytest.raises(ValueError):
        fwd(x, x, x, g[:1])
    with pytest.raises(TypeError):
        fwd(x, x, x, g, torch.tensor([0, 8], device="cuda"))
    with pytest.raises(ValueError):
        fwd(x, x, x, g, S0=S[:, :, :32])
    with pytest.raises(ValueError):
        fwd(x, x, x, g, S0=S, S_out=torch.zeros(2, H, 64, 64, device="cuda"))
    with pytest.raises(ValueError):
        fwd(x, x, x, g, slots=i32([0]), return_state=True)
    with pytest.raises(K.KataError):
        fwd(x, x, x, g, i32([0, 4, 8]), S0=S)  # fewer states than sequences
    with pytest.raises(K.KataError):
        fwd(x, x, x, g, S0=S, S_out=torch.zeros(3, H, 64, 64, device="cuda").view(-1)[64:64 + S.numel()].view_as(S),
            o=torch.zeros(8 * H * 64 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(8, H, 64))  # misaligned o
    with pytest.raises(TypeError):
        K.kata_bwd_linear_decay(x, x, x, x.float(), g)
    with pytest.raises(ValueError):
        K.kata_bwd_linear_decay(x, x, x, x.transpose(0, 1).contiguous().transpose(0, 1), g)
    with pytest.raises(K.KataError):
        K.kata_decode_step_linear_decay(x, x, x, S, g)  # 8 streams, 1 state
    with pytest.raises(ValueError):
        K.kata_decode_step_linear_decay(x, x, x, S, g, slots=i32([0]))
    c, sc = torch.zeros(1, H, 64, 64, dtype=torch.int8, device="cuda"), torch.zeros(1, H, 64, device="cuda")
    with pytest.raises(ValueError):
        K.kata_state_store_q8(S, c, sc[:, :, :3])
    with pytest.raises(TypeError):
        K.kata_state_store_q8(S, c.float(), sc)
    with pytest.raises(ValueError):
        K.kata_state_store_q8(S, c, sc, z=sc)
    with pytest.raises(ValueError):
        K.kata_state_load_q8(c, sc, S, slots=i32([0]), entries=i32([0, 0]))


def test_streams_graphs_and_repeats():
    """Another stream, capture and replay with new inputs, and bitwise repeats (segments included)."""
    p = Problem([4500, 3, 600], 0, 0, H=2, d=64, dv=64, seed=11)
    q, k, v, g, cu = p.inputs()
    dO = bf(p.dO)

    def run(stream=None):
        S = torch.empty(3, 2, 64, 64, device="cuda")
        o = K.kata_fwd_linear_decay(q, k, v, g, cu, p.scale, S_out=S, stream=stream)
        return (o, S) + K.kata_bwd_linear_decay(q, k, v, dO, g, cu, p.scale, stream=stream)

    want = run()
    assert all(torch.equal(a, b) for a, b in zip(want, run()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    torch.cuda.synchronize()
    got = run(stream=side)  # the allocations are this stream's, the work the other's
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph, other = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run()
    with torch.cuda.graph(other):
        out2 = run()
    q.copy_(bf(np.random.default_rng(1).standard_normal(p.q.shape)))
    want = run()
    graph.replay()
    other.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))
    assert all(torch.equal(a, b) for a, b in zip(want, out2))
