"""How exact the states of linear attention with a per-head decay are, and its
gradients at strong decays where sequences are cut, against 64 bits.

A state of tokens of like magnitude agrees with fp32 arithmetic.  In the 2-norm,
relative to the state:
* keys times their decay as three bf16 values lose 2^-24; those of chunks that
  are less than a 16th of what leaves are two values, off by up to 2^-16, in the
  mean square 2^-16 / sqrt(3) of less than 1/16: 5.5e-7;
* the tensor cores truncate a chunk's sum 8 times (16 tokens a product) by up to
  one step of 2^-23 of what it has come to, half a step in the mean, sqrt(i / 8)
  of the chunk after i products: 8 * 0.71 * 2^-24 = 3.4e-7;
* the factors between chunks, and between 16 segments or more, are held as two
  fp32 values; that between fewer segments is off by up to 2^-25 the same way
  for each of up to 15, 9 in the mean square: 2.7e-7;
* the decays' powers and the additions of the chunks are off by a few 2^-25.
Independent of one another: 7.0e-7, below 1e-6.  Keys of two bf16 values alone
come to 3e-6 to 4.5e-6, and factors of one fp32 value to up to 2^-25 for every
chunk or segment walked.
"""
import numpy as np
import pytest
import torch

import kernelized_feature_map_b200 as K
from kernelized_feature_map_b200 import _abi

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


def worst_rounded(near, tokens):
    """A decay's logarithm near `near` whose power over `tokens` tokens fp32 rounds by almost half a step."""
    g = (near * (1 + np.arange(4096) / 8192)).astype(np.float32)
    x = np.exp(g.astype(np.float64) * tokens)
    return float(g[np.argmax(np.abs(x.astype(np.float32) - x) / x)])


def state(k, v, g, S0, reverse=False):
    """The state that leaves one sequence, in 64 bits: [x, H, d], [x, H, dv], S0 [H, d, dv]; reversed it is the
    gradient of the state that entered, of queries k and upstream gradients v."""
    x, out = k.shape[0], []
    t = torch.arange(x, device="cuda", dtype=torch.float64)
    for h in range(k.shape[1]):
        w = torch.exp(g[h].double() * (t + 1 if reverse else x - 1 - t))
        out.append(torch.exp(g[h].double() * x) * S0[h].double() + (k[:, h].double() * w[:, None]).T @ v[:, h].double())
    return torch.stack(out)


def error(got, want):
    """Largest relative error in the 2-norm over the heads."""
    n = lambda x: torch.linalg.vector_norm(x.double(), dim=(-2, -1))  # noqa: E731
    return float((n(got.double() - want) / n(want)).max())


def parts(T, H, N, walks):
    """T over the plan's length of segments, from the records it asks for (0: one segment)."""
    f = K.kata_fwd_linear_decay_workspace_size if walks == 1 else K.kata_bwd_linear_decay_workspace_size
    records = f(T, H, 64, 64, N) // (H * 64 * 64 * 4 * walks)
    return records // 2 if records <= 2 * N else records - N


RETENTION = [float(np.log1p(-2.0 ** -5)), float(np.log1p(-2.0 ** -12)), 0.0, -0.5, -0.1]
# (heads, d, dv, lengths, decays: RETENTION or one near this whose powers over a chunk or segment round worst)
CASES = {
    "short": (5, 128, 128, [16, 100, 128, 300], None),
    "uncut": (5, 64, 128, [1000] * 32, None),
    "uncut slow": (16, 64, 64, [16384] * 10, -2.0 ** -17),
    "folded": (16, 128, 64, [5000, 90, 1], None),
    "folded slow": (16, 64, 64, [32768], -2.0 ** -17),
    "scanned": (5, 128, 128, [5000, 90, 1], None),
    "scanned slow": (1, 64, 64, [131072], -2.0 ** -18),
}


def decays(case, walks):
    H, _, _, lens, slow = CASES[case]
    T, N = sum(lens), len(lens)
    if slow is None:
        return torch.tensor([RETENTION[h % 5] for h in range(H)], dtype=torch.float32, device="cuda")
    over = 128  # tokens whose power the state is multiplied by again and again
    if not case.startswith("uncut"):  # a segment's, a multiple of 128
        n = parts(T, H, N, walks)
        over = T // n // 128 * 128
        assert n > 1 and over > T / (n + 1)
    return torch.full((H,), worst_rounded(slow, over), device="cuda")


@pytest.mark.parametrize("case", list(CASES))
def test_states_agree_with_fp32_arithmetic(case):
    H, d, dv, lens, _ = CASES[case]
    N, T, r, g = len(lens), sum(lens), gen(len(case)), decays(case, 1)
    n = parts(T, H, N, 1)  # segments have at least T / (n + 1) tokens
    if case.startswith("scanned"):
        assert n >= 16
    elif case.startswith("folded"):
        assert 1 < n < 16
    else:
        assert n == 0 or max(lens) <= T / (n + 1)
    k, v = bf(r, T, H, d), bf(r, T, H, dv)
    S0 = torch.randn(N, H, d, dv, device="cuda", generator=r) * 4
    S = K.kata_fwd_linear_decay(torch.zeros_like(k), k, v, g, edges(lens), 1.0, S0=S0, return_state=True)[1]
    a = 0
    for n, x in enumerate(lens):
        e = error(S[n], state(k[a:a + x], v[a:a + x], g, S0[n]))
        assert e <= 1e-6, (n, x, e)
        a += x


@pytest.mark.parametrize("case", [c for c in CASES if c != "uncut slow"])
def test_gradients_of_entering_states_agree_with_fp32_arithmetic(case):
    H, d, dv, lens, _ = CASES[case]
    N, T, r, g = len(lens), sum(lens), gen(len(case)), decays(case, 3)
    q, dO = bf(r, T, H, d), bf(r, T, H, dv)
    dS = torch.randn(N, H, d, dv, device="cuda", generator=r) * 4
    dS0 = K.kata_bwd_linear_decay(q, torch.zeros_like(q), torch.zeros_like(dO), dO, g, edges(lens), 1.0, dS_out=dS,
                                  return_dS0=True)[3]
    a = 0
    for n, x in enumerate(lens):
        e = error(dS0[n], state(q[a:a + x], dO[a:a + x], g, dS[n], reverse=True))
        assert e <= 1e-6, (n, x, e)
        a += x


@pytest.mark.parametrize("lens", [[400], [9000]])
def test_a_state_whose_last_keys_are_zero(lens):
    """Which keys are held as three values goes by the decay alone.  Where the last tokens add nothing, the state
    that leaves is made of keys of two, off by up to 2^-16 each, 2^-16 / sqrt(3) = 8.8e-6 in the mean square."""
    r, T, H, d = gen(5), sum(lens), 2, 64
    g = torch.tensor([-0.1, -0.03], device="cuda")
    k, v = bf(r, T, H, d), bf(r, T, H, d)
    k[T - 200:] = 0
    S = K.kata_fwd_linear_decay(k, k, v, g, edges(lens), 1.0, return_state=True)[1][0]
    want = state(k, v, g, torch.zeros_like(S))
    assert error(S, want) <= 9e-6
    mag = state(k.abs(), v.abs(), g, torch.zeros_like(S))
    assert ((S.double() - want).abs() <= 2.0 ** -15 * mag).all()


# --------------------------------------------------------------------------
# gradients at strong decays, cut
# --------------------------------------------------------------------------
U = 2.0 ** -8


def pairs(q, k, v, dO, g, scale, S0, dS):
    """dq, dk, dv and dS0 of one sequence from the sums over pairs, nothing divided by the decay; [x, H, *] in."""
    x, out = q.shape[0], []
    t = torch.arange(x, device="cuda", dtype=torch.float64)
    away = t[:, None] - t[None, :]
    for h in range(q.shape[1]):
        a, b, c, d = (y[:, h].double() for y in (q, k, v, dO))
        d = scale * d
        gh = g[h].double()
        w = torch.where(away > 0, torch.exp(gh * away.clamp(min=1)), (away == 0).double())
        reach = torch.exp(gh * (t + 1))[:, None]
        share = torch.where(t == x - 1, 1.0, torch.exp(gh * (x - 1 - t).clamp(min=1)))[:, None]
        P = (d @ c.T) * w
        out.append((P @ b + reach * (d @ S0[h].double().T), P.T @ a + share * (c @ dS[h].double().T),
                    ((a @ b.T) * w).T @ d + share * (b @ dS[h].double()),
                    torch.exp(gh * x) * dS[h].double() + (reach * a).T @ d))
    return [torch.stack(y, 1) for y in list(zip(*out))[:3]] + [torch.stack([y[3] for y in out])]


@pytest.mark.parametrize("H,d,dv,lens", [(6, 64, 64, [1500, 900, 3]), (5, 128, 64, [2000, 1, 129]),
                                         (12, 64, 128, [1700])])
def test_gradients_cut_at_strong_decays(H, d, dv, lens):
    """Decays from none to one that keeps only the current token, in one call whose sequences are cut.  Tolerances: u
    = 2^-8 of the value and 1.02 u of the terms' magnitudes, for a state 2^-15 of these."""
    r, N, T = gen(H + d), len(lens), sum(lens)
    assert parts(T, H, N, 3) > 1
    kinds = [-30.0, -float("inf"), -1.0, float(np.log1p(-2.0 ** -12)), 0.0, -3.0]
    g = torch.tensor([kinds[h % 6] for h in range(H)], device="cuda")
    q, k, v, dO = bf(r, T, H, d), bf(r, T, H, d), bf(r, T, H, dv), bf(r, T, H, dv)
    S0, dS = (torch.randn(N, H, d, dv, device="cuda", generator=r) for _ in range(2))
    got = K.kata_bwd_linear_decay(q, k, v, dO, g, edges(lens), 0.3, S0=S0, dS_out=dS, return_dS0=True)
    a = 0
    for n, x in enumerate(lens):
        part = slice(a, a + x)
        a += x
        args = [y[part] for y in (q, k, v, dO)]
        want = pairs(*args, g, 0.3, S0[n], dS[n])
        mag = pairs(*[y.abs() for y in args], g, 0.3, S0[n].abs(), dS[n].abs())
        for y, w, m in zip(got[:3], want, mag):
            assert ((y[part].double() - w).abs() <= U * w.abs() + 1.02 * U * m + 1e-30).all()
        assert ((got[3][n].double() - want[3]).abs() <= 2.0 ** -15 * mag[3] + 1e-30).all()


@pytest.mark.parametrize("H,d,dv,lens", [(2, 64, 64, [90, 140]), (1, 128, 64, [2600])])
def test_gradients_against_differences(H, d, dv, lens):
    """(f(x + u) - f(x - u)) / 2 of f = sum(o dO) + sum(S dS), each input in turn, on small integers: x + u and x - u
    are bf16 values, and f is linear in each input, so that only the roundings of o, S and the gradients are off: 3 u
    of the terms' magnitudes each (2 u in o, both sides of the difference, and 2 u in the gradient), independent of
    one another: their sum is off by the root of the sum of their squares."""
    r, N, T = gen(d), len(lens), sum(lens)
    whole = lambda n, *shape: torch.randint(-n, n + 1, shape, device="cuda", generator=r).float()  # noqa: E731
    x = [whole(4, T, H, d), whole(4, T, H, d), whole(4, T, H, dv), whole(4, N, H, d, dv)]
    dO, dS = whole(3, T, H, dv).to(torch.bfloat16), whole(3, N, H, d, dv)
    g, cu, half = torch.tensor([-0.02, -0.3][:H], device="cuda"), edges(lens), torch.bfloat16

    def forward(q, k, v, S0):
        return K.kata_fwd_linear_decay(q.to(half), k.to(half), v.to(half), g, cu, 0.25, S0=S0, return_state=True)

    def backward(q, k, v, S0, dO, dS):
        return K.kata_bwd_linear_decay(q.to(half), k.to(half), v.to(half), dO, g, cu, 0.25, S0=S0, dS_out=dS,
                                       return_dS0=True)

    grads = backward(*x, dO, dS)
    sizes = backward(*[t.abs() for t in x], dO.abs(), dS.abs())
    mag_o, mag_S = forward(*[t.abs() + 2 for t in x])  # no smaller than those of x + u and x - u
    for i in range(4):
        u = whole(2, *x[i].shape)
        up, down = list(x), list(x)
        up[i], down[i] = x[i] + u, x[i] - u
        (o1, S1), (o0, S0) = forward(*up), forward(*down)
        dot = lambda a, b: (a.double() * b.double()).sum()  # noqa: E731
        diff = (dot(o1, dO) - dot(o0, dO) + dot(S1, dS) - dot(S0, dS)) / 2
        noise = torch.stack([dot(a * b, a * b) for a, b in ((3 * U * mag_o.double(), dO.double()),
                                                            (2.0 ** -14 * mag_S.double(), dS.double()),
                                                            (3 * U * sizes[i].double(), u.double()))]).sum().sqrt()
        assert abs(diff - dot(grads[i], u)) <= noise, (i, float(diff), float(dot(grads[i], u)), float(noise))
