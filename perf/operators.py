"""Linear attention with a per-head decay, and the 8-bit cache of its states: what is measured.

The operators, each in its plain form (elementary torch operations, 32 bits)
and as the calls a user makes of the package (``own = True``):

* ``prompt`` -- ``kata_fwd_linear_decay``: packed prompts of different lengths
  [T, H, d], per-head decay a_h = exp(log_decay_h),
      S_t = a S_{t-1} + k_t v_t^T,   o_t = scale * q_t^T S_t,
  each sequence starting from zero or from its slot of a pool of states and
  leaving its final state there;
* ``train`` -- ``kata_bwd_linear_decay``: the gradients of q, k, v (and of the
  initial state) for given gradients of o (and of the final state);
* ``step`` -- ``kata_decode_step_linear_decay``: one token for every active
  sequence, in place on the pool of states;
* ``store`` / ``load`` -- ``kata_state_store_q8`` / ``kata_state_load_q8``:
  states written to and read back from a cache that holds each state row as
  8-bit integers with one fp32 scale: scale = max|row| / 127 (held in fp32;
  a row whose scale would be below 2^-126 is held as zeros), value = the
  integer nearest to x / scale (ties to even) times scale.  A ``store`` pass
  also reads the whole cache back, into a second pool, since what 8 bits hold
  is compared by the values it stands for.
"""
import math
import random

import torch

own = False

CHUNK = 128
MIN_SCALE = 2.0 ** -126


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one short turn of a chat: latency
        {"name": "prompt_turn", "op": "prompt", "n": 1, "total": 75, "mix": "ragged", "cut": 1, "pad": 0, "heads": 16,
         "d": 64, "dv": 64, "resume": False, "slots": 4, "decay": "retention"},
        # a serving batch: packed prompts, some of which go on from an earlier turn, rows of padding behind them
        {"name": "prompt_packed", "op": "prompt", "n": 13, "total": 8115, "mix": "ragged", "cut": 2, "pad": 77,
         "heads": 16, "d": 128, "dv": 128, "resume": True, "slots": 32, "decay": "slopes"},
        # one long document
        {"name": "prompt_long", "op": "prompt", "n": 1, "total": 131072, "mix": "ragged", "cut": 3, "pad": 0,
         "heads": 16, "d": 128, "dv": 128, "resume": False, "slots": 1, "decay": "retention"},
        # a fine-tuning step on a few packed documents, state carried from the piece before
        {"name": "train_packed", "op": "train", "n": 5, "total": 1337, "mix": "ragged", "cut": 4, "pad": 0, "heads": 8,
         "d": 64, "dv": 128, "state": True, "decay": "slopes"},
        # a training step at B8 H16 T2048
        {"name": "train_b8_t2048", "op": "train", "n": 8, "total": 16384, "mix": "equal", "cut": 5, "pad": 0,
         "heads": 16, "d": 128, "dv": 128, "state": False, "decay": "retention"},
        # decoding a single stream: latency
        {"name": "step_1", "op": "step", "n": 1, "heads": 16, "d": 128, "dv": 128, "slots": 4, "holes": 0,
         "dtype": "bf16", "decay": "retention"},
        # a full decoding batch
        {"name": "step_64", "op": "step", "n": 64, "heads": 16, "d": 128, "dv": 128, "slots": 64, "holes": 0,
         "dtype": "bf16", "decay": "slopes"},
        # a large batch padded to its bucket, fp32 activations
        {"name": "step_333_f32", "op": "step", "n": 333, "heads": 8, "d": 64, "dv": 128, "slots": 400, "holes": 21,
         "dtype": "f32", "decay": "slopes"},
        # parking three squared-feature states (p = 16: 256 rows), denominators included
        {"name": "store_squared", "op": "store", "n": 3, "heads": 16, "rows": 256, "cols": 64, "slots": 8,
         "entries": 16, "z": True, "holes": 0},
        # the prefixes of a whole batch into the cache
        {"name": "store_batch", "op": "store", "n": 48, "heads": 16, "rows": 128, "cols": 128, "slots": 64,
         "entries": 96, "z": False, "holes": 3},
        # one sequence comes back
        {"name": "load_one", "op": "load", "n": 1, "heads": 16, "rows": 128, "cols": 128, "slots": 4, "entries": 8,
         "z": False, "holes": 0, "fork": False},
        # a batch starts from cached prefixes, several sequences from the same one
        {"name": "load_batch", "op": "load", "n": 48, "heads": 16, "rows": 128, "cols": 128, "slots": 64,
         "entries": 96, "z": False, "holes": 3, "fork": True},
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "train", "train", "step", "step", "store", "load"])
    heads = rng.choice([1, 2, 3, 4, 8, 16, 16, 24, 32])
    d, dv = rng.choice([64, 128]), rng.choice([64, 128])
    decay = rng.choice(["retention", "slopes", "mixed"])
    if op in ("prompt", "train"):
        cap = (131072 if op == "prompt" else 32768) * 16 // max(heads, 8)
        total = _log_uniform(rng, 40, cap)
        n = min(_log_uniform(rng, 1, 64), max(1, total // 8))
        case = {"op": op, "n": n, "total": total, "mix": "ragged", "cut": rng.randrange(1 << 20),
                "pad": rng.choice([0, 0, 1, 50]), "heads": heads, "d": d, "dv": dv, "decay": decay}
        if op == "prompt":
            case.update(resume=rng.random() < 0.5, slots=n + rng.randrange(8))
        else:
            case.update(state=rng.random() < 0.4)
        return case
    if op == "step":
        n = _log_uniform(rng, 1, 512)
        return {"op": op, "n": n, "heads": heads, "d": d, "dv": dv, "slots": n + rng.randrange(n + 4),
                "holes": rng.randrange(1 + n // 8), "dtype": rng.choice(["bf16", "f32"]), "decay": decay}
    n = _log_uniform(rng, 1, 64)
    rows, cols = rng.choice([(64, 64), (64, 128), (128, 64), (128, 128), (256, 64), (256, 16), (1024, 64), (16, 64)])
    case = {"op": op, "n": n, "heads": heads, "rows": rows, "cols": cols, "slots": n + rng.randrange(n + 4),
            "entries": n + rng.randrange(n + 4), "z": rows in (256, 1024), "holes": rng.randrange(1 + n // 8)}
    if op == "load":
        case["fork"] = rng.random() < 0.5
    return case


def _lengths(case):
    """Lengths of the packed sequences: equal, or cut at random places (zero and one occur)."""
    n, total = case["n"], case["total"]
    if case["mix"] == "equal":
        return [total // n] * n
    r = random.Random(case["cut"])
    cuts = sorted(r.randint(0, total) for _ in range(n - 1))
    edges = [0] + cuts + [total]
    return [b - a for a, b in zip(edges, edges[1:])]


def _log_decay(kind, heads):
    """Natural logarithms of the heads' decays: 1 - 2^-(5..12), exp(-2^-(0..8)), or both kinds and none at all."""
    ret = [math.log1p(-2.0 ** -(5 + 7 * h / heads)) for h in range(heads)]
    slo = [-2.0 ** -(8 * (h + 1) / heads) for h in range(heads)]
    if kind == "retention":
        return ret
    if kind == "slopes":
        return slo
    return [(ret[h], slo[h], 0.0)[h % 3] for h in range(heads)]


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _indices(r, count, size, holes):
    """`count` different indices below `size`, `holes` of them replaced by -1 (rows of padding)."""
    idx = r.sample(range(size), count)
    for i in r.sample(range(count), holes):
        idx[i] = -1
    return idx


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = random.Random(seed)

    def normal(*shape, dtype=torch.bfloat16, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    H = case["heads"]
    st = {"case": case}
    if case["op"] in ("prompt", "train"):
        lens = _lengths(case)
        n, T, d, dv = case["n"], case["total"] + case["pad"], case["d"], case["dv"]
        q, k, v = normal(T, H, d), normal(T, H, d), normal(T, H, dv)
        st.update(lens=lens, q=q, k=k, v=v, scale=d ** -0.5,
                  log_decay=torch.tensor(_log_decay(case["decay"], H), dtype=torch.float32, device="cuda"))
        edges = [0]
        for x in lens:
            edges.append(edges[-1] + x)
        st["cu_seqlens"] = ints(edges)
        # what stands behind the last sequence is left over from other batches
        for x in (q, k, v):
            x[case["total"]:] = float("nan")
        if case["op"] == "prompt":
            st["slot_list"] = r.sample(range(case["slots"]), n)
            st["slots"] = ints(st["slot_list"])
            st["S"] = normal(case["slots"], H, d, dv, dtype=torch.float32, std=4.0)
            st["resume_list"] = [case["resume"] and r.random() < 0.5 for _ in range(n)]
            st["resume"] = torch.tensor(st["resume_list"], dtype=torch.uint8, device="cuda")
        else:
            st["dO"] = normal(T, H, dv)
            st["dO"][case["total"]:] = float("nan")
            st["S0"] = normal(n, H, d, dv, dtype=torch.float32, std=4.0) if case["state"] else None
            st["dS"] = normal(n, H, d, dv, dtype=torch.float32, std=0.1) if case["state"] else None
        return st
    if case["op"] == "step":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        n, d, dv = case["n"], case["d"], case["dv"]
        st.update(q=normal(n, H, d, dtype=dt), k=normal(n, H, d, dtype=dt), v=normal(n, H, dv, dtype=dt),
                  S=normal(case["slots"], H, d, dv, dtype=torch.float32, std=4.0), scale=d ** -0.5,
                  log_decay=torch.tensor(_log_decay(case["decay"], H), dtype=torch.float32, device="cuda"))
        st["slot_list"] = _indices(r, n, case["slots"], case["holes"])
        st["slots"] = ints(st["slot_list"])
        return st
    # states and their cache; row magnitudes differ, as those of accumulated features do
    n, rows, cols = case["n"], case["rows"], case["cols"]
    ns, ne = case["slots"], case["entries"]

    def states(m):
        return normal(m, H, rows, cols, dtype=torch.float32) * torch.exp(normal(m, H, rows, 1, dtype=torch.float32))

    st["S"] = states(ns)
    st["z"] = states(ns)[..., 0].abs().contiguous() if case["z"] else None
    full = states(ne)
    st["scales"] = full.abs().amax(-1) / 127
    st["cache"] = torch.round(full / st["scales"][..., None]).clamp_(-127, 127).to(torch.int8)
    st["z_cache"] = full[..., 0].abs().contiguous() if case["z"] else None
    slots, entries = _indices(r, n, ns, 0), _indices(r, n, ne, 0)
    if case.get("fork"):
        entries = [entries[i // 3] for i in range(n)]
    for i in r.sample(range(n), case["holes"]):
        slots[i] = entries[i] = -1
    st.update(slot_list=slots, entry_list=entries, slots=ints(slots), entries=ints(entries))
    if case["op"] == "store":
        st["all"] = ints(range(ne))
        st["mirror"] = torch.empty_like(full)
        st["z_mirror"] = torch.empty_like(st["z_cache"]) if case["z"] else None
    return st


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------
def _chunked(q, k, v, log_decay, S0):
    """One sequence, heads first ([H, T, *], fp32): o_t = q_t^T S_t and the final state, chunk by chunk."""
    H, T, d = q.shape
    dv = v.shape[-1]
    C = min(CHUNK, T)
    n = (T + C - 1) // C
    fill = n * C - T
    if fill:
        q, k, v = (torch.nn.functional.pad(x, (0, 0, 0, fill)) for x in (q, k, v))
    q, k, v = (x.reshape(H, n, C, x.shape[-1]) for x in (q, k, v))
    i = torch.arange(C, device=q.device, dtype=torch.float32)
    g = log_decay[:, None, None]
    away = i[:, None] - i[None, :]
    weight = torch.where(away >= 0, torch.exp(g * away.clamp(min=0)), torch.zeros((), device=q.device))  # [H, C, C]
    o = torch.matmul(torch.matmul(q, k.transpose(-1, -2)) * weight[:, None], v)
    # tokens of each chunk: the last may be shorter
    count = torch.full((n,), float(C), device=q.device)
    count[-1] = T - (n - 1) * C
    left = (count[:, None] - 1 - i[None, :]).clamp(min=0)                                   # [n, C]
    add = torch.matmul((k * torch.exp(g * left)[..., None]).transpose(-1, -2), v)            # [H, n, d, dv]
    keep = torch.exp(log_decay[:, None] * count)                                            # [H, n]
    S = torch.zeros(H, d, dv, device=q.device) if S0 is None else S0
    before = torch.empty_like(add)
    for c in range(n):
        before[:, c] = S
        S = S * keep[:, c, None, None] + add[:, c]
    o = o + torch.exp(g * (i + 1))[..., None] * torch.matmul(q, before)
    return o.reshape(H, n * C, dv)[:, :T], S


def _heads_first(x):
    return x.float().transpose(0, 1)


def _plain_prompt(st):
    o = torch.zeros_like(st["v"])
    S = st["S"]
    a = 0
    for x, slot, resume in zip(st["lens"], st["slot_list"], st["resume_list"]):
        if x == 0:
            if not resume:
                S[slot] = 0
            continue
        q, k, v = (_heads_first(st[name][a:a + x]) for name in ("q", "k", "v"))
        y, S1 = _chunked(q, k, v, st["log_decay"], S[slot] if resume else None)
        o[a:a + x] = (y * st["scale"]).transpose(0, 1).to(o.dtype)
        S[slot] = S1
        a += x
    return o, S


def _plain_train(st):
    q_all, k_all, v_all, dO_all = st["q"], st["k"], st["v"], st["dO"]
    dq, dk, dv = torch.zeros_like(q_all), torch.zeros_like(k_all), torch.zeros_like(v_all)
    state = st["S0"] is not None
    dS0 = torch.empty_like(st["S0"]) if state else None
    g, scale = st["log_decay"], st["scale"]
    keep = torch.exp(g)[:, None, None]
    a = 0
    for s, x in enumerate(st["lens"]):
        if x == 0:
            if state:
                dS0[s] = st["dS"][s]
            continue
        part = slice(a, a + x)
        q, k, v, dO = (_heads_first(t[part]) for t in (q_all, k_all, v_all, dO_all))
        dO = dO * scale
        y, _ = _chunked(dO, v, k, g, st["S0"][s].transpose(-1, -2) if state else None)
        dq[part] = y.transpose(0, 1).to(dq.dtype)
        # backwards in time: R_t = a R_{t+1} + q_t dO_t^T with R_{T+1} = dS / a
        rq, rk, rv, rdO = (t.flip(1) for t in (q, k, v, dO))
        R = st["dS"][s] / keep if state else None
        y, _ = _chunked(rv, rdO, rq, g, R.transpose(-1, -2) if state else None)
        dk[part] = y.flip(1).transpose(0, 1).to(dk.dtype)
        y, R = _chunked(rk, rq, rdO, g, R)
        dv[part] = y.flip(1).transpose(0, 1).to(dv.dtype)
        if state:
            dS0[s] = R * keep
        a += x
    return (dq, dk, dv, dS0) if state else (dq, dk, dv)


def _plain_step(st):
    S = st["S"]
    live = st["slots"] >= 0
    slot = st["slots"][live].long()
    q, k, v = (st[name][live].float() for name in ("q", "k", "v"))
    new = S[slot] * torch.exp(st["log_decay"])[:, None, None] + k[..., :, None] * v[..., None, :]
    S[slot] = new
    o = torch.zeros_like(st["v"])
    o[live] = ((q[..., :, None] * new).sum(-2) * st["scale"]).to(o.dtype)
    return o, S


def _plain_store(st):
    live = st["slots"] >= 0
    slot, entry = st["slots"][live].long(), st["entries"][live].long()
    x = st["S"][slot]
    scale = (x.abs().amax(-1).double() / 127).float()
    scale = torch.where(scale < MIN_SCALE, torch.zeros_like(scale), scale)
    # next to a border between two integers 32 bits would round the quotient across it
    y = torch.round(x.double() / scale.double()[..., None]).nan_to_num(nan=0.0)
    st["cache"][entry] = y.to(torch.int8)
    st["scales"][entry] = scale
    torch.mul(st["cache"], st["scales"][..., None], out=st["mirror"])
    if st["z"] is None:
        return [st["scales"], st["mirror"]]
    st["z_cache"][entry] = st["z"][slot]
    st["z_mirror"].copy_(st["z_cache"])
    return [st["scales"], st["mirror"], st["z_mirror"]]


def _plain_load(st):
    live = st["slots"] >= 0
    slot, entry = st["slots"][live].long(), st["entries"][live].long()
    st["S"][slot] = st["cache"][entry].float() * st["scales"][entry][..., None]
    if st["z"] is None:
        return [st["S"]]
    st["z"][slot] = st["z_cache"][entry]
    return [st["S"], st["z"]]


# --------------------------------------------------------------------------
# the calls
# --------------------------------------------------------------------------
def _own(st):
    import kernelized_feature_map_b200 as K
    op = st["case"]["op"]
    if op == "prompt":
        o = K.kata_fwd_linear_decay(st["q"], st["k"], st["v"], st["log_decay"], cu_seqlens=st["cu_seqlens"],
                                    scale=st["scale"], S0=st["S"], S_out=st["S"], slots=st["slots"],
                                    resume=st["resume"])
        return o, st["S"]
    if op == "train":
        state = st["S0"] is not None
        return K.kata_bwd_linear_decay(st["q"], st["k"], st["v"], st["dO"], st["log_decay"],
                                       cu_seqlens=st["cu_seqlens"], scale=st["scale"], S0=st["S0"], dS_out=st["dS"],
                                       return_dS0=state)
    if op == "step":
        o = K.kata_decode_step_linear_decay(st["q"], st["k"], st["v"], st["S"], st["log_decay"], slots=st["slots"],
                                            scale=st["scale"])
        return o, st["S"]
    if op == "store":
        K.kata_state_store_q8(st["S"], st["cache"], st["scales"], st["slots"], st["entries"], z=st["z"],
                              z_cache=st["z_cache"])
        K.kata_state_load_q8(st["cache"], st["scales"], st["mirror"], st["all"], st["all"], z=st["z_mirror"],
                             z_cache=st["z_cache"])
        return [st["scales"], st["mirror"]] + ([] if st["z"] is None else [st["z_mirror"]])
    K.kata_state_load_q8(st["cache"], st["scales"], st["S"], st["entries"], st["slots"], z=st["z"],
                         z_cache=st["z_cache"])
    return [st["S"]] if st["z"] is None else [st["S"], st["z"]]


_PLAIN = {"prompt": _plain_prompt, "train": _plain_train, "step": _plain_step, "store": _plain_store,
          "load": _plain_load}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------
def work(case):
    H, op, n = case["heads"], case["op"], case["n"]
    if op in ("prompt", "train"):
        d, dv, tokens = case["d"], case["dv"], case["total"] * H
        state = 4 * n * H * d * dv
        if op == "prompt":
            moved = 2 * tokens * (2 * d + 2 * dv) + state * (1.5 if case["resume"] else 1)
            return {"bytes": int(moved + 4 * (n + 1 + H + n)), "flops": 4 * tokens * d * dv}
        moved = 2 * tokens * (4 * d + 3 * dv) + (3 * state if case["state"] else 0)
        return {"bytes": moved + 4 * (n + 1 + H), "flops": 10 * tokens * d * dv}
    live = n - case["holes"]
    if op == "step":
        d, dv = case["d"], case["dv"]
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": live * H * (8 * d * dv + size * (2 * d + 2 * dv)) + 4 * (n + H), "flops": 5 * live * H * d * dv}
    rows, cols = case["rows"], case["cols"]
    z = 8 if case["z"] else 0
    if op == "store":
        each = H * rows * (5 * cols + 4 + z)
        return {"bytes": (live + case["entries"]) * each + 8 * n, "flops": H * rows * cols * (3 * live + case["entries"])}
    read = (n + 2) // 3 if case["fork"] else live
    return {"bytes": H * rows * (read * (cols + 4 + z // 2) + live * (4 * cols + z // 2)) + 8 * n,
            "flops": live * H * rows * cols}


# --------------------------------------------------------------------------
# from the definitions, in 64 bits
# --------------------------------------------------------------------------
def _pair_blocks(x, H, log_decay):
    """The decays a^(t-s) of all pairs s <= t < x, in blocks of rows: (first row, end, [H, rows, end])."""
    step = max(16, min(2048, int(2e8 / (max(1, x) * H))))
    g = log_decay.double()[:, None, None]
    for t0 in range(0, x, step):
        t1 = min(x, t0 + step)
        away = (torch.arange(t0, t1, device=g.device)[:, None] - torch.arange(t1, device=g.device)[None, :]).double()
        yield t0, t1, torch.exp(g * away).masked_fill_(away < 0, 0.0)


def exact(case, seed):
    if case["op"] in ("prompt", "train") and sum(x * x for x in _lengths(case)) * case["heads"] > 3e11:
        return None
    st = prepare(case, seed)
    H, op = case["heads"], case["op"]
    if op in ("prompt", "train"):
        g = st["log_decay"].double()
        a = 0
        if op == "prompt":
            o, S = torch.zeros_like(st["v"], dtype=torch.float64), st["S"].double()
        else:
            dq, dk, dv = (torch.zeros_like(st[name], dtype=torch.float64) for name in ("q", "k", "v"))
            state = st["S0"] is not None
            dS0 = torch.zeros_like(st["S0"], dtype=torch.float64) if state else None
        for s, x in enumerate(st["lens"]):
            part = slice(a, a + x)
            a += x
            q, k, v = (st[name][part].double().transpose(0, 1) for name in ("q", "k", "v"))
            t = torch.arange(x, device=g.device, dtype=torch.float64)
            since = torch.exp(g[:, None] * (t + 1))[..., None]         # a^(t+1): reach of the initial state
            until = torch.exp(g[:, None] * (x - 1 - t))[..., None]     # a^(T-1-t): share in the final state
            if op == "prompt":
                slot = st["slot_list"][s]
                S0 = S[slot].clone() if st["resume_list"][s] else torch.zeros_like(S[slot])
                y = since * (q @ S0)
                for t0, t1, w in _pair_blocks(x, H, st["log_decay"]):
                    y[:, t0:t1] += (q[:, t0:t1] @ k[:, :t1].transpose(-1, -2) * w) @ v[:, :t1]
                o[part] = (y * st["scale"]).transpose(0, 1)
                S[slot] = torch.exp(g * x)[:, None, None] * S0 + (until * k).transpose(-1, -2) @ v
                continue
            dO = st["dO"][part].double().transpose(0, 1) * st["scale"]
            eq, ek, ev = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
            if state:
                S0, dS = st["S0"][s].double(), st["dS"][s].double()
                eq += since * (dO @ S0.transpose(-1, -2))
                ek += until * (v @ dS.transpose(-1, -2))
                ev += until * (k @ dS)
                dS0[s] = torch.exp(g * x)[:, None, None] * dS + (since * q).transpose(-1, -2) @ dO
            for t0, t1, w in _pair_blocks(x, H, st["log_decay"]):
                pair = dO[:, t0:t1] @ v[:, :t1].transpose(-1, -2) * w
                eq[:, t0:t1] += pair @ k[:, :t1]
                ek[:, :t1] += pair.transpose(-1, -2) @ q[:, t0:t1]
                pair = q[:, t0:t1] @ k[:, :t1].transpose(-1, -2) * w
                ev[:, :t1] += pair.transpose(-1, -2) @ dO[:, t0:t1]
            dq[part], dk[part], dv[part] = (e.transpose(0, 1) for e in (eq, ek, ev))
        if op == "prompt":
            return o, S
        return (dq, dk, dv, dS0) if state else (dq, dk, dv)
    if op == "step":
        S, o = st["S"].double(), torch.zeros_like(st["v"], dtype=torch.float64)
        a = torch.exp(st["log_decay"].double())[:, None, None]
        for i, slot in enumerate(st["slot_list"]):
            if slot >= 0:
                q, k, v = (st[name][i].double() for name in ("q", "k", "v"))
                S[slot] = a * S[slot] + k[:, :, None] * v[:, None, :]
                o[i] = st["scale"] * torch.einsum("hi,hij->hj", q, S[slot])
        return o, S
    pairs = [(s, e) for s, e in zip(st["slot_list"], st["entry_list"]) if s >= 0]
    if op == "load":
        S = st["S"].double()
        z = st["z"].double() if case["z"] else None
        for s, e in pairs:
            S[s] = st["cache"][e].double() * st["scales"][e].double()[..., None]
            if case["z"]:
                z[s] = st["z_cache"][e].double()
        return [S, z] if case["z"] else [S]
    scales = st["scales"].double()
    mirror = st["cache"].double() * scales[..., None]
    zc = st["z_cache"].double() if case["z"] else None
    for s, e in pairs:
        x = st["S"][s].double()
        scale = (x.abs().max(dim=-1).values / 127).float().double()
        scales[e] = scale.masked_fill(scale < MIN_SCALE, 0.0)
        mirror[e] = torch.round(x / scale[..., None]) * scale[..., None]
        if case["z"]:
            zc[e] = st["z"][s].double()
    return [scales, mirror, zc] if case["z"] else [scales, mirror]
