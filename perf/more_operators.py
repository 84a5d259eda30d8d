"""The gated delta rule and the query/key preparation as measured work: cases, inputs, plain forms and exact values.

Five operators. `qk` (norms of queries and keys for each head and their rotation by positions on several axes, in one
pass) and `qk_grad` (its backward pass); `delta` (the gated delta rule over whole sequences), `delta_grad` (its backward
pass) and `delta_step` (one token of each of several streams, on states that lie in a cache).

The gated delta rule, for each value head (a = exp(g), S [dk, dv] the head's fast weights):

    p_t = a_t S_{t-1}^T k_t,   u_t = beta_t (v_t - p_t),   S_t = a_t S_{t-1} + k_t u_t^T,   o_t = scale S_t^T q_t

Value head h reads key head h // (value heads / key heads). Rows of q, k [n, key heads * dk], v [n, value heads * dv],
g, beta [n, value heads]; sequence b is rows cu[b] .. cu[b + 1].
"""
import math
import random

import torch

own = False

DEV = "cuda"
VIEW = 1374  # tokens of one view: 5 special ones and 37 x 37 patches
SPECIAL, GRID = 5, 37
BASE = 100.0  # rotation: the slowest pair of an axis of 16 pairs turns by 0.013 a patch
EPS = {"l2": 1e-12, "rms": 1e-6, "layer": 1e-6, "none": 0.0}
CHUNK = 64  # the plain form's


# ----------------------------------------------------------------------------------------------------------- cases
def listed():
    rows = {"per_axis": True, "interleaved": False}
    heads = {"hk": 16, "hv": 16, "dk": 64, "dv": 64}
    return [
        # queries and keys of one view before the layer: L2 norms, rotation by patch row and column
        {"name": "qk_view", "op": "qk", "n": VIEW, "h": 16, "hk": 16, "d": 64, "dtype": "bf16", "norm": "l2",
         "axes": "yx", "start": 0, **rows},
        # the queries and keys of a 100-view scene: RMS norms with weights, rotation by view, row and column
        {"name": "qk_scene", "op": "qk", "n": 100 * VIEW, "h": 16, "hk": 16, "d": 64, "dtype": "bf16", "norm": "rms",
         "axes": "tyx", "start": 0, **rows},
        # the gradient for one view in fp32, layer norms with weights and biases
        {"name": "qk_grad_view", "op": "qk_grad", "n": VIEW, "h": 16, "hk": 16, "d": 64, "dtype": "f32",
         "norm": "layer", "axes": "yx", "start": 0, **rows},
        # the gradient for a training batch of 48 views
        {"name": "qk_grad_batch", "op": "qk_grad", "n": 48 * VIEW, "h": 16, "hk": 16, "d": 64, "dtype": "bf16",
         "norm": "rms", "axes": "tyx", "start": 0, **rows},
        # one more view of a stream, from the state that the views before it left
        {"name": "delta_view", "op": "delta", "n": VIEW, "seqs": 1, **heads, "dtype": "bf16", "gate": True, "state": True},
        # a 100-view scene as one sequence
        {"name": "delta_scene", "op": "delta", "n": 100 * VIEW, "seqs": 1, **heads, "dtype": "bf16", "gate": True,
         "state": False},
        # 24 views' worth of tokens in 10 ragged sequences, fp32, two value heads to a key head
        {"name": "delta_ragged", "op": "delta", "n": 24 * VIEW, "seqs": 10, "hk": 8, "hv": 16, "dk": 64, "dv": 64,
         "dtype": "f32", "gate": True, "state": True},
        # training on one short scene in fp32
        {"name": "delta_grad_view", "op": "delta_grad", "n": VIEW, "seqs": 1, **heads, "dtype": "f32", "gate": True,
         "state": True},
        # training on a batch of 48 views, each a sequence of about a view's length
        {"name": "delta_grad_batch", "op": "delta_grad", "n": 48 * VIEW, "seqs": 48, **heads, "dtype": "bf16",
         "gate": True, "state": False},
        # wide heads: 8 of 128 x 128, 16 ragged sequences
        {"name": "delta_grad_wide", "op": "delta_grad", "n": 12 * VIEW, "seqs": 16, "hk": 8, "hv": 8, "dk": 128,
         "dv": 128, "dtype": "bf16", "gate": True, "state": True},
        # one stream, one token: latency counts
        {"name": "step_one", "op": "delta_step", "rows": 1, "slots": 4, **heads, "dtype": "bf16", "gate": True},
        # 256 streams out of a cache of 320 states, one token each
        {"name": "step_many", "op": "delta_step", "rows": 256, "slots": 320, **heads, "dtype": "bf16", "gate": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk", "qk_grad", "delta", "delta", "delta_grad", "delta_step"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op in ("qk", "qk_grad"):
        d = rng.choice([32, 64, 64, 72, 96, 128])
        h = rng.choice([1, 3, 8, 12, 16])
        hk = rng.choice([h, 1, h if h % 4 else h // 4])
        most = 100 if op == "qk" else 48
        n = _log(rng, 1, most * VIEW * 1024 // (d * h * (2 if dtype == "f32" else 1)))
        return {"op": op, "n": min(n, 4 * most * VIEW), "h": h, "hk": hk, "d": d, "dtype": dtype,
                "norm": rng.choice(["l2", "l2", "rms", "layer", "none"]), "axes": rng.choice(["yx", "tyx", "t"]),
                "start": rng.choice([0, 0, _log(rng, 1, 1000000)]), "per_axis": rng.random() < 0.6,
                "interleaved": rng.random() < 0.4}
    hk, group = rng.choice([(16, 1), (8, 2), (4, 4), (3, 1), (16, 1)])
    dk, dv = rng.choice([(64, 64), (64, 64), (128, 128), (64, 128), (128, 64)])
    shape = {"hk": hk, "hv": hk * group, "dk": dk, "dv": dv, "dtype": dtype, "gate": rng.random() < 0.85}
    cost = hk * group * dk * dv / (16 * 64 * 64) * (2 if dtype == "f32" else 1)
    if op == "delta_step":
        rows = _log(rng, 1, max(1, int(256 / cost)))
        return {"op": op, "rows": rows, "slots": rows + _log(rng, 1, 64), **shape}
    n = _log(rng, 1, max(1, int((100 if op == "delta" else 40) * VIEW / cost)))
    seqs = _log(rng, 1, 64)
    if op == "delta_grad":
        seqs = max(seqs, -(-n // (4 * VIEW)))  # a training sequence is a few views long
    return {"op": op, "n": n, "seqs": seqs, **shape, "state": rng.random() < 0.5}


def _lens(case):
    """The lengths of a case's sequences: ragged, some of them empty where there are more sequences than tokens."""
    n, seqs = case["n"], case["seqs"]
    r = random.Random(n * 131 + seqs)
    w = [r.uniform(0.5, 1.0) for _ in range(seqs)]
    cuts = [round(n * sum(w[:i]) / sum(w)) for i in range(seqs + 1)]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _sections(case):
    """Pairs of channels that each axis turns: an eighth, or a third, of the head's channels."""
    axes, d = case["axes"], case["d"]
    each = d // 2 // len(axes) // 2 * 2
    return [each] * len(axes)


# ---------------------------------------------------------------------------------------------------------- inputs
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _randn(shape, seed, stream, std=1.0, dtype=torch.float32):
    g = torch.Generator(device=DEV).manual_seed(int(seed) * 64 + stream)
    return (torch.randn(shape, generator=g, device=DEV) * std).to(dtype)


def _unit(x, heads):
    x = x.view(x.shape[0], heads, -1)
    return (x / x.norm(dim=-1, keepdim=True).clamp(min=1e-12)).flatten(1)


def prepare(case, seed):
    dt, s = _dtype(case["dtype"]), dict(case)
    if case["op"] in ("qk", "qk_grad"):
        n, d = case["n"], case["d"]
        for i, (x, h) in enumerate((("q", case["h"]), ("k", case["hk"]))):
            s[x] = _randn((n, h * d), seed, 1 + i, 1.5, dt)
            s[x + "_w"] = _randn((d,), seed, 3 + i, 0.2) + 1 if case["norm"] in ("rms", "layer") else None
            s[x + "_b"] = _randn((d,), seed, 5 + i, 0.1) if case["norm"] == "layer" else None
            if case["op"] == "qk_grad":
                s["d" + x] = _randn((n, h * d), seed, 7 + i, 1.0, dt)
        # tokens view by view: special tokens at (0, 0), patches from (1, 1) on
        t = torch.arange(n, device=DEV)
        view, p = t // VIEW, t % VIEW - SPECIAL
        at = {"t": view if "y" in case["axes"] else t, "y": torch.where(p < 0, 0, p // GRID + 1),
              "x": torch.where(p < 0, 0, p % GRID + 1)}
        s["pos"] = torch.stack([at[a] + (case["start"] if a == "t" else 0) for a in case["axes"]], 1).to(torch.int32)
        return s
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    n = case["rows"] if case["op"] == "delta_step" else case["n"]
    s["q"] = _unit(_randn((n, hk * dk), seed, 1), hk).to(dt)
    s["k"] = _unit(_randn((n, hk * dk), seed, 2), hk).to(dt)
    s["v"] = _randn((n, hv * dv), seed, 3, 1.0, dt)
    # decays from almost none to a few tokens' memory, by head and token
    rate = torch.exp(_randn((1, hv), seed, 4, 1.5) - 3)
    s["g"] = -rate * torch.nn.functional.softplus(_randn((n, hv), seed, 5)) if case["gate"] else None
    s["beta"] = torch.sigmoid(_randn((n, hv), seed, 6))
    if case["op"] == "delta_step":
        s["state"] = _randn((case["slots"], hv, dk, dv), seed, 7, 0.3)
        g = torch.Generator(device=DEV).manual_seed(int(seed) * 64 + 8)
        s["slot"] = torch.randperm(case["slots"], generator=g, device=DEV)[:n].to(torch.int32)
        return s
    s["lens"] = _lens(case)
    s["cu"] = torch.tensor([0] + s["lens"], device=DEV).cumsum(0).to(torch.int32)
    s["state"] = _randn((case["seqs"], hv, dk, dv), seed, 7, 0.3) if case["state"] else None
    if case["op"] == "delta_grad":
        s["do"] = _randn((n, hv * dv), seed, 9, 1.0, dt)
        s["dstate"] = _randn((case["seqs"], hv, dk, dv), seed, 10, 0.3) if case["state"] else None
    return s


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["op"] in ("qk", "qk_grad"):
        values = case["n"] * (case["h"] + case["hk"]) * case["d"]
        return {"bytes": values * e * (2 if case["op"] == "qk" else 3) + 4 * case["n"] * len(case["axes"]), "flops": 0}
    hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
    n = case["rows"] if case["op"] == "delta_step" else case["n"]
    keys, values, scalars = n * hk * dk * e, n * hv * dv * e, 4 * n * hv * (2 if case["gate"] else 1)
    one = 4 * hv * dk * dv  # the fp32 state of a sequence
    rule = 6 * n * hv * dk * dv  # p, the update and o, a multiply and an add a weight each
    if case["op"] == "delta_step":
        return {"bytes": 2 * keys + 2 * values + scalars + 2 * n * one + 4 * n, "flops": rule}
    states = case["seqs"] * one
    if case["op"] == "delta":
        return {"bytes": 2 * keys + 2 * values + scalars + states * (1 + case["state"]), "flops": rule}
    return {"bytes": 4 * keys + 3 * values + 2 * scalars + states * 3 * case["state"], "flops": 3 * rule}


# -------------------------------------------------------------------------------------- queries and keys, plain form
def _rope_plan(s):
    """(first channel, second channel, turns a position step in 64 bits, axis) of each rotated pair."""
    sec = _sections(s)
    per, inter = s["per_axis"], s["interleaved"]
    a = torch.tensor([i for i, c in enumerate(sec) for _ in range(c)])
    within = torch.tensor([j for c in sec for j in range(c)])
    total = sum(sec)
    size = torch.tensor([c for c in sec for _ in range(c)]) if per else torch.full((total,), total)
    j = within if per else torch.arange(total)
    off = torch.tensor([2 * sum(sec[:i]) for i, c in enumerate(sec) for _ in range(c)]) if per else torch.zeros(total, dtype=torch.long)
    first = off + (2 * j if inter else j)
    second = first + 1 if inter else first + size
    freq = torch.pow(torch.tensor(BASE, dtype=torch.float64), -(j.double() / size.double()))
    return tuple(t.to(DEV) for t in (first, second, freq, a))


def _angles(s):
    first, second, freq, axis = _rope_plan(s)
    ang = s["pos"].double()[:, axis] * freq
    return first, second, torch.cos(ang).float(), torch.sin(ang).float()


def _rotate(x, plan, back=False):
    first, second, cos, sin = plan
    cos, sin = cos[:, None], -sin[:, None] if back else sin[:, None]
    y = x.clone()
    a, b = x[..., first], x[..., second]
    y[..., first] = a * cos - b * sin
    y[..., second] = b * cos + a * sin
    return y


def _head_norm(x, norm, w, b):
    """(normalised, 1 / deviation, weighted) of x [n, heads, d]."""
    eps = EPS[norm]
    if norm == "none":
        return x, None, x
    if norm == "l2":
        r = 1 / x.square().sum(-1, keepdim=True).sqrt().clamp(min=eps)
        return x * r, r, x * r
    if norm == "layer":
        x = x - x.mean(-1, keepdim=True)
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    return x * r, r, x * r * w if b is None else x * r * w + b


def _qk_plain(s):
    plan = _angles(s)
    out = {}
    for x, h in (("q", s["h"]), ("k", s["hk"])):
        v = s[x].float().view(s["n"], h, s["d"])
        y = _head_norm(v, s["norm"], s[x + "_w"], s[x + "_b"])[2]
        out[x] = _rotate(y, plan).flatten(1).to(s[x].dtype)
    return out


def _qk_grad_plain(s):
    plan = _angles(s)
    out = {}
    for x, h in (("q", s["h"]), ("k", s["hk"])):
        v = s[x].float().view(s["n"], h, s["d"])
        d = _rotate(s["d" + x].float().view(s["n"], h, s["d"]), plan, back=True)
        hat, r, _ = _head_norm(v, s["norm"], s[x + "_w"], s[x + "_b"])
        if s[x + "_b"] is not None:
            out["d" + x + "_b"] = d.sum((0, 1))
        if s[x + "_w"] is not None:
            out["d" + x + "_w"] = (d * hat).sum((0, 1))
            d = d * s[x + "_w"]
        if s["norm"] == "l2":
            d = (d - hat * (d * hat).sum(-1, keepdim=True)) * r
        elif s["norm"] != "none":
            d = d - hat * (d * hat).mean(-1, keepdim=True) - (d.mean(-1, keepdim=True) if s["norm"] == "layer" else 0)
            d = d * r
        out["d" + x] = d.flatten(1).to(s[x].dtype)
    return out


# ------------------------------------------------------------------------------------------- delta rule, plain form
def _padded(s):
    """(rows [sequences, chunks, CHUNK] with -1 where there is none, rows by index)"""
    lens = torch.tensor(s["lens"], device=DEV)
    m = max(1, -(-max(s["lens"]) // CHUNK))
    t = torch.arange(m * CHUNK, device=DEV)
    rows = torch.where(t < lens[:, None], s["cu"][:-1, None].long() + t, -1)
    return rows.view(len(s["lens"]), m, CHUNK)


def _take(x, rows, heads, group=1):
    """x [n, heads * d] as fp32 [sequences, chunks, heads, CHUNK, d], zeros where there is no row."""
    x = torch.cat([x.float(), x.new_zeros((1, x.shape[1]), dtype=torch.float32)])[rows]
    x = x.unflatten(-1, (heads, -1)).transpose(2, 3)
    return x.repeat_interleave(group, 2) if group > 1 else x


def _put(x, rows, n):
    """The rows of x [sequences, chunks, heads, CHUNK, d] back at their places [n, heads * d]."""
    y = x.new_empty((n + 1, x.shape[2] * x.shape[4]))
    y[rows] = x.transpose(2, 3).flatten(3)
    return y[:n]


def _chunk_parts(s):
    rows, group = _padded(s), s["hv"] // s["hk"]
    p = {"rows": rows, "q": _take(s["q"], rows, s["hk"], group), "k": _take(s["k"], rows, s["hk"], group),
         "v": _take(s["v"], rows, s["hv"]), "beta": _take(s["beta"], rows, s["hv"])}
    g = torch.zeros_like(p["beta"][..., 0]) if s["g"] is None else _take(s["g"], rows, s["hv"])[..., 0]
    G = g.double().cumsum(-1)
    low = torch.ones((CHUNK, CHUNK), dtype=torch.bool, device=DEV).tril()
    p["D"] = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -math.inf)).float()
    p["decay"] = torch.exp(G)[..., None].float()  # from the chunk's start to each token
    p["rest"] = torch.exp(G[..., -1:] - G)[..., None].float()  # from each token to the chunk's end
    p["N"] = p["D"] * torch.matmul(p["k"], p["k"].mT)
    p["N"] = p["N"].tril(-1)
    L = p["N"] * p["beta"].mT
    T = torch.eye(CHUNK, device=DEV).expand(L.shape).contiguous()
    for i in range(1, CHUNK):
        T[..., i, :i] = -torch.matmul(L[..., i:i + 1, :i], T[..., :i, :i])[..., 0, :]
    p["T"] = T
    p["B"] = p["D"] * torch.matmul(p["q"], p["k"].mT)
    return p


def _first_state(s, p):
    if s["state"] is not None:
        return s["state"].clone()
    return torch.zeros((len(s["lens"]), s["hv"], s["dk"], s["dv"]), device=DEV)


def _scan(s, p):
    """The chunks one after the other: (state before each, its y, the last state)."""
    S = _first_state(s, p)
    before, ys = [], []
    for c in range(p["k"].shape[1]):
        k = p["k"][:, c]
        y = torch.matmul(p["T"][:, c], p["v"][:, c] - p["decay"][:, c] * torch.matmul(k, S))
        before.append(S)
        ys.append(y)
        S = p["decay"][:, c, :, -1:] * S + torch.matmul((k * p["rest"][:, c]).mT, p["beta"][:, c] * y)
    return torch.stack(before, 1), torch.stack(ys, 1), S


def _delta_plain(s):
    p = _chunk_parts(s)
    S, y, last = _scan(s, p)
    o = p["decay"] * torch.matmul(p["q"], S) + torch.matmul(p["B"], p["beta"] * y)
    return {"o": _put(o, p["rows"], s["n"]).to(s["v"].dtype), "state": last}


def _delta_grad_plain(s):
    p = _chunk_parts(s)
    S, y, last = _scan(s, p)
    q, k, v, beta, D = p["q"], p["k"], p["v"], p["beta"], p["D"]
    do = _take(s["do"], p["rows"], s["hv"])
    u = beta * y
    dS = torch.zeros_like(last) if s["dstate"] is None else s["dstate"].clone()
    after, dus, dRs = [], [], []
    for c in reversed(range(k.shape[1])):
        du = torch.matmul(p["B"][:, c].mT, do[:, c]) + p["rest"][:, c] * torch.matmul(k[:, c], dS)
        dR = torch.matmul(p["T"][:, c].mT, beta[:, c] * du)
        after.append(dS)
        dus.append(du)
        dRs.append(dR)
        w = p["decay"][:, c]
        dS = w[:, :, -1:] * dS + torch.matmul((q[:, c] * w).mT, do[:, c]) - torch.matmul((k[:, c] * w).mT, dR)
    after, du, dR = (torch.stack(t[::-1], 1) for t in (after, dus, dRs))
    F = D * torch.matmul(do, u.mT)
    E = torch.tril(D * torch.matmul(dR, y.mT), -1)  # beta of its column left out
    Eb = E * beta.mT
    dq = p["decay"] * torch.matmul(do, S.mT) + torch.matmul(F, k)
    dk = torch.matmul(F.mT, q) + p["rest"] * torch.matmul(u, after.mT) - p["decay"] * torch.matmul(dR, S.mT)
    dk = dk - torch.matmul(Eb, k) - torch.matmul(Eb.mT, k)
    dbeta = (du * y).sum(-1) - (E * torch.matmul(k, k.mT)).sum(-2)
    out = {}
    group = s["hv"] // s["hk"]
    for name, x in (("dq", dq), ("dk", dk)):
        x = x.unflatten(2, (s["hk"], group)).sum(3)
        out[name] = _put(x, p["rows"], s["n"]).to(s["q"].dtype)
    out["dv"] = _put(dR, p["rows"], s["n"]).to(s["v"].dtype)
    out["dbeta"] = _put(dbeta.unsqueeze(-1), p["rows"], s["n"])
    if s["g"] is not None:
        # from each token to its chunk's end, and what the chunks behind it say
        end = p["decay"][..., -1:, :] * S + torch.matmul((k * p["rest"]).mT, u)
        dG = ((q * dq).sum(-1) - (v * dR).sum(-1)).double()
        dg = dG.flip(-1).cumsum(-1).flip(-1) + (after * end).double().sum((-1, -2)).unsqueeze(-1)
        out["dg"] = _put(dg.float().unsqueeze(-1), p["rows"], s["n"])
    if s["state"] is not None:
        out["dstate"] = dS
    return out


def _step_plain(s):
    n, group = s["rows"], s["hv"] // s["hk"]
    at = s["slot"].long()
    q, k = (s[x].float().view(n, s["hk"], s["dk"], 1).repeat_interleave(group, 1) for x in ("q", "k"))
    v = s["v"].float().view(n, s["hv"], 1, s["dv"])
    S = s["state"][at]
    if s["g"] is not None:
        S = S * torch.exp(s["g"])[..., None, None]
    S = S + k * (s["beta"][..., None, None] * (v - (S * k).sum(-2, keepdim=True)))
    s["state"][at] = S
    return {"o": (S * q).sum(-2).flatten(1).to(s["v"].dtype), "state": s["state"]}


# ------------------------------------------------------------------------------------------------------------ run
def _run_own(s):
    import test_layer_amd as tla

    op = s["op"]
    if op in ("qk", "qk_grad"):
        args = dict(n_heads=s["h"], n_heads_k=s["hk"], norm=s["norm"], q_w=s["q_w"], k_w=s["k_w"], eps=EPS[s["norm"]],
                    pos=s["pos"], sections=_sections(s), base=BASE, per_axis=s["per_axis"], interleaved=s["interleaved"])
        if op == "qk":
            q, k = tla.qk_norm_rope(s["q"], s["k"], q_b=s["q_b"], k_b=s["k_b"], **args)
            return {"q": q, "k": k}
        got = tla.qk_norm_rope_grad(s["q"], s["k"], s["dq"], s["dk"], bias=s["q_b"] is not None, **args)
        return {name: x for name, x in got._asdict().items() if x is not None}
    if op == "delta_step":
        o = tla.gated_delta_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["hk"], s["state"], slots=s["slot"])
        return {"o": o, "state": s["state"]}
    args = dict(n_heads=s["hk"], state=s["state"], cu_seqlens=s["cu"], max_seqlen=max(s["lens"]))
    if op == "delta":
        o, state = tla.gated_delta(s["q"], s["k"], s["v"], s["g"], s["beta"], **args)
        return {"o": o, "state": state}
    got = tla.gated_delta_grad(s["q"], s["k"], s["v"], s["g"], s["beta"], s["do"], dstate=s["dstate"], **args)
    return {name: x for name, x in got._asdict().items() if x is not None}


def run(state):
    if own:
        return _run_own(state)
    return {"qk": _qk_plain, "qk_grad": _qk_grad_plain, "delta": _delta_plain, "delta_grad": _delta_grad_plain,
            "delta_step": _step_plain}[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------- exact
def _exact_qk(s):
    """Norm and rotation in 64 bits as a complex product; the gradient by automatic differentiation."""
    sec = _sections(s)
    turn, where = [], []
    for a, c in enumerate(sec):
        for j in range(c):
            p = j + sum(sec[:a])
            if s["per_axis"]:
                size, i, off = c, j, 2 * sum(sec[:a])
            else:
                size, i, off = sum(sec), p, 0
            turn.append((a, BASE ** (-i / size)))
            where.append((off + 2 * i, off + 2 * i + 1) if s["interleaved"] else (off + i, off + size + i))
    ang = s["pos"].double()[:, [a for a, _ in turn]] * torch.tensor([f for _, f in turn], device=DEV, dtype=torch.float64)
    z = torch.polar(torch.ones_like(ang), ang)[:, None]
    re, im = [w[0] for w in where], [w[1] for w in where]
    rest = [c for c in range(s["d"]) if c not in re and c not in im]
    order = torch.tensor(re + im + rest, device=DEV).argsort()
    out = {}
    for x, h in (("q", s["h"]), ("k", s["hk"])):
        v = s[x].double()
        w, b = (None if s[x + e] is None else s[x + e].double() for e in ("_w", "_b"))
        wants = [("d" + x, v), ("d" + x + "_w", w), ("d" + x + "_b", b)] if s["op"] == "qk_grad" else []
        wants = [(name, t.requires_grad_()) for name, t in wants if t is not None]
        y = v.view(s["n"], h, s["d"])
        if s["norm"] == "l2":
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True)).clamp(min=EPS["l2"])
        elif s["norm"] == "rms":
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS["rms"]) * w
        elif s["norm"] == "layer":
            y = (y - y.mean(-1, keepdim=True)) / torch.sqrt(y.var(-1, unbiased=False, keepdim=True) + EPS["layer"]) * w + b
        r = torch.complex(y[..., re], y[..., im]) * z
        y = torch.cat([r.real, r.imag, y[..., rest]], -1)[..., order].flatten(1)
        if s["op"] == "qk":
            out[x] = y
        else:
            out.update(zip([name for name, _ in wants], torch.autograd.grad(y, [t for _, t in wants], s["d" + x].double())))
    return out


def _exact_delta(s):
    """Token by token in 64 bits, as the recurrence says; the gradient by its reverse, with every state kept."""
    hk, hv, dk, dv, n = s["hk"], s["hv"], s["dk"], s["dv"], s["n"]
    group, lens, grad = hv // hk, s["lens"], s["op"] == "delta_grad"
    longest = max(max(lens), 1)
    at = s["cu"][:-1].long()[:, None] + torch.arange(longest, device=DEV)
    live = torch.arange(longest, device=DEV) < torch.tensor(lens, device=DEV)[:, None]
    at = torch.where(live, at, 0)

    def heads(x, h, rep):  # [longest, sequences * value heads, d], zeros past a sequence's end
        x = (x.double()[at] * live[..., None]).unflatten(-1, (h, -1)).repeat_interleave(rep, 2)
        return x.transpose(0, 1).flatten(1, 2)

    q, k, v = heads(s["q"], hk, group), heads(s["k"], hk, group), heads(s["v"], hv, 1)
    beta = heads(s["beta"], hv, 1)
    a = torch.ones_like(beta) if s["g"] is None else torch.exp(heads(s["g"], hv, 1))
    pairs = q.shape[1]
    S0 = torch.zeros((pairs, dk, dv), dtype=torch.float64, device=DEV) if s["state"] is None else s["state"].double().flatten(0, 1)
    do = heads(s["do"], hv, 1) if grad else None
    dS1 = torch.zeros_like(S0) if not grad or s["dstate"] is None else s["dstate"].double().flatten(0, 1)
    some = pairs if not grad else max(1, int(16e9 / (8 * longest * dk * dv)))
    parts = []
    for lo in range(0, pairs, some):
        sl = slice(lo, lo + some)
        Q, K, V, A, Bt = (x[:, sl].unsqueeze(-1) for x in (q, k, v, a, beta))
        S, kept, us, outs = S0[sl], [], [], []
        for t in range(longest):
            P = A[t] * S
            if grad:
                kept.append(P)
            u = Bt[t] * (V[t] - torch.bmm(P.mT.contiguous(), K[t]))
            S = P + K[t] * u.mT
            us.append(u)
            outs.append(torch.bmm(S.mT.contiguous(), Q[t])[..., 0])
        if not grad:
            parts.append({"o": torch.stack(outs), "state": S})
            continue
        dS, got = dS1[sl], []
        DO = do[:, sl].unsqueeze(-1)
        for t in reversed(range(longest)):
            P, u = kept[t], us[t]
            dq = torch.bmm(P + K[t] * u.mT, DO[t])
            dS = dS + Q[t] * DO[t].mT
            du = torch.bmm(dS.mT.contiguous(), K[t])
            miss = V[t] - torch.bmm(P.mT.contiguous(), K[t])
            dv_ = Bt[t] * du
            dk_ = torch.bmm(dS, u) - torch.bmm(P, dv_)
            dS = dS - K[t] * dv_.mT
            got.append((dq[..., 0], dk_[..., 0], dv_[..., 0], (dS * P).sum((1, 2))[:, None], (du * miss).sum(1)))
            dS = A[t] * dS
        names = ("dq", "dk", "dv", "dg", "dbeta")
        parts.append({**{m: torch.stack([x[i] for x in got[::-1]]) for i, m in enumerate(names)}, "dstate": dS})
    out = {m: torch.cat([p[m] for p in parts], 0 if "state" in m else 1) for m in parts[0]}

    def rows(x, h, rep):  # back to [n, heads * d], value heads of a key head summed
        x = x.unflatten(1, (len(lens), h, rep)).sum(3).transpose(0, 1)
        y = torch.zeros((n,) + x.shape[2:], dtype=x.dtype, device=DEV)
        y[at[live]] = x[live]
        return y.flatten(1)

    final = {}
    for m, x in out.items():
        if "state" in m:
            final[m] = x.view(len(lens), hv, dk, dv)
        elif m in ("dq", "dk"):
            final[m] = rows(x, hk, group)
        else:
            final[m] = rows(x, hv, 1)
    if s["g"] is None:
        final.pop("dg", None)
    if grad and s["state"] is None:
        final.pop("dstate")
    return final


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] in ("qk", "qk_grad"):
        return _exact_qk(s)
    if s["op"] != "delta_step":
        return _exact_delta(s)
    S = s["state"].double()
    o = torch.zeros((s["rows"], s["hv"], s["dv"]), dtype=torch.float64, device=DEV)
    kh = torch.arange(s["hv"], device=DEV) // (s["hv"] // s["hk"])
    at = s["slot"].long()
    k, q = (s[x].double().view(s["rows"], s["hk"], s["dk"])[:, kh] for x in ("k", "q"))
    v = s["v"].double().view(s["rows"], s["hv"], s["dv"])
    P = S[at] if s["g"] is None else S[at] * s["g"].double().exp()[..., None, None]
    miss = v - torch.bmm(k.flatten(0, 1).unsqueeze(1), P.flatten(0, 1)).view_as(v)
    P = P + torch.bmm(k.flatten(0, 1).unsqueeze(2), (s["beta"].double()[..., None] * miss).flatten(0, 1).unsqueeze(1)).view_as(P)
    o = torch.bmm(q.flatten(0, 1).unsqueeze(1), P.flatten(0, 1)).view_as(o)
    S[at] = P
    return {"o": o.flatten(1), "state": S}
