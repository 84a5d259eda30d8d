"""The 4-bit and block-join operators as measured work: cases, inputs, plain forms and exact values.

Five operators: `quantize` (tokens or weights to microscaled 4-bit and back to the values they stand for),
`matmul` (the product with 4-bit weights), `read` (the full-width fast-weight MLP frozen in 4 bits), `join` (norm
after a block, gate, residual scale, residual, norm before the next block) and `join_grad` (its backward pass).

A 4-bit matrix [rows, k] is held as `codes` uint8 [rows, kp/2] (kp: k rounded up to 128; the low nibble is the even
column; bit 3 the sign, bits 0-2 index 0, .5, 1, 1.5, 2, 3, 4, 6) and `scales` uint8 [ceil(rows/64), kp/128, 64, 4]:
the scale byte (exponent + 127, one per row and 32 columns) of row 64 R + 16 i + r, block 4 B + g stands at
[R, B, 16 g + r, i].
"""
import math

import torch

own = False

DEV = "cuda"
MLP_D, MLP_M = 1024, 4096  # the full-width fast-weight MLP
VIEW = 1374  # tokens of one view: 5 special ones and 37 x 37 patches
EPS = 1e-6
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ----------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the tokens of one unseen view, before a product reads them
        {"name": "quantize_view", "op": "quantize", "rows": VIEW, "k": MLP_D, "dtype": "bf16", "transpose": False},
        # one fast-weight matrix W_g [1024][4096] as it is stored: the contraction runs along its first axis
        {"name": "quantize_weight", "op": "quantize", "rows": MLP_M, "k": MLP_D, "dtype": "f32", "transpose": True},
        # the tokens of a 100-view scene
        {"name": "quantize_scene", "op": "quantize", "rows": 100 * VIEW, "k": MLP_D, "dtype": "bf16", "transpose": False},
        # one token through one weight matrix: latency counts
        {"name": "matmul_token", "op": "matmul", "m": 1, "n": MLP_M, "k": MLP_D, "a": "bf16", "out": "bf16"},
        # one view into a head of odd width, in fp32
        {"name": "matmul_view_ragged", "op": "matmul", "m": VIEW, "n": 999, "k": 1000, "a": "f32", "out": "f32"},
        # the queries of 50 unseen views, quantised already
        {"name": "matmul_queries", "op": "matmul", "m": 50 * VIEW, "n": MLP_M, "k": MLP_D, "a": "mx4", "out": "bf16"},
        # query mode for a single token, and for 50 unseen views
        {"name": "read_token", "op": "read", "m": 1},
        {"name": "read_queries", "op": "read", "m": 50 * VIEW},
        # the camera tokens of 24 views (5 special tokens each), RMS norms, a gate for every token
        {"name": "join_camera", "op": "join", "n": 24 * 5, "c": MLP_D, "dtype": "f32", "post": "rms", "pre": "rms",
         "bias": False, "gate": "token", "per": 1, "scale": True, "mx4": False},
        # a 100-view scene: layer norms with biases, residual scale, a gate per view
        {"name": "join_scene", "op": "join", "n": 100 * VIEW, "c": MLP_D, "dtype": "bf16", "post": "layer",
         "pre": "layer", "bias": True, "gate": "group", "per": VIEW, "scale": True, "mx4": False},
        # the gradient for one view in fp32, a gate for every token
        {"name": "join_grad_view", "op": "join_grad", "n": VIEW, "c": MLP_D, "dtype": "f32", "post": "rms",
         "pre": "rms", "bias": False, "gate": "token", "per": 1, "scale": True},
        # the gradient for a training batch of 48 views, gates per view
        {"name": "join_grad_batch", "op": "join_grad", "n": 48 * VIEW, "c": MLP_D, "dtype": "bf16", "post": "layer",
         "pre": "layer", "bias": True, "gate": "group", "per": VIEW, "scale": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "read", "join", "join_grad"])
    dtype = rng.choice(["bf16", "f32"])
    if op == "quantize":
        transpose = rng.random() < 0.3
        rows = _log(rng, 1, 4096 if transpose else 100 * VIEW)
        k = _log(rng, 8, min(4096, max(8, 100 * VIEW * 512 // rows)))
        return {"op": op, "rows": rows, "k": k, "dtype": dtype, "transpose": transpose}
    if op == "matmul":
        m = _log(rng, 1, 50 * VIEW)
        most = 50 * VIEW * MLP_M * MLP_D // (2 * m)
        n = _log(rng, 8, min(8192, max(8, most // 512)))
        k = _log(rng, 32, max(32, min(8192, most // n)))
        return {"op": op, "m": m, "n": n, "k": k, "a": rng.choice(["mx4", "mx4", "bf16", "f32"]), "out": dtype}
    if op == "read":
        return {"op": op, "m": _log(rng, 1, 50 * VIEW)}
    c = _log(rng, 16, 8192)
    n = _log(rng, 1, max(1, (24 if op == "join_grad" else 50) * VIEW * MLP_D // c))
    gate = rng.choice(["none", "token", "group"])
    case = {"op": op, "n": n, "c": c, "dtype": dtype, "post": rng.choice(["none", "rms", "layer"]),
            "pre": rng.choice(["none", "rms", "layer", "layer"]), "bias": rng.random() < 0.5, "gate": gate,
            "per": _log(rng, 2, 2 * VIEW) if gate == "group" else 1, "scale": rng.random() < 0.6}
    if op == "join":
        case["mx4"] = case["pre"] != "none" and rng.random() < 0.3
    return case


# ---------------------------------------------------------------------------------------------------------- inputs
def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _gen(seed, stream):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 64 + stream)


def _randn(shape, seed, stream, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=_gen(seed, stream), device=DEV) * std).to(dtype)


def _tokens(rows, k, seed, stream, dtype):
    """Activations: rows of differing size, some channels that stand out, some rows all zero (padded views)."""
    g = _gen(seed, stream)
    x = torch.randn((rows, k), generator=g, device=DEV)
    x *= torch.exp(torch.randn((rows, 1), generator=g, device=DEV))
    x *= 1 + 15 * (torch.rand((1, k), generator=g, device=DEV) < 0.01)
    x *= torch.rand((rows, 1), generator=g, device=DEV) >= 0.01
    return x.to(dtype)


def prepare(case, seed):
    op = case["op"]
    if op == "quantize":
        dt = _dtype(case["dtype"])
        x = _tokens(case["rows"], case["k"], seed, 1, dt)
        return dict(case, x=x.t().contiguous() if case["transpose"] else x)
    if op == "matmul":
        a = _tokens(case["m"], case["k"], seed, 1, torch.float32 if case["a"] == "f32" else torch.bfloat16)
        w = _pack(*_to4(_randn((case["n"], case["k"]), seed, 2, case["k"] ** -0.5)))
        return dict(case, A=_pack(*_to4(a.float())) if case["a"] == "mx4" else a, W=w)
    if op == "read":
        q = _randn((case["m"], MLP_D), seed, 1, 1.0)
        std = 1.5 * MLP_D ** -0.5
        return dict(case, q=q.to(torch.bfloat16), gate=_pack(*_to4(_randn((MLP_M, MLP_D), seed, 2, std))),
                    up=_pack(*_to4(_randn((MLP_M, MLP_D), seed, 3, std))),
                    down=_pack(*_to4(_randn((MLP_D, MLP_M), seed, 4, MLP_M ** -0.5))))
    n, c, dt = case["n"], case["c"], _dtype(case["dtype"])
    s = dict(case)
    s["f"] = _randn((n, c), seed, 2, 0.7, dt)
    s["g"] = None
    if case["gate"] != "none":
        s["g"] = _randn((-(-n // case["per"]), c), seed, 3, 0.5, dt) + 1
    s["s"] = _randn((c,), seed, 4, 0.1) + 0.3 if case["scale"] else None
    s["post_w"] = _randn((c,), seed, 5, 0.2) + 1 if case["post"] != "none" else None
    s["pre_w"] = _randn((c,), seed, 6, 0.2) + 1 if case["pre"] != "none" else None
    s["post_b"] = _randn((c,), seed, 7, 0.1) if case["post"] == "layer" and case["bias"] else None
    s["pre_b"] = _randn((c,), seed, 8, 0.1) if case["pre"] == "layer" and case["bias"] else None
    s["x"] = _randn((n, c), seed, 1, 1.5, dt)  # the stream before the join, or (join_grad) after it
    if op == "join_grad":
        s["dr"] = _randn((n, c), seed, 9, 1.0, dt)
        s["dy"] = _randn((n, c), seed, 10, 1.0, dt) if case["pre"] != "none" else None
    return s


def work(case):
    op = case["op"]
    if op == "quantize":  # values in, the values they stand for out
        return {"bytes": 2 * case["rows"] * case["k"] * (2 if case["dtype"] == "bf16" else 4), "flops": 0}
    q4 = 0.5 + 1 / 32
    if op == "matmul":
        m, n, k = case["m"], case["n"], case["k"]
        a = {"mx4": q4, "bf16": 2, "f32": 4}[case["a"]]
        return {"bytes": m * k * a + n * k * q4 + m * n * (2 if case["out"] == "bf16" else 4), "flops": 2 * m * n * k}
    if op == "read":
        m, p = case["m"], 3 * MLP_D * MLP_M
        return {"bytes": 4 * m * MLP_D + p * q4, "flops": 2 * m * p}
    n, c, e = case["n"], case["c"], 2 if case["dtype"] == "bf16" else 4
    gates = 0 if case["gate"] == "none" else -(-n // case["per"])
    if op == "join":
        return {"bytes": e * c * (n * (3 + (case["pre"] != "none")) + gates), "flops": 0}
    return {"bytes": e * c * (n * (4 + 2 * (case["pre"] != "none")) + 2 * gates), "flops": 0}


# ----------------------------------------------------------------------------------------------- 4 bits, plain form
def _to4(x):
    """fp32 [rows, k] -> (signed values on the grid [rows, kb, 32], block exponents [rows, kb])."""
    rows, k = x.shape
    kb = -(-k // 32)
    b = torch.nn.functional.pad(x, (0, 32 * kb - k)).view(rows, kb, 32)
    amax = b.abs().amax(-1)
    e = torch.where(amax > 0, torch.frexp(amax).exponent - 3, torch.full_like(amax, -127, dtype=torch.int32)).clamp(min=-127)
    v = torch.ldexp(b, -e.unsqueeze(-1))
    a = v.abs()
    q = torch.where(a < 2, torch.round(2 * a) / 2, torch.where(a < 4, torch.round(a), 2 * torch.round(a / 2))).clamp(max=6)
    return torch.copysign(q, v), e


def _from4(q, e, k):
    """The fp32 values [rows, k] that grid values and block exponents stand for."""
    return torch.ldexp(q, e.unsqueeze(-1)).flatten(1)[:, :k]


def _pack(q, e):
    """Grid values [rows, kb, 32] and exponents [rows, kb] -> (codes, scales, k in whole blocks) as stored."""
    rows, kb = e.shape
    kp = -(-kb // 4) * 4
    grid = torch.tensor(GRID, device=q.device)
    code = torch.bucketize(q.abs(), grid) + 8 * torch.signbit(q)
    code = torch.nn.functional.pad(code.view(rows, -1), (0, 32 * (kp - kb))).to(torch.uint8)
    rp = -(-rows // 64) * 64
    s = torch.nn.functional.pad((e + 127).to(torch.uint8), (0, kp - kb, 0, rp - rows))
    s = s.view(rp // 64, 4, 16, kp // 4, 4).permute(0, 3, 4, 2, 1).reshape(rp // 64, kp // 4, 64, 4).contiguous()
    return (code[:, 0::2] | code[:, 1::2] << 4).contiguous(), s


def _unpack(m, dtype=torch.float32):
    """The values [rows, kp] that stored codes and scales stand for (columns past k are 0)."""
    codes, s = m
    rows, kp = codes.shape[0], 2 * codes.shape[1]
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device, dtype=dtype)
    code = torch.stack((codes & 15, codes >> 4), -1).view(rows, kp)
    e = s.view(s.shape[0], kp // 128, 4, 16, 4).permute(0, 4, 3, 1, 2).reshape(-1, kp // 32)[:rows].to(torch.int32) - 127
    return torch.ldexp(grid[code.to(torch.int32)].view(rows, kp // 32, 32), e.unsqueeze(-1)).flatten(1)


def _values4(x):
    """The fp32 values that x (fp32) stands for after quantisation."""
    return _from4(*_to4(x), x.shape[1])


# ------------------------------------------------------------------------------------------------ join, plain form
def _norm(v, kind, w, b):
    """(normalised v, 1 / its deviation, w * normalised + b), in v's type."""
    if kind == "layer":
        v = v - v.mean(-1, keepdim=True)
    rstd = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    h = v * rstd
    return h, rstd, h * w if b is None else h * w + b


def _norm_back(dh, h, rstd, kind):
    """Gradient of the norm's input from that of the normalised value h."""
    d = dh - h * (dh * h).mean(-1, keepdim=True)
    if kind == "layer":
        d = d - dh.mean(-1, keepdim=True)
    return d * rstd


def _rows_of_gate(s, n):
    g = s["g"].float()
    return g if s["per"] == 1 else g.repeat_interleave(s["per"], 0)[:n]


def _join_plain(s):
    dt = s["x"].dtype
    h = s["f"].float()
    if s["post"] != "none":
        h = _norm(h, s["post"], s["post_w"], s["post_b"])[2]
    if s["g"] is not None:
        h = h * _rows_of_gate(s, h.shape[0])
    if s["s"] is not None:
        h = h * s["s"]
    r = (s["x"].float() + h).to(dt)  # the stream as it is stored; the norm is that of the stored stream
    if s["pre"] == "none":
        return {"r": r}
    y = _norm(r.float(), s["pre"], s["pre_w"], s["pre_b"])[2].to(dt)
    return {"r": r, "y": _values4(y.float()).to(dt) if s["mx4"] else y}


def _join_grad_plain(s):
    r, f, dt = s["x"].float(), s["f"].float(), s["x"].dtype
    n, c = r.shape
    out = {}
    d = s["dr"].float()
    if s["pre"] != "none":
        dy = s["dy"].float()
        rh, rstd, _ = _norm(r, s["pre"], s["pre_w"], None)
        d = d + _norm_back(dy * s["pre_w"], rh, rstd, s["pre"])
        out["dpre_w"] = (dy * rh).sum(0)
        if s["pre_b"] is not None:
            out["dpre_b"] = dy.sum(0)
    out["dx"] = d.to(dt)
    h = f
    if s["post"] != "none":
        fh, frstd, h = _norm(f, s["post"], s["post_w"], s["post_b"])
    g = None if s["g"] is None else _rows_of_gate(s, n)
    dg = d if g is None else d * g
    if s["s"] is not None:
        out["dscale"] = (dg * h).sum(0)
    ds = d if s["s"] is None else d * s["s"]
    if g is not None:
        groups = s["g"].shape[0]
        p = torch.nn.functional.pad(ds * h, (0, 0, 0, groups * s["per"] - n))
        out["dgate"] = p.view(groups, s["per"], c).sum(1).to(dt)
    dh = ds if g is None else ds * g
    if s["post"] == "none":
        out["df"] = dh.to(dt)
        return out
    out["dpost_w"] = (dh * fh).sum(0)
    if s["post_b"] is not None:
        out["dpost_b"] = dh.sum(0)
    out["df"] = _norm_back(dh * s["post_w"], fh, frstd, s["post"]).to(dt)
    return out


# ------------------------------------------------------------------------------------------------------------ run
def _run_plain(s):
    op = s["op"]
    if op == "quantize":
        x = s["x"].t() if s["transpose"] else s["x"]
        return _values4(x.float()).to(s["x"].dtype)
    if op == "matmul":
        w = _unpack(s["W"])[:, :s["k"]]
        a = _unpack(s["A"])[:, :s["k"]] if s["a"] == "mx4" else _values4(s["A"].float())
        return (a @ w.t()).to(_dtype(s["out"]))
    if op == "read":
        q = _values4(s["q"].float())
        h = q @ _unpack(s["gate"]).t()
        h = h / (1 + torch.exp(-h)) * (q @ _unpack(s["up"]).t())
        return (_values4(h) @ _unpack(s["down"]).t()).to(torch.bfloat16)
    return _join_plain(s) if op == "join" else _join_grad_plain(s)


def _run_own(s):
    import test_layer_amd as tla

    op = s["op"]
    if op == "quantize":
        return tla.mx4_dequantize(tla.mx4_quantize(s["x"], transpose=s["transpose"]), dtype=s["x"].dtype)
    if op == "matmul":
        a = tla.Mx4(*s["A"], s["k"]) if s["a"] == "mx4" else s["A"]
        return tla.mx4_matmul(a, tla.Mx4(*s["W"], s["k"]), dtype=_dtype(s["out"]))
    if op == "read":
        frozen = tla.FrozenMx4(tla.Mx4(*s["gate"], MLP_D), tla.Mx4(*s["up"], MLP_D), tla.Mx4(*s["down"], MLP_M))
        return tla.ttt_read_mx4(s["q"], frozen)
    args = dict(gate=s["g"], gate_tokens=s["per"], scale=s["s"], post=s["post"], post_w=s["post_w"], post_b=s["post_b"],
                pre=s["pre"], pre_w=s["pre_w"], eps=EPS)
    if op == "join":
        r, y = tla.block_join(s["x"], s["f"], pre_b=s["pre_b"], mx4=s["mx4"], **args)
        if s["mx4"]:
            y = tla.mx4_dequantize(y, dtype=s["x"].dtype)
        return {"r": r} if y is None else {"r": r, "y": y}
    got = tla.block_join_grad(s["x"], s["f"], s["dr"], s["dy"], pre_bias=s["pre_b"] is not None, **args)
    return {k: v for k, v in got._asdict().items() if v is not None}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------------------------------------- exact
def _exact4(x):
    """fp64 [rows, k] -> the values after quantisation: the nearest grid value of each block's scale, ties to the
    even code, by comparison with the grid's midpoints."""
    rows, k = x.shape
    kb = -(-k // 32)
    b = torch.nn.functional.pad(x, (0, 32 * kb - k)).reshape(rows * kb, 32)
    top = b.abs().max(-1, keepdim=True).values
    e = torch.floor(torch.log2(top.clamp(min=2.0 ** -140)))
    e = e - (torch.exp2(e) > top).double() + (torch.exp2(e + 1) <= top).double()  # log2 may round across a power
    scale = torch.exp2((e - 2).clamp(min=-127))
    v = b / scale
    grid = torch.tensor(GRID, device=x.device, dtype=torch.float64)
    mid = (grid[1:] + grid[:-1]) / 2
    at = torch.bucketize(v.abs(), mid)  # a value on a midpoint goes to the lower code
    at = at + ((at < 7) & (v.abs() == mid[at.clamp(max=6)]) & (at % 2 == 1)).long()
    return (torch.sign(v) * grid[at] * scale).view(rows, 32 * kb)[:, :k]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "quantize":
        x = s["x"].t() if case["transpose"] else s["x"]
        return _exact4(x.double())
    if op == "matmul":
        k = case["k"]
        a = _unpack(s["A"], torch.float64)[:, :k] if case["a"] == "mx4" else _exact4(s["A"].double())
        return torch.mm(a, _unpack(s["W"], torch.float64)[:, :k].t())
    if op == "read":
        q = _exact4(s["q"].double())
        h = torch.mm(q, _unpack(s["gate"], torch.float64).t())
        h = torch.sigmoid(h) * h * torch.mm(q, _unpack(s["up"], torch.float64).t())
        return torch.mm(_exact4(h), _unpack(s["down"], torch.float64).t())

    # the join and, by automatic differentiation in 64 bits, its gradient
    def norm(v, kind, w, b):
        if kind == "none":
            return v
        if kind == "rms":
            y = v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
        else:
            y = (v - v.mean(1, keepdim=True)) / torch.sqrt(v.var(1, unbiased=False, keepdim=True) + EPS)
        return y * w if b is None else y * w + b

    p = {k: None if s[k] is None else s[k].double() for k in ("x", "f", "g", "s", "post_w", "post_b", "pre_w", "pre_b")}
    n, dt = case["n"], s["x"].dtype
    at = torch.arange(n, device=DEV) // case["per"]
    if op == "join_grad":
        p = {k: None if v is None else v.requires_grad_() for k, v in p.items()}
    h = norm(p["f"], case["post"], p["post_w"], p["post_b"])
    if p["g"] is not None:
        h = h * p["g"][at]
    if p["s"] is not None:
        h = h * p["s"]
    if op == "join":
        r = p["x"] + h
        if case["pre"] == "none":
            return {"r": r}
        y = norm(r.to(dt).double(), case["pre"], p["pre_w"], p["pre_b"])
        return {"r": r, "y": _exact4(y.to(dt).double()) if case["mx4"] else y}
    r = p["x"]  # given: the gradient at the joined stream, whose dependence on x is the identity
    loss = 0.0 if s["dy"] is None else (norm(r, case["pre"], p["pre_w"], p["pre_b"]) * s["dy"].double()).sum()
    total = s["dr"].double()
    out = {}
    if s["dy"] is not None:
        wants = [k for k in ("pre_w", "pre_b") if p[k] is not None]
        got = torch.autograd.grad(loss, [r] + [p[k] for k in wants])
        total = total + got[0]
        out.update({"d" + k: v for k, v in zip(wants, got[1:])})
    out["dx"] = total
    wants = [k for k in ("f", "g", "s", "post_w", "post_b") if p[k] is not None]
    got = torch.autograd.grad((h * total).sum(), [p[k] for k in wants])
    names = {"f": "df", "g": "dgate", "s": "dscale", "post_w": "dpost_w", "post_b": "dpost_b"}
    out.update({names[k]: v for k, v in zip(wants, got)})
    return out
