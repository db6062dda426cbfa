"""Timed cases of the operators that training a mixture-of-experts block needs.

With ``own`` false, ``run`` computes them from elementary torch operations; with ``own`` true it
calls this package.

 grouped           y_r = x_r W_e^T for the rows r of every group e (or silu(gate) * up of it, with
                   the pre-activation kept), sizes of the groups on the device
 grouped gradient  dx_r = dz_r W_e and dW_e = sum of dz_r^T x_r over the group's rows
 norm              p = RMS norm of a block's output x (or x);  s = a residual + b gate_t scale_c p;
                   y = RMS norm of s
 norm gradient     of x, the residual, the gate, and the three vectors
 clip              the 2-norm over many gradients and the gradients scaled down to a largest norm
"""

import math
import random

import numpy as np
import torch

own = False


def _pkg():
    import mixture_experts_layer_04_gb300 as moe
    return moe


# ------------------------------------------------------------------------------- cases ----

def _grouped(name, rows, used, groups, active, fin, fout, dtype, out, dx, act, keep, pad, skew,
             direction):
    c = dict(op="grouped", direction=direction, rows=rows, used=used, groups=groups,
             active=active, fin=fin, fout=fout, dtype=dtype, out=out, dx=dx, act=act, keep=keep,
             pad=pad, skew=skew)
    if name:
        c["name"] = name
    return c


def _norm(name, rows, width, dtype, post, gate, scale, residual, norm, pad, direction):
    c = dict(op="norm", direction=direction, rows=rows, width=width, dtype=dtype, post=post,
             gate=gate, scale=scale, residual=residual, norm=norm, pad=pad)
    if name:
        c["name"] = name
    return c


def _clip(name, tensors, total, dtype, out, scale, biggest, write):
    c = dict(op="clip", direction="forward", tensors=tensors, total=total, dtype=dtype, out=out,
             scale=scale, biggest=biggest, write=write)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token being decoded through the gate and up products of its 8 experts of 128
        # (Qwen3-shaped): the weights' read
        _grouped("grouped_token", 8, 8, 128, 8, 2048, 768, "bfloat16", "bfloat16", "bfloat16",
                 "swiglu", False, 0, 0.0, "forward"),
        # the down product of 64 sequences being decoded, float32 rows for the combine
        _grouped("grouped_batch", 512, 512, 128, 119, 768, 2048, "bfloat16", "float32",
                 "bfloat16", "none", False, 0, 1.0, "forward"),
        # the gate and up products of a training step over 8192 tokens, pre-activation kept;
        # uneven groups, some empty
        _grouped("grouped_step", 65536, 65536, 128, 125, 2048, 768, "bfloat16", "bfloat16",
                 "bfloat16", "swiglu", True, 0, 1.0, "forward"),
        # their gradients, float32 rows of dx for the sum over a token's experts; some
        # assignments were dropped, so the last rows belong to no group
        _grouped("grouped_step_grad", 65536, 63011, 128, 125, 2048, 768, "bfloat16", "bfloat16",
                 "float32", "swiglu", True, 0, 1.0, "backward"),
        # a few large experts (Mixtral-shaped): the down product's gradients
        _grouped("grouped_large_grad", 8192, 8192, 8, 8, 14336, 4096, "bfloat16", "bfloat16",
                 "bfloat16", "none", False, 0, 0.1, "backward"),
        # a small float32 layer of odd sizes
        _grouped("grouped_f32_odd", 517, 501, 7, 5, 333, 201, "float32", "float32", "float32",
                 "swiglu", True, 3, 0.7, "backward"),
        # one token between two blocks: latency only
        _norm("norm_token", 1, 7168, "bfloat16", True, "none", False, True, True, 0, "forward"),
        # 16384 tokens of prefill between two blocks: norm after, gate, residual, norm before
        _norm("norm_prefill", 16384, 7168, "bfloat16", True, "logistic", True, True, True, 0,
              "forward"),
        # the same in a training step's backward
        _norm("norm_step_grad", 8192, 2048, "bfloat16", True, "value", True, True, True, 0,
              "backward"),
        # a float32 backward of an odd width, x a slice of a wider array
        _norm("norm_grad_f32_odd", 999, 1001, "float32", True, "logistic", True, True, True, 5,
              "backward"),
        # the gradients of a router, its norms and a few small layers
        _clip("clip_small", 23, 300007, "mixed", "same", 1.0, 0.3, True),
        # those of a Qwen3-shaped layer with 128 experts, next to its attention
        _clip("clip_layer", 150, 640000000, "bfloat16", "same", 1.0, 0.6, True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_MAX_FLOPS = 4 * 8192 * 14336 * 4096
_MAX_WEIGHTS = 1 << 29


def _draw_grouped(rng):
    dtype = rng.choice(("bfloat16", "bfloat16", "float32"))
    groups = _log_int(rng, 1, 256)
    fin, fout = _log_int(rng, 64, 8192), _log_int(rng, 64, 8192)
    if rng.random() < 0.6:  # most layers have sizes that are multiples of 64
        fin, fout = max(64, fin // 64 * 64), max(64, fout // 64 * 64)
    act = rng.choice(("none", "swiglu"))
    direction = rng.choice(("forward", "backward"))
    nout = fout * (2 if act == "swiglu" else 1)
    small = 1 if dtype == "bfloat16" else 8
    groups = max(1, min(groups, _MAX_WEIGHTS // small // (nout * fin)))
    rows = _log_int(rng, 1, 65536)
    per_row = (2 if direction == "forward" else 4) * fin * nout
    rows = max(1, min(rows, _MAX_FLOPS // 2 // small // per_row))
    used = rows if rng.random() < 0.6 else max(1, int(rows * rng.uniform(0.7, 1.0)))
    active = max(1, min(groups, used, int(round(groups * rng.uniform(0.5, 1.0)))))
    out = dtype if rng.random() < 0.7 else "float32"
    dx = dtype if rng.random() < 0.7 else "float32"
    return _grouped(None, rows, used, groups, active, fin, fout, dtype, out, dx, act,
                    act == "swiglu" and (direction == "backward" or rng.random() < 0.5),
                    rng.choice((0, 0, 5, 64)), rng.choice((0.0, 0.5, 1.0, 1.5)), direction)


def draw(rng):
    op = rng.choice(("grouped", "grouped", "grouped", "norm", "norm", "clip"))
    if op == "grouped":
        return _draw_grouped(rng)
    if op == "norm":
        rows, width = _log_int(rng, 1, 16384), _log_int(rng, 64, 8192)
        if rng.random() < 0.6:
            width = max(64, width // 64 * 64)
        rows = max(1, min(rows, 16384 * 7168 // 2 // width))
        residual = rng.random() < 0.8
        return _norm(None, rows, width, rng.choice(("bfloat16", "bfloat16", "float32")),
                     rng.random() < 0.5, rng.choice(("none", "value", "logistic")),
                     rng.random() < 0.5, residual, rng.random() < 0.8 or not residual,
                     rng.choice((0, 0, 5, 64)), rng.choice(("forward", "backward")))
    total = _log_int(rng, 1000, 300000000)
    return _clip(None, min(total // 10, _log_int(rng, 1, 900)), total,
                 rng.choice(("bfloat16", "float32", "mixed")), rng.choice(("same", "float32")),
                 rng.choice((1.0, 1.0 / 1024)), rng.choice((0.1, 0.5, 0.9)), rng.random() < 0.8)


# -------------------------------------------------------------------------------- work ----

def _bytes(dtype):
    return 2 if dtype == "bfloat16" else 4


def _outputs(case):
    """Rows of a group's weights."""
    return case["fout"] * (2 if case["act"] == "swiglu" else 1)


def work(case):
    sz = _bytes(case["dtype"])
    if case["op"] == "grouped":
        M, G, I, F, N = case["used"], case["groups"], case["fin"], case["fout"], _outputs(case)
        weights = case["active"] * N * I * sz
        if case["direction"] == "forward":
            b = M * I * sz + weights + M * F * _bytes(case["out"])
            b += M * N * sz if case["keep"] else 0
            f = 2 * M * N * I
        else:
            b = M * F * sz + (M * N * sz if case["act"] == "swiglu" else 0)  # dy and z
            b += M * I * (sz + _bytes(case["dx"])) + weights + G * N * I * sz
            f = 4 * M * N * I
        return {"bytes": int(b + 4 * (G + 1)), "flops": int(f)}
    if case["op"] == "norm":
        T, W = case["rows"], case["width"]
        vectors = case["post"] + case["scale"] + case["norm"]
        gate = 4 * T if case["gate"] != "none" else 0
        if case["direction"] == "forward":
            n = 2 + case["residual"] + case["norm"]  # x, s; residual, y
            b = n * T * W * sz + vectors * 4 * W + gate
            f = 8 * T * W
        else:
            # x where the block's own vectors or gate need it, ds, dx; dres; s and dy
            needs_x = case["post"] or case["scale"] or case["gate"] != "none"
            n = 2 + needs_x + case["residual"] + 2 * case["norm"]
            b = n * T * W * sz + 2 * vectors * 4 * W + 2 * gate
            f = 20 * T * W
        return {"bytes": int(b), "flops": int(f)}
    ins = sum(n * _bytes(d) for n, d, _ in _clip_tensors(case))
    outs = sum(n * _bytes(o) for n, _, o in _clip_tensors(case))
    return {"bytes": int(ins + (outs if case["write"] else 0) + 4),
            "flops": int(3 * case["total"])}


# ----------------------------------------------------------------------------- prepare ----

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    x = torch.randn(*shape, generator=g, device="cuda")
    if std != 1.0:
        x *= std
    return x if dtype == torch.float32 else x.to(dtype)


def _dtype(name):
    return torch.bfloat16 if name == "bfloat16" else torch.float32


def prepare(case, seed):
    return {"grouped": _prepare_grouped, "norm": _prepare_norm,
            "clip": _prepare_clip}[case["op"]](case, seed)


def _bounds(case, seed):
    """The groups' first rows and the end of the last, from the case's uneven shares."""
    r = np.random.default_rng(int(seed))
    chosen = r.permutation(case["groups"])[:case["active"]]
    share = np.exp(case["skew"] * r.standard_normal(case["active"]))
    size = np.zeros(case["groups"], np.int64)
    size[chosen] = 1 + r.multinomial(case["used"] - case["active"], share / share.sum())
    return [0] + np.cumsum(size).tolist()


def _prepare_grouped(case, seed):
    g, dt = _gen(seed), _dtype(case["dtype"])
    M, G, I, F, N = case["rows"], case["groups"], case["fin"], case["fout"], _outputs(case)
    st = dict(case=case, bounds=_bounds(case, seed))
    st["offsets"] = torch.tensor(st["bounds"], dtype=torch.int32, device="cuda")
    # with `pad` x is a slice of a wider array
    st["x"] = _randn(g, M, I + case["pad"], dtype=dt)[:, :I]
    st["w"] = torch.empty(G, N, I, dtype=dt, device="cuda")
    for e in range(0, G, 16):
        st["w"][e:e + 16] = _randn(g, min(16, G - e), N, I, dtype=dt, std=I ** -0.5)
    if case["direction"] == "backward":
        st["dy"] = _randn(g, M, F, dtype=dt)
        st["z"] = _randn(g, M, N, dtype=dt) if case["act"] == "swiglu" else None
    if own:
        moe = _pkg()
        types = {"bfloat16": moe.BF16, "float32": moe.F32}
        st["cfg"] = cfg = moe.GroupedConfig.make(
            rows=M, groups=G, in_features=I, out_features=F, dtype=types[case["dtype"]],
            out_dtype=types[case["out"]], dx_dtype=types[case["dx"]],
            activation=moe.ACT_SWIGLU if case["act"] == "swiglu" else moe.ACT_NONE,
            x_stride=I + case["pad"])
        st["ws"] = torch.empty(moe.grouped_linear_workspace_size(cfg), dtype=torch.uint8,
                               device="cuda")
        # rows that belong to no group stay as they were: zeros here
        if case["direction"] == "forward":
            st["y"] = torch.zeros(M, F, dtype=_dtype(case["out"]), device="cuda")
            st["z"] = torch.zeros(M, N, dtype=dt, device="cuda") if case["keep"] else None
        else:
            st["dx"] = torch.zeros(M, I, dtype=_dtype(case["dx"]), device="cuda")
            st["dw"] = torch.empty(G, N, I, dtype=dt, device="cuda")
    return st


_EPS = 1e-6
_RESIDUAL_SCALE, _BRANCH_SCALE = 0.875, 0.75


def _prepare_norm(case, seed):
    g, dt = _gen(seed), _dtype(case["dtype"])
    T, W = case["rows"], case["width"]
    st = dict(case=case)
    # rows of unlike sizes, as the outputs of blocks are
    rows = lambda: torch.exp(_randn(g, T, 1, std=0.5))
    st["x"] = (_randn(g, T, W + case["pad"]) * rows()).to(dt)[:, :W]
    weight = lambda on: 1.0 + _randn(g, W, std=0.2) if on else None
    st["post"], st["scale"], st["norm"] = (weight(case[k]) for k in ("post", "scale", "norm"))
    st["gate"] = None
    if case["gate"] != "none":
        st["gate"] = _randn(g, T) + (0.0 if case["gate"] == "logistic" else 1.0)
    st["residual"] = _randn(g, T, W, dtype=dt) if case["residual"] else None
    if case["direction"] == "backward":
        st["sum"] = (_randn(g, T, W) * rows()).to(dt)
        st["dsum"] = _randn(g, T, W, dtype=dt)
        st["dy"] = _randn(g, T, W, dtype=dt) if case["norm"] else None
    if own:
        moe = _pkg()
        gate = {"none": moe.GATE_NONE, "value": moe.GATE_VALUE, "logistic": moe.GATE_LOGISTIC}
        st["cfg"] = cfg = moe.BlockNormConfig.make(
            rows=T, width=W, dtype=moe.BF16 if dt == torch.bfloat16 else moe.F32, eps=_EPS,
            residual_scale=_RESIDUAL_SCALE, branch_scale=_BRANCH_SCALE, gate=gate[case["gate"]],
            x_stride=W + case["pad"])
        empty = lambda on, *shape, dtype=torch.float32: (
            torch.empty(*shape, dtype=dtype, device="cuda") if on else None)
        if case["direction"] == "forward":
            st["sum"] = empty(True, T, W, dtype=dt)
            st["y"] = empty(case["norm"], T, W, dtype=dt)
        else:
            st["ws"] = torch.empty(moe.block_norm_workspace_size(cfg), dtype=torch.uint8,
                                   device="cuda")
            st["out"] = [empty(True, T, W, dtype=dt), empty(case["residual"], T, W, dtype=dt),
                         empty(case["gate"] != "none", T), empty(case["post"], W),
                         empty(case["scale"], W), empty(case["norm"], W)]
    return st


def _clip_tensors(case):
    """(elements, type, type of the result) of every tensor: one large share, the rest uneven."""
    r = random.Random(case["tensors"] * 1000003 + case["total"])
    n, total = case["tensors"], case["total"]
    share = [math.exp(r.gauss(0.0, 1.5)) for _ in range(n)]
    share[r.randrange(n)] += case["biggest"] / (1.0 - case["biggest"]) * sum(share)
    size = [max(1, int(total * s / sum(share))) for s in share]
    size[size.index(max(size))] += total - sum(size)
    kinds = {"mixed": ("bfloat16", "float32")}.get(case["dtype"], (case["dtype"],))
    types = [r.choice(kinds) for _ in range(n)]
    return [(s, t, t if case["out"] == "same" else case["out"]) for s, t in zip(size, types)]


_MAX_NORM = 1.0


def _buckets(case):
    """The results lie in one flat buffer a type, each from a multiple of 16 elements on: the
    buffers' sizes, and (type, place) of every result."""
    end, place = {}, []
    for n, _, out in _clip_tensors(case):
        at = end.get(out, 0)
        place.append((out, at))
        end[out] = at + (n + 15) // 16 * 16
    return end, place


def _prepare_clip(case, seed):
    g, st = _gen(seed), dict(case=case, grads=[])
    st["end"], st["place"] = _buckets(case)
    for n, dtype, _ in _clip_tensors(case):
        std = 1e-2 * math.exp(0.5 * torch.randn((), generator=g, device="cuda").item())
        x = torch.empty(n, dtype=_dtype(dtype), device="cuda")
        for at in range(0, n, 1 << 26):
            x[at:at + (1 << 26)] = _randn(g, min(1 << 26, n - at), std=std / case["scale"])
        st["grads"].append(x)
    if own:
        moe = _pkg()
        outs = None
        if case["write"]:
            st["flat"] = {t: torch.zeros(n, dtype=_dtype(t), device="cuda")
                          for t, n in st["end"].items()}
            outs = [st["flat"][t][at:at + x.numel()]
                    for (t, at), x in zip(st["place"], st["grads"])]
        st["list"] = moe.GradList(st["grads"], outs)
        st["norm"] = torch.empty(1, device="cuda")
        st["ws"] = torch.empty(moe.clip_grad_norm_workspace_size(st["list"]), dtype=torch.uint8,
                               device="cuda")
    return st


# --------------------------------------------------------------------------------- run ----

def run(state):
    c = state["case"]
    forward = c["direction"] == "forward"
    if c["op"] == "grouped":
        if forward:
            return _run_grouped_own(state) if own else _run_grouped(state)
        return _run_grouped_grad_own(state) if own else _run_grouped_grad(state)
    if c["op"] == "norm":
        if forward:
            return _run_norm_own(state) if own else _run_norm(state)
        return _run_norm_grad_own(state) if own else _run_norm_grad(state)
    return _run_clip_own(state) if own else _run_clip(state)


def _run_grouped_own(st):
    _pkg().grouped_linear(st["cfg"], st["x"], st["offsets"], st["w"], st["y"], st["z"], st["ws"])
    return [st["y"], st["z"]] if st["case"]["keep"] else [st["y"]]


def _run_grouped_grad_own(st):
    _pkg().grouped_linear_backward(st["cfg"], st["dy"], st["x"], st["offsets"], st["w"], st["z"],
                                   st["dx"], st["dw"], st["ws"])
    return [st["dx"], st["dw"]]


def _run_norm_own(st):
    _pkg().block_norm(st["cfg"], st["x"], st["residual"], st["post"], st["gate"], st["scale"],
                      st["norm"], st["sum"], st["y"])
    return [st["sum"], st["y"]] if st["case"]["norm"] else [st["sum"]]


def _run_norm_grad_own(st):
    _pkg().block_norm_backward(st["cfg"], st["dy"], st["dsum"], st["x"], st["sum"], st["post"],
                               st["gate"], st["scale"], st["norm"], *st["out"], st["ws"])
    return [t for t in st["out"] if t is not None]


def _run_clip_own(st):
    _pkg().clip_grad_norm(st["list"], _MAX_NORM, st["norm"], st["ws"],
                          grad_scale=st["case"]["scale"])
    return [st["norm"], *st["flat"].values()] if st["case"]["write"] else [st["norm"]]


def _run_grouped(st):
    c, x, w = st["case"], st["x"], st["w"]
    F, N = c["fout"], _outputs(c)
    y = torch.zeros(c["rows"], F, dtype=_dtype(c["out"]), device=x.device)
    z = torch.zeros(c["rows"], N, dtype=x.dtype, device=x.device) if c["keep"] else None
    for e, (a, b) in enumerate(zip(st["bounds"], st["bounds"][1:])):
        if a == b:
            continue
        v = x[a:b].float() @ w[e].float().t()
        if z is not None:
            z[a:b] = v
        if c["act"] == "swiglu":
            gate = v[:, :F]
            v = gate / (1.0 + torch.exp(-gate)) * v[:, F:]
        y[a:b] = v
    return [y] if z is None else [y, z]


def _run_grouped_grad(st):
    c, x, w = st["case"], st["x"], st["w"]
    F = c["fout"]
    dx = torch.zeros(c["rows"], c["fin"], dtype=_dtype(c["dx"]), device=x.device)
    dw = torch.zeros_like(w)
    for e, (a, b) in enumerate(zip(st["bounds"], st["bounds"][1:])):
        if a == b:
            continue
        dz = st["dy"][a:b].float()
        if c["act"] == "swiglu":
            gate, up = st["z"][a:b, :F].float(), st["z"][a:b, F:].float()
            s = 1.0 / (1.0 + torch.exp(-gate))
            dz = torch.cat([dz * up * s * (1.0 + gate * (1.0 - s)), dz * gate * s], dim=1)
        dx[a:b] = dz @ w[e].float()
        dw[e] = dz.t() @ x[a:b].float()
    return [dx, dw]


def _gate(c, gate):
    return 1.0 / (1.0 + torch.exp(-gate)) if c["gate"] == "logistic" else gate


def _unit(v):
    """v over its root mean square, and the reciprocal of that."""
    r = 1.0 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + _EPS)
    return v * r, r


def _run_norm(st):
    c, dt = st["case"], st["x"].dtype
    p = st["x"].float()
    if c["post"]:
        p = _unit(p)[0] * st["post"]
    p = p * _BRANCH_SCALE
    if c["gate"] != "none":
        p = p * _gate(c, st["gate"])[:, None]
    if c["scale"]:
        p = p * st["scale"]
    if c["residual"]:
        p = p + st["residual"].float() * _RESIDUAL_SCALE
    if not c["norm"]:
        return [p.to(dt)]
    return [p.to(dt), (_unit(p)[0] * st["norm"]).to(dt)]


def _run_norm_grad(st):
    c, dt = st["case"], st["x"].dtype
    ds = st["dsum"].float()
    sums = {}
    if c["norm"]:
        n, r = _unit(st["sum"].float())
        dy = st["dy"].float()
        sums["norm"] = (dy * n).double().sum(dim=0).float()
        dn = dy * st["norm"]
        ds = ds + r * (dn - n * (dn * n).mean(dim=1, keepdim=True))
    out = {"residual": (ds * _RESIDUAL_SCALE).to(dt)} if c["residual"] else {}
    p = x = st["x"].float()
    if c["post"]:
        n, r = _unit(x)
        p = n * st["post"]
    dp = ds * _BRANCH_SCALE
    dq = dp * st["scale"] if c["scale"] else dp
    if c["gate"] != "none":
        gate = _gate(c, st["gate"])
        slope = gate * (1.0 - gate) if c["gate"] == "logistic" else 1.0
        out["gate"] = (dq * p).sum(dim=1) * slope
        dp, dq = dp * gate[:, None], dq * gate[:, None]
    if c["scale"]:
        sums["scale"] = (dp * p).double().sum(dim=0).float()
    if c["post"]:
        sums["post"] = (dq * n).double().sum(dim=0).float()
        dn = dq * st["post"]
        dq = r * (dn - n * (dn * n).mean(dim=1, keepdim=True))
    return ([dq.to(dt)] + [out[k] for k in ("residual", "gate") if k in out]
            + [sums[k] for k in ("post", "scale", "norm") if k in sums])


def _run_clip(st):
    c = st["case"]
    # a sum over hundreds of millions of squares: 64 bits
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for g in st["grads"]:
        total = total + (g.float() * g.float()).sum(dtype=torch.float64)
    norm = torch.sqrt(total) * c["scale"]
    out = [norm.float().reshape(1)]
    if c["write"]:
        factor = (c["scale"] * torch.clamp(_MAX_NORM / (norm + 1e-6), max=1.0)).float()
        flat = {t: torch.zeros(n, dtype=_dtype(t), device="cuda") for t, n in st["end"].items()}
        for g, (t, at) in zip(st["grads"], st["place"]):
            flat[t][at:at + g.numel()] = g.float() * factor
        out += flat.values()
    return out


# ------------------------------------------------------------------------------- exact ----

def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    return {"grouped": _exact_grouped, "norm": _exact_norm, "clip": _exact_clip}[case["op"]](st)


def _exact_grouped(st):
    c, b = st["case"], st["bounds"]
    F, dev = c["fout"], st["x"].device
    new = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)
    M, N, I = c["rows"], _outputs(c), c["fin"]
    if c["direction"] == "forward":
        z, y = new(M, N), new(M, F)
        for e in range(c["groups"]):
            at = slice(b[e], b[e + 1])
            z[at] = torch.einsum("ri,ni->rn", st["x"][at].double(), st["w"][e].double())
        if c["act"] == "swiglu":
            y += torch.nn.functional.silu(z[:, :F]) * z[:, F:]
        else:
            y += z
        return [y, z] if c["keep"] else [y]
    dz = st["dy"].double()
    if c["act"] == "swiglu":
        gate, up = st["z"].double().split(F, dim=1)
        s = torch.sigmoid(gate)
        dz = torch.cat([dz * up * (s + gate * s * (1.0 - s)),
                        dz * torch.nn.functional.silu(gate)], dim=1)
    dx, dw = new(M, I), new(c["groups"], N, I)
    for e in range(c["groups"]):
        at = slice(b[e], b[e + 1])
        dx[at] = torch.einsum("rn,ni->ri", dz[at], st["w"][e].double())
        dw[e] = torch.einsum("rn,ri->ni", dz[at], st["x"][at].double())
    return [dx, dw]


def _exact_norm(st):
    c = st["case"]
    d = lambda t: None if t is None else t.double()
    x, res = d(st["x"]), d(st["residual"])
    wp, sc, wn, gate = d(st["post"]), d(st["scale"]), d(st["norm"]), d(st["gate"])
    ms = lambda t: torch.rsqrt(torch.einsum("tw,tw->t", t, t) / t.shape[1] + _EPS)[:, None]
    T, W = x.shape
    one = lambda t: torch.ones(W, dtype=torch.float64, device=x.device) if t is None else t
    g = torch.ones(T, dtype=torch.float64, device=x.device) if gate is None else gate
    if c["gate"] == "logistic":
        g = torch.sigmoid(g)
    rx = ms(x) if c["post"] else torch.ones(T, 1, dtype=torch.float64, device=x.device)
    column = one(sc) * _BRANCH_SCALE  # what multiplies a normalised, weighted column
    if c["direction"] == "forward":
        s = x * rx * (one(wp) * column) * g[:, None]
        if res is not None:
            s += _RESIDUAL_SCALE * res
        return [s, s * ms(s) * wn] if c["norm"] else [s]
    ds = d(st["dsum"])
    if c["norm"]:
        s, dy = d(st["sum"]), d(st["dy"])
        rs = ms(s)
        d_norm = torch.einsum("tw,tw->w", dy, s * rs)
        up = dy * wn
        ds = ds + rs * up - s * rs ** 3 * torch.einsum("tw,tw->t", up, s)[:, None] / W
    out = []
    if c["residual"]:
        out.append(_RESIDUAL_SCALE * ds)
    unit = x * rx
    if gate is not None:
        dg = torch.einsum("tw,tw,w->t", ds, unit, one(wp) * column)
        out.append(dg * g * (1.0 - g) if c["gate"] == "logistic" else dg)
    gds = ds * g[:, None]
    if c["post"]:
        out.append(torch.einsum("tw,tw->w", gds, unit) * column)
    if c["scale"]:
        out.append(torch.einsum("tw,tw->w", gds, unit) * one(wp) * _BRANCH_SCALE)
    if c["norm"]:
        out.append(d_norm)
    v = gds * (one(wp) * column)
    if c["post"]:
        v = rx * v - x * rx ** 3 * torch.einsum("tw,tw->t", v, x)[:, None] / W
    return [v] + out


def _exact_clip(st):
    c = st["case"]
    squares = [torch.linalg.vector_norm(g, dtype=torch.float64) ** 2 for g in st["grads"]]
    norm = c["scale"] * math.sqrt(sum(float(s) for s in squares))
    out = [torch.tensor([norm], dtype=torch.float64)]
    if c["write"]:
        factor = c["scale"] * min(1.0, _MAX_NORM / (norm + 1e-6))
        flat = {t: torch.zeros(n, dtype=torch.float64, device="cuda")
                for t, n in st["end"].items()}
        for g, (t, at) in zip(st["grads"], st["place"]):
            torch.mul(g.double(), factor, out=flat[t][at:at + g.numel()])
        out += flat.values()
    return out
