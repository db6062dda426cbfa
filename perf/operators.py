"""Timed cases of the routing, linear and combine-gradient operators.

Every case is one call (or a forward call and its backward call) as a program around a
mixture-of-experts layer makes it.  With ``own`` false, ``run`` computes the operators from
elementary torch operations; with ``own`` true it calls this package.

 route            logits -> expert ids and weights: softmax or sigmoid scores, a balance bias
                  that takes part in the choice only, expert groups, top-k, renormalisation
 route gradient   d weights -> d logits
 linear           y = act(x W^T + bias) + residual, the pre-activation kept for the backward
 linear gradient  dx, dW, d bias from dy, x, W and the kept pre-activation
 combine gradient d route weights and d expert rows from dy
"""

import math

import numpy as np
import torch

own = False

_ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def _pkg():
    import mixture_experts_layer_04_gb300 as moe
    return moe


# ------------------------------------------------------------------------------- cases ----

def _route(name, T, E, K, groups, top_groups, rank, score, bias, renorm, scale, dtype, masked,
           direction):
    c = dict(op="route", direction=direction, T=T, E=E, K=K, groups=groups,
             top_groups=top_groups, rank=rank, score=score, bias=bias, renorm=renorm,
             scale=scale, dtype=dtype, masked=masked)
    if name:
        c["name"] = name
    return c


def _linear(name, rows, fin, fout, dtype, act, bias, residual, keep, pad, direction):
    c = dict(op="linear", direction=direction, rows=rows, fin=fin, fout=fout, dtype=dtype,
             act=act, bias=bias, residual=residual, keep=keep, pad=pad)
    if name:
        c["name"] = name
    return c


def _combine(name, T, H, K, dtype):
    c = dict(op="combine", direction="backward", T=T, H=H, K=K, dtype=dtype)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one token being decoded through a DeepSeek-shaped router: latency only
        _route("route_token", 1, 256, 8, 8, 4, 2, "sigmoid", True, True, 2.5, "float32", False,
               "forward"),
        # the same router over a prefill of 16384 tokens
        _route("route_prefill", 16384, 256, 8, 8, 4, 2, "sigmoid", True, True, 2.5, "float32",
               False, "forward"),
        # a small expert count, plain softmax weights, bf16 logits, an odd number of tokens:
        # a training step's forward and backward
        _route("route_step_softmax", 4099, 60, 4, 1, 1, 1, "softmax", False, False, 1.0,
               "bfloat16", False, "both"),
        # the router's backward of a training step over 16384 tokens
        _route("route_grad", 16384, 256, 8, 8, 4, 2, "sigmoid", True, True, 2.5, "float32", False,
               "backward"),
        # one token through an attention output projection with its residual
        _linear("linear_token", 1, 4096, 4096, "bfloat16", "none", False, True, False, 0,
                "forward"),
        # 64 sequences being decoded through a dense projection; x is a column slice
        _linear("linear_batch", 64, 7168, 2048, "bfloat16", "silu", True, True, False, 64,
                "forward"),
        # the first product of a dense feed-forward layer in a training step's forward
        _linear("linear_prefill", 4096, 4096, 14336, "bfloat16", "gelu_tanh", True, False, True,
                0, "forward"),
        # a small float32 layer of odd sizes
        _linear("linear_f32_odd", 333, 1001, 777, "float32", "silu", True, True, True, 3,
                "forward"),
        # the backward of a dense layer in a training step
        _linear("linear_grad", 8192, 2048, 7168, "bfloat16", "gelu", True, False, True, 0,
                "backward"),
        # a small float32 backward of odd sizes
        _linear("linear_grad_f32_odd", 517, 515, 1001, "float32", "relu", True, False, True, 0,
                "backward"),
        # the combine's backward for a handful of tokens
        _combine("combine_grad_tokens", 16, 2048, 8, "bfloat16"),
        # and for a Qwen3-shaped training batch
        _combine("combine_grad_batch", 8192, 2048, 8, "bfloat16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


_MAX_FLOPS = 4 * 8192 * 2048 * 7168


def draw(rng):
    op = rng.choice(("route", "route", "linear", "linear", "linear", "combine"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        per = rng.randint(max(2, 16 // groups), 256 // groups)
        E = groups * per
        top_groups = rng.randint(max(1, (groups + 1) // 2), groups)
        K = rng.randint(1, min(10, top_groups * per))
        return _route(None, _log_int(rng, 1, 16384), E, K, groups, top_groups,
                      rng.choice((1, 2)), rng.choice(("softmax", "sigmoid")),
                      rng.random() < 0.5, rng.random() < 0.6, rng.choice((1.0, 2.5)),
                      rng.choice(("float32", "bfloat16")), rng.random() < 0.3,
                      rng.choice(("forward", "backward", "both")))
    if op == "combine":
        T = _log_int(rng, 1, 8192)
        return _combine(None, T, 64 * _log_int(rng, 4, 64), rng.randint(1, 10),
                        rng.choice(("bfloat16", "bfloat16", "float32")))
    direction = rng.choice(("forward", "forward", "backward"))
    dtype = rng.choice(("bfloat16", "bfloat16", "float32"))
    act = rng.choice(_ACTS)
    rows, fin, fout = _log_int(rng, 1, 8192), _log_int(rng, 64, 8192), _log_int(rng, 64, 14336)
    if rng.random() < 0.6:  # most layers have sizes that are multiples of 64
        fin, fout = max(64, fin // 64 * 64), max(64, fout // 64 * 64)
    cap = _MAX_FLOPS if dtype == "bfloat16" else _MAX_FLOPS // 8
    per_row = (2 if direction == "forward" else 4) * fin * fout
    rows = max(1, min(rows, cap // per_row))
    return _linear(None, rows, fin, fout, dtype, act, rng.random() < 0.7,
                   direction == "forward" and rng.random() < 0.5,
                   direction == "backward" or rng.random() < 0.5,
                   rng.choice((0, 0, 5, 64)), direction)


# -------------------------------------------------------------------------------- work ----

def _size(dtype):
    return 2 if dtype == "bfloat16" else 4


def work(case):
    b, f = 0, 0
    if case["op"] == "route":
        T, E, K, sz = case["T"], case["E"], case["K"], _size(case["dtype"])
        if case["direction"] != "backward":
            b += T * E * sz + T * K * 8 + (4 * E if case["bias"] else 0)
            f += 8 * T * E
        if case["direction"] != "forward":
            # the dense gradient is written; without renormalisation a softmax row is read too
            dense = case["score"] == "softmax" and not case["renorm"]
            b += T * E * sz + T * K * 8 + (T * E * sz if dense else T * K * sz)
            f += 8 * T * (E if dense else K)
    elif case["op"] == "linear":
        M, I, N, sz = case["rows"], case["fin"], case["fout"], _size(case["dtype"])
        if case["direction"] == "forward":
            b = (M * I + N * I + M * N * (1 + case["residual"] + case["keep"])) * sz
            f = 2 * M * N * I
        else:
            has_z = case["act"] != "none"
            b = (2 * M * I + 2 * N * I + M * N * (1 + has_z)) * sz
            f = 4 * M * N * I
        b += 4 * N if case["bias"] else 0
    else:
        T, H, K, sz = case["T"], case["H"], case["K"], _size(case["dtype"])
        b = T * K * H * (4 + sz) + T * H * sz + T * K * 12
        f = 3 * T * K * H
    return {"bytes": int(b), "flops": int(f)}


# ----------------------------------------------------------------------------- prepare ----

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    x = torch.randn(*shape, generator=g, device="cuda")
    if std != 1.0:
        x *= std
    return x if dtype == torch.float32 else x.to(dtype)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bfloat16" else torch.float32


def prepare(case, seed):
    return {"route": _prepare_route, "linear": _prepare_linear,
            "combine": _prepare_combine}[case["op"]](case, seed)


def _prepare_route(case, seed):
    g = _gen(seed)
    T, E, K = case["T"], case["E"], case["K"]
    logits = _randn(g, T, E, dtype=_dtype(case), std=1.5)
    if case["masked"]:
        # a quarter of the experts masked at each token, and now and then all of them
        gone = torch.rand(T, E, generator=g, device="cuda") < 0.25
        gone |= torch.rand(T, 1, generator=g, device="cuda") < 0.02
        logits[gone] = float("-inf")
    st = dict(case=case, logits=logits,
              bias=_randn(g, E, std=0.1) if case["bias"] else None)
    if case["direction"] != "forward":
        st["d_weights"] = _randn(g, T, K)
    if case["direction"] == "backward":
        # K distinct available experts a token; which ones the gradient does not mind
        top = logits.float().topk(K, dim=1)
        st["ids"] = torch.where(top.values > float("-inf"), top.indices,
                                -torch.ones_like(top.indices)).to(torch.int32)
    if own:
        moe = _pkg()
        st["cfg"] = moe.RouteConfig.make(
            T=T, E=E, K=K, groups=case["groups"], top_groups=case["top_groups"],
            group_rank=case["rank"],
            score=moe.SCORE_SIGMOID if case["score"] == "sigmoid" else moe.SCORE_SOFTMAX,
            renormalise=case["renorm"], scale=case["scale"],
            dtype=moe.BF16 if case["dtype"] == "bfloat16" else moe.F32)
        if case["direction"] != "backward":
            st["ids"] = torch.empty(T, K, dtype=torch.int32, device="cuda")
            st["weights"] = torch.empty(T, K, device="cuda")
        if case["direction"] != "forward":
            st["d_logits"] = torch.empty_like(logits)
    return st


def _prepare_linear(case, seed):
    g = _gen(seed)
    M, I, N, dt = case["rows"], case["fin"], case["fout"], _dtype(case)
    st = dict(case=case)
    # with `pad` x is a slice of a wider activation (a fused projection's output)
    st["x"] = _randn(g, M, I + case["pad"], dtype=dt)[:, :I]
    st["w"] = _randn(g, N, I, dtype=dt, std=I ** -0.5)
    st["bias"] = _randn(g, N, std=0.1) if case["bias"] else None
    st["residual"] = _randn(g, M, N, dtype=dt) if case["residual"] else None
    if case["direction"] == "backward":
        st["dy"] = _randn(g, M, N, dtype=dt)
        st["z"] = _randn(g, M, N, dtype=dt) if case["act"] != "none" else None
    if own:
        moe = _pkg()
        st["cfg"] = moe.LinearConfig.make(
            rows=M, in_features=I, out_features=N,
            dtype=moe.BF16 if dt == torch.bfloat16 else moe.F32,
            activation=getattr(moe, "ACT_" + case["act"].upper()), x_stride=I + case["pad"])
        st["ws"] = torch.empty(moe.linear_workspace_size(st["cfg"]), dtype=torch.uint8,
                               device="cuda")
        if case["direction"] == "forward":
            st["y"] = torch.empty(M, N, dtype=dt, device="cuda")
            st["z_out"] = torch.empty(M, N, dtype=dt, device="cuda") if case["keep"] else None
        else:
            st["dx"] = torch.empty(M, I, dtype=dt, device="cuda")
            st["dw"] = torch.empty(N, I, dtype=dt, device="cuda")
            st["dbias"] = torch.empty(N, device="cuda") if case["bias"] else None
    return st


def _prepare_combine(case, seed):
    g = _gen(seed)
    T, H, K, dt = case["T"], case["H"], case["K"], _dtype(case)
    st = dict(case=case)
    st["dy"] = _randn(g, T, H, dtype=dt)
    st["rows"] = _randn(g, T * K, H)
    st["weights"] = torch.softmax(_randn(g, T, K), dim=1)
    st["inv"] = torch.randperm(T * K, generator=g, device="cuda").to(torch.int32).view(T, K)
    if own:
        moe = _pkg()
        st["cfg"] = moe.MoEConfig.make(T=T, H=H, E=max(K, 16), K=K, I=64,
                                       dtype=moe.BF16 if dt == torch.bfloat16 else moe.F32)
        st["d_rows"] = torch.empty(T * K, H, dtype=dt, device="cuda")
        st["d_weights"] = torch.empty(T, K, device="cuda")
    return st


# --------------------------------------------------------------------------------- run ----

def run(state):
    c = state["case"]
    if c["op"] == "route":
        return _run_route_own(state) if own else _run_route(state)
    if c["op"] == "linear":
        if c["direction"] == "forward":
            return _run_linear_own(state) if own else _run_linear(state)
        return _run_linear_grad_own(state) if own else _run_linear_grad(state)
    return _run_combine_own(state) if own else _run_combine(state)


def _run_route_own(st):
    moe, c, out = _pkg(), st["case"], []
    if c["direction"] != "backward":
        moe.route_scored(st["cfg"], st["logits"], st["bias"], st["ids"], st["weights"])
        out += [st["ids"], st["weights"]]
    if c["direction"] != "forward":
        moe.route_scored_backward(st["cfg"], st["logits"], st["ids"], st["d_weights"],
                                  st["d_logits"])
        out.append(st["d_logits"])
    return out


def _run_linear_own(st):
    moe = _pkg()
    moe.linear(st["cfg"], st["x"], st["w"], st["bias"], st["residual"], st["y"], st["z_out"],
               st["ws"])
    return [st["y"], st["z_out"]] if st["case"]["keep"] else [st["y"]]


def _run_linear_grad_own(st):
    moe = _pkg()
    moe.linear_backward(st["cfg"], st["dy"], st["x"], st["w"], st["z"], st["dx"], st["dw"],
                        st["dbias"], st["ws"])
    return [st["dx"], st["dw"]] + ([st["dbias"]] if st["case"]["bias"] else [])


def _run_combine_own(st):
    moe = _pkg()
    moe.combine_backward(st["cfg"], st["dy"], st["rows"], st["inv"], st["weights"], st["d_rows"],
                         st["d_weights"])
    return [st["d_rows"], st["d_weights"]]


def _scores(c, logits):
    """Scores of every expert in 64 bits (0 where the expert is masked)."""
    l = logits.double()
    if c["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    m = l.amax(dim=1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = torch.exp(l - m)
    return p / p.sum(dim=1, keepdim=True).clamp_min(1e-300)


def _run_route(st):
    c, logits = st["case"], st["logits"]
    T, E, K, G = c["T"], c["E"], c["K"], c["groups"]
    minus = float("-inf")
    s = _scores(c, logits)
    out = []
    if c["direction"] != "backward":
        key = s if st["bias"] is None else s + st["bias"].double()
        key = torch.where(logits == minus, torch.full_like(key, minus), key)
        if c["top_groups"] < G:
            best = key.view(T, G, E // G).sort(dim=2, descending=True).values
            best = best[:, :, :c["rank"]]
            some = best[:, :, 0] > minus
            total = torch.where(best > minus, best, torch.zeros_like(best)).sum(dim=2)
            total = torch.where(some, total, torch.full_like(total, minus))
            order = total.sort(dim=1, descending=True, stable=True).indices
            live = torch.zeros(T, G, dtype=torch.bool, device=key.device)
            live.scatter_(1, order[:, :c["top_groups"]], True)
            live = live.repeat_interleave(E // G, dim=1)
            key = torch.where(live, key, torch.full_like(key, minus))
        top = key.sort(dim=1, descending=True, stable=True)
        ids = top.indices[:, :K]
        have = top.values[:, :K] > minus
        w = torch.where(have, s.gather(1, ids), torch.zeros_like(ids, dtype=s.dtype))
        if c["renorm"]:
            w = w / w.sum(dim=1, keepdim=True).clamp_min(1e-300)
        ids = torch.where(have, ids, torch.full_like(ids, -1)).to(torch.int32)
        out += [ids, (w * c["scale"]).float()]
    else:
        ids = st["ids"]
    if c["direction"] != "forward":
        have = ids >= 0
        at = ids.clamp_min(0).long()
        dw = torch.where(have, st["d_weights"].double() * c["scale"], 0.0)
        sk = torch.where(have, s.gather(1, at), torch.zeros_like(dw))
        if c["renorm"]:
            total = sk.sum(dim=1, keepdim=True).clamp_min(1e-300)
            dw = (dw - (dw * sk).sum(dim=1, keepdim=True) / total) / total
        ds = torch.zeros_like(s).scatter_add_(1, at, torch.where(have, dw, torch.zeros_like(dw)))
        if c["score"] == "sigmoid":
            dl = ds * s * (1.0 - s)
        else:
            dl = s * (ds - (ds * s).sum(dim=1, keepdim=True))
        out.append(dl.to(logits.dtype))
    return out


def _act(name, z):
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    if name == "gelu_tanh":
        u = (2.0 / math.pi) ** 0.5 * (z + 0.044715 * z * z * z)
        return 0.5 * z * (1.0 + torch.tanh(u))
    if name == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return (0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5))
                + z * torch.exp(-0.5 * z * z) * (1.0 / (2.0 * math.pi) ** 0.5))
    if name == "gelu_tanh":
        a = (2.0 / math.pi) ** 0.5
        t = torch.tanh(a * (z + 0.044715 * z * z * z))
        return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * a * (1.0 + 3.0 * 0.044715 * z * z)
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return torch.ones_like(z)


def _run_linear(st):
    c, dt = st["case"], st["x"].dtype
    z = st["x"].float() @ st["w"].float().t()
    if st["bias"] is not None:
        z = z + st["bias"]
    y = _act(c["act"], z)
    if st["residual"] is not None:
        y = y + st["residual"].float()
    return [y.to(dt), z.to(dt)] if c["keep"] else [y.to(dt)]


def _run_linear_grad(st):
    c, dt = st["case"], st["x"].dtype
    dz = st["dy"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(c["act"], st["z"].float())
    out = [(dz @ st["w"].float()).to(dt), (dz.t() @ st["x"].float()).to(dt)]
    if c["bias"]:
        out.append(dz.double().sum(dim=0).float())
    return out


def _run_combine(st):
    T, K = st["inv"].shape
    dy, at = st["dy"].float(), st["inv"].long()
    d_rows = torch.empty(st["rows"].shape, dtype=st["dy"].dtype, device=dy.device)
    d_weights = torch.empty(T, K, device=dy.device)
    for k in range(K):
        d_weights[:, k] = (dy * st["rows"][at[:, k]]).sum(dim=1)
        d_rows[at[:, k]] = (st["weights"][:, k:k + 1] * dy).to(d_rows.dtype)
    return [d_rows, d_weights]


# ------------------------------------------------------------------------------- exact ----

def exact(case, seed):
    global own
    keep, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = keep
    if case["op"] == "route":
        return _exact_route(case, st)
    if case["op"] == "linear":
        return _exact_linear(case, st)
    return _exact_combine(st)


def _exact_route(c, st):
    """By the definition, one row after another, in numpy's 64 bits."""
    L = st["logits"].double().cpu().numpy()
    T, E = L.shape
    K, G = c["K"], c["groups"]
    per = E // G
    bias = np.zeros(E) if st["bias"] is None else st["bias"].double().cpu().numpy()
    fwd, bwd = c["direction"] != "backward", c["direction"] != "forward"
    ids = np.full((T, K), -1, np.int64)
    w = np.zeros((T, K))
    dl = np.zeros((T, E))
    given = None if fwd else st["ids"].cpu().numpy()
    dw_all = st["d_weights"].double().cpu().numpy() if bwd else None
    for t in range(T):
        ok = np.flatnonzero(L[t] > -np.inf)
        if ok.size == 0:
            continue
        score = np.zeros(E)
        if c["score"] == "sigmoid":
            score[ok] = 1.0 / (1.0 + np.exp(-L[t, ok]))
        else:
            p = np.exp(L[t, ok] - L[t, ok].max())
            score[ok] = p / p.sum()
        if fwd:
            cand = ok
            key = score + bias
            if c["top_groups"] < G:
                ranked = []
                for g in range(G):
                    mine = key[ok[(ok >= g * per) & (ok < (g + 1) * per)]]
                    if mine.size:
                        ranked.append((-np.sort(mine)[::-1][:c["rank"]].sum(), g))
                chosen = {g for _, g in sorted(ranked)[:c["top_groups"]]}
                cand = np.array([e for e in ok if e // per in chosen])
            pick = cand[np.argsort(-key[cand], kind="stable")][:K]
            ids[t, :pick.size] = pick
        else:
            pick = given[t][given[t] >= 0]
        kept = score[pick]
        total = kept.sum() if c["renorm"] else 1.0
        if fwd:
            w[t, :pick.size] = c["scale"] * kept / total
        if bwd:
            up = c["scale"] * dw_all[t, :pick.size]
            # d w_k / d s_j = (delta_kj - w_k/scale) / total with renormalisation
            d_score = np.zeros(E)
            if c["renorm"]:
                d_score[pick] = up / total - (up @ kept) / total ** 2
            else:
                d_score[pick] = up
            if c["score"] == "sigmoid":
                dl[t] = d_score * score * (1.0 - score)
            else:
                dl[t] = score * d_score - score * (score @ d_score)
    out = []
    if fwd:
        out += [torch.from_numpy(ids).to(torch.int32), torch.from_numpy(w)]
    if bwd:
        out.append(torch.from_numpy(dl))
    return out


def _exact_linear(c, st):
    x, w = st["x"].double(), st["w"].double()
    name = c["act"]
    if c["direction"] == "forward":
        z = torch.einsum("mi,ni->mn", x, w)
        if st["bias"] is not None:
            z += st["bias"].double()[None, :]
        if name == "relu":
            y = z.clamp(min=0.0)
        elif name == "gelu":
            y = 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
        elif name == "gelu_tanh":
            # (1 + tanh u) / 2 is the logistic function of 2u
            y = z * torch.sigmoid(math.sqrt(8.0 / math.pi) * (z + 0.044715 * z ** 3))
        elif name == "silu":
            y = z * torch.sigmoid(z)
        else:
            y = z.clone()
        if st["residual"] is not None:
            y += st["residual"].double()
        return [y, z] if c["keep"] else [y]
    dz = st["dy"].double()
    if name != "none":
        z = st["z"].double()
        if name == "relu":
            slope = torch.heaviside(z, torch.zeros((), dtype=z.dtype, device=z.device))
        elif name == "gelu":
            slope = (0.5 * torch.special.erfc(-z / math.sqrt(2.0))
                     + z * torch.exp(-z * z / 2.0) / math.sqrt(2.0 * math.pi))
        elif name == "gelu_tanh":
            a = math.sqrt(8.0 / math.pi)
            p = torch.sigmoid(a * (z + 0.044715 * z ** 3))
            slope = p + z * p * (1.0 - p) * a * (1.0 + 0.134145 * z * z)
        else:
            p = torch.sigmoid(z)
            slope = p + z * p * (1.0 - p)
        dz = dz * slope
    out = [torch.einsum("mn,ni->mi", dz, w), torch.einsum("mn,mi->ni", dz, x)]
    if c["bias"]:
        out.append(torch.einsum("mn->n", dz))
    return out


def _exact_combine(st):
    T, K = st["inv"].shape
    owner = torch.empty(T * K, dtype=torch.long, device=st["dy"].device)
    flat = st["inv"].long().flatten()
    owner[flat] = torch.arange(T * K, device=owner.device)  # row -> its assignment
    dots = torch.empty(T * K, dtype=torch.float64, device=owner.device)
    d_rows = torch.empty(st["rows"].shape, dtype=torch.float64, device=owner.device)
    wts = st["weights"].double().flatten()
    step = 8192
    for r in range(0, T * K, step):
        a = owner[r:r + step]
        grad = st["dy"][a // K].double()
        dots[a] = torch.einsum("rh,rh->r", grad, st["rows"][r:r + step].double())
        d_rows[r:r + step] = grad * wts[a][:, None]
    return [d_rows, dots.view(T, K)]
