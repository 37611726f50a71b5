"""Workloads of the operators around an expert layer: the choice of experts
(scores, balance bias, groups, top-k, renormalised weights) and the norms
before and after a block with its gate and residual, each with its gradient.

``run`` computes them with elementary torch operations in 32 bits, or, with
``own`` set, with the library's ``ExpertRouter`` and ``BlockNorm``.  ``exact``
evaluates the definitions in 64 bits.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_EPS_SUM = 1e-20          # added to the sum of the chosen scores
_LOWEST = -3.0e38         # ranks an excluded expert below every other one

# Largest listed sizes; drawn cases stay within their cost.
_MAX_LOGITS = 131072 * 256
_MAX_NORM = 16384 * 8192


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _route(name, T, E, K, score="softmax", groups=1, top_groups=1, group_score="max", bias=False, renorm=True,
           scale=1.0, dtype="f32", pad=0, mask=0.0, backward=False):
    return {"name": name, "op": "route_backward" if backward else "route", "T": T, "E": E, "K": K, "score": score,
            "groups": groups, "top_groups": top_groups, "group_score": group_score, "bias": bias, "renorm": renorm,
            "scale": scale, "dtype": dtype, "pad": pad, "mask": mask}


def _norm(name, T, H, kind="rms", dtype="bf16", residual="same", weights="same", gate="none", gate_sigmoid=False,
          post=True, pre=True, offset=0.0, scale=1.0, eps=1e-6, pad=0, backward=False):
    return {"name": name, "op": "norm_backward" if backward else "norm", "T": T, "H": H, "kind": kind, "dtype": dtype,
            "residual": residual, "weights": weights, "gate": gate, "gate_sigmoid": gate_sigmoid, "post": post,
            "pre": pre, "offset": offset, "scale": scale, "eps": eps, "pad": pad}


def listed():
    return [
        # One decode step of 64 sequences through a layer of 256 experts in 8
        # groups, scored by sigmoid with a balance bias: latency only.
        _route("route_decode", 64, 256, 8, "sigmoid", 8, 4, "top2", bias=True, scale=2.5),
        # A prefill chunk of the 128-expert layer, 4073 tokens: softmax over
        # bf16 logits with no groups, some experts closed to some tokens.
        _route("route_prefill", 4073, 128, 8, "softmax", dtype="bf16", mask=0.1),
        # A training batch with 160 experts in groups of 20 (no power of
        # two), the best expert of a group scoring it, weights left as they are.
        _route("route_groups_160", 32768, 160, 6, "softmax", 8, 3, "max", renorm=False, scale=16.0),
        # The largest training batch: 131072 tokens, 256 experts, 8 groups.
        _route("route_train", 131072, 256, 8, "sigmoid", 8, 4, "top2", bias=True, scale=2.5),
        # Router gradients: a small odd batch whose softmax reaches every
        # expert, and the largest batch, where only chosen experts get one.
        _route("route_grad_odd", 4073, 97, 5, "softmax", renorm=False, pad=3, backward=True),
        _route("route_grad_train", 131072, 256, 8, "sigmoid", 8, 4, "top2", bias=True, scale=2.5, backward=True),
        # One decoded token between two blocks: post-norm, residual, pre-norm.
        _norm("norm_decode", 1, 2048),
        # A ragged prefill with an odd width (no vector loads line up),
        # centred norms, a per-token sigmoid gate and a scaled branch.
        _norm("norm_odd_layer", 1777, 2047, "layer", "f16", gate="token", gate_sigmoid=True, scale=0.22, eps=1e-5),
        # The prefill chunk of 4096 tokens: 32-bit residual stream, a
        # per-channel gate.
        _norm("norm_prefill", 4096, 2048, residual="f32", gate="channel", weights="f32"),
        # The largest batch, wide rows, weights stored as offsets from one.
        _norm("norm_train", 16384, 8192, offset=1.0),
        # Gradients: a ragged chunk with a full gate and centred norms, and
        # the largest batch.
        _norm("norm_grad_layer", 4073, 4096, "layer", gate="full", residual="f32", weights="f32", scale=0.5,
              eps=1e-5, backward=True),
        _norm("norm_grad_train", 16384, 8192, offset=1.0, backward=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    backward = rng.random() < 0.4
    if rng.random() < 0.5:
        groups = rng.choice([1, 1, 2, 4, 5, 8, 16])
        size = max(1, _log_int(rng, 8, 512) // groups)
        E = groups * size
        top_groups = rng.randint(1, groups)
        K = rng.randint(1, max(1, min(16, top_groups * size)))
        T = max(1, min(_log_int(rng, 1, 131072), _MAX_LOGITS // E))
        score = rng.choice(["softmax", "sigmoid"])
        renorm = K > 1 and rng.random() < 0.6  # (one renormalised weight is the scale itself)
        return _route(None, T, E, K, score, groups, top_groups, rng.choice(["max", "top2"]), rng.random() < 0.5,
                      renorm, rng.choice([1.0, 2.5]), rng.choice(["f32", "bf16", "f16"]),
                      rng.choice([0, 0, 3, 8]), rng.choice([0.0, 0.0, 0.1]), backward)
    H = _log_int(rng, 64, 8192)
    if rng.random() < 0.7:
        H = max(64, H // 64 * 64)
    T = max(1, min(_log_int(rng, 1, 65536), _MAX_NORM // H))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if dtype == "f32":  # twice the bytes of a 16-bit case
        T = max(1, T // 2)
    residual = rng.choice(["same", "f32"])
    if residual == "f32" and dtype != "f32":
        T = max(1, T * 2 // 3)
    post, pre = rng.choice([(True, True), (True, True), (True, False), (False, True)])
    gate = rng.choice(["none", "none", "channel", "token", "full"])
    if gate == "full":
        T = max(1, T * 2 // 3)
    return _norm(None, T, H, rng.choice(["rms", "rms", "layer"]), dtype, residual, rng.choice(["same", "f32"]), gate,
                 gate != "none" and rng.random() < 0.5, post, pre, rng.choice([0.0, 1.0]), rng.choice([1.0, 0.22]),
                 1e-5, rng.choice([0, 0, 1, 8]), backward)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _padded(t, pad):
    """The same values in rows `pad` elements longer than they need be."""
    if not pad:
        return t
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _draw_logits(case, rows, g):
    # router logits of a trained layer: a few units wide, each token with a
    # sharpness of its own
    E = case["E"]
    sharp = 0.5 + 1.5 * torch.rand(rows, 1, generator=g, device="cuda")
    logits = torch.randn(rows, E, generator=g, device="cuda") * sharp
    if case["mask"]:
        closed = torch.rand(rows, E, generator=g, device="cuda") < case["mask"]
        closed |= torch.rand(rows, 1, generator=g, device="cuda") < 1.0 / 512  # padding tokens: nothing open
        logits = logits.masked_fill(closed, -math.inf)
    return logits.to(_TYPES[case["dtype"]])


def _by_score(case):
    """Whether the choice compares scores (else logits, which order alike)."""
    return case["bias"] or (case["groups"] > 1 and case["group_score"] == "top2")


def _near_ties(case, logits, bias):
    """Rows whose choice hangs on a difference near 32-bit rounding."""
    if not _by_score(case):
        return torch.zeros(logits.shape[0], dtype=torch.bool, device=logits.device)
    choice, open_ = _exact_choice(case, logits, bias)
    tol = 4e-6
    bad = torch.zeros(logits.shape[0], dtype=torch.bool, device=logits.device)
    if case["groups"] > 1 and case["top_groups"] < case["groups"]:
        gs = _exact_group_scores(case, choice).sort(dim=1, descending=True).values
        gap = gs[:, case["top_groups"] - 1] - gs[:, case["top_groups"]]
        bad |= (gap > 0) & (gap < tol)
        choice, open_ = _exact_group_limit(case, choice, open_)
    top = choice.sort(dim=1, descending=True).values[:, :case["K"] + 1]
    gap = top[:, :-1] - top[:, 1:]
    return bad | ((gap > 0) & (gap < tol)).any(dim=1)


def _route_inputs(case, seed):
    g = _gen(seed)
    T, E = case["T"], case["E"]
    # balance biases move by steps of 0.001, so many experts share a value
    bias = None
    if case["bias"]:
        spread = 0.1 if case["score"] == "sigmoid" else 0.02
        bias = (torch.randn(E, generator=g, device="cuda") * spread * 1000).round() / 1000
    logits = _draw_logits(case, T, g)
    for _ in range(12):
        rows = _near_ties(case, logits, bias).nonzero().squeeze(1)
        if rows.numel() == 0:
            break
        logits[rows] = _draw_logits(case, rows.numel(), g)
    st = {"logits": _padded(logits, case["pad"]), "bias": bias}
    if case["op"] == "route_backward":
        ids, w = _plain_route(case, logits, bias)
        st["ids"], st["weights"] = ids, w
        st["dweights"] = torch.randn(T, case["K"], generator=g, device="cuda")
    return st


def _norm_inputs(case, seed):
    g = _gen(seed)
    T, H = case["T"], case["H"]
    dt = _TYPES[case["dtype"]]
    rt = torch.float32 if case["residual"] == "f32" else dt
    wt = torch.float32 if case["weights"] == "f32" else dt

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # a residual stream with a few loud channels; block outputs whose size
    # differs from token to token; 1% padding tokens, all zero
    dead = torch.rand(T, 1, generator=g, device="cuda") < 0.01
    loud = torch.ones(H, device="cuda")
    loud[torch.randint(0, H, (max(1, H // 512),), generator=g, device="cuda")] = 20.0
    residual = (randn(T, H) * loud).masked_fill(dead, 0.0).to(rt)
    size = torch.exp(torch.rand(T, 1, generator=g, device="cuda") * 3.0 - 2.0)
    y = (randn(T, H) * size + 0.1).masked_fill(dead, 0.0).to(dt)
    near_one = 1.0 - case["offset"]
    st = {"residual": _padded(residual, case["pad"]), "y": _padded(y, case["pad"]), "gate": None}
    st["post_weight"] = (near_one + 0.2 * randn(H)).to(wt) if case["post"] else None
    st["pre_weight"] = (near_one + 0.2 * randn(H)).to(wt) if case["pre"] else None
    shape = {"channel": (H,), "token": (T, 1), "full": (T, H)}.get(case["gate"])
    if shape:
        gate = (0.5 + 0.5 * randn(*shape)).to(dt)
        st["gate"] = _padded(gate, case["pad"]) if case["gate"] == "full" else gate
    if case["op"] == "norm_backward":
        st["residual_out"] = _padded(_plain_norm(case, st)[0].to(rt), case["pad"])
        del st["residual"]
        st["dresidual_out"] = _padded((randn(T, H) * 0.5).masked_fill(dead, 0.0).to(rt), case["pad"])
        st["dh"] = _padded(randn(T, H).masked_fill(dead, 0.0).to(dt), case["pad"]) if case["pre"] else None
    return st


def _inputs(case, seed):
    return _route_inputs(case, seed) if case["op"].startswith("route") else _norm_inputs(case, seed)


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if own:
        import nvfp4_token_quantized_gb300 as lib

        if case["op"].startswith("route"):
            state["router"] = lib.ExpertRouter(case["E"], case["K"], score=case["score"], num_groups=case["groups"],
                                               top_groups=case["top_groups"], group_score=case["group_score"],
                                               renormalize=case["renorm"], scale=case["scale"])
        else:
            state["norm"] = lib.BlockNorm(case["H"], kind=case["kind"], eps=case["eps"], post=case["post"],
                                          pre=case["pre"], gate=case["gate"], gate_sigmoid=case["gate_sigmoid"],
                                          weight_offset=case["offset"], branch_scale=case["scale"])
    return state


# ---------------------------------------------------------------------------
# plain forms, 32 bits
# ---------------------------------------------------------------------------

def _plain_scores(case, l):
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    m = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = e.sum(dim=1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total)


def _first_largest(v, n):
    """Indices of the n largest of each row, the first of equal ones first."""
    v = v.clone()
    out = []
    for _ in range(n):
        i = v.max(dim=1, keepdim=True).indices
        out.append(i)
        v.scatter_(1, i, -math.inf)
    return torch.cat(out, dim=1)


def _plain_route(case, logits, bias):
    T, E, G = case["T"], case["E"], case["groups"]
    l = logits.float()
    s = _plain_scores(case, l)
    choice = l
    if _by_score(case):
        choice = s if bias is None else s + bias
    choice = choice.masked_fill(l == -math.inf, _LOWEST)
    if G > 1 and case["top_groups"] < G:
        grouped = choice.view(T, G, E // G)
        best = grouped.amax(dim=2)
        if case["group_score"] == "top2" and E // G > 1:
            first = grouped.max(dim=2, keepdim=True).indices
            second = grouped.scatter(2, first, _LOWEST).amax(dim=2)
            best = torch.where(second > _LOWEST, best + second, best)
        keep = torch.zeros(T, G, dtype=torch.bool, device=l.device)
        keep.scatter_(1, _first_largest(best, case["top_groups"]), True)
        choice = grouped.masked_fill(~keep[:, :, None], _LOWEST).view(T, E)
    ids = _first_largest(choice, case["K"])
    w = torch.where(choice.gather(1, ids) > _LOWEST, s.gather(1, ids), torch.zeros((), device=l.device))
    if case["renorm"]:
        w = w / (w.sum(dim=1, keepdim=True) + _EPS_SUM)
    return ids.int(), w * case["scale"]


def _plain_route_backward(case, st):
    l = st["logits"].float()
    ids = st["ids"].long()
    dw = st["dweights"] * case["scale"]
    s = _plain_scores(case, l)
    live = st["weights"] != 0
    sk = torch.where(live, s.gather(1, ids), torch.zeros((), device=l.device))
    if case["renorm"]:
        total = sk.sum(dim=1, keepdim=True) + _EPS_SUM
        dw = (dw - (dw * sk).sum(dim=1, keepdim=True) / total) / total
    dsk = torch.where(live, dw, torch.zeros((), device=l.device))
    ds = torch.zeros_like(s).scatter_(1, ids, dsk)
    if case["score"] == "sigmoid":
        dl = ds * s * (1.0 - s)
    else:
        dl = s * (ds - (dsk * sk).sum(dim=1, keepdim=True))
    return dl.to(st["logits"].dtype)


def _plain_stats(case, x):
    if case["kind"] == "layer":
        x = x - x.mean(dim=1, keepdim=True)
    rstd = 1.0 / torch.sqrt((x * x).mean(dim=1, keepdim=True) + case["eps"])
    return x * rstd, rstd


def _plain_weight(case, w):
    return w.float() + case["offset"]


def _plain_gate(case, gate):
    if gate is None:
        return None
    g = gate.float()
    return 1.0 / (1.0 + torch.exp(-g)) if case["gate_sigmoid"] else g


def _plain_norm(case, st):
    """The new residual in 32 bits and the normed rows (or None)."""
    b = st["y"].float()
    if case["post"]:
        b = _plain_stats(case, b)[0] * _plain_weight(case, st["post_weight"])
    g = _plain_gate(case, st["gate"])
    if g is not None:
        b = b * g
    r = st["residual"].float() + case["scale"] * b
    h = _plain_stats(case, r)[0] * _plain_weight(case, st["pre_weight"]) if case["pre"] else None
    return r, h


def _plain_norm_grad(case, dout, x, w):
    """Gradients of a norm's input and weight."""
    xhat, rstd = _plain_stats(case, x)
    a = dout * _plain_weight(case, w)
    dx = a - xhat * (a * xhat).mean(dim=1, keepdim=True)
    if case["kind"] == "layer":
        dx = dx - a.mean(dim=1, keepdim=True)
    return dx * rstd, (dout * xhat).sum(dim=0)


def _plain_norm_backward(case, st):
    dt, rt = st["y"].dtype, st["residual_out"].dtype
    dr = st["dresidual_out"].float()
    dpre = None
    if case["pre"]:
        dx, dpre = _plain_norm_grad(case, st["dh"].float(), st["residual_out"].float(), st["pre_weight"])
        dr = dr + dx
    y = st["y"].float()
    g = _plain_gate(case, st["gate"])
    db = case["scale"] * dr
    dgate = None
    if g is not None:
        u = _plain_stats(case, y)[0] * _plain_weight(case, st["post_weight"]) if case["post"] else y
        dgate = db * u
        if case["gate_sigmoid"]:
            dgate = dgate * g * (1.0 - g)
        if case["gate"] == "channel":
            dgate = dgate.sum(dim=0)
        elif case["gate"] == "token":
            dgate = dgate.sum(dim=1, keepdim=True).to(dt)
        else:
            dgate = dgate.to(dt)
        db = db * g
    dpost = None
    if case["post"]:
        db, dpost = _plain_norm_grad(case, db, y, st["post_weight"])
    return _present(dr.to(rt), db.to(dt), dgate, dpost, dpre)


def _present(*outs):
    return [o for o in outs if o is not None]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _run_own(case, st):
    if case["op"] == "route":
        return list(st["router"].select(st["logits"], bias=st["bias"]))
    if case["op"] == "route_backward":
        return [st["router"].select_backward(st["logits"], st["ids"], st["weights"], st["dweights"])]
    if case["op"] == "norm":
        return _present(*st["norm"].forward(st["residual"], st["y"], gate=st["gate"], post_weight=st["post_weight"],
                                            pre_weight=st["pre_weight"]))
    grads = st["norm"].backward(st["dresidual_out"], st["dh"], st["residual_out"], st["y"], gate=st["gate"],
                                post_weight=st["post_weight"], pre_weight=st["pre_weight"])
    return _present(*grads)


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "route":
        return list(_plain_route(case, state["logits"], state["bias"]))
    if case["op"] == "route_backward":
        return [_plain_route_backward(case, state)]
    if case["op"] == "norm":
        r, h = _plain_norm(case, state)
        dt = state["y"].dtype
        return _present(r.to(state["residual"].dtype), None if h is None else h.to(dt))
    return _plain_norm_backward(case, state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    T = case["T"]
    if case["op"].startswith("route"):
        E, K, b = case["E"], case["K"], _BYTES[case["dtype"]]
        if case["op"] == "route":
            return {"bytes": T * E * b + T * K * 8 + (E * 4 if case["bias"] else 0), "flops": T * E * 6}
        # the gradient of a sigmoid reads the chosen logits only
        read = T * K * b if case["score"] == "sigmoid" else T * E * b
        return {"bytes": read + T * E * b + T * K * 12, "flops": T * (E * 6 if case["score"] == "softmax" else K * 10)}
    H, b = case["H"], _BYTES[case["dtype"]]
    rb = 4 if case["residual"] == "f32" else b
    wb = 4 if case["weights"] == "f32" else b
    n = T * H
    gate = {"none": 0, "channel": H * b, "token": T * b, "full": n * b}[case["gate"]]
    vectors = H * wb * (case["post"] + case["pre"])
    if case["op"] == "norm":
        return {"bytes": n * (b + 2 * rb + (b if case["pre"] else 0)) + gate + vectors, "flops": n * 12}
    dgate = {"none": 0, "channel": H * 4, "token": T * b, "full": n * b}[case["gate"]]
    grads = H * 4 * (case["post"] + case["pre"])
    # read: y, the residual's gradient and, with a pre-norm, its rows and the
    # gradient of h; written: the gradients of the residual and of y
    moved = n * (b + rb + (rb + b if case["pre"] else 0)) + n * (rb + b)
    return {"bytes": moved + gate + dgate + vectors + grads, "flops": n * 30}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_choice(case, logits, bias):
    """What experts are chosen by (closed ones at -inf), and which are open."""
    l = logits.double()
    open_ = l != -math.inf
    if not _by_score(case):
        return l, open_
    v = _exact_score(case, l)
    return (v if bias is None else v + bias.double()).masked_fill(~open_, -math.inf), open_


def _exact_score(case, l):
    if case["score"] == "sigmoid":
        return torch.sigmoid(l)
    return torch.nan_to_num(torch.softmax(l, dim=1), nan=0.0)  # (a row with nothing open)


def _exact_group_scores(case, choice):
    c = choice.view(choice.shape[0], case["groups"], -1)
    n = 2 if case["group_score"] == "top2" else 1
    best = c.sort(dim=2, descending=True).values[:, :, :n]
    empty = best[:, :, 0] == -math.inf
    total = torch.where(best == -math.inf, torch.zeros_like(best), best).sum(dim=2)
    return total.masked_fill(empty, -math.inf)


def _exact_group_limit(case, choice, open_):
    T, G = choice.shape[0], case["groups"]
    order = _exact_group_scores(case, choice).sort(dim=1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, torch.arange(G, device=order.device).expand(T, G).contiguous())
    keep = (rank < case["top_groups"])[:, :, None].expand(T, G, choice.shape[1] // G).reshape(T, -1)
    open_ = open_ & keep
    return choice.masked_fill(~open_, -math.inf), open_


def _exact_route(case, st):
    choice, open_ = _exact_choice(case, st["logits"], st["bias"])
    if case["groups"] > 1:
        choice, open_ = _exact_group_limit(case, choice, open_)
    ids = choice.sort(dim=1, descending=True, stable=True).indices[:, :case["K"]]
    s = _exact_score(case, st["logits"].double())
    w = (s * open_).gather(1, ids)
    if case["renorm"]:
        w = w / (w.sum(dim=1, keepdim=True) + _EPS_SUM)
    return [ids.int(), w * case["scale"]]


def _exact_route_backward(case, st):
    l = st["logits"].double().requires_grad_()
    s = torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1)
    w = s.gather(1, st["ids"].long()) * (st["weights"] != 0)
    if case["renorm"]:
        w = w / (w.sum(dim=1, keepdim=True) + _EPS_SUM)
    loss = (w * st["dweights"].double()).sum() * case["scale"]
    (dl,) = torch.autograd.grad(loss, l)
    if case["score"] == "softmax":  # a row with nothing open has no gradient
        dl = dl.masked_fill((st["logits"] == -math.inf).all(dim=1, keepdim=True), 0.0)
    return [dl]


def _exact_normed(case, x, w):
    mean = x.mean(dim=1, keepdim=True) if case["kind"] == "layer" else 0.0
    return (x - mean) * torch.rsqrt((x - mean).square().mean(dim=1, keepdim=True) + case["eps"]) * (case["offset"] + w)


def _exact_branch(case, y, gate, w):
    b = _exact_normed(case, y, w) if case["post"] else y
    if gate is not None:
        b = b * (torch.sigmoid(gate) if case["gate_sigmoid"] else gate)
    return b * case["scale"]


def _double(t):
    return None if t is None else t.double()


def _exact_norm(case, st):
    r = st["residual"].double() + _exact_branch(case, st["y"].double(), _double(st["gate"]), _double(st["post_weight"]))
    return _present(r, _exact_normed(case, r, st["pre_weight"].double()) if case["pre"] else None)


def _exact_norm_backward(case, st):
    dr = st["dresidual_out"].double()
    dpre = None
    if case["pre"]:
        x, w = st["residual_out"].double().requires_grad_(), st["pre_weight"].double().requires_grad_()
        dx, dpre = torch.autograd.grad(_exact_normed(case, x, w), (x, w), st["dh"].double())
        dr = dr + dx
        del x, dx
    leaves = {"y": st["y"].double().requires_grad_()}
    if st["gate"] is not None:
        leaves["gate"] = st["gate"].double().requires_grad_()
    if case["post"]:
        leaves["w"] = st["post_weight"].double().requires_grad_()
    b = _exact_branch(case, leaves["y"], leaves.get("gate"), leaves.get("w"))
    grads = dict(zip(leaves, torch.autograd.grad(b, tuple(leaves.values()), dr)))
    return _present(dr, grads["y"], grads.get("gate"), grads.get("w"), dpre)


def exact(case, seed):
    st = _inputs(case, seed)
    return {"route": _exact_route, "route_backward": _exact_route_backward, "norm": _exact_norm,
            "norm_backward": _exact_norm_backward}[case["op"]](case, st)
