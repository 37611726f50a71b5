"""Workloads of training and serving around quantized experts: the balance loss
of the expert choice with its counts and gradient, the global gradient norm and
clipping over many tensors, and low-rank adapters of many requests beside a
shared projection with their gradients.

``run`` computes them with elementary torch operations in 32 bits, or, with
``own`` set, with the library's ``ExpertRouter``, ``GradientClip`` and
``LowRankAdapters``.  ``exact`` evaluates the definitions in 64 bits.
"""

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f16": 2, "f32": 4}
_EPS_SUM = 1e-20   # added to the sum of a token's sigmoid scores
_EPS_NORM = 1e-6   # added to the norm that a clipping divides by

# Largest listed sizes; drawn cases stay within their cost.
_MAX_LOGITS = 131072 * 256
_MAX_GRADIENTS = 400_000_000
_MAX_ADAPTED = 16384 * (4096 + 4096)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _balance(name, T, E, K, score="softmax", sequences=0, mask=0.0, closed=0.0, tail=0, dtype="f32", pad=0, add=False,
             coefficient=0.01, kind="loss"):
    # kind: the loss, its gradient alone, or a training step's both
    return {"name": name, "op": {"loss": "balance", "gradient": "balance_backward", "step": "balance_step"}[kind], "T": T, "E": E, "K": K, "score": score,
            "sequences": sequences, "mask": mask, "closed": closed, "tail": tail, "dtype": dtype, "pad": pad,
            "add": add, "coefficient": coefficient}


def _clip(name, layers, hidden, experts, rank, blocks, dtype="bf16", limit=0.1, in_place=False, norm_only=False):
    return {"name": name, "op": "clip", "layers": layers, "hidden": hidden, "experts": experts, "rank": rank,
            "blocks": blocks, "dtype": dtype, "limit": limit, "in_place": in_place, "norm_only": norm_only}


def _adapt(name, T, inp, out, rank, adapters, requests, dtype="bf16", none=0.1, base=True, scales=True, pad=0,
           backward=False):
    return {"name": name, "op": "adapt_backward" if backward else "adapt", "T": T, "in": inp, "out": out,
            "rank": rank, "adapters": adapters, "requests": requests, "dtype": dtype, "none": none, "base": base,
            "scales": scales, "pad": pad}


def listed():
    return [
        # A small odd micro-batch of a model of 97 experts: latency only.
        _balance("balance_micro", 257, 97, 5, "sigmoid", pad=3),
        # A training batch of 41 ragged sequences, balanced one by one, with
        # padding tokens inside and behind them; 160 experts, bf16 logits: the
        # loss and its gradient.
        _balance("balance_sequences", 32768, 160, 6, "softmax", sequences=41, mask=0.03, closed=0.02, tail=219,
                 dtype="bf16", kind="step"),
        # The largest training batch: 131072 tokens, 256 experts, one balance.
        _balance("balance_train", 131072, 256, 8, "sigmoid", kind="step"),
        # A gradient alone, added to the gradient that the choice passes back.
        _balance("balance_grad_train", 131072, 256, 8, "softmax", add=True, kind="gradient"),
        # The routers, norms and small adapters of two layers, as tensors of
        # one to some thousand elements: latency and the list's handling.
        _clip("clip_small", 2, 512, 32, 4, 0, limit=0.02),
        # A stack whose norms and routers are FP32, with odd widths and some
        # gradients of zero, not clipped: most steps of a stable run.
        _clip("clip_quiet_odd", 36, 2047, 97, 16, 0, dtype="mixed", limit=6.0, in_place=True),
        # The largest set: dense blocks of 4096 x 4096 beside the rest, clipped.
        _clip("clip_large", 16, 4096, 64, 16, 22),
        # One decode step of 64 requests on 16 adapters of rank 16.
        _adapt("adapters_decode", 64, 2048, 2048, 16, 16, 64),
        # A ragged prefill of 13 requests: FP16, rank 24, outputs of another
        # width, rows of a wider buffer.
        _adapt("adapters_prefill_odd", 4073, 2048, 1536, 24, 8, 13, dtype="f16", pad=8),
        # The largest prefill: 16384 tokens of 32 requests, rank 64.
        _adapt("adapters_prefill", 16384, 4096, 4096, 64, 8, 32),
        # Gradients: a small batch with an odd width (no vector loads line
        # up) and the largest, 16384 tokens on four adapters of rank 32.
        _adapt("adapters_grad_odd", 777, 1001, 520, 8, 5, 9, dtype="f16", backward=True),
        _adapt("adapters_grad_train", 16384, 4096, 4096, 32, 4, 16, none=0.0, backward=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["balance", "clip", "adapt"])
    backward = rng.random() < 0.4
    if kind == "balance":
        E = _log_int(rng, 8, 512)
        if rng.random() < 0.5:
            E = max(8, E // 8 * 8)
        K = rng.randint(1, min(16, E))
        T = max(1, min(_log_int(rng, 1, 131072), _MAX_LOGITS // E))
        sequences = rng.choice([0, 0, 1, _log_int(rng, 1, 200)])
        return _balance(None, T, E, K, rng.choice(["softmax", "sigmoid"]), sequences, rng.choice([0.0, 0.05]),
                        rng.choice([0.0, 0.05]), rng.choice([0, T // 50]) if sequences else 0,
                        rng.choice(["f32", "bf16", "f16"]), rng.choice([0, 0, 3, 8]),
                        rng.random() < 0.5, rng.choice([0.01, 1.0]), rng.choice(["loss", "step", "gradient"]))
    if kind == "clip":
        hidden = _log_int(rng, 64, 4096)
        if rng.random() < 0.6:
            hidden = max(64, hidden // 64 * 64)
        layers = _log_int(rng, 1, 48)
        experts, rank = _log_int(rng, 8, 256), rng.choice([4, 8, 13, 16, 32])
        rest = layers * hidden * (experts + 2 * rank + 2)
        blocks = rng.randint(0, 24)
        blocks = max(0, min(blocks, (_MAX_GRADIENTS // 2 - rest) // (hidden * hidden)))
        return _clip(None, layers, hidden, experts, rank, blocks, rng.choice(["bf16", "f16", "f32", "mixed"]),
                     rng.choice([0.02, 0.1, 6.0]), False, rng.random() < 0.3)
    inp, out = _log_int(rng, 64, 4096), _log_int(rng, 64, 4096)
    if rng.random() < 0.7:
        inp, out = max(64, inp // 64 * 64), max(64, out // 64 * 64)
    rank = rng.choice([4, 8, 13, 16, 24, 32, 64, 128])
    T = _log_int(rng, 1, 16384)
    T = max(1, min(T, _MAX_ADAPTED // (inp + out) * 32 // max(32, rank)))
    adapters = max(1, min(_log_int(rng, 1, 64), 512 // rank))
    requests = rng.choice([min(T, 64), min(T, 9), T if T <= 256 else 33])
    return _adapt(None, T, inp, out, rank, adapters, requests, rng.choice(["bf16", "bf16", "f16"]),
                  rng.choice([0.0, 0.1, 0.5]), rng.random() < 0.7, rng.random() < 0.7, rng.choice([0, 0, 1, 8]), backward)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _rand(g, *shape):
    return torch.rand(*shape, generator=g, device="cuda")


def _padded(t, pad):
    """The same values in rows `pad` elements longer than they need be."""
    if not pad:
        return t
    wide = torch.zeros(t.shape[0], t.shape[1] + pad, dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _cuts(g, total, parts):
    """Bounds of `parts` ragged runs of `total` items (some may be empty)."""
    inner = (_rand(g, parts - 1) * (total + 1)).floor().clamp(max=total).sort().values
    ends = torch.tensor([0.0], device="cuda"), torch.tensor([float(total)], device="cuda")
    return torch.cat([ends[0], inner, ends[1]]).int()


def _balance_inputs(case, seed):
    g = _gen(seed)
    T, E, K = case["T"], case["E"], case["K"]
    # logits of a router whose experts differ in popularity, each token with
    # a sharpness of its own; some experts closed to some tokens
    logits = _randn(g, T, E) * (0.5 + 1.5 * _rand(g, T, 1)) + 0.5 * _randn(g, E)
    if case["closed"]:
        logits = logits.masked_fill(_rand(g, T, E) < case["closed"], -math.inf)
        logits = logits.masked_fill(_rand(g, T, 1) < 1.0 / 1024, -math.inf)  # tokens with nothing open
    ids = logits.topk(K, dim=1).indices.int()
    st = {"logits": _padded(logits.to(_TYPES[case["dtype"]]), case["pad"]), "ids": ids, "offsets": None, "mask": None}
    if case["sequences"]:
        st["offsets"] = _cuts(g, T - case["tail"], case["sequences"])
    if case["mask"]:
        st["mask"] = _rand(g, T) >= case["mask"]
    if case["op"] != "balance":
        if case["op"] == "balance_backward":
            st["slope"] = _plain_balance(case, st)[2]
        st["dloss"] = 0.5 + _rand(g, 1)[0]
        st["add"] = None
        if case["add"]:  # the gradient of the choice reaches the chosen experts
            passed = torch.zeros(T, E, device="cuda").scatter_(1, ids.long(), _randn(g, T, K) * 1e-3)
            st["add"] = _padded(passed.to(_TYPES[case["dtype"]]), case["pad"])
    return st


def _clip_shapes(case):
    H, E, r = case["hidden"], case["experts"], case["rank"]
    small = "f32" if case["dtype"] == "mixed" else case["dtype"]
    large = "bf16" if case["dtype"] == "mixed" else case["dtype"]
    layer = [((H,), small), ((H,), small), ((E, H), small), ((E,), small), ((4, r, H), large), ((4, r, H), large)]
    return layer * case["layers"] + [((H, H), large)] * case["blocks"]


def _clip_inputs(case, seed):
    g = _gen(seed)
    # each type's gradients lie in one buffer, as a trainer's buckets hold them
    flat = _clip_buffers(case)
    grads = _clip_views(case, flat)
    for t in grads:
        # tensors differ in size by orders of magnitude; a few got no token
        size = torch.exp(_rand(g, 1) * 6.0 - 9.0) * (_rand(g, 1) >= 0.04)
        t.copy_(_randn(g, *t.shape) * size)
    # the limit is a multiple of the norm that such gradients have
    expected = math.sqrt(sum(t.numel() for t in grads) * 0.96 * (math.exp(-6.0) - math.exp(-18.0)) / 12.0)
    return {"flat": flat, "grads": grads, "max_norm": case["limit"] * expected}


def _clip_buffers(case):
    sizes = {}
    for shape, dtype in _clip_shapes(case):
        sizes[dtype] = sizes.get(dtype, 0) + math.prod(shape)
    return {dtype: torch.empty(n, dtype=_TYPES[dtype], device="cuda") for dtype, n in sizes.items()}


def _clip_views(case, flat):
    views, at = [], dict.fromkeys(flat, 0)
    for shape, dtype in _clip_shapes(case):
        n = math.prod(shape)
        views.append(flat[dtype][at[dtype]:at[dtype] + n].view(shape))
        at[dtype] += n
    return views


def _adapt_inputs(case, seed):
    g = _gen(seed)
    T, K, N, r, L = case["T"], case["in"], case["out"], case["rank"], case["adapters"]
    dt = _TYPES[case["dtype"]]
    # requests hold runs of tokens, each request an adapter or none; one token
    # a request in a decode step
    which = torch.randint(0, L, (case["requests"],), generator=g, device="cuda")
    which = which.masked_fill(_rand(g, case["requests"]) < case["none"], -1)
    if case["requests"] == T:
        ids = which
    else:
        cuts = _cuts(g, T, case["requests"])
        ids = which[torch.searchsorted(cuts[1:-1].contiguous(), torch.arange(T, device="cuda", dtype=torch.int32),
                                       right=True)]
    size = torch.exp(_rand(g, T, 1) * 2.0 - 1.0)
    st = {"ids": ids.int().contiguous(), "x": _padded((_randn(g, T, K) * size).to(dt), case["pad"]),
          "down": (_randn(g, L, r, K) / math.sqrt(K)).to(dt), "up": (_randn(g, L, r, N) * 0.3 / math.sqrt(r)).to(dt)}
    st["scales"] = 0.5 + 1.5 * _rand(g, L) if case["scales"] else None
    width = K if case["op"] == "adapt_backward" else N
    st["base"] = _padded(_randn(g, T, width).to(dt), case["pad"]) if case["base"] else None
    if case["op"] == "adapt_backward":
        st["dout"] = _padded((_randn(g, T, N) * 0.1).to(dt), case["pad"])
        st["hidden"] = _plain_hidden(st["x"], st["ids"], st["down"], st["scales"]).sum(dim=1)
    return st


def _inputs(case, seed):
    if case["op"].startswith("balance"):
        return _balance_inputs(case, seed)
    return _clip_inputs(case, seed) if case["op"] == "clip" else _adapt_inputs(case, seed)


def prepare(case, seed):
    state = _inputs(case, seed)
    state["case"] = case
    if case["op"] == "clip" and not case["in_place"] and not case["norm_only"]:
        state["into"] = _clip_buffers(case)  # (the gradients stay as they are)
        state["clipped"] = _clip_views(case, state["into"])
    if own:
        import nvfp4_token_quantized_gb300 as lib

        if case["op"].startswith("balance"):
            state["router"] = lib.ExpertRouter(case["E"], case["K"], score=case["score"])
        elif case["op"] == "clip":
            state["clip"] = lib.GradientClip(state["max_norm"], eps=_EPS_NORM)
        else:
            state["adapters"] = lib.LowRankAdapters(case["in"], case["out"], case["rank"])
    return state


# ---------------------------------------------------------------------------
# plain forms, 32 bits
# ---------------------------------------------------------------------------

def _plain_scores(case, logits):
    """A token's scores as shares of one, and (sigmoid) their raw values and
    their sum."""
    l = logits.float()
    if case["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
        total = s.sum(dim=1, keepdim=True) + _EPS_SUM
        return s / total, s, total
    m = l.amax(dim=1, keepdim=True)
    e = torch.exp(l - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = e.sum(dim=1, keepdim=True)
    return e / torch.where(total == 0, torch.ones_like(total), total), None, None


def _plain_places(case, st):
    """Each token's sequence, S for one that is not counted, and S."""
    T = case["T"]
    S = max(1, case["sequences"])
    place = torch.zeros(T, dtype=torch.long, device="cuda")
    if st["offsets"] is not None:
        row = torch.arange(T, device="cuda", dtype=torch.int32)
        place = torch.searchsorted(st["offsets"][1:].contiguous(), row, right=True).clamp(max=S)
        place = place.masked_fill(row < st["offsets"][0], S)
    if st["mask"] is not None:
        place = place.masked_fill(~st["mask"], S)
    return place, S


def _plain_balance(case, st):
    E, K = case["E"], case["K"]
    place, S = _plain_places(case, st)
    p = _plain_scores(case, st["logits"])[0]
    tokens = torch.zeros(S + 1, device="cuda").index_add_(0, place, torch.ones(place.shape[0], device="cuda"))[:S]
    slots = (place[:, None] * E + st["ids"].long()).reshape(-1)
    counts = torch.zeros((S + 1) * E, dtype=torch.int32, device="cuda")
    counts = counts.index_add_(0, slots, torch.ones_like(slots, dtype=torch.int32)).view(S + 1, E)[:S]
    # (long sums: thousands of tokens an expert)
    if st["offsets"] is None:
        total = (p * (place < S)[:, None]).sum(dim=0, keepdim=True, dtype=torch.float64).float()
    else:
        total = torch.zeros(S + 1, E, dtype=torch.float64, device="cuda").index_add_(0, place, p.double())[:S].float()
    n = tokens.clamp(min=1.0)[:, None]
    used = (tokens > 0).sum().clamp(min=1)
    share = counts * (E / K) / n
    loss = case["coefficient"] * (share * (total / n)).sum() / used
    return loss, counts, case["coefficient"] * share / n / used


def _plain_balance_backward(case, st, slope):
    place, S = _plain_places(case, st)
    slope = torch.cat([slope, torch.zeros(1, case["E"], device="cuda")])[place] * st["dloss"]
    p, s, total = _plain_scores(case, st["logits"])
    d = slope - (p * slope).sum(dim=1, keepdim=True)
    d = p * d if s is None else s * (1.0 - s) * (d / total)
    d = torch.where((place < S)[:, None], d, torch.zeros_like(d))
    if st["add"] is not None:
        d = d + st["add"].float()
    return d.to(st["logits"].dtype)


def _plain_clip(case, st):
    sums = torch.stack([t.float().square().sum() for t in st["grads"]])
    norm = sums.double().sum().sqrt().float()
    if case["norm_only"]:
        return [norm]
    factor = (st["max_norm"] / (norm + _EPS_NORM)).clamp(max=1.0)
    for o, t in zip(st["grads"] if case["in_place"] else st["clipped"], st["grads"]):
        o.copy_(t.float() * factor)
    return [norm, *st["flat" if case["in_place"] else "into"].values()]


def _plain_hidden(x, ids, first, scales):
    """x through every adapter's first factor, scaled, kept where the row has
    that adapter: [T, adapters, rank]."""
    L, r, _ = first.shape
    h = (x.float() @ first.float().flatten(0, 1).t()).view(x.shape[0], L, r)
    if scales is not None:
        h = h * scales[None, :, None]
    mine = ids[:, None] == torch.arange(L, device="cuda", dtype=torch.int32)
    return torch.where(mine[:, :, None], h, torch.zeros_like(h))


def _plain_adapt(x, ids, first, second, scales, base):
    h = _plain_hidden(x, ids, first, scales)
    out = h.flatten(1) @ second.float().flatten(0, 1)
    return (out if base is None else out + base.float()).to(x.dtype), h


def _plain_adapt_backward(st):
    L, r, _ = st["down"].shape
    dx, dh = _plain_adapt(st["dout"], st["ids"], st["up"], st["down"], st["scales"], st["base"])
    mine = st["ids"][:, None] == torch.arange(L, device="cuda", dtype=torch.int32)
    h = torch.where(mine[:, :, None], st["hidden"][:, None, :], torch.zeros_like(dh))
    ddown = (dh.flatten(1).t() @ st["x"].float()).view(L, r, -1)
    dup = (h.flatten(1).t() @ st["dout"].float()).view(L, r, -1)
    return [dx, ddown.to(dx.dtype), dup.to(dx.dtype)]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def _run_own(case, st):
    if case["op"].startswith("balance"):
        outs, slope = [], st.get("slope")
        if slope is None:
            outs = list(st["router"].balance_loss(st["logits"], st["ids"], coefficient=case["coefficient"],
                                                  offsets=st["offsets"], mask=st["mask"]))
            slope = outs[2]
        if case["op"] != "balance":
            outs.append(st["router"].balance_backward(st["logits"], slope, dloss=st["dloss"], offsets=st["offsets"],
                                                      mask=st["mask"], add=st["add"]))
        return outs
    if case["op"] == "clip":
        if case["norm_only"]:
            return [st["clip"].norm(st["grads"])]
        norm, _ = st["clip"].clip(st["grads"], out=None if case["in_place"] else st["clipped"])
        return [norm, *st["flat" if case["in_place"] else "into"].values()]
    if case["op"] == "adapt":
        return [st["adapters"].forward(st["x"], st["ids"], st["down"], st["up"], scales=st["scales"],
                                       base=st["base"])[0]]
    return list(st["adapters"].backward(st["dout"], st["x"], st["hidden"], st["ids"], st["down"], st["up"],
                                        scales=st["scales"], base=st["base"]))


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    if case["op"] == "balance":
        return list(_plain_balance(case, state))
    if case["op"] == "balance_backward":
        return [_plain_balance_backward(case, state, state["slope"])]
    if case["op"] == "balance_step":
        outs = _plain_balance(case, state)
        return [*outs, _plain_balance_backward(case, state, outs[2])]
    if case["op"] == "clip":
        return _plain_clip(case, state)
    if case["op"] == "adapt":
        return [_plain_adapt(state["x"], state["ids"], state["down"], state["up"], state["scales"], state["base"])[0]]
    return _plain_adapt_backward(state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    if case["op"].startswith("balance"):
        T, E, K, b = case["T"], case["E"], case["K"], _BYTES[case["dtype"]]
        S = max(1, case["sequences"])
        around = (S + 1) * 4 * bool(case["sequences"]) + T * bool(case["mask"])
        if case["op"] == "balance":
            return {"bytes": T * E * b + T * K * 4 + S * E * 8 + 4 + around, "flops": T * E * 6}
        step = case["op"] == "balance_step"
        moved = T * E * b * (3 if case["add"] else 2) + (T * K * 4 + S * E * 8 if step else S * E * 4) + 8 + around
        return {"bytes": moved, "flops": T * E * (16 if step else 10)}
    if case["op"] == "clip":
        n = b = 0
        for shape, dtype in _clip_shapes(case):
            n += math.prod(shape)
            b += math.prod(shape) * _BYTES[dtype]
        # not clipped in place: nothing has to be written
        writes = not case["norm_only"] and not case["in_place"]
        return {"bytes": b * (2 if writes else 1) + 4, "flops": n * (3 if writes else 2)}
    T, K, N, r, b = case["T"], case["in"], case["out"], case["rank"], _BYTES[case["dtype"]]
    busy = T * (1.0 - case["none"])
    factors = min(case["adapters"], case["requests"]) * r * (K + N) * b
    if case["op"] == "adapt":
        moved = busy * K * b + T * N * b * (2 if case["base"] else 1) + T * 4
        return {"bytes": int(moved + factors), "flops": int(2 * busy * r * (K + N))}
    moved = busy * (K + N) * b + T * K * b * (2 if case["base"] else 1) + busy * r * 4 + T * 4
    written = case["adapters"] * r * (K + N) * b
    return {"bytes": int(moved + factors + written), "flops": int(4 * busy * r * (K + N))}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_shares(case, l):
    if case["score"] == "sigmoid":
        s = torch.sigmoid(l)
        return s / (s.sum(dim=1, keepdim=True) + _EPS_SUM)
    return torch.softmax(l, dim=1)


def _exact_rows(case, st):
    """The counted rows of each sequence."""
    bounds = [0, case["T"]] if st["offsets"] is None else st["offsets"].tolist()
    for lo, hi in zip(bounds, bounds[1:]):
        rows = torch.arange(lo, hi, device="cuda")
        yield rows if st["mask"] is None else rows[st["mask"][lo:hi]]


def _exact_balance(case, st):
    E, K = case["E"], case["K"]
    sequences = list(_exact_rows(case, st))
    used = max(1, sum(rows.numel() > 0 for rows in sequences))
    loss = torch.zeros((), dtype=torch.float64, device="cuda")
    counts, slope = [], []
    for rows in sequences:
        n = max(1, rows.numel())
        shares = torch.nan_to_num(_exact_shares(case, st["logits"][rows].double()), nan=0.0)
        count = torch.bincount(st["ids"][rows].reshape(-1).long(), minlength=E)
        f = count.double() * E / (K * n)
        loss = loss + (f * shares.sum(dim=0)).sum() * case["coefficient"] / (n * used)
        counts.append(count.int())
        slope.append(f * case["coefficient"] / (n * used))
    return [loss, torch.stack(counts), torch.stack(slope)]


def _exact_balance_backward(case, st, slope):
    out = torch.zeros(case["T"], case["E"], dtype=torch.float64, device="cuda")
    for s, rows in enumerate(_exact_rows(case, st)):
        l = st["logits"][rows].double().requires_grad_()
        value = (_exact_shares(case, l) * slope[s].double()).sum() * st["dloss"].double()
        (d,) = torch.autograd.grad(value, l)
        nothing = (l == -math.inf).all(dim=1, keepdim=True)
        out[rows] = d.masked_fill(nothing, 0.0)
    return [out if st["add"] is None else out + st["add"].double()]


def _exact_clip(case, st):
    norm = torch.sqrt(sum(torch.linalg.vector_norm(t.double()) ** 2 for t in st["grads"]))
    if case["norm_only"]:
        return [norm]
    factor = min(1.0, st["max_norm"] / (norm.item() + _EPS_NORM))
    return [norm] + [t.double() * factor for t in st["flat"].values()]


def _exact_adapt(st, x, first, second):
    """The rows that the adapters give, and what lies between the factors."""
    out = torch.zeros(x.shape[0], second.shape[2], dtype=torch.float64, device="cuda")
    h = torch.zeros(x.shape[0], first.shape[1], dtype=torch.float64, device="cuda")
    for a in range(first.shape[0]):
        rows = (st["ids"] == a).nonzero().squeeze(1)
        scale = 1.0 if st["scales"] is None else st["scales"][a].double()
        h[rows] = torch.einsum("tk,rk->tr", x[rows].double(), first[a].double()) * scale
        out[rows] = torch.einsum("tr,rn->tn", h[rows], second[a].double())
    return out if st["base"] is None else out + st["base"].double(), h


def _exact_adapt_backward(st):
    dx, dh = _exact_adapt(st, st["dout"], st["up"], st["down"])
    ddown = torch.zeros(st["down"].shape, dtype=torch.float64, device="cuda")
    dup = torch.zeros(st["up"].shape, dtype=torch.float64, device="cuda")
    for a in range(ddown.shape[0]):
        rows = (st["ids"] == a).nonzero().squeeze(1)
        ddown[a] = torch.einsum("tr,tk->rk", dh[rows], st["x"][rows].double())
        dup[a] = torch.einsum("tr,tn->rn", st["hidden"][rows].double(), st["dout"][rows].double())
    return [dx, ddown, dup]


def exact(case, seed):
    st = _inputs(case, seed)
    if case["op"] == "balance":
        return _exact_balance(case, st)
    if case["op"] == "balance_backward":
        return _exact_balance_backward(case, st, st["slope"])
    if case["op"] == "balance_step":
        outs = _exact_balance(case, st)
        return outs + _exact_balance_backward(case, st, outs[2])
    if case["op"] == "clip":
        return _exact_clip(case, st)
    if case["op"] == "adapt":
        return [_exact_adapt(st, st["x"], st["down"], st["up"])[0]]
    return _exact_adapt_backward(st)
