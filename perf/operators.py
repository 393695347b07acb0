"""Cases of the 4-bit expert operators, with their plain forms.

Operators: projections with integer 4-bit weights and group scales (`w4g_proj`), the same product grouped by
expert with ragged sizes (`w4g_proj_grouped`), the router that makes the groups (`moe_route`), the weighted sum of
the experts' rows (`moe_combine`), and the expert MLP that runs them together (`w4g_moe_mlp`).
"""
import math

import torch

own = False

DEV = "cuda"


def _dense(name, m, n, k, group, zero=False, half=False):
    return {"name": name, "op": "dense", "m": m, "n": n, "k": k, "group": group, "zero": zero, "half": half}


def _grouped(name, tokens, topk, experts, n, k, group, zero=False, half=False, skew=0.0):
    return {"name": name, "op": "grouped", "tokens": tokens, "topk": topk, "experts": experts, "n": n, "k": k,
            "group": group, "zero": zero, "half": half, "skew": skew}


def _route(name, tokens, experts, topk, bf16, renorm, pad=0):
    return {"name": name, "op": "route", "tokens": tokens, "experts": experts, "topk": topk, "bf16": bf16,
            "renorm": renorm, "pad": pad}


def _combine(name, tokens, topk, n, residual, drop=False):
    return {"name": name, "op": "combine", "tokens": tokens, "topk": topk, "n": n, "residual": residual,
            "drop": drop}


def _mlp(name, tokens, topk, experts, inner, k, group, skew=0.0):
    return {"name": name, "op": "mlp", "tokens": tokens, "topk": topk, "experts": experts, "inner": inner, "k": k,
            "group": group, "skew": skew}


def listed():
    return [
        # one token through an attention-sized projection: the latency of a decode step
        _dense("dense_decode_1", 1, 4096, 4096, 128),
        # a few tokens (speculative decode) through the up projection, zero points, an odd number of rows
        _dense("dense_decode_5_zero", 5, 14333, 4096, 64, zero=True, half=True),
        # a prompt through the up projection
        _dense("dense_prefill_2048", 2048, 14336, 4096, 128),
        # one token's eight experts
        _grouped("grouped_decode_1x8", 1, 8, 64, 2048, 2048, 128),
        # a decode batch: a few rows for each of many experts
        _grouped("grouped_batch_48x8", 48, 8, 128, 1536, 2048, 64, zero=True),
        # a prompt over many small experts, ragged, with popular and nearly idle experts
        _grouped("grouped_prefill_4099x6", 4099, 6, 64, 1408, 2048, 32, half=True, skew=2.0),
        # the router for one decode batch, and for a padded batch of prompts
        _route("route_decode_33", 33, 64, 8, False, True),
        _route("route_prefill_16384", 16384, 128, 8, True, False, pad=1000),
        # the weighted sum for a decode batch, and for prompts with a residual and dropped pairs
        _combine("combine_decode_16", 16, 8, 2048, False),
        _combine("combine_prefill_8192", 8192, 8, 2048, True, drop=True),
        # the whole expert MLP: a decode batch of four, and a prompt through eight large experts
        _mlp("mlp_decode_4", 4, 2, 8, 14336, 4096, 128),
        _mlp("mlp_prefill_4096", 4096, 2, 8, 14336, 4096, 128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["dense", "dense", "grouped", "grouped", "route", "combine", "mlp"])
    group = rng.choice([32, 64, 128])
    zero, half = rng.random() < 0.5, rng.random() < 0.5
    if op == "dense":
        m = _log(rng, 1, 16) if rng.random() < 0.5 else _log(rng, 17, 2048)
        case = _dense("", m, _log(rng, 256, 14336), group * _log(rng, 512 // group, 14336 // group), group, zero, half)
    elif op == "grouped":
        experts = rng.randint(3, 128)
        tokens = _log(rng, 1, 64) if rng.random() < 0.5 else _log(rng, 65, 4096)
        case = _grouped("", tokens, rng.randint(1, min(8, experts)), experts, _log(rng, 128, 2048),
                        group * _log(rng, 256 // group, 2048 // group), group, zero, half,
                        rng.choice([0.0, 0.0, 2.0]))
    elif op == "route":
        experts = rng.randint(2, 384)
        tokens = _log(rng, 1, 16384)
        case = _route("", tokens, experts, rng.randint(1, min(8, experts)), rng.random() < 0.5, rng.random() < 0.5,
                      rng.choice([0, tokens // 5]))
    elif op == "combine":
        case = _combine("", _log(rng, 1, 8192), rng.randint(1, 8), _log(rng, 129, 4096), rng.random() < 0.5,
                        rng.random() < 0.5)
    else:
        experts = rng.randint(2, 32)
        case = _mlp("", _log(rng, 1, 1024), rng.randint(1, min(8, experts)), experts,
                    group * _log(rng, 256 // group, 2048 // group), group * _log(rng, 256 // group, 2048 // group),
                    group, rng.choice([0.0, 2.0]))
    case.pop("name")
    return case


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _weight(gen, lead, n, k, group, zero, half):
    shape = lead + (n, k // group)
    codes = torch.randint(0, 256, lead + (n, k // 2), dtype=torch.uint8, device=DEV, generator=gen)
    scale = (torch.rand(shape, device=DEV, generator=gen) + 0.5) * (0.3 / math.sqrt(k))
    zeros = torch.randint(4, 13, shape, dtype=torch.uint8, device=DEV, generator=gen) if zero else None
    return codes, scale.to(torch.float16 if half else torch.bfloat16), zeros


def _acts(gen, rows, k):
    # one channel in a hundred is an outlier channel
    a = torch.randn(rows, k, device=DEV, generator=gen)
    loud = torch.rand(k, device=DEV, generator=gen) < 0.01
    return (a * torch.where(loud, 20.0, 1.0)).bfloat16()


def _logits(gen, tokens, experts, skew):
    x = torch.randn(tokens, experts, device=DEV, generator=gen)
    return x + skew * torch.randn(experts, device=DEV, generator=gen)


def prepare(case, seed):
    gen = _generator(seed)
    op = case["op"]
    if op == "dense":
        weight = _weight(gen, (), case["n"], case["k"], case["group"], case["zero"], case["half"])
        return {"op": op, "a": _acts(gen, case["m"], case["k"]), "weight": weight}
    if op == "route":
        logits = _logits(gen, case["tokens"], case["experts"], 0.5)
        if case["pad"]:  # padding tokens choose no expert
            logits[case["tokens"] - case["pad"]:] = -math.inf
        return {"op": op, "logits": logits.bfloat16() if case["bf16"] else logits, "topk": case["topk"],
                "renorm": case["renorm"]}
    if op == "combine":
        tokens, topk, n = case["tokens"], case["topk"], case["n"]
        pairs = tokens * topk
        pos = torch.randperm(pairs, device=DEV, generator=gen).to(torch.int32).reshape(tokens, topk)
        weights = torch.rand(tokens, topk, device=DEV, generator=gen) + 0.05
        weights = weights / weights.sum(1, keepdim=True)
        if case["drop"]:
            lost = torch.rand(tokens, topk, device=DEV, generator=gen) < 0.1
            pos, weights = torch.where(lost, -1, pos), torch.where(lost, 0.0, weights)
        y = torch.randn(pairs, n, device=DEV, generator=gen).bfloat16()
        residual = torch.randn(tokens, n, device=DEV, generator=gen).bfloat16() if case["residual"] else None
        return {"op": op, "y": y, "pos": pos, "weights": weights, "residual": residual}
    logits = _logits(gen, case["tokens"], case["experts"], case["skew"])
    ids, _, offsets, rows, _ = _plain_route(logits, case["topk"], True)
    capacity = int((offsets[1:] - offsets[:-1]).max())  # the most rows of one expert
    x = _acts(gen, case["tokens"], case["k"])
    if op == "grouped":
        weight = _weight(gen, (case["experts"],), case["n"], case["k"], case["group"], case["zero"], case["half"])
        return {"op": op, "a": x, "weight": weight, "offsets": offsets, "rows": rows, "capacity": capacity}
    up = [_weight(gen, (case["experts"],), case["inner"], case["k"], case["group"], False, False) for _ in range(2)]
    down = _weight(gen, (case["experts"],), case["k"], case["inner"], case["group"], False, False)
    return {"op": op, "x": x, "logits": logits, "gate": up[0], "up": up[1], "down": down, "topk": case["topk"],
            "capacity": capacity}


def _values(weight):
    """The weight's values (q - z) * s in 32 bits."""
    codes, scale, zeros = weight
    q = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).float()
    q = q.unflatten(-1, (scale.shape[-1], -1))
    z = 8.0 if zeros is None else zeros.float().unsqueeze(-1)
    return ((q - z) * scale.float().unsqueeze(-1)).flatten(-2)


def _plain_route(logits, topk, renorm):
    x = logits.float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    experts = x.shape[1]
    ordered, index = torch.sort(x, dim=1, descending=True, stable=True)
    chosen, ids = ordered[:, :topk], index[:, :topk]
    none = chosen == -math.inf
    ids = torch.where(none, -1, ids)
    top = torch.where(ordered[:, :1] == -math.inf, 0.0, ordered[:, :1])
    p = torch.exp(chosen - top)
    total = (p if renorm else torch.exp(x - top)).sum(1, keepdim=True)
    weights = torch.where(none, 0.0, p / torch.where(total > 0, total, 1.0))
    key = torch.where(ids < 0, experts, ids).reshape(-1)
    key, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=key.device))
    rows = torch.where(key < experts, order // topk, -1)
    pos = torch.empty_like(order)
    pos[order] = torch.arange(order.numel(), device=order.device)
    pos = torch.where(ids < 0, -1, pos.reshape(ids.shape))
    return ids.int(), weights, offsets.int(), rows.int(), pos.int()


def _plain_grouped(a, offsets, rows, weight, capacity):
    """All experts in one batched product over rows padded to the largest group."""
    experts = offsets.numel() - 1
    row = torch.arange(rows.numel(), device=rows.device)
    expert = torch.searchsorted(offsets[1:], row, right=True).clamp(max=experts - 1)
    place = expert * capacity + row - offsets[expert]
    padded = torch.zeros(experts * capacity, a.shape[1], device=a.device)
    padded[place] = a.float()[rows.long()]
    out = torch.bmm(padded.unflatten(0, (experts, capacity)), _values(weight).transpose(1, 2))
    return out.flatten(0, 1)[place].bfloat16()


def _plain_combine(y, pos, weights, residual):
    terms = y[pos.clamp(min=0).long()].float() * torch.where(pos < 0, 0.0, weights).unsqueeze(-1)
    out = terms.sum(1)
    return (out if residual is None else out + residual.float()).bfloat16()


def run(state):
    op = state["op"]
    if own:
        import block_scaled_precision_requant_b200 as bsr

        if op == "dense":
            return bsr.w4g_proj(state["a"], *state["weight"])
        if op == "grouped":
            return bsr.w4g_proj_grouped(state["a"], state["offsets"], *state["weight"], rows=state["rows"])
        if op == "route":
            return tuple(bsr.moe_route(state["logits"], state["topk"], renormalize=state["renorm"]))
        if op == "combine":
            return bsr.moe_combine(state["y"], state["pos"], state["weights"], residual=state["residual"])
        return bsr.w4g_moe_mlp(state["x"], state["logits"], state["gate"], state["up"], state["down"],
                               state["topk"])
    if op == "dense":
        return (state["a"].float() @ _values(state["weight"]).T).bfloat16()
    if op == "grouped":
        return _plain_grouped(state["a"], state["offsets"], state["rows"], state["weight"], state["capacity"])
    if op == "route":
        return _plain_route(state["logits"], state["topk"], state["renorm"])
    if op == "combine":
        return _plain_combine(state["y"], state["pos"], state["weights"], state["residual"])
    # the tensors between the operators are BF16
    _, weights, offsets, rows, pos = _plain_route(state["logits"], state["topk"], True)
    gate = _plain_grouped(state["x"], offsets, rows, state["gate"], state["capacity"]).float()
    up = _plain_grouped(state["x"], offsets, rows, state["up"], state["capacity"]).float()
    hidden = (gate / (1 + torch.exp(-gate)) * up).bfloat16()
    every = torch.arange(rows.numel(), device=rows.device)
    y = _plain_grouped(hidden, offsets, every, state["down"], state["capacity"])
    return _plain_combine(y, pos, weights, None)


def _weight_bytes(case, n, k):
    return n * k // 2 + n * (k // case["group"]) * (3 if case.get("zero") else 2)


def work(case):
    op = case["op"]
    if op == "dense":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": _weight_bytes(case, n, k) + 2 * m * (n + k), "flops": 2 * m * n * k}
    if op == "route":
        t, k = case["tokens"], case["topk"]
        return {"bytes": t * case["experts"] * (2 if case["bf16"] else 4) + t * k * 16 + 4 * case["experts"] + 4,
                "flops": 3 * t * case["experts"]}
    t, topk = case["tokens"], case["topk"]
    if op == "combine":
        n = case["n"]
        kept = 0.9 if case["drop"] else 1.0
        return {"bytes": int(kept * t * topk) * n * 2 + (4 if case["residual"] else 2) * t * n + 8 * t * topk,
                "flops": 2 * int(kept * t * topk) * n}
    # experts that any of the tokens chooses, for choices without preference
    used = case["experts"] * (1 - (1 - topk / case["experts"]) ** t)
    if op == "grouped":
        n, k = case["n"], case["k"]
        return {"bytes": int(used * _weight_bytes(case, n, k)) + 2 * t * k + 2 * t * topk * n + 4 * t * topk,
                "flops": 2 * t * topk * n * k}
    n, k = case["inner"], case["k"]
    return {"bytes": int(used * (2 * _weight_bytes(case, n, k) + _weight_bytes(case, k, n))) + 4 * t * k
            + 4 * t * case["experts"], "flops": 6 * t * topk * n * k}


def _exact_weight(weight, e=None):
    codes, scale, zeros = [None if t is None else (t if e is None else t[e]) for t in weight]
    n, half_k = codes.shape
    value = torch.empty(n, 2 * half_k, dtype=torch.float64, device=codes.device)
    value[:, 0::2] = (codes & 15).double()
    value[:, 1::2] = (codes >> 4).double()
    size = 2 * half_k // scale.shape[1]
    value -= 8.0 if zeros is None else zeros.double().repeat_interleave(size, dim=1)
    value *= scale.double().repeat_interleave(size, dim=1)
    return value


def _exact_groups(logits, topk):
    """(expert, score) of every pair, by repeated search for the first largest score."""
    x = logits.double().clone()
    x[torch.isnan(x)] = -math.inf
    index = torch.arange(x.shape[1], device=x.device)
    ids, scores = [], []
    for _ in range(topk):
        best = x.amax(1, keepdim=True)
        first = torch.where(x == best, index, x.shape[1]).amin(1, keepdim=True)
        scores.append(best)
        ids.append(torch.where(best == -math.inf, -1, first))
        x.scatter_(1, first, -math.inf)
    return torch.cat(ids, 1), torch.cat(scores, 1)


def _exact_route(logits, topk, renorm):
    ids, scores = _exact_groups(logits, topk)
    x = logits.double()
    x = torch.where(torch.isnan(x), -math.inf, x)
    weights = torch.softmax(scores, 1) if renorm else torch.exp(scores - torch.logsumexp(x, 1, keepdim=True))
    weights = torch.where(ids < 0, 0.0, weights)
    flat = ids.reshape(-1)
    experts = logits.shape[1]
    pos = torch.full_like(flat, -1)
    rows = torch.full_like(flat, -1)
    offsets = [0]
    for e in range(experts):
        pairs = (flat == e).nonzero().squeeze(1)
        start, stop = offsets[-1], offsets[-1] + pairs.numel()
        pos[pairs] = torch.arange(start, stop, device=flat.device)
        rows[start:stop] = pairs // topk
        offsets.append(stop)
    return ids, weights, torch.tensor(offsets, device=flat.device), rows, pos.reshape(ids.shape)


def _exact_product(a, offsets, weight):
    bounds = offsets.tolist()
    out = torch.zeros(a.shape[0], weight[0].shape[1], dtype=torch.float64, device=a.device)
    for e in range(len(bounds) - 1):
        if bounds[e + 1] > bounds[e]:
            out[bounds[e]:bounds[e + 1]] = a[bounds[e]:bounds[e + 1]] @ _exact_weight(weight, e).T
    return out


def _exact_sum(y, pos, weights, residual):
    out = torch.zeros(pos.shape[0], y.shape[1], dtype=torch.float64, device=y.device)
    for j in range(pos.shape[1]):
        kept = (pos[:, j] >= 0).nonzero().squeeze(1)
        out[kept] += weights[kept, j].double().unsqueeze(1) * y[pos[kept, j].long()].double()
    return out if residual is None else out + residual.double()


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "dense":
        return state["a"].double() @ _exact_weight(state["weight"]).T
    if op == "route":
        ids, weights, offsets, rows, pos = _exact_route(state["logits"], state["topk"], state["renorm"])
        return ids.int(), weights, offsets.int(), rows.int(), pos.int()
    if op == "combine":
        return _exact_sum(state["y"], state["pos"], state["weights"], state["residual"])
    if op == "grouped":
        return _exact_product(state["a"].double()[state["rows"].long()], state["offsets"], state["weight"])
    ids, weights, offsets, rows, pos = _exact_route(state["logits"], state["topk"], True)
    a = state["x"].double()[rows.clamp(min=0)]
    gate = _exact_product(a, offsets, state["gate"])
    up = _exact_product(a, offsets, state["up"])
    y = _exact_product(gate * torch.sigmoid(gate) * up, offsets, state["down"])
    return _exact_sum(y, pos, weights, None)
