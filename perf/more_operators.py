"""Products whose weights depend on the row, as cases to be measured: routing to experts, the experts' products with their gradients, and
low-rank adapters beside a shared projection.

  "route"     scores of each token's logits (softmax or sigmoid), a bias for balance, groups of experts, the `top` largest, their gates
  "unroute"   the same, and the gradient of the logits from that of the gates
  "experts"   y[t] = sum_s gates[t][s] W2[e] (silu(W1[e][:I] x[t]) * W1[e][I:] x[t]), e = ids[t][s]
  "train"     the same, and the gradients of x, the gates and both weights
  "adapters"  y[t] = W x[t] + scales[r] B[r] (A[r] x[t]), r = ids[t], or W x[t] alone where ids[t] is -1

`own` false: the plain forms, in elementary torch operations and 32 bits (scores in 64, so that the choice next to a tie is the same).
`own` true: the package's operators.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # One token on its way through a layer of many small experts: what counts is the latency.
        {"name": "route one token", "op": "route", "t": 1, "e": 64, "top": 8, "type": "bf16", "score": "softmax", "bias": False, "groups": 1, "keep": 1,
         "by": "max", "renorm": True},
        # A long prompt, sigmoid scores balanced by a bias, four of eight groups of experts kept.
        {"name": "route prompt groups", "op": "route", "t": 16384, "e": 256, "top": 8, "type": "f32", "score": "sigmoid", "bias": True, "groups": 8, "keep": 4,
         "by": "top2", "renorm": True},
        # A training batch, softmax over all experts, an odd number of tokens and experts: the gradient reaches every logit.
        {"name": "route training odd", "op": "unroute", "t": 4097, "e": 63, "top": 6, "type": "bf16", "score": "softmax", "bias": False, "groups": 1, "keep": 1,
         "by": "max", "renorm": False},
        # One token's experts, weights in 16 bits, the choice made before.
        {"name": "experts one token", "op": "experts", "t": 1, "e": 64, "top": 8, "h": 2048, "i": 1024, "type": "bf16"},
        # A short prompt, no size a multiple of anything.
        {"name": "experts odd prompt", "op": "experts", "t": 333, "e": 8, "top": 2, "h": 2049, "i": 1025, "type": "f16"},
        # A long prompt through few wide experts.
        {"name": "experts long prompt", "op": "experts", "t": 8192, "e": 8, "top": 2, "h": 4096, "i": 4096, "type": "bf16"},
        # A training step of a layer of many small experts.
        {"name": "train small experts", "op": "train", "t": 4096, "e": 64, "top": 4, "h": 2048, "i": 1024, "type": "bf16"},
        # A training step of odd sizes: an uneven batch, few experts.
        {"name": "train odd", "op": "train", "t": 1021, "e": 7, "top": 3, "h": 1000, "i": 517, "type": "f16"},
        # One token of one request.
        {"name": "adapters one token", "op": "adapters", "t": 1, "n": 4096, "k": 4096, "r": 16, "count": 8, "type": "bf16"},
        # A batch of single tokens, each of a request with an adapter of its own choice, odd sizes.
        {"name": "adapters 61 tokens odd", "op": "adapters", "t": 61, "n": 4095, "k": 2049, "r": 17, "count": 30, "type": "f16"},
        # The widest batch of single tokens, through a wide projection.
        {"name": "adapters 64 tokens wide", "op": "adapters", "t": 64, "n": 16384, "k": 8192, "r": 64, "count": 32, "type": "bf16"},
        # Several requests' prompts together.
        {"name": "adapters prompts", "op": "adapters", "t": 8192, "n": 4096, "k": 4096, "r": 32, "count": 16, "type": "bf16"},
    ]


def _size(rng, low, high):
    """A size between low and high, even over the logarithm; half of them as drawn, half rounded to a multiple of 32."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    if rng.random() < 0.5 and n >= 48:
        n = min(high, 32 * ((n + 16) // 32))
    return max(low, min(high, n))


def draw(rng):
    op = rng.choice(("route", "unroute", "experts", "train", "adapters"))
    while True:
        if op in ("route", "unroute"):
            groups = rng.choice((1, 1, 2, 4, 8))
            e = groups * max(2, _size(rng, 4, 256) // groups)
            keep = rng.randint(1, groups)
            c = {"op": op, "t": _size(rng, 1, 16384), "e": e, "top": rng.randint(1, min(8, keep * (e // groups))), "type": rng.choice(("bf16", "f16", "f32")),
                 "score": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5, "groups": groups, "keep": keep, "by": rng.choice(("max", "top2")),
                 "renorm": rng.random() < 0.5}
            if c["t"] * e * (3 if op == "unroute" else 1) <= 16384 * 256:
                return c
        elif op in ("experts", "train"):
            e = _size(rng, 2, 64)
            c = {"op": op, "t": _size(rng, 1 if op == "experts" else 64, 8192), "e": e, "top": rng.randint(1, min(8, e)), "h": _size(rng, 64, 4096),
                 "i": _size(rng, 32, 4096), "type": rng.choice(("bf16", "f16"))}
            if c["t"] * c["top"] * c["h"] * c["i"] * (3 if op == "train" else 1) <= 8192 * 2 * 4096 * 2048 and e * c["h"] * c["i"] <= 64 * 2048 * 1024:
                return c
        else:
            c = {"op": op, "t": rng.choice((1, rng.randint(2, 64), _size(rng, 65, 8192))), "n": _size(rng, 64, 16384), "k": _size(rng, 64, 8192),
                 "r": rng.choice((8, 16, 32, 64, rng.randint(4, 64))), "count": _size(rng, 1, 64), "type": rng.choice(("bf16", "f16"))}
            if c["t"] * c["n"] * c["k"] <= 8192 * 4096 * 4096:
                return c


# ---- inputs ---------------------------------------------------------------


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda shape, scale=1.0: torch.randn(shape, generator=g, device="cuda") * scale  # noqa: E731
    s, dtype, t = dict(case), TYPES[case["type"]], case["t"]
    if case["op"] in ("route", "unroute"):
        e = case["e"]
        # some experts are liked more than others
        s["logits"] = (normal((t, e)) + normal((1, e), 0.5)).to(dtype)
        s["b"] = normal((e,), 0.1) if case["bias"] else None
        if case["op"] == "unroute":
            s["dgates"] = normal((t, case["top"]))
    elif case["op"] in ("experts", "train"):
        e, h, i = case["e"], case["h"], case["i"]
        s["x"] = normal((t, h)).to(dtype)
        s["w1"] = normal((e, 2 * i, h), 1 / math.sqrt(h)).to(dtype)
        s["w2"] = normal((e, h, i), 1 / math.sqrt(i)).to(dtype)
        # the choice of a router that likes some experts more than others
        gates, ids = torch.topk(torch.softmax(normal((t, e)) + normal((1, e), 0.5), -1), case["top"], dim=-1)
        s["ids"], s["gates"] = ids.int(), gates / gates.sum(-1, keepdim=True)
        if case["op"] == "train":
            s["dy"] = normal((t, h)).to(dtype)
    else:
        n, k, r, count = case["n"], case["k"], case["r"], case["count"]
        s["x"] = normal((t, k)).to(dtype)
        s["w"] = normal((n, k), 1 / math.sqrt(k)).to(dtype)
        s["a"] = normal((count, r, k), 1 / math.sqrt(k)).to(dtype)
        s["bb"] = normal((count, n, r), 1 / math.sqrt(r)).to(dtype)
        s["scales"] = torch.rand((count,), generator=g, device="cuda") + 0.5
        # single tokens: a request each; prompts: runs of tokens of one request; one request in count + 1 has no adapter
        runs = t if t <= 64 else max(1, t // 256)
        of = torch.randint(-1, count, (runs,), generator=g, device="cuda", dtype=torch.int32)
        cuts = torch.randint(0, t, (runs - 1,), generator=g, device="cuda").sort().values
        s["ids"] = of if t <= 64 else of[torch.searchsorted(cuts, torch.arange(t, device="cuda"), right=True)].contiguous()
        if t == 1:
            s["ids"] = s["ids"].clamp(min=0)
    return s


# ---- the plain forms --------------------------------------------------------


def _lowest_first(v, top):
    """Places of the `top` largest of each row, in falling order; of equal ones the lower first."""
    return torch.sort(v, dim=-1, descending=True, stable=True).indices[:, :top]


def _plain_route(s):
    z = s["logits"].double()
    t, e = z.shape
    score = torch.softmax(z, -1) if s["score"] == "softmax" else torch.sigmoid(z)
    key = score if s["b"] is None else score + s["b"].double()
    if s["groups"] > 1:
        by = key.reshape(t, s["groups"], -1)
        of = by.amax(-1) if s["by"] == "max" else by.topk(min(2, by.shape[-1]), -1).values.sum(-1)
        kept = torch.zeros_like(of, dtype=torch.bool).scatter_(1, _lowest_first(of, s["keep"]), True)
        key = by.masked_fill(~kept.unsqueeze(-1), -math.inf).reshape(t, e)
    ids = _lowest_first(key, s["top"])
    gates = score.gather(1, ids)
    if s["renorm"]:
        gates = gates / gates.sum(-1, keepdim=True)
    if s["op"] == "route":
        return ids.int(), gates.float()
    dg = s["dgates"].double()
    picked = score.gather(1, ids)
    if s["renorm"]:
        dg = (dg - (dg * gates).sum(-1, keepdim=True)) / picked.sum(-1, keepdim=True)
    ds = torch.zeros_like(score).scatter_(1, ids, dg)
    if s["score"] == "softmax":
        dz = score * (ds - (dg * picked).sum(-1, keepdim=True))
    else:
        dz = score * (1 - score) * ds
    return ids.int(), gates.float(), dz.to(s["logits"].dtype)


def _plain_experts(s):
    x, gates = s["x"].float(), s["gates"]
    t, top = s["ids"].shape
    e, h, i = s["w2"].shape
    if s["op"] == "experts" and t * top < e:  # fewer choices than experts: their weights alone
        pick = s["ids"].reshape(-1).long()
        a = torch.matmul(s["w1"][pick].float(), x.repeat_interleave(top, 0).unsqueeze(-1)).squeeze(-1)
        u = a[:, :i] * torch.sigmoid(a[:, :i]) * a[:, i:]
        y = torch.matmul(s["w2"][pick].float(), u.unsqueeze(-1)).reshape(t, top, h)
        return (y * gates.unsqueeze(-1)).sum(1).to(s["x"].dtype)
    w1, w2 = s["w1"].float(), s["w2"].float()
    # the pairs (token, choice) by expert, each expert's padded to the most that one has
    flat = s["ids"].reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    counts = torch.zeros(e, dtype=torch.long, device=x.device).index_add_(0, flat, torch.ones_like(flat))
    most = int(counts.max())
    of = flat[order]
    place = of * most + torch.arange(t * top, device=x.device) - (counts.cumsum(0) - counts)[of]

    def spread(rows):
        return torch.zeros((e * most, rows.shape[1]), device=x.device).index_copy_(0, place, rows).reshape(e, most, -1)

    def gather(rows):  # by pair
        return torch.empty((t * top, rows.shape[-1]), device=x.device).index_copy_(0, order, rows.reshape(e * most, -1)[place])

    token = order // top
    xs = spread(x[token])
    a = torch.matmul(xs, w1.transpose(1, 2))
    p, q = a[..., :i], a[..., i:]
    sg = torch.sigmoid(p)
    u = p * sg * q
    y = (gather(torch.matmul(u, w2.transpose(1, 2))).reshape(t, top, h) * gates.unsqueeze(-1)).sum(1).to(s["x"].dtype)
    if s["op"] == "experts":
        return y
    dys = spread(s["dy"].float()[token])
    gs = spread(gates.reshape(-1, 1)[order])
    du = torch.matmul(dys, w2)
    dgates = gather((du * u).sum(-1, keepdim=True)).reshape(t, top)
    du = du * gs
    da = torch.cat((du * q * sg * (1 + p * (1 - sg)), du * p * sg), -1)
    dx = gather(torch.matmul(da, w1)).reshape(t, top, h).sum(1)
    dw1 = torch.matmul(da.transpose(1, 2), xs)
    dw2 = torch.matmul(dys.transpose(1, 2), u * gs)
    dtype = s["x"].dtype
    return y, dx.to(dtype), dgates, dw1.to(dtype), dw2.to(dtype)


def _plain_adapters(s):
    x, ids = s["x"].float(), s["ids"]
    count, r, k = s["a"].shape
    # every adapter on every row, the others' products dropped
    v = torch.matmul(x, s["a"].float().reshape(count * r, k).t()).reshape(-1, count, r)
    share = torch.where(ids.unsqueeze(1) == torch.arange(count, device=x.device), s["scales"], 0.0)
    v = (v * share.unsqueeze(-1)).reshape(-1, count * r)
    y = torch.matmul(x, s["w"].float().t()) + torch.matmul(v, s["bb"].float().transpose(1, 2).reshape(count * r, -1))
    return y.to(s["x"].dtype)


def run(state):
    s = state
    if own:
        import tiled_fp32_gemm_03_amd as g

        if s["op"] in ("route", "unroute"):
            ids, gates = g.moe_route(s["logits"], s["top"], score=s["score"], bias=s["b"], groups=s["groups"], top_groups=s["keep"], group_score=s["by"],
                                     renormalize=s["renorm"])
            if s["op"] == "route":
                return ids, gates
            return ids, gates, g.moe_route_backward(s["dgates"], s["logits"], ids, score=s["score"], renormalize=s["renorm"])
        if s["op"] == "experts":
            return g.moe_experts(s["x"], s["ids"], s["gates"], s["w1"], s["w2"])
        if s["op"] == "train":
            y, saved = g.moe_experts(s["x"], s["ids"], s["gates"], s["w1"], s["w2"], save=True)
            return (y, *g.moe_experts_backward(s["dy"], s["x"], s["ids"], s["gates"], s["w1"], s["w2"], saved))
        return g.matmul_adapters(s["x"], s["w"], s["a"], s["bb"], s["ids"], s["scales"])
    if s["op"] in ("route", "unroute"):
        return _plain_route(s)
    if s["op"] in ("experts", "train"):
        return _plain_experts(s)
    return _plain_adapters(s)


# ---- what cannot be done without --------------------------------------------


def work(case):
    width = {"bf16": 2, "f16": 2, "f32": 4}[case["type"]]
    t = case["t"]
    if case["op"] in ("route", "unroute"):
        back = case["op"] == "unroute"
        return {"bytes": t * case["e"] * width * (2 if back else 1) + t * case["top"] * (12 if back else 8) + (4 * case["e"] if case["bias"] else 0),
                "flops": t * case["e"] * (12 if back else 6)}
    if case["op"] in ("experts", "train"):
        e, top, h, i = (case[x] for x in ("e", "top", "h", "i"))
        asked = e * (1 - (1 - top / e) ** t)  # experts that at least one token asks, for even routing
        if case["op"] == "experts":
            return {"bytes": asked * 3 * h * i * width + 2 * t * h * width + t * top * 8, "flops": 6 * t * top * h * i}
        return {"bytes": (asked + e) * 3 * h * i * width + 4 * t * h * width + t * top * 12, "flops": 18 * t * top * h * i}
    n, k, r, count = (case[x] for x in ("n", "k", "r", "count"))
    runs = t if t <= 64 else max(1, t // 256)
    asked = 1 if t == 1 else count * (1 - (1 - 1 / (count + 1)) ** runs)
    return {"bytes": (n * k + asked * r * (n + k) + t * (n + k)) * width + t * 4, "flops": 2 * t * n * k + 2 * t * r * (n + k)}


# ---- the definitions in 64 bits -----------------------------------------------


def _exact_route(case, s):
    z = s["logits"].double()
    t, e = z.shape
    rows = torch.arange(t, device=z.device)
    if case["score"] == "softmax":
        score = torch.exp(z - z.max(1, keepdim=True).values)
        score = score / score.sum(1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-z))
    key = score.clone()
    if case["bias"]:
        key = key + s["b"].double()
    if case["groups"] > 1:
        size, totals = e // case["groups"], []
        for j in range(case["groups"]):
            part = key[:, j * size:(j + 1) * size].sort(dim=1, descending=True).values
            totals.append(part[:, 0] if case["by"] == "max" or size == 1 else part[:, 0] + part[:, 1])
        totals = torch.stack(totals, 1)
        out = torch.ones_like(totals, dtype=torch.bool)
        for _ in range(case["keep"]):
            best = totals.max(1, keepdim=True).values
            at = (totals == best).int().argmax(1)  # the first of equals
            out[rows, at] = False
            totals[rows, at] = -math.inf
        key[out.repeat_interleave(size, 1)] = -math.inf
    ids = []
    for _ in range(case["top"]):
        best = key.max(1, keepdim=True).values
        at = (key == best).int().argmax(1)
        ids.append(at)
        key[rows, at] = -math.inf
    ids = torch.stack(ids, 1)
    picked = score[rows.unsqueeze(1), ids]
    gates = picked / picked.sum(1, keepdim=True) if case["renorm"] else picked
    if case["op"] == "route":
        return ids.int(), gates
    # d gate / d z, one gate at a time
    dz = torch.zeros_like(z)
    for j in range(case["top"]):
        w = s["dgates"].double()[:, j] * gates[:, j]
        if case["renorm"]:
            for m in range(case["top"]):
                mine = 1 - picked[:, m] if case["score"] == "sigmoid" else 1.0
                dz[rows, ids[:, m]] += w * mine * ((1.0 if m == j else 0.0) - gates[:, m])
        elif case["score"] == "sigmoid":
            dz[rows, ids[:, j]] += w * (1 - picked[:, j])
        else:
            dz -= w.unsqueeze(1) * score
            dz[rows, ids[:, j]] += w
    return ids.int(), gates, dz


def _exact_experts(case, s):
    x, gates, ids, i = s["x"].double(), s["gates"].double(), s["ids"].long(), case["i"]
    train = case["op"] == "train"
    y = torch.zeros_like(x)
    if train:
        dy, dx, dgates = s["dy"].double(), torch.zeros_like(x), torch.zeros_like(gates)
        dw1, dw2 = torch.zeros(s["w1"].shape, dtype=torch.float64, device="cuda"), torch.zeros(s["w2"].shape, dtype=torch.float64, device="cuda")
    for e in range(case["e"]):
        tok, slot = torch.nonzero(ids == e, as_tuple=True)
        if tok.numel() == 0:
            continue
        w1, w2 = s["w1"][e].double(), s["w2"][e].double()
        p, q = x[tok] @ w1[:i].t().contiguous(), x[tok] @ w1[i:].t().contiguous()
        bend = 1 + torch.exp(-p)
        u, w = p / bend * q, gates[tok, slot].unsqueeze(1)
        y.index_add_(0, tok, w * (u @ w2.t().contiguous()))
        if train:
            du = dy[tok] @ w2
            dgates[tok, slot] = (du * u).sum(1)
            dp = w * du * q * (1 / bend + p * torch.exp(-p) / bend ** 2)
            dq = w * du * p / bend
            dx.index_add_(0, tok, dp @ w1[:i] + dq @ w1[i:])
            dw1[e, :i], dw1[e, i:] = dp.t().contiguous() @ x[tok], dq.t().contiguous() @ x[tok]
            dw2[e] = dy[tok].t().contiguous() @ (w * u)
    return (y, dx, dgates, dw1, dw2) if train else y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("route", "unroute"):
        return _exact_route(case, s)
    if case["op"] in ("experts", "train"):
        return _exact_experts(case, s)
    y = s["x"].double() @ s["w"].double().t().contiguous()
    for r in range(case["count"]):
        tok = torch.nonzero(s["ids"] == r).squeeze(1)
        if tok.numel():
            v = s["x"][tok].double() @ s["a"][r].double().t().contiguous()
            y[tok] += s["scales"][r].double() * (v @ s["bb"][r].double().t().contiguous())
    return y
