"""The operators of a decoder layer with experts as a serving loop calls them: the norm that adds the
residual (with an output in 8 bits where asked), the choice of each token's experts, and the experts'
gated products over Q4_0 weights.

``own`` chooses between the library's entry points and the plain form: the same operators in
elementary torch operations on f32 values.  Sizes are the library's decoder sweep's (hidden 4096,
feed-forward 14336) or generic ones.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _norm(name, **more):
    c = {"name": name, "op": "norm", "dtype": "f32", "rows": 1, "width": 4096, "residual": True, "q8": False, "offset": 0.0}
    c.update(more)
    return c


def _route(name, **more):
    c = {"name": name, "op": "route", "dtype": "f32", "tokens": 1, "experts": 64, "top_k": 8, "sigmoid": False, "bias": False,
         "groups": 1, "top_groups": 1, "group_top": 2, "renormalize": True, "scale": 1.0}
    c.update(more)
    return c


def _experts(name, **more):
    c = {"name": name, "op": "experts", "dtype": "f32", "tokens": 1, "experts": 8, "top_k": 2, "hidden": 4096, "inner": 14336,
         "gated": True, "skew": 0.5, "idle": 0.0}
    c.update(more)
    return c


def listed():
    return [
        # One token of one request between two blocks: latency counts.
        _norm("norm step"),
        # A serving batch's tokens, with 8-bit rows for the products that take them.
        _norm("norm batch to 8 bits", dtype="bf16", rows=64, q8=True),
        # A chunk of prompts; the norm's weights are held as their distance from 1.
        _norm("norm prompts", dtype="bf16", rows=8192, offset=1.0),
        # One token's experts.
        _route("route step", experts=64, top_k=8),
        # A chunk of prompts under grouped routing with a bias that balances the load.
        _route("route prompts in groups", tokens=4096, experts=256, top_k=8, sigmoid=True, bias=True, groups=8, top_groups=4,
               scale=2.5),
        # One token of one request through two large experts of the decoder sweep's size.
        _experts("experts step"),
        # One token through eight of many small experts of a size that is no multiple of 256.
        _experts("experts step small", dtype="bf16", experts=64, top_k=8, hidden=2048, inner=1408),
        # A serving batch's step: most experts get a token or a few.
        _experts("experts batch", dtype="bf16", tokens=48, experts=64, top_k=6, hidden=4096, inner=1024, skew=1.0),
        # Short prompts, f32 rows, large experts.
        _experts("experts prompt", tokens=500, experts=8, top_k=2),
        # Prompts packed to a fixed number of rows (some of them padding), many experts of uneven popularity.
        _experts("experts prompts ragged", dtype="bf16", tokens=2048, experts=64, top_k=8, hidden=4096, inner=1024, skew=1.0,
                 idle=0.1),
        # Long prompts through large experts.
        _experts("experts prompts large", dtype="bf16", tokens=4096, experts=8, top_k=2),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "experts", "experts"])
    dtype = rng.choice(["f32", "bf16"])
    if op == "norm":
        c = _norm("", dtype=dtype, rows=_log(rng, 1, 6000), width=_log(rng, 96, 16384), residual=rng.random() < 0.7,
                  offset=rng.choice([0.0, 1.0]))
        if dtype == "bf16" and rng.random() < 0.5:  # (of f32 rows, a value next to a rounding border would differ by a whole step)
            c.update(q8=True, width=32 * max(1, c["width"] // 32))
    elif op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 8, 512 // groups)
        c = _route("", dtype=dtype, tokens=_log(rng, 1, 8000), experts=experts, sigmoid=rng.random() < 0.5, groups=groups,
                   bias=rng.random() < 0.5, top_groups=rng.randint(1, groups), group_top=rng.choice([1, 2]),
                   renormalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]))
        c["top_k"] = rng.randint(1, min(10, c["top_groups"] * experts // groups))
    else:
        c = _experts("", dtype=dtype, tokens=_log(rng, 1, 1500), experts=_log(rng, 2, 96), gated=rng.random() < 0.8,
                     skew=rng.choice([0.0, 0.5, 1.0]), idle=rng.choice([0.0, 0.0, 0.2]))
        step = rng.choice([32, 128, 256, 256])
        c.update(hidden=step * max(1, _log(rng, 512, 4096) // step), inner=step * max(1, _log(rng, 256, 4096) // step),
                 top_k=rng.randint(1, min(8, c["experts"])))
    del c["name"]
    return c


# ---- what a pass cannot do without


def work(case):
    c = case
    item = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "norm":
        n = c["rows"] * c["width"]
        streams = 4 if c["residual"] else 2  # x and the residual in, their sum and the norm out
        return {"bytes": n * streams * item + c["width"] * 4 + (n * (34 / 32 + item) if c["q8"] else 0), "flops": 6 * n}
    if c["op"] == "route":
        n = c["tokens"] * c["experts"]
        return {"bytes": n * item + c["tokens"] * c["top_k"] * 8 + (4 * c["experts"] if c["bias"] else 0), "flops": 8 * n}
    rows = c["tokens"] * (1.0 - c["idle"]) * c["top_k"]
    chosen = c["experts"] * (1.0 - (1.0 - c["top_k"] / c["experts"]) ** (c["tokens"] * (1.0 - c["idle"])))
    each = (3 if c["gated"] else 2) * c["hidden"] * c["inner"]
    return {"bytes": chosen * each * 9 / 16 + c["tokens"] * (2 * c["hidden"] * item + 8 * c["top_k"]), "flops": 2 * rows * each}


# ---- inputs


def _blocks(shape, k, gen):
    """Random Q4_0 rows of k elements: uniform nibbles, scales that keep the products of rows near 1 near 1."""
    x = torch.randint(0, 256, (*shape, k // 32, 18), dtype=torch.uint8, device="cuda", generator=gen)
    d = (0.5 + torch.rand((*shape, k // 32), device="cuda", generator=gen)) * (0.2 / math.sqrt(k))
    d = torch.where(torch.rand(d.shape, device="cuda", generator=gen) < 0.5, d, -d).half()
    x[..., :2] = d.unsqueeze(-1).view(torch.uint8)
    return x.reshape(*shape, k // 32 * 18)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def normal(*shape):
        return torch.randn(shape, device="cuda", generator=gen)

    dtype = DTYPES[c["dtype"]]
    s = {"case": dict(c)}
    if c["op"] == "norm":
        size = torch.exp(normal(c["rows"], 1))  # rows of different sizes, a few strong channels
        strong = 1.0 + 20.0 * (torch.rand(c["width"], device="cuda", generator=gen) < 0.005)
        s["x"] = (normal(c["rows"], c["width"]) * size).to(dtype)
        if c["residual"]:
            s["residual"] = (normal(c["rows"], c["width"]) * size * strong).to(dtype)
        s["weight"] = 1.0 - c["offset"] + 0.2 * normal(c["width"])
        return s
    if c["op"] == "route":
        s["logits"] = (1.5 * normal(c["tokens"], c["experts"]) + 0.5 * normal(c["experts"])).to(dtype)
        s["bias"] = 0.1 * normal(c["experts"]) if c["bias"] else None
        return s
    s["x"] = normal(c["tokens"], c["hidden"]).to(dtype)
    liking = normal(c["tokens"], c["experts"]) + c["skew"] * normal(c["experts"])
    top = torch.topk(liking, c["top_k"], dim=-1)
    s["ids"], s["weights"] = top.indices.to(torch.int32), torch.softmax(top.values, -1)
    if c["idle"]:  # rows of padding have no experts
        s["ids"][torch.rand(c["tokens"], device="cuda", generator=gen) < c["idle"]] = -1
    for name in ("w_gate", "w_up") if c["gated"] else ("w_up",):
        s[name] = _blocks((c["experts"], c["inner"]), c["hidden"], gen)
    s["w_down"] = _blocks((c["experts"], c["hidden"]), c["inner"], gen)
    return s


# ---- the library's form


def _run_own(s):
    import bit_block_quantized_qm_gb300 as qm
    c = s["case"]
    if c["op"] == "norm":
        out, total, q8 = qm.qm_add_rmsnorm(s["x"], s["weight"], residual=s.get("residual"), eps=1e-6, weight_offset=c["offset"],
                                           want_q8=c["q8"])
        got = {"out": out}
        if c["residual"]:
            got["sum"] = total
        if c["q8"]:
            got["q8"] = qm.qm_dequant_q8_0(q8).view(c["rows"], c["width"]).to(DTYPES[c["dtype"]])
        return got
    if c["op"] == "route":
        ids, weights = qm.qm_route_experts(s["logits"], c["top_k"], bias=s["bias"],
                                           scoring=qm.QM_SCORE_SIGMOID if c["sigmoid"] else qm.QM_SCORE_SOFTMAX,
                                           n_groups=c["groups"], top_groups=c["top_groups"], group_top=c["group_top"],
                                           renormalize=c["renormalize"], scale=c["scale"])
        return {"ids": ids, "weights": weights}
    if "handle" not in s:  # the layer that a program keeps
        s["handle"] = qm.Experts(s.get("w_gate"), s["w_up"], s["w_down"], activation=qm.QM_ACT_SILU)
    return {"out": qm.qm_experts_q4_0(s["handle"], s["x"], s["ids"], s["weights"])}


# ---- the plain form


def _plain_norm(s):
    c, dtype = s["case"], DTYPES[s["case"]["dtype"]]
    x = s["x"].float()
    got = {}
    if c["residual"]:
        x = x + s["residual"].float()
        got["sum"] = x.to(dtype)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * (c["offset"] + s["weight"])
    got["out"] = y.to(dtype)
    if c["q8"]:
        b = y.reshape(c["rows"], -1, 32)
        d = b.abs().amax(-1, keepdim=True) / 127.0
        t = b / torch.where(d == 0, torch.ones_like(d), d)
        q = torch.sign(t) * torch.floor(t.abs() + 0.5)
        got["q8"] = (torch.clamp(q, -127.0, 127.0) * d.half().float()).reshape(c["rows"], c["width"]).to(dtype)
    return {k: got[k] for k in ("out", "sum", "q8") if k in got}


def _top(c, k, dim=-1):
    """The k largest of a dimension and where they are; of equal ones the first."""
    v, i = torch.sort(c, dim=dim, descending=True, stable=True)
    return v[..., :k], i[..., :k]


def _plain_route(s):
    c = s["case"]
    x = s["logits"].double()  # (two choices next to each other have to keep their order)
    if c["sigmoid"]:
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        score = torch.exp(x - x.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if c["groups"] > 1:
        per = choice.reshape(c["tokens"], c["groups"], -1)
        _, best = _top(_top(per, c["group_top"])[0].sum(-1), c["top_groups"])
        stays = torch.zeros((c["tokens"], c["groups"]), dtype=torch.bool, device="cuda").scatter_(-1, best, True)
        choice = per.masked_fill(~stays.unsqueeze(-1), -math.inf).reshape(c["tokens"], -1)
    _, ids = _top(choice, c["top_k"])
    w = score.gather(-1, ids)
    if c["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.to(torch.int32), "weights": (w * c["scale"]).float()}


def _values(w):
    """Q4_0 rows as f32."""
    b = w.reshape(*w.shape[:-1], -1, 18)
    q = b[..., 2:]
    d = b[..., :2].contiguous().view(torch.float16).float()
    return (torch.cat([q & 15, q >> 4], -1).float().sub_(8.0)).mul_(d).reshape(*w.shape[:-1], -1)


def _plain_experts(s):
    c = s["case"]
    x, ids = s["x"].float(), s["ids"].reshape(-1).long()
    token = torch.arange(len(ids), device="cuda") // c["top_k"]
    weight = torch.where(ids < 0, torch.zeros((), device="cuda"), s["weights"].reshape(-1))
    names = [n for n in ("w_gate", "w_up", "w_down") if n in s]
    if len(ids) <= c["experts"]:  # each pair's expert by itself
        w = {n: _values(s[n][ids.clamp(min=0)]) for n in names}
        rows, back = x[token].unsqueeze(1), None
    else:  # rows in batches of their experts, padded to the longest
        ids = ids.clamp(min=0)
        order = torch.argsort(ids, stable=True)
        count = torch.bincount(ids, minlength=c["experts"])
        place = torch.empty_like(order)
        place[order] = torch.arange(len(ids), device="cuda") - (count.cumsum(0) - count)[ids[order]]
        longest = int(count.max())
        back = ids * longest + place
        rows = torch.zeros((c["experts"] * longest, c["hidden"]), device="cuda")
        rows[back] = x[token]
        rows = rows.reshape(c["experts"], longest, c["hidden"])
        w = {n: _values(s[n]) for n in names}
    h = torch.matmul(rows, w["w_up"].transpose(1, 2))
    if c["gated"]:
        g = torch.matmul(rows, w["w_gate"].transpose(1, 2))
        h = g / (1.0 + torch.exp(-g)) * h
    else:
        h = h / (1.0 + torch.exp(-h))
    y = torch.matmul(h, w["w_down"].transpose(1, 2)).reshape(-1, c["hidden"])
    if back is not None:
        y = y[back]
    y = (y * weight.unsqueeze(-1)).reshape(c["tokens"], c["top_k"], c["hidden"]).sum(1)
    return {"out": y.to(DTYPES[c["dtype"]])}


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _plain_norm, "route": _plain_route, "experts": _plain_experts}[state["case"]["op"]](state)


# ---- the definition in 64 bits


def _expert_rows(w):
    """One expert's Q4_0 rows in f64, nibble by nibble."""
    n = w.shape[0]
    b = w.reshape(n, -1, 18)
    d = (b[:, :, 0].to(torch.int32) + 256 * b[:, :, 1].to(torch.int32)).to(torch.int16).view(torch.float16).double()
    v = torch.empty((n, b.shape[1], 32), dtype=torch.float64, device="cuda")
    v[:, :, :16] = (b[:, :, 2:] % 16).double() - 8.0
    v[:, :, 16:] = torch.div(b[:, :, 2:], 16, rounding_mode="floor").double() - 8.0
    return (v * d.unsqueeze(-1)).reshape(n, -1)


def exact(case, seed):
    c = case
    if work(c)["flops"] > 4e12:
        return None
    s = prepare(c, seed)
    if c["op"] == "norm":
        t = s["x"].double()
        if c["residual"]:
            t = t + s["residual"].double()
        y = t / torch.sqrt((t ** 2).sum(-1, keepdim=True) / c["width"] + 1e-6) * (s["weight"].double() + c["offset"])
        got = {"out": y}
        if c["residual"]:
            got["sum"] = t
        if c["q8"]:
            got["q8"] = None  # its steps are a rounding in 32 bits by definition
        return got
    if c["op"] == "route":
        # The ids are whole numbers.  (Experts with equal choices have equal weights, whichever comes first.)
        x = s["logits"].double()
        p = torch.sigmoid(x) if c["sigmoid"] else torch.softmax(x, -1)
        a = p if s["bias"] is None else p + s["bias"].double()
        if c["groups"] > 1:
            g = a.unflatten(1, (c["groups"], -1))
            border = g.topk(min(c["group_top"], g.shape[-1]), -1).values.sum(-1)
            out = border < border.topk(c["top_groups"], -1).values[:, -1:]
            a = torch.where(out.unsqueeze(-1), -math.inf, g).flatten(1)
        ids = a.topk(c["top_k"], -1).indices
        w = torch.gather(p, 1, ids)
        return {"ids": None, "weights": c["scale"] * (w / w.sum(1, keepdim=True) if c["renormalize"] else w)}
    out = torch.zeros((c["tokens"], c["hidden"]), dtype=torch.float64, device="cuda")
    for e in range(c["experts"]):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if len(t) == 0:
            continue
        x = s["x"][t].double()
        u = x @ _expert_rows(s["w_up"][e]).T
        if c["gated"]:
            g = x @ _expert_rows(s["w_gate"][e]).T
            h = g * torch.sigmoid(g) * u
        else:
            h = u * torch.sigmoid(u)
        out.index_add_(0, t, (h @ _expert_rows(s["w_down"][e]).T) * s["weights"][t, j].double().unsqueeze(-1))
    return {"out": out}
