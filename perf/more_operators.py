"""The operators of a mixture-of-experts layer in 8-bit integers: routing by softmax or sigmoid scores
with a balance bias, expert groups and scaled weights, and its gradient; the copy of tokens into the
experts' order as int8 rows with a scale each; and the int8 product with a scale per token and per
channel, of one matrix or of every expert's.

`run` takes one pass through one operator: in its plain form, elementary torch operations, or (`own`)
through the library's entry points.  `exact` is the same in 64 bits.
"""
import math

import torch

own = False

INT8_MAX = 127.0
TINY = 2.0 ** -96    # rows whose largest magnitude is below this share its scale
COEF = 0.001         # weight of the balance loss
CHUNK = 1024         # int8 products that FP32 adds exactly: 1024 * 2^14 = 2^24


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a decoding step, 256 experts in eight groups, scores biased for balance: pure latency
        _route("route_one_token", tokens=1, size=32, groups=8, top_groups=4, top_k=8, score="sigmoid", best=2, bias=True, dtype="f32"),
        # a padded batch of prompts, softmax scores in BF16 (many ties), the best of three of four groups, some experts closed
        _route("route_padded_bf16", tokens=4099, size=15, groups=4, top_groups=3, top_k=4, score="softmax", best=1, bias=False, dtype="bf16",
               masked=True, normalize=False, scale=16.0),
        # a training micro-batch of 128 Ki tokens over 256 experts
        _route("route_train_128k", tokens=131071, size=32, groups=8, top_groups=4, top_k=8, score="sigmoid", best=2, bias=True, dtype="f32"),
        # its gradient: from the weights and from the balance loss
        _route("route_grad_64k", tokens=65536, size=32, groups=8, top_groups=4, top_k=8, score="sigmoid", best=2, bias=True, dtype="f32", op="route_grad"),
        # sixteen tokens of a decoding batch into int8 rows
        _quantize_case("quantize_decode", tokens=16, experts=64, top_k=8, hidden=4096, dtype="bf16"),
        # the rows between two products, in order already, from FP32; a width that is not a power of two
        _quantize_case("quantize_rows_f32", tokens=8190, experts=0, top_k=1, hidden=1424, dtype="f32"),
        # a prompt batch of 16 Ki tokens, eight experts each
        _quantize_case("quantize_prompt", tokens=16384, experts=64, top_k=8, hidden=4096, dtype="bf16"),
        # one token through a square projection: latency and the weights' bytes
        _product("product_one_token", groups=0, rows=1, n=4096, k=4096, out="bf16"),
        # the FP8 benchmark's size in int8
        _product("product_8192", groups=0, rows=8192, n=8192, k=8192, out="bf16"),
        # a decoding batch's experts: two rows each, every weight read once
        _product("product_experts_decode", groups=32, rows=64, n=4096, k=4096, out="bf16"),
        # fine-grained experts with uneven loads (some without rows), ragged sizes, with a bias and ReLU into FP32
        _product("product_experts_ragged", groups=60, rows=2047, n=1416, k=2064, out="f32", skew=1.0, bias=True, relu=True),
        # the grouped benchmark's layer: 16 experts of 4096 x 4096 over 16384 rows
        _product("product_experts_prompt", groups=16, rows=16384, n=4096, k=4096, out="bf16", skew=0.5),
    ]


def _route(name, *, tokens, size, groups, top_groups, top_k, score, best, bias, dtype, masked=False, normalize=True, scale=2.5, op="route"):
    return {"name": name, "op": op, "tokens": tokens, "experts": size * groups, "groups": groups, "top_groups": top_groups, "top_k": top_k, "score": score,
            "best": best, "bias": bias, "dtype": dtype, "masked": masked, "normalize": normalize, "scale": scale}


def _quantize_case(name, *, tokens, experts, top_k, hidden, dtype):
    return {"name": name, "op": "quantize", "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden, "dtype": dtype}


def _product(name, *, groups, rows, n, k, out, skew=0.0, bias=False, relu=False):
    return {"name": name, "op": "product", "groups": groups, "rows": rows, "n": n, "k": k, "out": out, "skew": skew, "bias": bias, "relu": relu}


def _spread(rng, low, high, step=1):
    """A size between `low` and `high`, even over its logarithm, a multiple of `step`."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return max(max(low, min(high, v)) // step * step, step)


def draw(rng):
    op = rng.choice(["route", "route", "route", "route_grad", "quantize", "quantize", "product", "product", "product", "product"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 2, 4, 5, 8, 16])
        size = _spread(rng, 2, 512 // (16 if groups == 5 else groups))
        top_groups = rng.randint(1, groups)
        most = (131071 if op == "route" else 65536) * 256
        case = _route("", tokens=_spread(rng, 1, min(131071, most // (size * groups))), size=size, groups=groups, top_groups=top_groups,
                      top_k=rng.randint(1, min(10, top_groups * size)), score=rng.choice(["sigmoid", "sigmoid", "softmax"]), best=rng.randint(1, 2),
                      bias=rng.random() < 0.7, dtype=rng.choice(["f32", "bf16"]), masked=rng.random() < 0.3, normalize=rng.random() < 0.6,
                      scale=rng.choice([1.0, 2.5]), op=op)
    elif op == "quantize":
        hidden = _spread(rng, 64, 8192, 16)
        experts = rng.choice([0, _spread(rng, 4, 256)])
        top_k = rng.randint(1, min(8, experts)) if experts else 1
        case = _quantize_case("", tokens=_spread(rng, 1, 16384 * 8 * 4096 // (top_k * 8192)), experts=experts, top_k=top_k, hidden=hidden,
                              dtype=rng.choice(["f32", "bf16"]))
    else:
        groups = rng.choice([0, 0, _spread(rng, 2, 64)])
        n, k = _spread(rng, 64, 8192 if groups == 0 else 4096), _spread(rng, 64, 8192 if groups == 0 else 4096, 16)
        rows = _spread(rng, max(1, groups // 4), min(16384, 8192 ** 3 // (n * k)))
        case = _product("", groups=groups, rows=rows, n=n, k=k, out=rng.choice(["bf16", "bf16", "f32"]),
                        skew=rng.choice([0.0, 0.5, 1.0]), bias=rng.random() < 0.3, relu=rng.random() < 0.3)
    del case["name"]
    return case


# ------------------------------------------------------------------------------------ inputs
def _dtype(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _live_tokens(case):
    return case["tokens"] - (case["tokens"] // 16 if case.get("masked") else 0)


def _loads(case):
    """Rows of each group: shares falling as 1 / rank^skew, the same for every seed up to their order."""
    share = [(g + 1.0) ** -case["skew"] for g in range(max(1, case["groups"]))]
    total = sum(share)
    want = [case["rows"] * v / total for v in share]
    rows = [int(v) for v in want]
    order = sorted(range(len(rows)), key=lambda g: rows[g] - want[g])
    for g in order[:case["rows"] - sum(rows)]:
        rows[g] += 1
    return rows


def _route_inputs(case, gen):
    """Logits with a spread of means, as a router in training gives; a bias of whole update steps of 0.001; padding rows that hold
    what memory held, and experts that a token may not use."""
    t, e = case["tokens"], case["experts"]
    x = torch.randn(t, e, generator=gen, device="cuda") + 0.5 * torch.randn(e, generator=gen, device="cuda")
    s = {"mask": None, "bias": None}
    if case["masked"]:
        mask = torch.ones(t, dtype=torch.uint8, device="cuda")
        mask[torch.randperm(t, generator=gen, device="cuda")[:t - _live_tokens(case)]] = 0
        x = x.masked_fill(torch.rand(t, e, generator=gen, device="cuda") < 0.1, float("-inf"))
        x[mask == 0] = float("nan")
        s["mask"] = mask
    s["logits"] = x.to(_dtype(case["dtype"]))
    if case["bias"]:
        s["bias"] = 0.001 * torch.randint(-100, 101, (e,), generator=gen, device="cuda").float()
    return s


def _quantize(x):
    """int8 values and FP32 scales of the rows of x: scale = amax / 127, value = x * (127 / amax) to the nearest, ties to even.
    The quotient is one IEEE division (a number over a tensor is a reciprocal and a product in torch)."""
    amax = x.abs().amax(-1).clamp(min=TINY)
    inv = torch.div(torch.full_like(amax, INT8_MAX), amax)
    return torch.round(x * inv[..., None]).clamp(-INT8_MAX, INT8_MAX).to(torch.int8), amax / INT8_MAX


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    new = lambda *shape: torch.randn(*shape, generator=gen, device="cuda")  # noqa: E731
    if case["op"] in ("route", "route_grad"):
        s = _route_inputs(case, gen)
        if case["op"] == "route_grad":
            first = _plain_route(case, s)
            s.update(expert=first["expert"], counts=first["counts"], totals=first["totals"])
            s["d_weight"] = new(case["tokens"], case["top_k"]) / case["tokens"]
            s["d_loss"] = 0.5 + torch.rand(1, generator=gen, device="cuda")
        return s
    if case["op"] == "quantize":
        t, e, k = case["tokens"], case["experts"], case["top_k"]
        # a few channels far larger than the others, as hidden states have
        x = new(t, case["hidden"]) * torch.where(torch.rand(case["hidden"], generator=gen, device="cuda") < 0.01, 8.0, 1.0)
        s = {"x": x.to(_dtype(case["dtype"])), "row": None, "total": t * k}
        if e:
            expert = (new(t, e) + 0.5 * new(e)).topk(k, dim=1).indices.reshape(-1)
            s["row"] = torch.empty(t * k, dtype=torch.int32, device="cuda")
            s["row"][torch.argsort(expert, stable=True)] = torch.arange(t * k, dtype=torch.int32, device="cuda")
            s["row"] = s["row"].reshape(t, k)
        return s
    rows = _loads(case)
    rows = [rows[g] for g in torch.randperm(len(rows), generator=gen, device="cuda").tolist()]
    s = {"rows_host": rows, "counts": torch.tensor(rows, dtype=torch.int32, device="cuda") if case["groups"] else None, "bias": None}
    s["a"], s["a_scale"] = _quantize(new(case["rows"], case["k"]))
    b = [_quantize(0.02 * new(case["n"], case["k"])) for _ in rows]
    s["b"], s["b_scale"] = torch.cat([v for v, _ in b]), torch.cat([v for _, v in b])   # one group's N rows after another's
    if case["bias"]:
        s["bias"] = 0.1 * new(len(rows) * case["n"])
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        _prepare_own(case, s)
    return s


def _prepare_own(case, s):
    """The plan and the output buffers that a program keeps."""
    import tile_scheduled_tensor_gb300 as tst
    s["tst"], op = tst, case["op"]
    new = lambda *shape, dt=torch.float32: torch.empty(*shape, dtype=dt, device="cuda")  # noqa: E731
    if op == "product":
        s["plan"] = tst.gemm_int8_plan_create(case["rows"], case["n"], case["k"], groups=case["groups"], out_dtype=case["out"],
                                              has_bias=case["bias"], relu=case["relu"])
        s["o"] = {"d": new(case["rows"], case["n"], dt=_dtype(case["out"]))}
        return
    t, k = case["tokens"], case["top_k"]
    if op == "quantize":
        s["plan"] = tst.moe_plan_create(t, max(case["experts"], 1), k)
        s["o"] = {"rows": new(s["total"], case["hidden"], dt=torch.int8), "scales": new(s["total"])}
        return
    s["plan"] = tst.moe_plan_create(t, case["experts"], k, normalize=case["normalize"], balance_coef=COEF, score=case["score"],
                                    groups=case["groups"], top_groups=case["top_groups"], group_best=case["best"], weight_scale=case["scale"])
    if op == "route":
        s["o"] = {"expert": new(t, k, dt=torch.int32), "weight": new(t, k), "row": new(t, k, dt=torch.int32),
                  "counts": new(case["experts"], dt=torch.int32), "totals": new(2, dt=torch.int32), "loss": new(1)}
    else:
        s["o"] = {"d_logits": torch.empty_like(s["logits"])}


# ------------------------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        return _run_own(case["op"], s)
    return {"route": _plain_route, "route_grad": _plain_route_grad, "quantize": _plain_quantize, "product": _plain_product}[case["op"]](case, s)


def _run_own(op, s):
    tst, o = s["tst"], s["o"]
    if op == "product":
        tst.gemm_int8_run(s["plan"], s["a"], s["b"], o["d"], s["a_scale"], s["b_scale"], bias=s["bias"], group_rows=s["counts"])
    elif op == "quantize":
        tst.moe_dispatch(s["plan"], s["x"], s["row"], o["rows"], scales=o["scales"])
    elif op == "route":
        tst.moe_route(s["plan"], s["logits"], o["expert"], o["weight"], o["row"], o["counts"], o["totals"], o["loss"], mask=s["mask"], bias=s["bias"])
    else:
        tst.moe_route_backward(s["plan"], s["logits"], s["expert"], s["counts"], s["totals"], o["d_logits"], d_weight=s["d_weight"],
                               d_loss=s["d_loss"], mask=s["mask"])
    return o


def _open_logits(s, dt):
    """The logits as `dt`, padding rows closed, and the rows with an open expert."""
    x = s["logits"].to(dt)
    if s["mask"] is not None:
        x = torch.where(s["mask"].bool()[:, None], x, float("-inf"))
    return x, (x > float("-inf")).any(1, keepdim=True)


def _scores(case, x, live):
    """Sigmoid or softmax scores of the open logits x, in x's type; 0 where closed."""
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-x))
    e = torch.exp(x - torch.where(live, x.amax(1, keepdim=True), 0.0))
    return torch.where(live, e / e.sum(1, keepdim=True), 0.0)


def _plain_route(case, s):
    t, n_experts, k, groups = case["tokens"], case["experts"], case["top_k"], case["groups"]
    # what is compared lies close together at the borders of the choice: 64 bits
    x, live = _open_logits(s, torch.float64)
    value = _scores(case, x, live)
    if s["bias"] is not None:
        value = value + s["bias"].double()
    value = torch.where(x > float("-inf"), value, float("-inf"))
    by_group = value.reshape(t, groups, -1)
    best = by_group.topk(min(case["best"], by_group.shape[2]), dim=2).values
    total = torch.where(best[:, :, 0] > float("-inf"), torch.where(best > float("-inf"), best, 0.0).sum(2), float("-inf"))
    order = torch.sort(total, dim=1, descending=True, stable=True).indices[:, :case["top_groups"]]   # ties to the lower group
    kept = torch.zeros_like(total, dtype=torch.bool).scatter_(1, order, True)
    value = torch.where(kept[:, :, None], by_group, float("-inf")).reshape(t, n_experts)
    best, expert = torch.sort(value, dim=1, descending=True, stable=True)                            # ties to the lower expert
    best, expert = best[:, :k], expert[:, :k]
    chosen = best > float("-inf")
    # the weights and the loss in 32 bits
    x, live = _open_logits(s, torch.float32)
    score = _scores(case, x, live)
    weight = torch.where(chosen, score.gather(1, expert), 0.0)
    if case["normalize"]:
        weight = torch.where(chosen, weight / weight.sum(1, keepdim=True), 0.0)
    weight = weight * case["scale"]
    p = torch.where(live, score / score.sum(1, keepdim=True), 0.0)
    slot = torch.where(chosen, expert, n_experts).reshape(-1)
    counts = torch.zeros(n_experts + 1, dtype=torch.int32, device=x.device).scatter_add_(0, slot, torch.ones_like(slot, dtype=torch.int32))[:-1]
    row = torch.empty_like(slot, dtype=torch.int32)
    row[torch.argsort(slot, stable=True)] = torch.arange(slot.numel(), dtype=torch.int32, device=x.device)
    totals = torch.stack([counts.sum(), live.sum()]).to(torch.int32)
    share = counts / totals[0].clamp(min=1)
    loss = COEF * n_experts * (share * (p.sum(0) / totals[1].clamp(min=1))).sum()
    return {"expert": torch.where(chosen, expert, -1).to(torch.int32), "weight": weight,
            "row": torch.where(chosen, row.reshape(chosen.shape), -1), "counts": counts, "totals": totals, "loss": loss.reshape(1)}


def _plain_route_grad(case, s):
    x, live = _open_logits(s, torch.float32)
    score = _scores(case, x, live)
    all_scores = torch.where(live, score.sum(1, keepdim=True), 1.0)
    chosen = s["expert"] >= 0
    expert = s["expert"].clamp(min=0).long()
    dw = torch.where(chosen, s["d_weight"], 0.0) * case["scale"]
    factor = s["d_loss"] * (COEF * case["experts"]) / (s["totals"][0].clamp(min=1).float() * s["totals"][1].clamp(min=1).float())
    g = (s["counts"].float() * factor)[None, :]
    d = (g - (score / all_scores * g).sum(1, keepdim=True)) / all_scores   # the loss's part of the scores' gradient
    if case["normalize"]:
        w = torch.where(chosen, score.gather(1, expert), 0.0)
        z = torch.where(chosen.any(1, keepdim=True), w.sum(1, keepdim=True), 1.0)
        dw = torch.where(chosen, (dw - (w / z * dw).sum(1, keepdim=True)) / z, 0.0)
    d = d.scatter_add(1, expert, dw)
    d = d * score * (1.0 - score) if case["score"] == "sigmoid" else score * (d - (score * d).sum(1, keepdim=True))
    return {"d_logits": torch.where(x > float("-inf"), d, 0.0).to(s["logits"].dtype)}


def _plain_quantize(case, s):
    q, scales = _quantize(s["x"].float())
    if s["row"] is None:
        return {"rows": q, "scales": scales}
    rows = torch.empty(s["total"], case["hidden"], dtype=torch.int8, device="cuda")
    out = torch.empty(s["total"], device="cuda")
    at = s["row"].reshape(-1).long()
    token = torch.arange(case["tokens"], device="cuda").repeat_interleave(case["top_k"])
    rows[at], out[at] = q[token], scales[token]
    return {"rows": rows, "scales": out}


def _plain_product(case, s):
    n, k = case["n"], case["k"]
    out = torch.empty(case["rows"], n, dtype=_dtype(case["out"]), device="cuda")
    at = 0
    for g, rows in enumerate(s["rows_host"]):   # library products for each group that has rows
        if rows:
            a, b, here = s["a"][at:at + rows].float(), s["b"][g * n:(g + 1) * n].float(), slice(g * n, (g + 1) * n)
            total = torch.zeros(rows, n, dtype=torch.int32, device="cuda")
            for c in range(0, k, CHUNK):        # FP32 adds the integers of a chunk exactly
                total += torch.matmul(a[:, c:c + CHUNK], b[:, c:c + CHUNK].t()).to(torch.int32)
            z = total.float() * s["a_scale"][at:at + rows, None] * s["b_scale"][None, here]
            if s["bias"] is not None:
                z = z + s["bias"][None, here]
            out[at:at + rows] = z.clamp(min=0.0) if case["relu"] else z
        at += rows
    return {"d": out}


# ------------------------------------------------------------------------------------ floors
def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2}
    if op == "product":
        m, n, k = case["rows"], case["n"], case["k"]
        used = sum(1 for v in _loads(case) if v)
        return {"bytes": m * k + 4 * m + used * n * (k + (8 if case["bias"] else 4)) + m * n * size[case["out"]] + 4 * case["groups"], "flops": 2 * m * n * k}
    if op == "quantize":
        t, h, rows = case["tokens"], case["hidden"], case["tokens"] * case["top_k"]
        return {"bytes": t * h * size[case["dtype"]] + rows * (h + 4) + (4 * rows if case["experts"] else 0), "flops": 3 * t * h}
    t, e, k = case["tokens"], case["experts"], case["top_k"]
    if op == "route":
        return {"bytes": t * e * size[case["dtype"]] + 12 * t * k + 8 * e + (t if case["masked"] else 0), "flops": 8 * t * e}
    return {"bytes": 2 * t * e * size[case["dtype"]] + 8 * t * k + 4 * e + (t if case["masked"] else 0), "flops": 12 * t * e}


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "product":
        group = torch.repeat_interleave(torch.arange(len(s["rows_host"]), device="cuda"), torch.tensor(s["rows_host"], device="cuda"))
        out = torch.empty(case["rows"], case["n"], dtype=torch.float64, device="cuda")
        b = s["b"].reshape(len(s["rows_host"]), case["n"], case["k"])
        scale = s["b_scale"].reshape(len(s["rows_host"]), case["n"]).double()
        for g in group.unique().tolist():
            mine = group == g
            z = torch.einsum("ik,jk->ij", s["a"][mine].double(), b[g].double())
            z *= torch.outer(s["a_scale"][mine].double(), scale[g])
            if s["bias"] is not None:
                z += s["bias"].double().reshape(scale.shape)[g]
            out[mine] = torch.relu(z) if case["relu"] else z
        return {"d": out}
    if case["op"] == "quantize":   # the int8 values are whole numbers by FP32 steps; the scales have a value in 64 bits
        scale = torch.linalg.vector_norm(s["x"].double(), ord=float("inf"), dim=1).clamp(min=TINY) / INT8_MAX
        if s["row"] is None:
            return {"rows": None, "scales": scale}
        out = torch.empty(s["total"], dtype=torch.float64, device="cuda")
        out.scatter_(0, s["row"].reshape(-1).long(), scale.repeat_interleave(case["top_k"]))
        return {"rows": None, "scales": out}
    return _exact_route(case, s)


def _exact_route(case, s):
    e, k, groups = case["experts"], case["top_k"], case["groups"]
    x = s["logits"].double()
    rows = torch.arange(case["tokens"], device="cuda") if s["mask"] is None else torch.nonzero(s["mask"]).reshape(-1)
    rows = rows[(x[rows] != float("-inf")).any(1)]
    x = x[rows]
    shut = x == float("-inf")
    score = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    p = score / torch.linalg.vector_norm(score, ord=1, dim=1, keepdim=True)
    if case["op"] == "route":
        v = (score if s["bias"] is None else score + s["bias"].double()).masked_fill(shut, float("-inf"))
        g = torch.sort(v.unflatten(1, (groups, -1)), dim=2, descending=True).values
        rank = g[:, :, 0]
        if case["best"] == 2 and g.shape[2] > 1:
            rank = rank + g[:, :, 1].clamp(min=0.0).where(g[:, :, 1] == float("-inf"), g[:, :, 1])
        gone = torch.argsort(rank, dim=1, descending=True, stable=True)[:, case["top_groups"]:]
        drop = torch.zeros_like(rank).scatter_(1, gone, 1.0).bool().repeat_interleave(e // groups, 1)
        v = v.masked_fill(drop, float("-inf"))
        expert = torch.argsort(v, dim=1, descending=True, stable=True)[:, :k]
        used = v.gather(1, expert) != float("-inf")
        w = score.gather(1, expert) * used
        if case["normalize"]:
            w = w / w.sum(1, keepdim=True)
        weight = torch.zeros(case["tokens"], k, dtype=torch.float64, device="cuda")
        weight[rows] = w * case["scale"]
        share = torch.bincount(expert[used], minlength=e).double() / max(1, int(used.sum()))
        loss = COEF * e * torch.dot(share, p.sum(0) / max(1, rows.numel()))
        return {"expert": None, "weight": weight, "row": None, "counts": None, "totals": None, "loss": loss.reshape(1)}
    # the gradient by the chain of log-derivatives: d log s = (1 - s) dl, or dl - <p, dl>
    expert = s["expert"][rows].long()
    used = (expert >= 0).double()
    expert = expert.clamp(min=0)
    dw = s["d_weight"][rows].double() * used * case["scale"]
    r, n = s["totals"].tolist()
    g = s["counts"].double() * (float(s["d_loss"].double()) * COEF * e / (max(1, r) * max(1, n)))
    up = p * (g - (p @ g)[:, None])                       # s dL/ds
    w = score.gather(1, expert) * used
    if case["normalize"]:
        q = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        up.scatter_add_(1, expert, q * (dw - torch.linalg.vecdot(q, dw)[:, None]))
    else:
        up.scatter_add_(1, expert, w * dw)
    d = up * (1.0 - score) if case["score"] == "sigmoid" else up - score * up.sum(1, keepdim=True)
    out = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
    out[rows] = d.masked_fill(shut, 0.0)
    return {"d_logits": out}
