"""The operators around a mixture of experts whose products run as grouped GEMMs: the router with
its balance loss and per-expert counts, the copy of tokens into the experts' order (block-scaled
e4m3 or unchanged), the block-scaled e4m3 product of every expert, and the weighted return to
token order; with the gradients of the router and of the return.

`run` takes one pass through one operator: in its plain form, elementary torch operations in
32 bits, or (`own`) through the library's entry points.  `exact` is the same in 64 bits.
"""
import math

import torch

own = False

BLOCK = 128          # elements of K per scale
E4M3_MAX = 448.0
TINY = 2.0 ** -96    # blocks whose largest magnitude is below this share its scale
COEF = 0.01          # weight of the balance loss


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token of a decoding step, through a layer of many small experts: pure latency
        _route("route_one_token", tokens=1, experts=128, top_k=8, dtype="f32", masked=False, normalize=True),
        # a padded batch of prompts with BF16 logits (many ties), some experts closed to a token
        _route("route_padded_bf16", tokens=4099, experts=60, top_k=4, dtype="bf16", masked=True, normalize=False),
        # a training micro-batch of 128 Ki tokens over 256 experts
        _route("route_train_128k", tokens=131071, experts=256, top_k=8, dtype="f32", masked=False, normalize=True),
        # its gradient: from the weights and from the balance loss
        _route("route_grad_64k", tokens=65536, experts=256, top_k=8, dtype="f32", masked=False, normalize=True, op="route_grad"),
        # sixteen tokens of a decoding batch into e4m3 rows with one scale per 128 elements
        _rows("dispatch_decode_e4m3", "dispatch", tokens=16, experts=64, top_k=8, hidden=4096, dtype="bf16", out="e4m3", masked=False),
        # a prompt batch of 16 Ki tokens, eight experts each
        _rows("dispatch_prompt_e4m3", "dispatch", tokens=16384, experts=64, top_k=8, hidden=4096, dtype="bf16", out="e4m3", masked=False),
        # a decoding batch's products: two rows per expert, every weight read once
        _product("product_decode", rows=64, experts=32, n=4096, k=4096, out="bf16", skew=0.0),
        # fine-grained experts with uneven loads (some without rows), ragged N and K
        _product("product_ragged", rows=2047, experts=60, n=1416, k=2064, out="bf16", skew=1.0),
        # the grouped benchmark's layer: 16 experts of 4096 x 4096 over 16384 rows
        _product("product_prompt", rows=16384, experts=16, n=4096, k=4096, out="bf16", skew=0.5),
        # return of a small padded batch, FP32 rows, a hidden size that is not a whole vector
        _rows("combine_small_f32", "combine", tokens=100, experts=16, top_k=2, hidden=1021, dtype="f32", out="f32", masked=True),
        # return of the prompt batch
        _rows("combine_prompt_bf16", "combine", tokens=16384, experts=64, top_k=8, hidden=4096, dtype="bf16", out="bf16", masked=False),
        # its gradient in training: every expert row's and every weight's
        _rows("combine_grad_8k", "combine_grad", tokens=8192, experts=64, top_k=8, hidden=4096, dtype="bf16", out="bf16", masked=False),
    ]


def _route(name, *, tokens, experts, top_k, dtype, masked, normalize, op="route"):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "dtype": dtype, "masked": masked, "normalize": normalize}


def _rows(name, op, *, tokens, experts, top_k, hidden, dtype, out, masked, weighted=True):
    return {"name": name, "op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "hidden": hidden, "dtype": dtype, "out": out, "masked": masked, "weighted": weighted}


def _product(name, *, rows, experts, n, k, out, skew):
    return {"name": name, "op": "product", "rows": rows, "experts": experts, "n": n, "k": k, "out": out, "skew": skew}


def _spread(rng, low, high, step=1):
    """A size between `low` and `high`, even over its logarithm, a multiple of `step`."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    v = max(low, min(high, v)) // step * step
    v = max(v, step)
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["route", "route", "route_grad", "dispatch", "dispatch", "product", "product", "product", "combine", "combine", "combine_grad"])
    if op in ("route", "route_grad"):
        most = 131071 * 256 if op == "route" else 65536 * 256
        experts = _spread(rng, 4, 512)
        top_k = rng.randint(1, min(10, experts))
        tokens = _spread(rng, 1, min(131071, most // experts))
        case = _route("", tokens=tokens, experts=experts, top_k=top_k, dtype=rng.choice(["f32", "bf16"]),
                      masked=rng.random() < 0.3, normalize=rng.random() < 0.6, op=op)
    elif op == "product":
        experts = _spread(rng, 2, 64)
        k = _spread(rng, 128, 4096, 16)
        n = _spread(rng, 128, min(4096, 16 * 4096 * 4096 // (experts * k)), 8)
        rows = _spread(rng, 1, 16384)
        case = _product("", rows=rows, experts=experts, n=n, k=k, out=rng.choice(["bf16", "bf16", "f32"]), skew=rng.choice([0.0, 0.5, 1.0]))
    else:
        dtype, top_k = rng.choice(["bf16", "bf16", "f32"]), rng.randint(1, 8)
        tokens = _spread(rng, 1, 8192 if dtype == "bf16" else 4096)
        out = dtype if op != "dispatch" or rng.random() < 0.3 else "e4m3"
        hidden = _spread(rng, 64, 4096, 16 if out == "e4m3" else rng.choice([1, 8]))
        case = _rows("", op, tokens=tokens, experts=_spread(rng, 8, 256), top_k=top_k, hidden=hidden, dtype=dtype, out=out,
                     masked=rng.random() < 0.3, weighted=op != "combine" or rng.random() < 0.7)
    del case["name"]
    if case.get("tokens", 0) * case.get("top_k", 0) == 3072:
        case["tokens"] += 1
    return case


# ------------------------------------------------------------------------------------ inputs
def _dtype(name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[name]


def _live_tokens(case):
    return case["tokens"] - (case["tokens"] // 16 if case["masked"] else 0)


def _loads(case):
    """Rows of each expert: shares falling as 1 / rank^skew, the same for every seed up to their order."""
    share = [(e + 1.0) ** -case["skew"] for e in range(case["experts"])]
    total = sum(share)
    exact_rows = [case["rows"] * v / total for v in share]
    rows = [int(v) for v in exact_rows]
    order = sorted(range(len(rows)), key=lambda e: rows[e] - exact_rows[e])
    for e in order[:case["rows"] - sum(rows)]:
        rows[e] += 1
    return rows


def _mask(case, gen):
    """One byte per token, 0 for padding."""
    if not case["masked"]:
        return None
    t = case["tokens"]
    mask = torch.ones(t, dtype=torch.uint8, device="cuda")
    mask[torch.randperm(t, generator=gen, device="cuda")[:t - _live_tokens(case)]] = 0
    return mask


def _logits(case, mask, gen):
    t, e = case["tokens"], case["experts"]
    x = torch.randn(t, e, generator=gen, device="cuda") + 0.5 * torch.randn(e, generator=gen, device="cuda")
    if case["masked"]:   # experts that a token may not use, and padding rows holding what memory held
        x = x.masked_fill(torch.rand(t, e, generator=gen, device="cuda") < 0.1, float("-inf"))
        x[mask == 0] = float("nan")
    return x.to(_dtype(case["dtype"]))


def _assign(case, mask, gen):
    """Each token's row for each of its experts in the experts' order (-1 for padding), and the number of rows."""
    t, e, k = case["tokens"], case["experts"], min(case["top_k"], case["experts"])
    like = torch.randn(t, e, generator=gen, device="cuda") + 0.5 * torch.randn(e, generator=gen, device="cuda")
    expert = like.topk(k, dim=1).indices
    if mask is not None:
        expert = torch.where(mask.bool()[:, None], expert, e)
    order = torch.argsort(expert.reshape(-1), stable=True)
    row = torch.empty(t * k, dtype=torch.int32, device="cuda")
    row[order] = torch.arange(t * k, dtype=torch.int32, device="cuda")
    total = _live_tokens(case) * k
    row = torch.where(row < total, row, -1)
    return row.reshape(t, k), total


def _blocks(x, rows, cols):
    """x (... x R x C) cut into rows x cols blocks, padded with zeros: ... x R' x rows x C' x cols."""
    r, c = x.shape[-2:]
    pr, pc = -r % rows, -c % cols
    x = torch.nn.functional.pad(x, (0, pc, 0, pr))
    return x.reshape(*x.shape[:-2], (r + pr) // rows, rows, (c + pc) // cols, cols)


def _quantize(x, rows):
    """e4m3 values and FP32 scales of x in rows x 128 blocks: scale = amax / 448, value = x * (448 / amax)."""
    b = _blocks(x, rows, BLOCK)
    amax = b.abs().amax(dim=(-3, -1)).clamp(min=TINY)
    q = (b * (E4M3_MAX / amax)[..., :, None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
    q = q.reshape(*x.shape[:-2], b.shape[-4] * rows, b.shape[-2] * BLOCK)[..., :x.shape[-2], :x.shape[-1]]
    return q.to(torch.float8_e4m3fn).contiguous(), (amax / E4M3_MAX).contiguous()


def _inputs(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    if op in ("route", "route_grad"):
        mask = _mask(case, gen)
        s = {"mask": mask, "logits": _logits(case, mask, gen)}
        if op == "route_grad":
            first = _plain_route(case, s)
            s.update(expert=first["expert"], counts=first["counts"], totals=first["totals"])
            s["d_weight"] = torch.randn(case["tokens"], case["top_k"], generator=gen, device="cuda") / case["tokens"]
            s["d_loss"] = 0.5 + torch.rand(1, generator=gen, device="cuda")
        return s
    if op == "product":
        rows = _loads(case)
        order = torch.randperm(len(rows), generator=gen, device="cuda").tolist()
        rows = [rows[e] for e in order]
        x = torch.randn(case["rows"], case["k"], generator=gen, device="cuda")
        s = {"rows_host": rows, "counts": torch.tensor(rows, dtype=torch.int32, device="cuda")}
        s["a"], s["a_scales"] = _quantize(x, 1)
        b = [_quantize(torch.randn(case["n"], case["k"], generator=gen, device="cuda") * 0.02, BLOCK) for _ in rows]
        s["b"] = torch.stack([v.view(torch.uint8) for v, _ in b]).view(torch.float8_e4m3fn)
        s["b_scales"] = torch.stack([v for _, v in b])
        return s
    mask = _mask(case, gen)
    row, total = _assign(case, mask, gen)
    t, k = row.shape
    s = {"row": row, "total": total}
    dt = _dtype(case["dtype"])
    if op in ("dispatch", "combine_grad"):
        s["x" if op == "dispatch" else "d_out"] = torch.randn(t, case["hidden"], generator=gen, device="cuda").to(dt)
    if op != "dispatch":
        s["rows"] = torch.randn(max(total, 1), case["hidden"], generator=gen, device="cuda").to(dt)
        w = torch.rand(t, k, generator=gen, device="cuda") + 0.05
        s["weight"] = w / w.sum(1, keepdim=True) if case["weighted"] else None
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
    if op == "product":
        s["plan"] = tst.gemm_grouped_plan_create(case["experts"], case["rows"], case["n"], case["k"], dtype="e4m3",
                                                 out_dtype=case["out"], ab_block=(1, BLOCK, BLOCK))
        s["d"] = torch.empty(case["rows"], case["n"], dtype=_dtype(case["out"]), device="cuda")
        return
    t, k = case["tokens"], min(case["top_k"], case["experts"])
    s["plan"] = tst.moe_plan_create(t, case["experts"], k, normalize=case.get("normalize", True), balance_coef=COEF)
    new = lambda *shape, dt=torch.float32: torch.empty(*shape, dtype=dt, device="cuda")  # noqa: E731
    if op == "route":
        s["o"] = {"expert": new(t, k, dt=torch.int32), "weight": new(t, k), "row": new(t, k, dt=torch.int32),
                  "counts": new(case["experts"], dt=torch.int32), "totals": new(2, dt=torch.int32), "loss": new(1)}
    elif op == "route_grad":
        s["o"] = {"d_logits": torch.empty_like(s["logits"])}
    elif op == "dispatch":
        s["o"] = {"rows": new(s["total"], case["hidden"], dt=_dtype(case["out"]))}
        if case["out"] == "e4m3":
            s["o"]["scales"] = new(s["total"], -(-case["hidden"] // BLOCK))
    elif op == "combine":
        s["o"] = {"out": new(t, case["hidden"], dt=_dtype(case["out"]))}
    else:
        s["o"] = {"d_rows": torch.empty_like(s["rows"]), "d_weight": new(t, k)}


# ------------------------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        return _run_own(op, s)
    return {"route": _plain_route, "route_grad": _plain_route_grad, "dispatch": _plain_dispatch, "product": _plain_product,
            "combine": _plain_combine, "combine_grad": _plain_combine_grad}[op](case, s)


def _run_own(op, s):
    tst = s["tst"]
    if op == "product":
        tst.gemm_grouped_run(s["plan"], s["counts"], s["a"], s["b"], s["d"], a_block_scales=s["a_scales"], b_block_scales=s["b_scales"])
        return {"d": s["d"]}
    o = s["o"]
    if op == "route":
        tst.moe_route(s["plan"], s["logits"], o["expert"], o["weight"], o["row"], o["counts"], o["totals"], o["loss"], mask=s["mask"])
    elif op == "route_grad":
        tst.moe_route_backward(s["plan"], s["logits"], s["expert"], s["counts"], s["totals"], o["d_logits"], d_weight=s["d_weight"],
                               d_loss=s["d_loss"], mask=s["mask"])
    elif op == "dispatch":
        tst.moe_dispatch(s["plan"], s["x"], s["row"], o["rows"], scales=o.get("scales"))
    elif op == "combine":
        tst.moe_combine(s["plan"], s["rows"], s["row"], o["out"], weight=s["weight"])
    else:
        tst.moe_combine_backward(s["plan"], s["rows"], s["row"], s["weight"], s["d_out"], o["d_rows"], o["d_weight"])
    return o


def _softmax(s):
    """FP32 logits with padding rows closed, their shifted exponentials and the probabilities (rows without an open expert: 0)."""
    x = s["logits"].float()
    if s["mask"] is not None:
        x = torch.where(s["mask"].bool()[:, None], x, float("-inf"))
    top = x.amax(1, keepdim=True)
    live = top > float("-inf")
    e = torch.exp(x - torch.where(live, top, 0.0))
    return x, e, torch.where(live, e / e.sum(1, keepdim=True), 0.0), live


def _plain_route(case, s):
    k, n_experts = case["top_k"], case["experts"]
    x, e, p, live = _softmax(s)
    # the k largest, ties to the lowest expert: integers in the logits' order with the expert in the low digits
    bits = (x + 0.0).view(torch.int32)
    order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64)
    order = order * n_experts + torch.arange(n_experts - 1, -1, -1, device=x.device)
    expert = n_experts - 1 - torch.remainder(order.topk(k, dim=1).values, n_experts)
    chosen = x.gather(1, expert) > float("-inf")
    weight = torch.where(chosen, (e if case["normalize"] else p).gather(1, expert), 0.0)
    if case["normalize"]:
        weight = torch.where(live, weight / weight.sum(1, keepdim=True), 0.0)
    slot = torch.where(chosen, expert, n_experts).reshape(-1)
    counts = torch.zeros(n_experts + 1, dtype=torch.int32, device=x.device).scatter_add_(0, slot, torch.ones_like(slot, dtype=torch.int32))[:-1]
    row = torch.empty_like(slot, dtype=torch.int32)
    row[torch.argsort(slot, stable=True)] = torch.arange(slot.numel(), dtype=torch.int32, device=x.device)
    totals = torch.stack([counts.sum(), live.sum()]).to(torch.int32)
    share = counts / totals[0].clamp(min=1)
    mean = p.sum(0) / totals[1].clamp(min=1)
    loss = COEF * n_experts * (share * mean).sum()
    return {"expert": torch.where(chosen, expert, -1).to(torch.int32), "weight": weight,
            "row": torch.where(chosen, row.reshape(chosen.shape), -1), "counts": counts, "totals": totals, "loss": loss.reshape(1)}


def _plain_route_grad(case, s):
    x, e, p, live = _softmax(s)
    chosen = s["expert"] >= 0
    expert = s["expert"].clamp(min=0).long()
    dw = torch.where(chosen, s["d_weight"], 0.0)
    scale = s["d_loss"] * (COEF * case["experts"]) / (s["totals"][0].clamp(min=1).float() * s["totals"][1].clamp(min=1).float())
    g = (s["counts"].float() * scale)[None, :]
    if case["normalize"]:
        w = torch.where(chosen, e.gather(1, expert), 0.0)
        w = torch.where(live, w / w.sum(1, keepdim=True), 0.0)
        d = p * (g - (p * g).sum(1, keepdim=True))
        d = d.scatter_add(1, expert, w * (dw - (w * dw).sum(1, keepdim=True)))
    else:
        g = g.expand_as(p).scatter_add(1, expert, dw)
        d = p * (g - (p * g).sum(1, keepdim=True))
    return {"d_logits": d.to(s["logits"].dtype)}


def _place(v, s):
    """v (T x k x ...) at its rows; what has no row goes to one more row that is left out."""
    at = torch.where(s["row"] >= 0, s["row"], s["total"]).reshape(-1).long()
    out = torch.empty(s["total"] + 1, v.shape[-1], dtype=v.dtype, device=v.device)
    out.index_copy_(0, at, v.reshape(-1, v.shape[-1]))
    return out[:s["total"]]


def _plain_dispatch(case, s):
    t, k = s["row"].shape
    each = lambda v: v[:, None, :].expand(t, k, v.shape[1])  # noqa: E731
    if case["out"] != "e4m3":
        return {"rows": _place(each(s["x"]), s)}
    q, scales = _quantize(s["x"].float(), 1)
    return {"rows": _place(each(q.view(torch.uint8)), s).view(torch.float8_e4m3fn), "scales": _place(each(scales), s)}


def _spread_scales(v, rows, n, k):
    return v.repeat_interleave(rows, 0)[:n].repeat_interleave(BLOCK, 1)[:, :k]


def _plain_product(case, s):
    n, k = case["n"], case["k"]
    a = s["a"].float() * _spread_scales(s["a_scales"], 1, case["rows"], k)
    out = torch.empty(case["rows"], n, dtype=torch.float32, device="cuda")
    at = 0
    for g, rows in enumerate(s["rows_host"]):   # one library product per expert that has rows
        if rows:
            b = s["b"][g].float() * _spread_scales(s["b_scales"][g], BLOCK, n, k)
            torch.matmul(a[at:at + rows], b.t(), out=out[at:at + rows])
        at += rows
    return {"d": out.to(_dtype(case["out"]))}


def _gathered(s):
    """The FP32 rows of every token (T x k x H), 0 where it has none."""
    return torch.where((s["row"] >= 0)[:, :, None], s["rows"][s["row"].clamp(min=0).long()].float(), 0.0)


def _plain_combine(case, s):
    v = _gathered(s)
    if s["weight"] is not None:
        v = v * s["weight"][:, :, None]
    return {"out": v.sum(1).to(_dtype(case["out"]))}


def _plain_combine_grad(case, s):
    d = s["d_out"].float()
    d_rows = _place((s["weight"][:, :, None] * d[:, None, :]).to(s["rows"].dtype), s)
    d_weight = (_gathered(s) * d[:, None, :]).sum(2)
    return {"d_rows": d_rows, "d_weight": d_weight}


# ------------------------------------------------------------------------------------ floors
def work(case):
    op, size = case["op"], {"f32": 4, "bf16": 2, "e4m3": 1}
    if op == "product":
        m, n, k = case["rows"], case["n"], case["k"]
        used = sum(1 for v in _loads(case) if v)
        blocks = -(-k // BLOCK)
        return {"bytes": m * k + 4 * m * blocks + used * (n * k + 4 * -(-n // BLOCK) * blocks) + m * n * size[case["out"]] + 4 * case["experts"],
                "flops": 2 * m * n * k}
    t, e, k = case["tokens"], case["experts"], min(case["top_k"], case["experts"])
    if op == "route":
        return {"bytes": t * e * size[case["dtype"]] + 12 * t * k + 4 * e + (t if case["masked"] else 0), "flops": 5 * t * e}
    if op == "route_grad":
        return {"bytes": 2 * t * e * size[case["dtype"]] + 8 * t * k + 4 * e + (t if case["masked"] else 0), "flops": 9 * t * e}
    h, rows = case["hidden"], _live_tokens(case) * k
    into, out = size[case["dtype"]], size[case["out"]]
    if op == "dispatch":
        live = _live_tokens(case)
        return {"bytes": live * h * into + rows * h * out + (4 * rows * -(-h // BLOCK) if case["out"] == "e4m3" else 0) + 4 * t * k, "flops": 3 * live * h}
    if op == "combine":
        return {"bytes": rows * h * into + t * h * out + (8 if case["weighted"] else 4) * t * k, "flops": 2 * rows * h}
    return {"bytes": 2 * rows * h * into + t * h * into + 12 * t * k, "flops": 3 * rows * h}


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "product":
        out = torch.empty(case["rows"], case["n"], dtype=torch.float64, device="cuda")
        kb = torch.arange(case["k"], device="cuda") // BLOCK
        nb = torch.arange(case["n"], device="cuda") // BLOCK
        at = 0
        for g, rows in enumerate(s["rows_host"]):
            a = s["a"][at:at + rows].double() * s["a_scales"][at:at + rows].double()[:, kb]
            b = s["b"][g].double() * s["b_scales"][g].double()[nb][:, kb]
            out[at:at + rows] = torch.einsum("ik,jk->ij", a, b)
            at += rows
        return {"d": out}
    if op in ("route", "route_grad"):
        return _exact_route(case, s)
    at = s["row"].reshape(-1).long()
    has = at >= 0
    token = torch.arange(case["tokens"], device="cuda").repeat_interleave(s["row"].shape[1])[has]
    at = at[has]
    if op == "dispatch":
        source = torch.empty(s["total"], dtype=torch.long, device="cuda")
        source[at] = token
        x = s["x"].double()
        if case["out"] != "e4m3":
            return {"rows": x[source]}
        pad = torch.nn.functional.pad(x, (0, -case["hidden"] % BLOCK)).unflatten(1, (-1, BLOCK))
        scale = pad.abs().amax(2).clamp(min=TINY) / E4M3_MAX
        v = (pad / scale[:, :, None]).flatten(1)[:, :case["hidden"]]
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)   # e4m3: 3 mantissa bits, least exponent -6
        return {"rows": (torch.round(v / step) * step)[source], "scales": scale[source]}
    if op == "combine":
        out = torch.zeros(case["tokens"], case["hidden"], dtype=torch.float64, device="cuda")
        w = torch.ones(at.numel(), device="cuda") if s["weight"] is None else s["weight"].reshape(-1)[has]
        for part in torch.arange(at.numel(), device="cuda").split(16384):
            out.index_add_(0, token[part], s["rows"][at[part]].double() * w[part].double()[:, None])
        return {"out": out}
    d_rows = torch.empty(s["rows"].shape, dtype=torch.float64, device="cuda")
    d_weight = torch.zeros(s["weight"].numel(), dtype=torch.float64, device="cuda")
    where = torch.nonzero(has).reshape(-1)
    for part in torch.arange(at.numel(), device="cuda").split(16384):
        d = s["d_out"][token[part]].double()
        d_rows[at[part]] = d * s["weight"].reshape(-1)[where[part]].double()[:, None]
        d_weight[where[part]] = torch.linalg.vecdot(d, s["rows"][at[part]].double())
    return {"d_rows": d_rows, "d_weight": d_weight.reshape(s["weight"].shape)}


def _exact_route(case, s):
    n_experts = case["experts"]
    x = s["logits"].double()
    if s["mask"] is not None:
        x[s["mask"] == 0] = float("-inf")
    open_rows = torch.isfinite(x).any(1)
    logp = x[open_rows] - torch.logsumexp(x[open_rows], 1, keepdim=True)
    p = torch.exp(logp)
    if case["op"] == "route":
        best, expert = torch.sort(x[open_rows], dim=1, descending=True, stable=True)
        best, expert = best[:, :case["top_k"]], expert[:, :case["top_k"]]
        w = torch.softmax(best, 1) if case["normalize"] else torch.exp(logp.gather(1, expert))
        weight = torch.zeros(case["tokens"], case["top_k"], dtype=torch.float64, device="cuda")
        weight[open_rows] = w
        used = expert[best > float("-inf")]
        share = torch.bincount(used, minlength=n_experts).double() / max(1, used.numel())
        loss = COEF * n_experts * torch.dot(share, p.sum(0) / max(1, p.shape[0]))
        return {"expert": None, "weight": weight, "row": None, "counts": None, "totals": None, "loss": loss.reshape(1)}
    expert = s["expert"][open_rows].long()
    used = (expert >= 0).double()
    expert = expert.clamp(min=0)
    dw = s["d_weight"][open_rows].double() * used
    rows, live = s["totals"].tolist()
    g = s["counts"].double() * (float(s["d_loss"].double()) * COEF * n_experts / (max(1, rows) * max(1, live)))
    d = p * (g - (p @ g)[:, None])
    if case["normalize"]:
        w = torch.exp(logp.gather(1, expert)) * used
        w = w / w.sum(1, keepdim=True)
        back = w * (dw - (w * dw).sum(1, keepdim=True))
        d.scatter_add_(1, expert, back)
    else:
        ps = p.gather(1, expert) * used
        d = d - p * (ps * dw).sum(1, keepdim=True)
        d.scatter_add_(1, expert, ps * dw)
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")
    out[open_rows] = d
    return {"d_logits": out}
