"""Cases of the operators around the compressed projections, and their plain form.

Four operators, chosen by a case's ``op``:

* ``route``: router logits to each token's experts and their weights;
* ``dispatch``: rows grouped by expert (a stable counting sort) and the
  activations copied to their experts' rows;
* ``combine``: the experts' output rows weighted and summed back per token;
* ``lora``: many requests' low-rank adapters beside one or two projections
  that read the same activations.

``run`` computes them from elementary torch operations, or, where ``own`` is
true, makes the calls of this package that a serving program makes.
"""
import torch

own = False

NONE = -1  # an entry without an expert, a token without an adapter

# The projection shapes are those of bench.py's 8B-shaped layer (hidden 4096,
# intermediate 14336); 8 experts with 2 per token are its --moe settings.


def listed():
    return [
        # one decode step of one request: latency only
        dict(name="route-1x8", op="route", tokens=1, experts=8, top_k=2, score="softmax", bias=False, groups=1,
             top_groups=1, pairs=False, renorm=True, scale=1.0, dtype="f32", pad=0, masked=False),
        # a decode batch on a many-expert layer with a balance bias and expert groups
        dict(name="route-64x256-groups", op="route", tokens=64, experts=256, top_k=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, pairs=True, renorm=True, scale=2.5, dtype="f32", pad=0, masked=False),
        # a prompt chunk, bf16 logits cut out of a wider row, some experts switched off per token
        dict(name="route-4099x60-bf16", op="route", tokens=4099, experts=60, top_k=4, score="softmax", bias=False,
             groups=1, top_groups=1, pairs=False, renorm=False, scale=1.0, dtype="bf16", pad=4, masked=True),
        # the largest prompt batch on the many-expert layer
        dict(name="route-16384x256-groups", op="route", tokens=16384, experts=256, top_k=8, score="sigmoid", bias=True,
             groups=8, top_groups=4, pairs=True, renorm=True, scale=2.5, dtype="f32", pad=0, masked=False),
        # a decode batch over 8 experts, 2 per token
        dict(name="dispatch-64x4096", op="dispatch", tokens=64, experts=8, top_k=2, cols=4096, pad=0, dropped=0.0),
        # a long prompt over many experts, some entries without an expert
        dict(name="dispatch-8191x2048-of-256", op="dispatch", tokens=8191, experts=256, top_k=8, cols=2048, pad=64,
             dropped=0.03),
        # the way back of the decode batch, onto a shared branch's output
        dict(name="combine-64x4096", op="combine", tokens=64, top_k=2, cols=4096, base=True, out="f32", dropped=0.0),
        # the way back of the long prompt, rounded for the next layer's product
        dict(name="combine-8191x2048-bf16", op="combine", tokens=8191, top_k=8, cols=2048, base=False, out="bf16",
             dropped=0.03),
        # one request with an adapter on gate and up, one token
        dict(name="lora-1tok-gate-up", op="lora", tokens=1, slots=4, max_rank=16, ragged=False, rows=14336, cols=4096,
             projections=2, runs=False, without=0.0),
        # a decode batch in which every request has an adapter of its own, gate and up
        dict(name="lora-64tok-64adapters-gate-up", op="lora", tokens=64, slots=64, max_rank=16, ragged=False,
             rows=14336, cols=4096, projections=2, runs=False, without=0.0),
        # prompts and decode tokens mixed on the down projection: ragged ranks, some requests without an adapter
        dict(name="lora-777tok-ragged-down", op="lora", tokens=777, slots=23, max_rank=64, ragged=True, rows=4096,
             cols=14336, projections=1, runs=True, without=0.15),
        # long prompts of few requests on the gate projection
        dict(name="lora-8192tok-gate", op="lora", tokens=8192, slots=8, max_rank=64, ragged=True, rows=14336,
             cols=4096, projections=1, runs=True, without=0.1),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "lora"])
    if op == "route":
        experts = rng.choice([4, 8, 16, 60, 64, 96, 128, 160, 256, 384, 512])
        tokens = _log(rng, 1, 16384 * 256 // max(256, experts))
        groups = rng.choice([g for g in (1, 1, 2, 4, 8) if experts % g == 0 and experts // g >= 2])
        top_groups = rng.randint(1, groups)
        top_k = rng.randint(1, min(16, experts // groups * top_groups))
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, score=rng.choice(["softmax", "sigmoid"]),
                    bias=rng.random() < 0.5, groups=groups, top_groups=top_groups, pairs=rng.random() < 0.5,
                    renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "f32", "bf16"]),
                    pad=rng.choice([0, 0, 1, 4]), masked=rng.random() < 0.3)
    if op in ("dispatch", "combine"):
        cols = 64 * _log(rng, 4, 112)
        top_k = rng.randint(1, 8)
        tokens = _log(rng, 1, 8191 * 2048 * 8 // (cols * max(4, top_k) * 2))
        case = dict(op=op, tokens=tokens, top_k=top_k, cols=cols, dropped=rng.choice([0.0, 0.03, 0.3]))
        if op == "dispatch":
            case.update(experts=rng.choice([e for e in (8, 16, 60, 64, 128, 256) if e >= top_k]),
                        pad=rng.choice([0, 0, 8, 64]))
        else:
            case.update(base=rng.random() < 0.5, out=rng.choice(["f32", "bf16"]))
        return case
    rows, cols = 16 * _log(rng, 16, 896), 64 * _log(rng, 4, 224)
    projections = rng.randint(1, 2)
    tokens = _log(rng, 1, min(8192, 8192 * 14336 * 4096 // (projections * max(rows, 2048) * max(cols, 4096))))
    return dict(op=op, tokens=tokens, slots=_log(rng, 1, 64 if tokens <= 1024 else 8),
                max_rank=rng.choice([4, 8, 16, 24, 32, 64]), ragged=rng.random() < 0.5, rows=rows, cols=cols,
                projections=projections, runs=rng.random() < 0.6, without=rng.choice([0.0, 0.0, 0.15]))


def _ranks(case):
    r = case["max_rank"]
    return [max(1, (r, r // 2, r - 3, r // 4 + 1)[i % 4]) if case["ragged"] else r for i in range(case["slots"])]


def work(case):
    t = case["tokens"]
    if case["op"] == "route":
        size = 4 if case["dtype"] == "f32" else 2
        e = case["experts"]
        return {"bytes": t * e * size + (4 * e if case["bias"] else 0) + 8 * t * case["top_k"], "flops": 4 * t * e}
    if case["op"] == "dispatch":
        n = t * case["top_k"]
        rows = n * (1 - case["dropped"])
        return {"bytes": 2 * case["cols"] * (t + rows) + 12 * n + 4 * case["experts"], "flops": 0}
    if case["op"] == "combine":
        n = t * case["top_k"]
        rows = n * (1 - case["dropped"])
        out = (4 if case["out"] == "f32" else 2) + (4 if case["base"] else 0)
        return {"bytes": case["cols"] * (4 * rows + out * t) + 8 * n, "flops": 2 * rows * case["cols"]}
    with_adapter = max(1, round(t * (1 - case["without"])))
    ranks = _ranks(case)
    used = ranks[:min(len(ranks), with_adapter)]
    p, k, n = case["projections"], case["cols"], case["rows"]
    mean = sum(ranks) / len(ranks)
    return {"bytes": 2 * t * k + p * (2 * sum(used) * (k + n) + 8 * t * n) + 4 * t,
            "flops": p * 2 * with_adapter * mean * (k + n)}


# ---- inputs ----


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _choices(case, g, experts):
    """Distinct experts per token, some far more popular than others, the best first; NONE where dropped."""
    t, k = case["tokens"], case["top_k"]
    popular = torch.randn(experts, generator=g, device="cuda")
    noise = torch.rand((t, experts), generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
    index = (popular - torch.log(-torch.log(noise))).argsort(dim=1, descending=True)[:, :k].to(torch.int32)
    if case["dropped"]:
        gone = torch.rand((t, k), generator=g, device="cuda") < case["dropped"]
        index = torch.where(gone, NONE, index)
    return index.contiguous()


def prepare(case, seed):
    g = _generator(seed)
    dev = "cuda"
    t = case["tokens"]
    s = {"case": case}
    if case["op"] == "route":
        e = case["experts"]
        wide = torch.randn((t, e + case["pad"]), generator=g, device=dev) * 1.5
        if case["masked"]:  # a quarter of the tokens may use half of the experts, one in 64 none at all
            some = torch.rand((t, 1), generator=g, device=dev)
            off = (some < 0.25) & (torch.rand(wide.shape, generator=g, device=dev) < 0.5) | (some < 1 / 64)
            wide = wide.masked_fill(off, float("-inf"))
        s["logits"] = wide.to(torch.float32 if case["dtype"] == "f32" else torch.bfloat16)[:, :e]
        s["bias"] = torch.randn(e, generator=g, device=dev) * 0.1 if case["bias"] else None
        if own:
            s["experts"] = torch.empty((t, case["top_k"]), dtype=torch.int32, device=dev)
            s["weights"] = torch.empty((t, case["top_k"]), dtype=torch.float32, device=dev)
    elif case["op"] == "dispatch":
        n, c = t * case["top_k"], case["cols"]
        s["index"] = _choices(case, g, case["experts"])
        s["x"] = torch.randn((t, c + case["pad"]), generator=g, device=dev).to(torch.bfloat16)[:, :c]
        if own:
            import decode_gemm_bf16_amd as uw
            s["offsets"] = torch.empty(case["experts"] + 1, dtype=torch.int32, device=dev)
            s["order"] = torch.empty(n, dtype=torch.int32, device=dev)
            s["slot"] = torch.empty((t, case["top_k"]), dtype=torch.int32, device=dev)
            s["xs"] = torch.zeros((n, c), dtype=torch.bfloat16, device=dev)  # rows without an entry stay as they are
            s["work"] = torch.empty(uw.group_rows_workspace_bytes(n, case["experts"]), dtype=torch.uint8, device=dev)
    elif case["op"] == "combine":
        k, c = case["top_k"], case["cols"]
        n = t * k
        there = torch.rand((t, k), generator=g, device=dev) >= case["dropped"]
        place = torch.randperm(n, generator=g, device=dev).reshape(t, k)  # where a sort by expert put the entries
        s["slot"] = torch.where(there, place, NONE).to(torch.int32).contiguous()
        s["weights"] = torch.rand((t, k), generator=g, device=dev)
        s["ys"] = torch.randn((n, c), generator=g, device=dev)
        s["base"] = torch.randn((t, c), generator=g, device=dev) if case["base"] else None
        if own:
            s["y"] = torch.empty((t, c), dtype=torch.float32 if case["out"] == "f32" else torch.bfloat16, device=dev)
    else:
        k, n, slots, r = case["cols"], case["rows"], case["slots"], case["max_rank"]
        ranks = _ranks(case)
        if case["runs"]:  # tokens of one request stand together, requests of all lengths
            cuts = (torch.rand(slots - 1, generator=g, device=dev) * t).sort()[0]
            index = torch.searchsorted(cuts, torch.arange(t, device=dev, dtype=torch.float32), right=True)
            index = torch.randperm(slots, generator=g, device=dev)[index]
        else:  # every adapter is used where there are tokens enough
            index = (torch.arange(t, device=dev) % slots)[torch.randperm(t, generator=g, device=dev)]
        if case["without"]:
            index = torch.where(torch.rand(t, generator=g, device=dev) < case["without"], NONE, index)
        s["index"] = index.to(torch.int32)
        s["x"] = torch.randn((t, k), generator=g, device=dev).to(torch.bfloat16)
        s["base"] = [torch.randn((t, n), generator=g, device=dev) for _ in range(case["projections"])]
        # [slots, r, cols] and [slots, rows, r]; ranks beyond an adapter's own are zero
        live = torch.arange(r, device=dev) < torch.tensor(ranks, device=dev)[:, None]
        s["a"], s["b"] = [], []
        for _ in range(case["projections"]):
            a = torch.randn((slots, r, k), generator=g, device=dev) * live[:, :, None] / k ** 0.5
            b = torch.randn((slots, n, r), generator=g, device=dev) * live[:, None, :] * 0.3
            s["a"].append(a.to(torch.bfloat16))
            s["b"].append(b.to(torch.bfloat16))
        s["scale"] = torch.tensor([0.5 + i % 4 * 0.5 for i in range(slots)], device=dev)
        if own:
            import decode_gemm_bf16_amd as uw
            s["adapters"] = []
            for a, b in zip(s["a"], s["b"]):
                h = uw.Adapters(slots, n, k, r)
                for i, rank in enumerate(ranks):
                    h.load(i, a[i, :rank].contiguous(), b[i, :, :rank].contiguous(), 0.5 + i % 4 * 0.5)
                s["adapters"].append(h)
            s["y"] = [torch.empty_like(b) for b in s["base"]]
            s["plan"] = torch.empty(uw.lora_plan_bytes(t, slots), dtype=torch.uint8, device=dev)
            s["work"] = torch.empty(uw.lora_workspace_bytes(s["adapters"], t), dtype=torch.uint8, device=dev)
            del s["a"], s["b"]
    return s


# ---- one pass ----


def run(s):
    case = s["case"]
    if own:
        return {"route": _own_route, "dispatch": _own_dispatch, "combine": _own_combine, "lora": _own_lora}[case["op"]](s)
    return {"route": _route, "dispatch": _dispatch, "combine": _combine, "lora": _lora}[case["op"]](s)


def _own_route(s):
    import decode_gemm_bf16_amd as uw
    c = s["case"]
    uw.route(s["logits"], s["experts"], s["weights"],
             score=uw.SCORE_SIGMOID if c["score"] == "sigmoid" else uw.SCORE_SOFTMAX, bias=s["bias"],
             groups=c["groups"], top_groups=c["top_groups"], group_score=uw.GROUP_TOP2 if c["pairs"] else uw.GROUP_MAX,
             renormalise=c["renorm"], scale=c["scale"])
    return {"experts": s["experts"], "weights": s["weights"]}


def _own_dispatch(s):
    import decode_gemm_bf16_amd as uw
    uw.group_rows(s["index"], s["case"]["experts"], s["offsets"], s["order"], s["slot"], s["work"])
    uw.dispatch_rows(s["x"], s["slot"], s["xs"])
    return {"offsets": s["offsets"], "order": s["order"], "slot": s["slot"], "xs": s["xs"]}


def _own_combine(s):
    import decode_gemm_bf16_amd as uw
    uw.combine_rows(s["ys"], s["slot"], s["weights"], s["y"], base=s["base"])
    return {"y": s["y"]}


def _own_lora(s):
    import decode_gemm_bf16_amd as uw
    uw.lora_plan(s["index"], s["case"]["slots"], s["plan"])
    uw.lora_apply(s["adapters"], s["plan"], s["x"], s["y"], s["work"], bases=s["base"])
    return {"y": s["y"]}


def _route(s):
    c = s["case"]
    # 64 bits: a choice between two experts must not hang on a rounding
    low = float("-inf")
    logits = s["logits"].double()
    if c["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-logits))
    else:
        top = logits.amax(dim=1, keepdim=True)
        e = torch.where(logits > low, torch.exp(logits - torch.where(top > low, top, 0.0)), 0.0)
        total = e.sum(dim=1, keepdim=True)
        score = e / torch.where(total > 0, total, 1.0)
    valued = score + s["bias"].double() if c["bias"] else score
    choice = torch.where(logits > low, valued if c["bias"] else logits, low)
    if c["groups"] > 1:
        t, e = choice.shape
        value = torch.where(logits > low, valued, low) if c["pairs"] else choice
        best = value.reshape(t, c["groups"], e // c["groups"]).sort(dim=2, descending=True)[0]
        merit = best[:, :, 0] + torch.where(best[:, :, 1] > low, best[:, :, 1], 0.0) if c["pairs"] else best[:, :, 0]
        rank = merit.sort(dim=1, descending=True, stable=True)[1]
        kept = torch.zeros_like(merit, dtype=torch.bool).scatter_(1, rank[:, :c["top_groups"]], True)
        choice = torch.where(kept.repeat_interleave(e // c["groups"], dim=1), choice, low)
    value, index = choice.sort(dim=1, descending=True, stable=True)
    value, index = value[:, :c["top_k"]], index[:, :c["top_k"]]
    chosen = value > low
    weight = torch.where(chosen, score.gather(1, index), 0.0)
    if c["renorm"]:
        total = weight.sum(dim=1, keepdim=True)
        weight = weight / torch.where(total > 0, total, 1.0)
    return {"experts": torch.where(chosen, index, NONE).to(torch.int32), "weights": (weight * c["scale"]).float()}


def _dispatch(s):
    c = s["case"]
    index = s["index"].reshape(-1)
    n, experts = index.numel(), c["experts"]
    label = torch.where(index >= 0, index, experts)
    order = label.sort(stable=True)[1]
    counts = (index[:, None] == torch.arange(experts, device=index.device)).sum(dim=0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    slot = torch.empty_like(order)
    slot[order] = torch.arange(n, device=index.device)
    slot = torch.where(index >= 0, slot, NONE).reshape(c["tokens"], c["top_k"])
    there = label[order] < experts
    xs = torch.where(there[:, None], s["x"][order // c["top_k"]], 0.0)
    return {"offsets": offsets.to(torch.int32), "order": order.to(torch.int32), "slot": slot.to(torch.int32), "xs": xs}


def _combine(s):
    slot = s["slot"].long()
    rows = s["ys"][slot.clamp(min=0)]
    y = torch.where((slot >= 0)[:, :, None], s["weights"][:, :, None] * rows, 0.0).sum(dim=1)
    if s["base"] is not None:
        y = s["base"] + y
    return {"y": y.to(torch.float32 if s["case"]["out"] == "f32" else torch.bfloat16)}


def _lora(s):
    c = s["case"]
    x = s["x"].float()
    # every token against every adapter's ranks, and zero where the adapter is not the token's
    mine = s["index"][:, None] == torch.arange(c["slots"], device=x.device)
    factor = mine * s["scale"]
    ys = []
    for a, b, base in zip(s["a"], s["b"], s["base"]):
        v = (x @ a.float().reshape(-1, c["cols"]).t()).reshape(c["tokens"], c["slots"], -1) * factor[:, :, None]
        ys.append(base + v.reshape(c["tokens"], -1) @ b.float().permute(0, 2, 1).reshape(-1, c["rows"]))
    return {"y": ys}


# ---- the definition, in 64 bits ----


def _inputs(case, seed):
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "dispatch":
        return {"offsets": None, "order": None, "slot": None, "xs": _exact_rows(case, s)}
    if case["op"] == "combine":
        y = torch.zeros((case["tokens"], case["cols"]), dtype=torch.float64, device="cuda")
        for j in range(case["top_k"]):
            slot = s["slot"][:, j].long()
            t = (slot >= 0).nonzero()[:, 0]
            y[t] += s["weights"][t, j, None].double() * s["ys"][slot[t]].double()
        return {"y": y if s["base"] is None else y + s["base"].double()}
    ys = []
    for a, b, base in zip(s["a"], s["b"], s["base"]):
        y = base.double()
        for i in range(case["slots"]):
            t = (s["index"] == i).nonzero()[:, 0]
            if t.numel():
                delta = s["x"][t].double() @ a[i].double().t().contiguous()
                y[t] += float(s["scale"][i]) * (delta @ b[i].double().t().contiguous())
        ys.append(y)
    return {"y": ys}


def _exact_rows(case, s):
    index = s["index"].reshape(-1).cpu()
    xs = torch.zeros((index.numel(), case["cols"]), dtype=torch.float64, device="cuda")
    at = 0
    for e in range(case["experts"]):
        rows = (index == e).nonzero()[:, 0].cuda() // case["top_k"]
        xs[at:at + rows.numel()] = s["x"][rows].double()
        at += rows.numel()
    return xs


def _exact_route(case, s):
    """The weights of the chosen experts, on the host, by choosing one expert after the other."""
    logits = s["logits"].cpu().double()
    live = logits > float("-inf")
    if case["score"] == "sigmoid":
        score = torch.special.expit(logits)
    else:
        score = torch.exp(logits - torch.logsumexp(logits, dim=1, keepdim=True)).nan_to_num(0.0)
    value = score + s["bias"].cpu().double() if case["bias"] else logits
    merit = score + s["bias"].cpu().double() if case["bias"] else score
    value = value.masked_fill(~live, float("-inf"))
    per = case["experts"] // case["groups"]
    if case["groups"] > 1:
        members = (merit if case["pairs"] else value).masked_fill(~live, float("-inf"))
        members = members.reshape(-1, case["groups"], per)
        first = members.amax(dim=2)
        if case["pairs"]:
            rest = members.scatter(2, members.argmax(dim=2, keepdim=True), float("-inf")).amax(dim=2)
            first = first + rest.masked_fill(rest == float("-inf"), 0.0)
        open_ = torch.zeros_like(first, dtype=torch.bool)
        for _ in range(case["top_groups"]):
            g = first.argmax(dim=1, keepdim=True)
            open_.scatter_(1, g, True)
            first = first.scatter(1, g, float("-inf"))
        value = value.masked_fill(~open_.repeat_interleave(per, dim=1), float("-inf"))
    chosen, weights = [], []
    for _ in range(case["top_k"]):
        best, e = value.max(dim=1, keepdim=True)
        there = best > float("-inf")
        chosen.append(torch.where(there, e, NONE))
        weights.append(torch.where(there, score.gather(1, e), 0.0))
        value = value.scatter(1, e, float("-inf"))
    w = torch.cat(weights, dim=1)
    if case["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).masked_fill(w.sum(dim=1, keepdim=True) == 0, 1.0)
    return {"experts": torch.cat(chosen, dim=1).to(torch.int32), "weights": w * case["scale"]}
