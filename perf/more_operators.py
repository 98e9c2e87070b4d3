"""Cases of the operators around a paged cache of keys and values, and their plain form.

Four operators, chosen by a case's ``op``:

* ``write``: queries and keys turned by their rotary positions (one or several
  axes), keys and values written to the cache's pages;
* ``attend``: attention of each sequence's new tokens over its pages: prompts,
  chunks of prompts, single tokens and trees of drafted tokens;
* ``copy``: pages copied within the cache, all layers at once;
* ``keep``: the rows of accepted drafted tokens moved to their places, all layers
  at once.

``run`` computes them from elementary torch operations, or, where ``own`` is
true, makes the calls of this package that a serving program makes.

A cache is two bfloat16 tensors [layers, pages, kv_heads, page, dim].  Within a
page of one head, element d of the key at place o stands at
((o / 32 * dim / 8 + d / 8) * 32 + o % 32) * 8 + d % 8, that of the value at
((o / 16 * 2 + o / 4 % 2) * dim + d) * 8 + o / 8 % 2 * 4 + o % 4.
"""
import torch

own = False

# Head layouts: 32 and 8 heads of 128 and 64 and 8 of 128 are those of the 4096 and
# 8192 wide layers that bench.py measures; the others are generic.


def listed():
    write = dict(op="write", axes=1, turned=128, adjacent=False, type="f32", padding=0.0, spread=False)
    attend = dict(op="attend", ragged=False, cap=0.0, window=0, slopes=False, prefix=0, docs=0, tree=False)
    return [
        # one decode step of one request: latency only
        dict(write, name="write-1", tokens=1, heads=32, kv_heads=8, dim=128, page=64, far=8000),
        # a long prompt of images and video (time, height, width), half of each head turned, bf16 projections
        dict(write, name="write-8191-3axes", tokens=8191, heads=32, kv_heads=8, dim=128, page=64, far=300000, axes=3,
             turned=64, adjacent=True, type="bf16"),
        # one request, one token, a short context: latency only
        dict(attend, name="attend-1x700", seqs=1, tokens=1, least=700, length=700, heads=32, kv_heads=8, dim=128, page=64),
        # a decode batch of contexts of all lengths
        dict(attend, name="attend-64x1-ragged", seqs=64, tokens=1, least=1, length=8192, heads=32, kv_heads=8, dim=128,
             page=64),
        # few requests with very long contexts
        dict(attend, name="attend-2x1-long", seqs=2, tokens=1, least=120001, length=131072, heads=64, kv_heads=8, dim=128,
             page=128),
        # verification of drafted trees, scores capped
        dict(attend, name="attend-16x61-tree", seqs=16, tokens=61, least=200, length=6000, heads=32, kv_heads=8, dim=128,
             page=64, cap=50.0, tree=True),
        # one long prompt
        dict(attend, name="attend-prompt-8192", seqs=1, tokens=8192, least=8192, length=8192, heads=32, kv_heads=8,
             dim=128, page=64),
        # chunks of prompts and single tokens mixed; small heads of their own keys, distance slopes, a window
        dict(attend, name="attend-chunks-slopes", seqs=24, tokens=700, least=700, length=3000, heads=16, kv_heads=16,
             dim=64, page=32, ragged=True, slopes=True, window=1500),
        # a fork: a long shared context gets a copy of its own, all layers
        dict(op="copy", name="copy-160-pages", layers=32, pages=400, copies=160, kv_heads=8, dim=128, page=64),
        # a fork that copies a partial page only: latency
        dict(op="copy", name="copy-1-page", layers=16, pages=64, copies=1, kv_heads=8, dim=128, page=64),
        # accepted tokens after a verification, all layers
        dict(op="keep", name="keep-1-of-8", layers=16, seqs=1, drafts=8, most=4, length=900, kv_heads=8, dim=128, page=64),
        dict(op="keep", name="keep-64-of-61", layers=32, seqs=64, drafts=61, most=7, length=4000, kv_heads=8, dim=128,
             page=64),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["write", "attend", "attend", "attend", "copy", "keep"])
    kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
    dim = rng.choice([64, 96, 128, 128, 256])
    case = dict(op=op, kv_heads=kv_heads, dim=dim, page=rng.choice([32, 64, 128, 256]))
    wide = max(1, kv_heads * dim // 1024)  # against 8 heads of 128
    if op in ("write", "attend"):
        case["heads"] = kv_heads * rng.choice([g for g in (1, 2, 3, 4, 6, 8) if g * kv_heads <= 64])
    if op == "write":
        axes = rng.randint(1, 4)
        case.update(tokens=_log(rng, 1, 8191 * 4096 // max(4096, case["heads"] * dim)), axes=axes,
                    turned=rng.choice([dim, dim, dim // 2, 2 * rng.randint(axes, dim // 2)]), far=_log(rng, 100, 1000000),
                    adjacent=rng.random() < 0.5, type=rng.choice(["f32", "bf16"]), padding=rng.choice([0.0, 0.05]),
                    spread=rng.random() < 0.4)
    elif op == "attend":
        kind = rng.choice(["decode", "decode", "tree", "chunks", "chunks"])
        case.update(cap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.25,
                    window=rng.choice([0, 0, _log(rng, 1, 8192)]), prefix=0, docs=0, tree=kind == "tree", ragged=False)
        if kind == "decode":
            seqs = _log(rng, 1, 256)
            length = _log(rng, 16, min(131072, 64 * 8192 // (seqs * wide)))
            tokens = rng.choice([1, 1, 1, rng.randint(2, 8)])
        elif kind == "tree":
            seqs = _log(rng, 1, 32)
            tokens = rng.randint(2, 100)
            length = _log(rng, tokens, max(tokens, min(32768, 65536 // (seqs * wide))))
        else:
            seqs = _log(rng, 1, 32)
            tokens = _log(rng, 9, max(9, 4096 // seqs))
            length = _log(rng, tokens, max(tokens, min(16384, 8192 * 8192 * 32 // (seqs * tokens * case["heads"] * 2),
                                                       65536 // (seqs * wide))))
            case.update(ragged=rng.random() < 0.6, docs=rng.choice([0, 0, _log(rng, 16, 2000)]))
            if not case["docs"]:
                case["prefix"] = rng.choice([0, 0, rng.randint(1, length)])
        tokens = min(tokens, length)
        case.update(seqs=seqs, tokens=tokens, length=length, least=rng.choice([tokens, length]))
    elif op == "copy":
        copies = _log(rng, 1, max(1, 160 * 64 // (case["page"] * wide)))
        case.update(layers=rng.randint(1, 32), copies=copies, pages=2 * copies + rng.randint(0, 50))
    else:
        drafts = rng.randint(2, 64)
        case.update(layers=rng.randint(1, 32), seqs=_log(rng, 1, max(1, 64 // wide)), drafts=drafts,
                    most=rng.randint(1, max(1, drafts // 2)), length=rng.randint(0, 4000))
    return case


# ---- what follows from a case alone ----


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, hi among them, in no order."""
    return [hi if i == 0 else lo + int((hi - lo + 1) * (i * 0.6180339887 % 1.0)) for i in range(n)]


def _counts(case):
    """New tokens and whole length of each sequence."""
    lengths = _spread(case["seqs"], case["least"], case["length"])
    counts = [case["tokens"]] * case["seqs"]
    if case["ragged"]:  # every third sequence decodes, the others have chunks of all lengths
        counts = [1 if i % 3 == 2 else c for i, c in enumerate(_spread(case["seqs"], 1, case["tokens"]))]
    return [min(c, n) for c, n in zip(counts, lengths)], lengths


def _kept(case):
    """How many drafted tokens each sequence keeps."""
    return _spread(case["seqs"], 1, case["most"])


def _pairs(case, count, length):
    """Visible (query, key) pairs of a sequence, as near as the sizes alone say."""
    pairs = 0
    start = length - count
    if case["tree"]:
        return count * min(start, case["window"] or start) + count * min(count, 8)
    for i in range(count):
        seen = max(start + i + 1, min(case["prefix"], length))
        pairs += min(seen, case["window"] or seen, case["docs"] or seen)
    return pairs


def work(case):
    if case["op"] == "write":
        t, size = case["tokens"], 4 if case["type"] == "f32" else 2
        q, k = case["heads"] * case["dim"], case["kv_heads"] * case["dim"]
        return {"bytes": t * (q + 2 * k) * (size + 2) + t * 4 * (case["axes"] + 1), "flops": 3 * t * (q + k)}
    if case["op"] == "attend":
        counts, lengths = _counts(case)
        tokens = sum(counts)
        row = case["kv_heads"] * case["dim"] * 4
        seen = 0
        for c, n in zip(counts, lengths):
            far = max(0, n - c + 1 - case["window"]) if case["window"] and not case["prefix"] else 0
            seen += n - far
        pairs = sum(_pairs(case, c, n) for c, n in zip(counts, lengths))
        return {"bytes": seen * row + tokens * case["heads"] * (4 * case["dim"] + 4),
                "flops": 4 * case["dim"] * case["heads"] * pairs}
    row = case["layers"] * case["kv_heads"] * case["dim"] * 4
    rows = case["copies"] * case["page"] if case["op"] == "copy" else sum(_kept(case))
    return {"bytes": 2 * rows * row, "flops": 0}


# ---- inputs ----


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)


def _cache(case, g, layers, pages):
    shape = (layers, pages, case["kv_heads"], case["page"], case["dim"])
    return _normal(g, shape), _normal(g, shape)


def _tables(g, need, spare=3):
    """A table of pages for sequences that need so many, in no order, -1 behind them; pages in all."""
    need = torch.tensor(need, device="cuda")
    total = int(need.sum())
    at = torch.arange(int(need.max()), device="cuda")[None, :]
    there = at < need[:, None]
    table = torch.full(there.shape, -1, dtype=torch.int32, device="cuda")
    table[there] = torch.randperm(total + spare, generator=g, device="cuda")[:total].to(torch.int32)
    return table, total + spare


def _tree(case, g, counts):
    """Each drafted token's ancestors and itself as bits of 64-bit words; tokens come after their parents."""
    n, width = len(counts), max(counts)
    words = (width + 63) // 64
    parent = torch.rand((n, width), generator=g, device="cuda").cpu()
    sees = torch.zeros((n, width, words * 64), dtype=torch.bool)
    for i in range(width):  # one in five hangs on the context itself, the others on one of the 12 before
        lo = max(0, i - 12)
        p = (lo + (parent[:, i] * 1.25 * (i - lo)).long())
        if i:
            sees[:, i] = torch.where((p < i)[:, None], sees[torch.arange(n), p.clamp(max=i - 1)], False)
        sees[:, i, i] = True
    mask = (sees.reshape(n, width, words, 64).long() << torch.arange(64)).sum(dim=3)
    there = torch.arange(width)[None, :] < torch.tensor(counts)[:, None]
    return mask[there].cuda().contiguous()


def prepare(case, seed):
    g = _generator(seed)
    dev, op = "cuda", case["op"]
    s = {"case": case}
    if op == "write":
        t, dim, page = case["tokens"], case["dim"], case["page"]
        type_ = torch.float32 if case["type"] == "f32" else torch.bfloat16
        s["q"] = torch.randn((t, case["heads"] * dim), generator=g, device=dev).to(type_)
        s["k"] = torch.randn((t, case["kv_heads"] * dim), generator=g, device=dev).to(type_)
        s["v"] = torch.randn((t, case["kv_heads"] * dim), generator=g, device=dev).to(type_)
        first = torch.randint(0, case["far"], (case["axes"], 1), generator=g, device=dev)
        s["positions"] = (first + (torch.randint(0, case["far"], (case["axes"], t), generator=g, device=dev)
                                   if case["spread"] else torch.arange(t, device=dev))).to(torch.int32)
        pairs = case["turned"] // 2
        s["freqs"] = (10000.0 ** (-torch.arange(pairs, device=dev, dtype=torch.float64) / pairs)).float()
        s["axis"] = (torch.arange(pairs, device=dev) * case["axes"] // pairs).to(torch.int32)
        table, pages = _tables(g, [(t + page - 1) // page + 1])
        place = torch.arange(t, device=dev) + int(seed) % page  # a prompt goes on where the last chunk ended
        if case["spread"]:
            place = torch.randperm(table.shape[1] * page, generator=g, device=dev)[:t]
        slot = table[0, place // page] * page + place % page
        gone = torch.rand(t, generator=g, device=dev) < case["padding"]
        s["slots"] = torch.where(gone, -1, slot).to(torch.int32)
        kc, vc = _cache(case, g, 1, pages)
        s["kc"], s["vc"] = kc[0], vc[0]
        s["qr"] = torch.empty_like(s["q"], dtype=torch.bfloat16)
    elif op == "attend":
        counts, lengths = _counts(case)
        n, total, cols = len(counts), sum(counts), case["heads"] * case["dim"]
        s["tables"], pages = _tables(g, [(v + case["page"] - 1) // case["page"] for v in lengths])
        kc, vc = _cache(case, g, 1, pages)
        s["kc"], s["vc"] = kc[0], vc[0]
        s["q"] = _normal(g, (total, cols)) * 2  # some keys far more seen than others
        s["counts"] = torch.tensor(counts, device=dev)
        s["offsets"] = torch.cat([s["counts"].new_zeros(1), s["counts"].cumsum(0)]).to(torch.int32)
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
        h = torch.arange(1, case["heads"] + 1, device=dev)
        s["slopes"] = 2.0 ** (-8.0 * h / case["heads"]) if case["slopes"] else None
        s["prefix"] = (torch.full((n,), case["prefix"], dtype=torch.int32, device=dev) if case["prefix"] else None)
        s["mask"] = _tree(case, g, counts) if case["tree"] else None
        s["first"] = None
        if case["docs"]:  # a token's document begins at a multiple of docs
            seq = torch.repeat_interleave(torch.arange(n, device=dev), s["counts"])
            place = torch.arange(total, device=dev) - s["offsets"][seq] + (s["lengths"] - s["counts"])[seq]
            s["first"] = (place // case["docs"] * case["docs"]).to(torch.int32)
        s["y"] = torch.empty((total, cols), dtype=torch.bfloat16, device=dev)
        s["lse"] = torch.empty((total, case["heads"]), dtype=torch.float32, device=dev)
        if own:
            import decode_gemm_bf16_amd as uw
            s["work"] = torch.empty(uw.attend_workspace_bytes(total, n, case["heads"], case["kv_heads"], case["dim"],
                                                              max(counts), max(lengths)), dtype=torch.uint8, device=dev)
    elif op == "copy":
        s["kc"], s["vc"] = _cache(case, g, case["layers"], case["pages"])
        order = torch.randperm(case["pages"], generator=g, device=dev).to(torch.int32)
        s["src"], s["dst"] = order[:case["copies"]].contiguous(), order[case["copies"]:2 * case["copies"]].contiguous()
    else:
        n, d, most, page = case["seqs"], case["drafts"], case["most"], case["page"]
        # only the pages that hold drafted tokens are there: the others' entries name a page that is not touched
        start = torch.randint(case["length"] // 2, case["length"] + 1, (n,), generator=g, device=dev)
        per = (d + page - 1) // page + 1
        width = (case["length"] + d) // page + 2
        pages = torch.randperm(n * per + 1, generator=g, device=dev).to(torch.int32)
        table = pages[-1].repeat(n, width)
        col = start[:, None] // page + torch.arange(per, device=dev)
        s["tables"] = table.scatter_(1, col.clamp(max=width - 1), pages[:n * per].reshape(n, per)).contiguous()
        s["starts"] = start.to(torch.int32)
        s["kc"], s["vc"] = _cache(case, g, case["layers"], n * per + 1)
        # the first drafted token, then some behind the places that are filled
        later = torch.rand((n, max(1, d - most)), generator=g, device=dev).argsort(dim=1)[:, :most - 1].sort(dim=1)[0] + most
        kept = torch.cat([later.new_zeros((n, 1)), later], dim=1)
        live = torch.arange(kept.shape[1], device=dev) < torch.tensor(_kept(case), device=dev)[:, None]
        s["kept"] = torch.where(live, kept, -1).to(torch.int32).contiguous()
        s["lengths"] = torch.empty(n, dtype=torch.int32, device=dev)
    return s


# ---- one pass ----


def run(s):
    op = s["case"]["op"]
    if own:
        return {"write": _own_write, "attend": _own_attend, "copy": _own_copy, "keep": _own_keep}[op](s)
    return {"write": _write, "attend": _attend, "copy": _copy, "keep": _keep}[op](s)


def _own_write(s):
    import decode_gemm_bf16_amd as uw
    uw.cache_write(s["q"], s["k"], s["v"], s["positions"], s["freqs"], s["slots"], s["qr"], s["kc"], s["vc"],
                   axis=s["axis"], adjacent=s["case"]["adjacent"])
    return {"q": s["qr"], "k": s["kc"], "v": s["vc"]}


def _own_attend(s):
    import decode_gemm_bf16_amd as uw
    c = s["case"]
    uw.attend(s["q"], s["kc"], s["vc"], s["offsets"], s["lengths"], s["tables"], s["y"], s["work"], cap=c["cap"],
              window=c["window"], slopes=s["slopes"], prefix=s["prefix"], first=s["first"], mask=s["mask"], lse=s["lse"],
              max_tokens=c["tokens"], max_length=c["length"])
    return {"y": s["y"], "lse": s["lse"]}


def _own_copy(s):
    import decode_gemm_bf16_amd as uw
    uw.cache_copy_pages(s["kc"], s["vc"], s["src"], s["dst"])
    return {"k": s["kc"], "v": s["vc"]}


def _own_keep(s):
    import decode_gemm_bf16_amd as uw
    uw.cache_keep(s["kc"], s["vc"], s["tables"], s["starts"], s["kept"], s["lengths"])
    return {"k": s["kc"], "v": s["vc"], "lengths": s["lengths"]}


def _key_view(kc):
    """[..., page / 32, 32 places, dim / 8, 8]"""
    page, dim = kc.shape[-2:]
    return kc.view(*kc.shape[:-2], page // 32, dim // 8, 32, 8).transpose(-3, -2)


def _value_view(vc):
    """[..., page / 16, 2, 2, 4 places in this order, dim]"""
    page, dim = vc.shape[-2:]
    return vc.view(*vc.shape[:-2], page // 16, 2, dim, 2, 4).permute(*range(vc.dim() - 2), -5, -2, -4, -1, -3)


def _put(kc, vc, page, at, k, v):
    """Rows k and v [n, ..., dim] to their places; kc and vc [pages, kv_heads, ...] or with layers before."""
    lead = (slice(None),) * (kc.dim() - 4)
    kv, vv = _key_view(kc), _value_view(vc)
    kv[lead + (page, slice(None), at // 32, at % 32)] = k.reshape(*k.shape[:-1], -1, 8)
    vv[lead + (page, slice(None), at // 16, at // 8 % 2, at // 4 % 2, at % 4)] = v


def _write(s):
    c = s["case"]
    t, dim, pairs = c["tokens"], c["dim"], c["turned"] // 2
    # 64 bits: 32 lose the angle of a far position
    angle = s["positions"][s["axis"].long()].double().t() * s["freqs"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

    def turn(x):
        x = x.float().reshape(t, -1, dim)
        part, rest = x[:, :, :2 * pairs], x[:, :, 2 * pairs:]
        if c["adjacent"]:
            a, b = part[:, :, 0::2], part[:, :, 1::2]
            return torch.cat([torch.stack([a * cos - b * sin, a * sin + b * cos], dim=3).flatten(2), rest], dim=2)
        a, b = part[:, :, :pairs], part[:, :, pairs:]
        return torch.cat([a * cos - b * sin, a * sin + b * cos, rest], dim=2)

    s["qr"].copy_(turn(s["q"]).reshape(t, -1))
    slot = s["slots"].long()
    page, at = slot.clamp(min=0) // c["page"], slot.clamp(min=0) % c["page"]
    k, v = turn(s["k"]).to(torch.bfloat16), s["v"].reshape(t, -1, dim).to(torch.bfloat16)
    if c["padding"]:
        live = (slot >= 0).nonzero()[:, 0]
        page, at, k, v = page[live], at[live], k[live], v[live]
    _put(s["kc"], s["vc"], page, at, k, v)
    return {"q": s["qr"], "k": s["kc"], "v": s["vc"]}


def _attend(s):
    c = s["case"]
    n, heads, kv, dim = c["seqs"], c["heads"], c["kv_heads"], c["dim"]
    group, most = heads // kv, c["tokens"]
    table = s["tables"].long().clamp(min=0)
    keys = _key_view(s["kc"])[table].float().reshape(n, -1, kv, c["page"], dim).transpose(1, 2).reshape(n, kv, -1, dim)
    values = _value_view(s["vc"])[table].float().reshape(n, -1, kv, c["page"], dim).transpose(1, 2).reshape(n, kv, -1, dim)
    places = keys.shape[2]
    counts, lengths = s["counts"][:, None], s["lengths"].long()[:, None]
    start = lengths - counts
    i = torch.arange(most, device=table.device)
    row = (s["offsets"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1)  # [n, most]
    q = s["q"][row].float().reshape(n, most, kv, group, dim).permute(0, 2, 3, 1, 4).reshape(n, kv, group * most, dim)
    score = (q @ keys.transpose(2, 3) / dim ** 0.5).reshape(n, kv, group, most, places)
    if c["cap"]:
        score = c["cap"] * torch.tanh(score / c["cap"])
    k = torch.arange(places, device=table.device)
    at = start + i  # places of the queries
    seen = k <= at[:, :, None]
    near, far = at, k.expand(n, places)  # positions of the queries and the keys
    if c["tree"]:
        mask = s["mask"][row]  # [n, most, words]
        draft = k - start  # [n, places]
        words = mask[:, :, :, None] >> torch.arange(64, device=k.device) & 1
        bits = words.flatten(2)
        seen = torch.where((draft < 0)[:, None], True, bits.gather(2, draft.clamp(0, bits.shape[2] - 1)[:, None].expand(
            n, most, places)) > 0) & (draft < counts)[:, None]
        depth = bits.sum(dim=2) - 1
        near = start + depth
        far = torch.where(draft < 0, far, start + depth.gather(1, draft.clamp(0, most - 1)))
    distance = near[:, :, None] - far[:, None]
    if s["prefix"] is not None:
        seen = seen | (k < s["prefix"][:, None])[:, None]
    seen = seen & (k < lengths)[:, None]
    if s["first"] is not None:
        seen = seen & (k >= s["first"][row][:, :, None])
    if c["window"]:
        seen = seen & (distance < c["window"])
    if s["slopes"] is not None:
        score = score - s["slopes"].reshape(1, kv, group, 1, 1) * distance.abs()[:, None, None]
    score = torch.where(seen[:, None, None], score, float("-inf"))
    top = score.amax(dim=4, keepdim=True)
    weight = torch.exp(score - torch.where(top > float("-inf"), top, 0.0))
    total = weight.sum(dim=4, keepdim=True)
    y = weight.reshape(n, kv, group * most, places) @ values
    y = y.reshape(n, kv, group, most, dim) / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).squeeze(4)
    live = i < counts
    s["y"].copy_(y.permute(0, 3, 1, 2, 4)[live].reshape(-1, heads * dim))
    s["lse"].copy_(lse.permute(0, 3, 1, 2)[live].reshape(-1, heads))
    return {"y": s["y"], "lse": s["lse"]}


def _copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    s["kc"][:, dst] = s["kc"][:, src]
    s["vc"][:, dst] = s["vc"][:, src]
    return {"k": s["kc"], "v": s["vc"]}


def _keep(s):
    page = s["case"]["page"]
    kept, start = s["kept"].long(), s["starts"].long()[:, None]
    to = torch.arange(kept.shape[1], device=kept.device).expand(kept.shape)
    # places past a list's end keep what they hold
    src, dst = (start + torch.where(kept >= 0, kept, to)).reshape(-1), (start + to).reshape(-1)
    seq = torch.arange(kept.shape[0], device=kept.device).repeat_interleave(kept.shape[1])
    sp, dp = s["tables"][seq, src // page].long(), s["tables"][seq, dst // page].long()
    a, b = src % page, dst % page
    k = _key_view(s["kc"])[:, sp, :, a // 32, a % 32].flatten(-2)
    v = _value_view(s["vc"])[:, sp, :, a // 16, a // 8 % 2, a // 4 % 2, a % 4]
    _put(s["kc"], s["vc"], dp, b, k, v)
    s["lengths"].copy_(s["starts"] + (kept >= 0).sum(dim=1))
    return {"k": s["kc"], "v": s["vc"], "lengths": s["lengths"]}


# ---- the definition, in 64 bits ----


def _flat(case, key):
    """Where each (place, element) of a page of one head stands."""
    page, dim = case["page"], case["dim"]
    o, d = torch.arange(page, device="cuda")[:, None], torch.arange(dim, device="cuda")[None, :]
    if key:
        return ((o // 32 * (dim // 8) + d // 8) * 32 + o % 32) * 8 + d % 8
    return ((o // 16 * 2 + o // 4 % 2) * dim + d) * 8 + o // 8 % 2 * 4 + o % 4


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(case, s)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    return None  # copies


def _exact_write(case, s):
    t, dim, pairs = case["tokens"], case["dim"], case["turned"] // 2
    j = torch.arange(pairs, device="cuda")
    a, b = (2 * j, 2 * j + 1) if case["adjacent"] else (j, j + pairs)
    angle = torch.stack([s["positions"][int(x)].double() for x in s["axis"].tolist()], dim=1) * s["freqs"].double()
    unit = torch.polar(torch.ones_like(angle), angle)

    def turn(x):
        x = x.double().reshape(t, -1, dim).clone()
        z = torch.complex(x[:, :, a], x[:, :, b]) * unit[:, None]
        x[:, :, a], x[:, :, b] = z.real, z.imag
        return x

    out = {"q": turn(s["q"]).reshape(t, -1)}
    slot = s["slots"].long()
    live = (slot >= 0).nonzero()[:, 0]
    for name, cache, rows in (("k", s["kc"], turn(s["k"])), ("v", s["vc"], s["v"].double().reshape(t, -1, dim))):
        flat = cache.double().flatten(2)  # [pages, kv_heads, page * dim]
        where = _flat(case, name == "k")[slot[live] % case["page"]]
        index = where[:, None].expand(-1, case["kv_heads"], -1)
        page = (slot[live] // case["page"])[:, None, None].expand_as(index)
        head = torch.arange(case["kv_heads"], device="cuda")[None, :, None].expand_as(index)
        flat[page, head, index] = rows[live]
        out[name] = flat.reshape(cache.shape)
    return out


def _exact_attend(case, s):
    dim, kv, group = case["dim"], case["kv_heads"], case["heads"] // case["kv_heads"]
    total = s["q"].shape[0]
    y = torch.zeros((total, case["heads"], dim), dtype=torch.float64, device="cuda")
    lse = torch.zeros((total, case["heads"]), dtype=torch.float64, device="cuda")
    q = s["q"].double().reshape(total, case["heads"], dim)
    order = {True: _flat(case, True).reshape(-1), False: _flat(case, False).reshape(-1)}
    counts, lengths = _counts(case)
    at = 0
    for b, (m, n) in enumerate(zip(counts, lengths)):
        pages = s["tables"][b][:(n + case["page"] - 1) // case["page"]].long()
        # a row of the cache at a time: [length, kv_heads, dim]
        rows = [c[pages].flatten(2)[:, :, order[key]].reshape(len(pages), kv, case["page"], dim).permute(0, 2, 1, 3).reshape(
            -1, kv, dim)[:n] for c, key in ((s["kc"], True), (s["vc"], False))]
        place = torch.arange(n, device="cuda")
        query = place[n - m:, None]
        hidden = place[None, :] > query
        position = place
        if s["mask"] is not None:
            bits = torch.stack([s["mask"][at:at + m, j // 64] >> j % 64 & 1 for j in range(m)], dim=1)
            hidden = torch.cat([bits.new_zeros((m, n - m)), 1 - bits], dim=1).bool()
            position = torch.cat([place[:n - m], n - m + bits.sum(dim=1) - 1])
        far = position[n - m:, None] - position[None, :]
        if s["prefix"] is not None:
            hidden = hidden & (place >= int(s["prefix"][b]))[None, :]
        if s["first"] is not None:
            hidden = hidden | (place[None, :] < s["first"][at:at + m, None])
        if case["window"]:
            hidden = hidden | (far >= case["window"])
        for h in range(case["heads"]):
            z = q[at:at + m, h] @ rows[0][:, h // group].double().t() / dim ** 0.5
            if case["cap"]:
                z = case["cap"] * torch.tanh(z / case["cap"])
            if s["slopes"] is not None:
                z -= s["slopes"][h].double() * far.abs()
            z = z.masked_fill_(hidden, float("-inf"))
            lse[at:at + m, h] = torch.logsumexp(z, dim=1)
            y[at:at + m, h] = torch.softmax(z, dim=1).nan_to_num(0.0) @ rows[1][:, h // group].double()
        at += m
    return {"y": y.reshape(total, -1), "lse": lse}
