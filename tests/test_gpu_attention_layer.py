"""The attention layer on compressed projections, and the cache's calls together as a
server makes them: prompts, single tokens, forks, drafted trees, compacted pages, graphs
(GPU)."""
import numpy as np
import pytest

import oracle
import synth
from oracle import attention as att

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import decode_gemm_bf16_amd as uw
    return torch, uw


def i32(env, a):
    return env[0].from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Layer:
    def __init__(self, env, seed, hidden, heads, kv, dim, formats=None):
        uw = env[1]
        self.heads, self.kv, self.dim, self.hidden = heads, kv, dim, hidden
        self.w = [synth.weights(r, c, seed + j, 0.002, 10) for j, (r, c) in
                  enumerate(((heads * dim, hidden), (kv * dim, hidden), (kv * dim, hidden), (hidden, heads * dim)))]
        self.m = [uw.Matrix(w, formats or uw.FMT_PALETTE) for w in self.w]
        for m in self.m:
            m.set_variant(1)  # no K split with atomic sums: one order of summation

    def free(self):
        for m in self.m:
            m.free()


def batch(env, rng, counts, lengths, page, extra=2):
    """Offsets, lengths, tables, slots and positions of the last counts[b] places of sequences."""
    need = [-(-n // page) for n in lengths]
    order = rng.permutation(sum(need) + extra)
    tables = np.full((len(lengths), max(need)), -1)
    at = 0
    for b, n in enumerate(need):
        tables[b, :n], at = order[at:at + n], at + n
    places = [np.arange(n - c, n) for c, n in zip(counts, lengths)]
    slots = np.concatenate([tables[b, p // page] * page + p % page for b, p in enumerate(places)])
    return dict(offsets=i32(env, np.concatenate([[0], np.cumsum(counts)])), lengths=i32(env, lengths), tables=i32(env, tables),
                slots=i32(env, slots), positions=i32(env, np.concatenate(places)[None])), len(order), places


def formula(layer, xb, freqs, counts, lengths, old_k, old_v, cap=0.0, window=0):
    """The layer in float64 from the weights (old_k, old_v: per sequence the rows [length -
    count, kv, dim] that were in the cache), and how far it may be off: every rounding to
    bf16 half a step, float32 sums of n terms in any order n steps of the terms' sizes."""
    heads, kv, dim, hidden, half = layer.heads, layer.kv, layer.dim, layer.hidden, att.BF16_HALF
    w = [oracle.bf16_to_f64(a) for a in layer.w]
    x = oracle.bf16_to_f64(xb)
    tokens = len(x)
    angles = np.concatenate([np.arange(n - c, n) for c, n in zip(counts, lengths)])[:, None] * freqs.astype(np.float64)
    q, k, v = x @ w[0].T, x @ w[1].T, x @ w[2].T
    # what float32 sums and (for q and k) the turn add to half a step: hidden + 16 steps of
    # the sums' absolute terms
    more = [(hidden + 16) * att.U * (np.abs(x) @ np.abs(a).T) for a in w[:3]]
    q, k = (att.turn(a.reshape(tokens, -1, dim), angles, False) for a in (q, k))
    spread = lambda a: np.abs(a) + np.roll(np.abs(a), dim // 2, axis=-1)  # noqa: E731 (turned pairs mix)
    dq, dk = half * np.abs(q) + spread(more[0].reshape(q.shape)), half * np.abs(k) + spread(more[1].reshape(k.shape))
    v = v.reshape(tokens, kv, dim)
    dv = half * np.abs(v) + more[2].reshape(v.shape)
    rows, drows = np.zeros((tokens, heads, dim)), np.zeros((tokens, heads, dim))
    t = 0
    for c, n, ok, ov in zip(counts, lengths, old_k, old_v):
        s = slice(t, t + c)
        keys, values = np.concatenate([ok, k[s]]), np.concatenate([ov, v[s]])
        dkeys, dvalues = (np.concatenate([np.zeros(ok.shape), d[s]]) for d in (dk, dv))
        for i in range(c):
            at, _ = att.visible(i, c, n, window)
            for h in range(heads):
                g = h * kv // heads
                score = dim ** -0.5 * (keys[at, g] @ q[t, h])
                e = dim ** -0.5 * (np.abs(keys[at, g]) @ dq[t, h] + dkeys[at, g] @ (np.abs(q[t, h]) + dq[t, h]))
                e += 2 * dim * att.U * dim ** -0.5 * (np.abs(keys[at, g]) @ np.abs(q[t, h])) + 16 * att.U * (1 + np.abs(score))
                if cap:  # (its slope is at most 1)
                    score, e = cap * np.tanh(score / cap), e + 8 * att.U * cap
                p = np.exp(score - score.max())
                p /= p.sum()
                rows[t, h] = p @ values[at, g]
                # each weight off by exp(e + max e) at most, and by half a step; sums of len(at) terms
                f = np.minimum(np.exp(e + e.max()) * (1 + half) - 1 + (len(at) + 16) * att.U, 1 / np.maximum(p, 1e-300))
                drows[t, h] = (f * p) @ (np.abs(values[at, g]) + dvalues[at, g]) + p @ dvalues[at, g]
            t += 1
    drows += half * (np.abs(rows) + drows)
    rows, drows = rows.reshape(tokens, -1), drows.reshape(tokens, -1)
    return rows @ w[3].T, (drows + heads * dim * att.U * (np.abs(rows) + drows)) @ np.abs(w[3]).T


@pytest.mark.parametrize("pipelines", [(4, 4, 4, 4), (0, 0, 0, 0), (3, 4, 3, 4)])
@pytest.mark.parametrize("counts", [[1], [1, 1, 1], [5, 0, 11], [40, 1], [200]])
def test_layer_equals_its_parts(env, counts, pipelines):
    """Bit for bit where the products add in one order (k and v in one launch or in two);
    against the formula where K is split over atomic sums, whose order differs from call to
    call."""
    torch, uw = env
    rng = np.random.default_rng(sum(counts))
    layer = Layer(env, 300, 512, 8, 2, 64, uw.FMT_PALETTE | uw.FMT_HUFFMAN)
    tokens, page = sum(counts), 32
    lengths = [c + 30 for c in counts]
    b, pages, _ = batch(env, rng, counts, lengths, page)
    xb = synth.activations(tokens, 512, xseed=5)
    x = uw.bf16_tensor(xb)
    freqs = torch.from_numpy((10000.0 ** -(np.arange(32) / 32)).astype(np.float32)).cuda()
    old = torch.from_numpy(rng.standard_normal((2, pages, 2, page, 64), dtype=np.float32)).bfloat16().cuda()
    kinds = [layer.m[j].variant_in_use(tokens, pipelines[j])[1] for j in range(4)]
    print(f"layer {counts} {pipelines} {kinds}", flush=True)
    new = old.clone()
    y = torch.empty((tokens, 512), device="cuda")
    need = uw.attention_workspace_bytes(tokens, len(counts), 8, 2, 64, max(counts), max(counts) + 30)
    work = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    uw.attention_forward(*layer.m, pipelines, x, y, work[:need], new[0], new[1], freqs=freqs, cap=30.0, window=50,
                         max_tokens=max(counts), max_length=max(counts) + 30, **b)
    ref, out = old.clone(), torch.empty_like(y)
    q, k, v = (torch.empty((tokens, n), device="cuda") for n in (512, 128, 128))
    for m, t, p in zip(layer.m, (q, k, v), pipelines):
        m.matmul(x, t, tokens, p)
    turned = torch.empty((tokens, 512), dtype=torch.bfloat16, device="cuda")
    rows = torch.empty_like(turned)
    uw.cache_write(q, k, v, b["positions"], freqs, b["slots"], turned, ref[0], ref[1])
    part = torch.empty(uw.attend_workspace_bytes(tokens, len(counts), 8, 2, 64, max(counts), max(counts) + 30),
                       dtype=torch.uint8, device="cuda")
    uw.attend(turned, ref[0], ref[1], b["offsets"], b["lengths"], b["tables"], rows, part, cap=30.0, window=50,
              max_tokens=max(counts), max_length=max(counts) + 30)
    layer.m[3].matmul(rows, out, tokens, pipelines[3])
    torch.cuda.synchronize()
    assert not torch.equal(new, old) and torch.isfinite(y).all() and (work[need:] == 255).all()
    if pipelines == (4, 4, 4, 4):
        assert torch.equal(new.view(torch.int16), ref.view(torch.int16)) and torch.equal(y, out)
    tables = b["tables"].cpu().numpy()
    ok, ov = ([att.read_cache(f64(old[j]), tables[s], n - c, j == 0) for s, (c, n) in enumerate(zip(counts, lengths))]
              for j in range(2))
    want, bound = formula(layer, xb, freqs.cpu().numpy(), counts, lengths, ok, ov, 30.0, 50)
    for a in (y, out):
        assert (np.abs(f64(a) - want) <= bound).all()
    layer.free()


def test_layer_against_its_formula(env):
    """Whole prompts: every key is this call's."""
    torch, uw = env
    rng = np.random.default_rng(3)
    heads, kv, dim, hidden, page, counts = 4, 2, 64, 256, 32, [1, 37, 20]
    layer = Layer(env, 500, hidden, heads, kv, dim)
    b, pages, _ = batch(env, rng, counts, counts, page)
    tokens = sum(counts)
    xb = synth.activations(tokens, hidden, xseed=9)
    freqs = (10000.0 ** -(np.arange(32) / 32)).astype(np.float32)
    kc, vc = (torch.zeros((pages, kv, page, dim), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    y = torch.empty((tokens, hidden), device="cuda")
    work = torch.empty(uw.attention_workspace_bytes(tokens, 3, heads, kv, dim, 37, 37), dtype=torch.uint8, device="cuda")
    uw.attention_forward(*layer.m, [4] * 4, uw.bf16_tensor(xb), y, work, kc, vc, freqs=torch.from_numpy(freqs).cuda(),
                         max_tokens=37, max_length=37, **b)
    torch.cuda.synchronize()
    none = [np.zeros((0, kv, dim))] * 3
    want, bound = formula(layer, xb, freqs, counts, counts, none, none)
    assert (np.abs(f64(y) - want) <= bound).all()
    layer.free()


class Server:
    """Sequences over one paged cache of `layers` layers, with every written row kept on the
    host; each step's attention is compared with the rows kept."""

    def __init__(self, env, seed, layers, heads, kv, dim, page, pages):
        torch, uw = env
        self.env, self.rng = env, np.random.default_rng(seed)
        self.heads, self.kv, self.dim, self.page = heads, kv, dim, page
        self.kc, self.vc = (torch.full((layers, pages, kv, page, dim), NAN, dtype=torch.bfloat16, device="cuda")
                            for _ in range(2))
        self.pages = uw.Pages(pages)
        self.freqs = torch.from_numpy((1000.0 ** -(np.arange(dim // 2) / (dim // 2))).astype(np.float32)).cuda()
        self.tables, self.rows = [], []  # per sequence: pages; per layer kept rows [(key, value)]
        self.layers = layers

    def add(self):
        self.tables.append([])
        self.rows.append([[] for _ in range(self.layers)])
        return len(self.tables) - 1

    def copy(self, src, dst):
        if len(src):
            self.env[1].cache_copy_pages(self.kc, self.vc, i32(self.env, src), i32(self.env, dst))

    def fork(self, b):
        """A second sequence with b's rows: whole pages shared, the last one its own."""
        t = self.tables[b]
        self.pages.share(t)
        new = list(t)
        if len(self.rows[b][0]) % self.page:
            new[-1] = self.pages.own(new[-1])
            self.copy([t[-1]], [new[-1]])
        self.tables.append(new)
        self.rows.append([list(r) for r in self.rows[b]])
        return len(self.tables) - 1

    def compact(self):
        src, dst = self.pages.compact()
        self.copy(src, dst)
        name = dict(zip(src.tolist(), dst.tolist()))
        self.tables = [[name.get(p, p) for p in t] for t in self.tables]
        return len(src)

    def drop(self, b):
        self.pages.drop(self.tables[b])
        self.tables[b], self.rows[b] = [], [[] for _ in range(self.layers)]

    def table(self):
        t = np.full((len(self.tables), max(1, max(map(len, self.tables)))), -1)
        for b, p in enumerate(self.tables):
            t[b, :len(p)] = p
        return i32(self.env, t)

    def step(self, counts, masks=None, words=1):
        """counts[b] new tokens for each sequence (drafts if masks), in every layer."""
        torch, uw = self.env
        starts = [len(r[0]) for r in self.rows]
        slots, positions, n = [], [], sum(counts)
        for b, c in enumerate(counts):
            t = self.tables[b]
            more = -(-(starts[b] + c) // self.page) - len(t)
            if more > 0:
                t.extend(self.pages.take(more).tolist())
            p = np.arange(starts[b], starts[b] + c)
            slots += [t[i // self.page] * self.page + i % self.page for i in p]
            depth = [bin(m).count("1") - 1 for m in masks[b]] if masks else range(c)
            positions += [starts[b] + d for d in depth]
        lengths = [s + c for s, c in zip(starts, counts)]
        off, ln, tb, sl = i32(self.env, np.concatenate([[0], np.cumsum(counts)])), i32(self.env, lengths), self.table(), i32(self.env, slots)
        pos = i32(self.env, [positions])
        mask = None
        if masks:
            mask = torch.tensor([[m >> 64 * w & ((1 << 64) - 1) for w in range(words)] for b in masks for m in b],
                                dtype=torch.uint64).view(torch.int64).cuda()
        h, kv, dim = self.heads, self.kv, self.dim
        print("step", counts, "of", lengths, flush=True)
        for layer in range(self.layers):
            q, k, v = (torch.from_numpy(self.rng.standard_normal((n, c * dim), dtype=np.float32)).cuda() for c in (h, kv, kv))
            qr = torch.empty((n, h * dim), dtype=torch.bfloat16, device="cuda")
            y = torch.empty_like(qr)
            kc, vc = self.kc[layer], self.vc[layer]
            uw.cache_write(q, k, v, pos, self.freqs, sl, qr, kc, vc)
            work = torch.empty(uw.attend_workspace_bytes(n, len(counts), h, kv, dim, max(counts), max(lengths)),
                               dtype=torch.uint8, device="cuda")
            uw.attend(qr, kc, vc, off, ln, tb, y, work, mask=mask, max_tokens=max(counts), max_length=max(lengths))
            # the rows that are new, as they were written (and near what they have to be)
            angles = np.array(positions)[:, None] * f64(self.freqs)
            turned = att.turn(f64(k).reshape(n, kv, dim), angles, False)
            kb, vb = (synth.bf16_bits_to_f32(uw.bits_of(c)).astype(np.float64) for c in (kc, vc))
            at = 0
            for b, c in enumerate(counts):
                new_k = att.read_cache(kb, self.tables[b], lengths[b], True)[starts[b]:]
                new_v = att.read_cache(vb, self.tables[b], lengths[b], False)[starts[b]:]
                assert (np.abs(new_k - turned[at:at + c]) <= att.BF16_HALF * np.abs(turned[at:at + c]) + 2.0 ** -16).all()
                kept = self.rows[b][layer] + list(zip(new_k, new_v))
                if c:
                    keys, values = np.stack([r[0] for r in kept]), np.stack([r[1] for r in kept])
                    want, _, dy, _ = att.attend(f64(qr)[at:at + c].reshape(c, h, dim), keys, values, c, lengths[b],
                                                np.float64(np.float32(dim ** -0.5)), masks=masks[b] if masks else None)
                    assert (np.abs(f64(y)[at:at + c].reshape(c, h, dim) - want) <= dy).all(), (layer, b)
                self.rows[b][layer] = kept
                at += c

    def keep(self, kept, counts):
        """Keep drafts kept[b] of the counts[b] that were written last."""
        torch, uw = self.env
        starts = [len(r[0]) - c for r, c in zip(self.rows, counts)]
        lists = np.full((len(kept), max(1, max(map(len, kept)))), -1)
        for b, l in enumerate(kept):
            lists[b, :len(l)] = l
            for layer in range(self.layers):
                r = self.rows[b][layer]
                self.rows[b][layer] = r[:starts[b]] + [r[starts[b] + i] for i in l]
        lengths = i32(self.env, np.zeros(len(kept)))
        uw.cache_keep(self.kc, self.vc, self.table(), i32(self.env, starts), i32(self.env, lists), lengths)
        assert lengths.cpu().tolist() == [len(r[0]) for r in self.rows]
        for b, t in enumerate(self.tables):  # pages behind the kept rows go back
            n = -(-len(self.rows[b][0]) // self.page)
            self.pages.drop(t[n:])
            del t[n:]


@pytest.mark.parametrize("heads,kv,dim,page", [(4, 2, 64, 32), (6, 2, 128, 64)])
def test_a_server(env, heads, kv, dim, page):
    s = Server(env, heads, 2, heads, kv, dim, page, 40)
    for _ in range(3):
        s.add()
    s.step([70, 1, 33])
    s.step([1, 1, 1])
    s.fork(0)
    s.step([1, 2, 0, 1])  # the fork and its source go apart
    rng = s.rng
    counts = [7, 61, 12, 1]
    masks = []
    for c in counts:
        rows = []
        for i in range(c):
            p = rng.integers(-1, i) if i else -1
            rows.append((rows[p] if p >= 0 else 0) | 1 << i)
        masks.append(rows)
    s.step(counts, masks)
    path = [[i for i in range(c) if rows[j] >> i & 1] for c, rows, j in zip(counts, masks, (6, 60, 3, 0))]
    path[2] = []  # nothing was accepted
    s.keep(path, counts)
    s.step([1] * 4)
    s.drop(0)
    assert s.compact() > 0
    s.step([0, 3, 1, 40])
    f = s.fork(3)
    s.step([0, 0, 0, 1, 5])
    assert s.pages.left == 40 - len({p for t in s.tables for p in t}) and f == 4


def test_graphs(env):
    """Steps of single tokens as graphs (rows written, attention with split keys, drafts
    kept): what tables, lengths and rows hold counts at each replay.  Two graphs share one
    workspace, one after the other; eager work between the replays."""
    torch, uw = env
    rng = np.random.default_rng(8)
    heads, kv, dim, page, n, reach, longest = 8, 2, 64, 32, 3, 100, 100 * 32
    pages = n * reach + 4
    kc, vc = (torch.from_numpy(rng.standard_normal((1, pages, kv, page, dim), dtype=np.float32)).bfloat16().cuda()
              for _ in range(2))
    freqs = torch.from_numpy((1000.0 ** -(np.arange(32) / 32)).astype(np.float32)).cuda()
    tables = torch.empty((n, reach), dtype=torch.int32, device="cuda")
    lengths, starts = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
    kept = torch.empty((n, 4), dtype=torch.int32, device="cuda")
    work = torch.empty(uw.attend_workspace_bytes(4 * n, n, heads, kv, dim, 4, longest), dtype=torch.uint8, device="cuda")
    assert work.numel() > 0

    def step(count):
        """The buffers of a step of count tokens per sequence, and the step."""
        t = n * count
        q, k, v = (torch.empty((t, c * dim), device="cuda") for c in (heads, kv, kv))
        pos, slots = torch.empty((1, t), dtype=torch.int32, device="cuda"), torch.empty(t, dtype=torch.int32, device="cuda")
        off = i32(env, np.arange(n + 1) * count)
        qr = torch.empty((t, heads * dim), dtype=torch.bfloat16, device="cuda")
        y = torch.empty_like(qr)

        def run(k_cache, v_cache, y):
            stream = torch.cuda.current_stream()
            uw.cache_write(q, k, v, pos, freqs, slots, qr, k_cache[0], v_cache[0], stream=stream)
            uw.attend(qr, k_cache[0], v_cache[0], off, lengths, tables, y, work, max_tokens=count, max_length=longest,
                      stream=stream)
            if count > 1:
                uw.cache_keep(k_cache, v_cache, tables, starts, kept, lengths, stream=stream)
        return (q, k, v, pos, slots, y), run

    graphs = []
    for count in (1, 4):
        buffers, run = step(count)
        for b in buffers + (tables, lengths, starts, kept):
            b.zero_()
        kept.fill_(-1)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(kc, vc, buffers[5])
        graphs.append((count, g, buffers, run))
    for replay in range(6):
        count, g, (q, k, v, pos, slots, y), run = graphs[replay % 2]
        tb = rng.permutation(pages)[:n * reach].reshape(n, reach)
        ln = rng.integers(count, longest + 1, size=n)
        at = np.concatenate([np.arange(x - count, x) for x in ln])
        who = np.repeat(np.arange(n), count)
        for t in (q, k, v):
            t.normal_()
        tables.copy_(torch.from_numpy(tb))
        lengths.copy_(torch.from_numpy(ln))
        starts.copy_(torch.from_numpy(ln - count))
        pos.copy_(torch.from_numpy(at[None]))
        slots.copy_(torch.from_numpy(tb[who, at // page] * page + at % page))
        kept.copy_(torch.from_numpy(np.array([[0, 2, -1, -1], [1, 2, 3, -1], [-1] * 4])))
        ek, ev, ey = kc.clone(), vc.clone(), torch.empty_like(y)
        run(ek, ev, ey)
        after = lengths.clone()
        lengths.copy_(torch.from_numpy(ln))
        torch.cuda.synchronize()
        y.fill_(NAN)
        print(f"replay {replay}, {count} tokens each of {ln}", flush=True)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ey) and torch.equal(kc, ek) and torch.equal(vc, ev) and torch.equal(lengths, after)
        assert torch.isfinite(y).all()


def test_layer_on_its_stream_and_in_a_graph(env):
    torch, uw = env
    rng = np.random.default_rng(5)
    layer = Layer(env, 700, 256, 4, 2, 64)
    b, pages, _ = batch(env, rng, [1, 1], [100, 33], 32)
    freqs = torch.ones(16, device="cuda")
    x = uw.bf16_tensor(synth.activations(2, 256, xseed=3))
    kc, vc = (torch.from_numpy(rng.standard_normal((pages, 2, 32, 64), dtype=np.float32)).bfloat16().cuda() for _ in range(2))
    work = torch.empty(uw.attention_workspace_bytes(2, 2, 4, 2, 64, 1, 100), dtype=torch.uint8, device="cuda")
    y, want = torch.zeros((2, 256), device="cuda"), torch.empty((2, 256), device="cuda")
    call = lambda x, y: uw.attention_forward(*layer.m, [4] * 4, x, y, work, kc, vc, freqs=freqs, max_tokens=1,  # noqa: E731
                                             max_length=100, **b)
    call(x, want)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for m in layer.m:
        m.set_streams(side)
    with torch.cuda.stream(side):
        late = torch.zeros_like(x)
        big = torch.ones(1 << 26, device="cuda")
        for _ in range(10):
            big.mul_(1.0001)
        late.copy_(x)
        call(late, y)
        twice = y * 2
    torch.cuda.synchronize()
    assert torch.equal(twice, want * 2)
    late.copy_(x)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for m in layer.m:
            m.set_streams(torch.cuda.current_stream())
        call(late, y)
    for m in layer.m:
        m.set_streams()
    for _ in range(4):
        late.copy_(torch.randn(2, 256, device="cuda"))
        call(late, want)
        torch.cuda.synchronize()
        y.fill_(NAN)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.isfinite(y).all()
    layer.free()


def test_layer_refuses_before_any_launch(env):
    """What only a layer with device copies comes to: nothing is launched by a refused call."""
    import ctypes as C
    torch, uw = env
    rng = np.random.default_rng(6)
    layer = Layer(env, 800, 128, 2, 1, 64)
    b, pages, _ = batch(env, rng, [2], [40], 32)
    freqs, x = torch.ones(32, device="cuda"), uw.bf16_tensor(synth.activations(2, 128, xseed=1))
    y = torch.full((2, 128), 7.0, device="cuda")
    kc, vc = (torch.zeros((pages, 1, 32, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    need = uw.attention_workspace_bytes(2, 1, 2, 1, 64, 2, 40)
    work = torch.zeros(need, dtype=torch.uint8, device="cuda")
    good = {k: b[k].data_ptr() for k in ("positions", "slots", "offsets", "lengths", "tables")}
    good.update(freqs=freqs.data_ptr(), tokens=2, seqs=1, max_tokens=2, max_length=40, ldt=2, max_pages=2)

    def call(rotary=uw.Rotary(1, 32, 0), options=uw.AttendConfig(0.125, 0, 0), x=x.data_ptr(), kc=kc.data_ptr(),
             vc=vc.data_ptr(), y=y.data_ptr(), **kw):
        return uw._lib.uw_attention_forward(*[m._h for m in layer.m], (C.c_int32 * 4)(4, 4, 4, 4),
                                            uw.CacheConfig(2, 1, 64, 32, pages), rotary, options,
                                            uw.AttentionBatch(**dict(good, **kw)), x, kc, vc, y, work.data_ptr(), need)

    w = work.data_ptr()
    for kw, status in [(dict(rotary=None), uw.ERR_INVALID_ARG), (dict(options=None), uw.ERR_INVALID_ARG),
                       (dict(rotary=uw.Rotary(5, 32, 0)), uw.ERR_INVALID_ARG), (dict(rotary=uw.Rotary(1, 33, 0)), uw.ERR_SHAPE),
                       (dict(options=uw.AttendConfig(-1.0, 0, 0)), uw.ERR_INVALID_ARG), (dict(kc=None), uw.ERR_INVALID_ARG),
                       (dict(slots=None), uw.ERR_INVALID_ARG), (dict(tables=None), uw.ERR_INVALID_ARG),
                       (dict(max_pages=3), uw.ERR_SHAPE), (dict(mask=b["slots"].data_ptr(), mask_words=0), uw.ERR_SHAPE),
                       (dict(vc=kc.data_ptr()), uw.ERR_INVALID_ARG), (dict(y=w), uw.ERR_INVALID_ARG), (dict(x=w + 64), uw.ERR_INVALID_ARG),
                       (dict(kc=w), uw.ERR_INVALID_ARG), (dict(y=kc.data_ptr()), uw.ERR_INVALID_ARG),
                       (dict(x=vc.data_ptr() + 256), uw.ERR_INVALID_ARG), (dict(y=x.data_ptr()), uw.ERR_INVALID_ARG),
                       (dict(lengths=w + 512), uw.ERR_INVALID_ARG), (dict(slots=y.data_ptr()), uw.ERR_INVALID_ARG),
                       (dict(freqs=kc.data_ptr() + 64), uw.ERR_INVALID_ARG), (dict(first=vc.data_ptr()), uw.ERR_INVALID_ARG)]:
        assert call(**kw) == status, (kw, uw.last_error())
    torch.cuda.synchronize()
    assert (y == 7.0).all() and not kc.any() and not vc.any() and not work.any()
    assert call() == 0
    torch.cuda.synchronize()
    assert not (y == 7.0).any() and vc.any()
    layer.free()
