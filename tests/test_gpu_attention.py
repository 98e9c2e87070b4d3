"""The paged cache of keys and values and attention over it on the GPU against the
64-bit oracle, within bounds that the oracle derives from the float32 steps and the
roundings to bf16."""
import numpy as np
import pytest

import synth
from oracle import attention as att

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import decode_gemm_bf16_amd as uw
    return torch, uw


def bf16(rng, *shape):
    """bf16 bit patterns of standard normal values, and the values."""
    bits = synth.f32_to_bf16_bits(rng.standard_normal(shape, dtype=np.float32))
    return bits, synth.bf16_bits_to_f32(bits).astype(np.float64)


def i32(env, a):
    return env[0].from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Cache:
    """Pages of random old rows (bits), with sequences' keys and values at their places and
    garbage (NaN) in the places of their pages that were never written."""

    def __init__(self, rng, lengths, kv, dim, page, extra=2, garbage=True, reach=None):
        need = [max(1, -(-n // page)) for n in lengths]
        total = sum(need) + extra
        self.k, self.v = (bf16(rng, total, kv, page, dim)[0] for _ in range(2))
        order = rng.permutation(total)
        self.tables = np.full((len(lengths), reach or max(need) + 1), -1, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.tables[b, :n] = order[at:at + n]
            at += n
        if garbage:
            d = np.arange(dim)
            for b, n in enumerate(lengths):
                for p in range(n, need[b] * page):
                    pg = self.tables[b, p // page]
                    self.k[pg].reshape(kv, -1)[:, att.key_index(p % page, d, dim)] = 0x7FC1
                    self.v[pg].reshape(kv, -1)[:, att.value_index(p % page, d, dim)] = 0xFFC1

    def rows(self, b, length):
        k = att.read_cache(synth.bf16_bits_to_f32(self.k).astype(np.float64), self.tables[b], length, True)
        v = att.read_cache(synth.bf16_bits_to_f32(self.v).astype(np.float64), self.tables[b], length, False)
        return k, v

    def set_row(self, b, p, head, key, bits):
        """Write one head's row at place p of sequence b."""
        page, dim = self.k.shape[2:]
        c, index = (self.k, att.key_index) if key else (self.v, att.value_index)
        c[self.tables[b, p // page], head].reshape(-1)[index(p % page, np.arange(dim), dim)] = bits


def run(env, rng, counts, lengths, heads, kv, dim, page, cache=None, q=None, cap=0.0, window=0, slopes=None, prefix=None,
        first=None, masks=None, words=1, out="bf16", scale=None, max_tokens=None, max_length=None, stream=None, lse=True,
        compare=True):
    """One call of attend; compares with the oracle and returns y, lse (float64)."""
    torch, uw = env
    c = cache or Cache(rng, lengths, kv, dim, page)
    n, total = len(counts), sum(counts)
    qb, qv = bf16(rng, total + 1, heads * dim) if q is None else q  # a token behind the last sequence
    offsets = np.concatenate([[0], np.cumsum(counts)])
    mask = None
    if masks is not None:
        mask = np.zeros((total + 1, words), dtype=np.uint64)
        for i, m in enumerate(masks):
            for w in range(words):
                mask[i, w] = (m >> (64 * w)) & ((1 << 64) - 1)
        mask = torch.from_numpy(mask.view(np.int64)).cuda()
    scale = dim ** -0.5 if scale is None else scale
    max_tokens = max(1, max(counts)) if max_tokens is None else max_tokens
    max_length = max(1, max(lengths)) if max_length is None else max_length
    work = torch.full((uw.attend_workspace_bytes(total + 1, n, heads, kv, dim, max_tokens, max_length),), 255,
                      dtype=torch.uint8, device="cuda")
    y = torch.full((total + 1, heads * dim), 7.0, dtype=torch.bfloat16 if out == "bf16" else torch.float32, device="cuda")
    l = torch.full((total + 1, heads), 7.0, device="cuda") if lse else None
    kc, vc = uw.bf16_tensor(c.k), uw.bf16_tensor(c.v)
    print(f"attend {counts} of {lengths}, heads {heads}/{kv} of {dim}, page {page}, workspace {work.numel()}", flush=True)
    dev = lambda a, t: None if a is None else torch.from_numpy(np.asarray(a, dtype=t)).cuda()  # noqa: E731
    args = (uw.bf16_tensor(qb), kc, vc, i32(env, offsets), i32(env, lengths), i32(env, c.tables), y, work)
    kw = dict(scale=scale, cap=cap, window=window, slopes=dev(slopes, np.float32), prefix=dev(prefix, np.int32),
              first=dev(None if first is None else list(first) + [0], np.int32), mask=mask, lse=l, max_tokens=max_tokens,
              max_length=max_length, stream=stream)
    torch.cuda.synchronize()
    uw.attend(*args, **kw)
    torch.cuda.synchronize()
    got, gl = y.float().cpu().numpy().astype(np.float64), None if l is None else l.cpu().numpy().astype(np.float64)
    assert (got[total] == 7.0).all() and (l is None or (gl[total] == 7.0).all())  # the token of no sequence
    if compare:
        half = att.BF16_HALF if out == "bf16" else 2.0 ** -24
        for b in range(n):
            t0, t1 = offsets[b], offsets[b + 1]
            k, v = c.rows(b, lengths[b])
            want, wl, dy, dl = att.attend(qv[t0:t1].reshape(counts[b], heads, dim), k, v, counts[b], lengths[b],
                                          np.float64(np.float32(scale)), np.float64(np.float32(cap)), window,
                                          None if slopes is None else np.asarray(slopes, dtype=np.float32).astype(np.float64),
                                          0 if prefix is None else prefix[b], None if first is None else first[t0:t1],
                                          None if masks is None else masks[t0:t1], half)
            g = got[t0:t1].reshape(want.shape)
            assert (np.abs(g - want) <= dy).all(), (b, np.max(np.abs(g - want) / np.maximum(dy, 1e-300)))
            if l is not None:
                e = gl[t0:t1]
                none = wl == -np.inf
                assert (e[none] == -np.inf).all() and (g[none] == 0).all()
                assert (np.abs(e - np.where(none, 0, wl))[~none] <= dl[~none]).all()
    return got[:total], None if l is None else gl[:total]


def tree(rng, count, roots=0.2, words=1):
    """Drafted tokens' rows of bits: each after its parent."""
    rows = []
    for i in range(count):
        p = rng.integers(0, i) if i and rng.random() > roots else -1
        rows.append((rows[p] if p >= 0 else 0) | 1 << i)
    return rows


# ---- attention ----

@pytest.mark.parametrize("heads,kv,dim,page", [(4, 2, 64, 32), (8, 2, 128, 64), (6, 2, 96, 32), (4, 1, 256, 128),
                                               (3, 3, 128, 256), (64, 1, 64, 64), (5, 1, 128, 32)])
@pytest.mark.parametrize("counts,lengths", [([1], [1]), ([1], [31]), ([1], [257]), ([1, 1, 1], [33, 1, 128]),
                                            ([3, 2], [70, 2]), ([40], [40]), ([37, 1, 0, 5], [101, 64, 17, 5])])
def test_sizes(env, heads, kv, dim, page, counts, lengths):
    rng = np.random.default_rng(heads * 1000 + dim + sum(lengths))
    run(env, rng, counts, lengths, heads, kv, dim, page)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("count", [1, 20])
def test_split_keys(env, out, dim, count):
    """Long keys in parts that are joined (2 to more than 16 of them), both kernels."""
    rng = np.random.default_rng(dim + count)
    run(env, rng, [count], [1500], 4, 1, dim, 64, out=out)
    run(env, rng, [count, 1], [6000, 700], 2, 1, dim, 128, out=out)


@pytest.mark.parametrize("counts,lengths,max_tokens,max_length", [
    ([5, 1], [300, 2], 1, 1), ([40, 2], [100, 2], 1, 5000), ([1, 1], [90, 1000], 2, 64), ([3], [2000], 3, 33)])
def test_other_sizes_than_laid_out_for(env, counts, lengths, max_tokens, max_length):
    rng = np.random.default_rng(3)
    run(env, rng, counts, lengths, 8, 2, 64, 32, max_tokens=max_tokens, max_length=max_length)


def test_nothing_to_see(env):
    """Empty sequences, lengths of zero, more tokens than keys, documents that begin
    behind a token: zeros and -inf."""
    rng = np.random.default_rng(4)
    y, lse = run(env, rng, [1, 0, 2, 4], [0, 0, 0, 2], 4, 2, 64, 32)
    assert (y[:5] == 0).all() and (lse[:5] == -INF).all() and np.isfinite(lse[5:]).all()
    run(env, rng, [3], [40], 4, 2, 64, 32, first=[0, 39, 40])
    run(env, rng, [20], [40], 8, 2, 64, 32, first=[k % 41 for k in range(0, 60, 3)])
    run(env, rng, [2], [50], 4, 2, 64, 32, masks=[0, 0])  # the context alone
    y, lse = run(env, rng, [2], [2], 4, 2, 64, 32, masks=[0, 2])
    assert (y[0] == 0).all() and (lse[0] == -INF).all()


@pytest.mark.parametrize("counts,lengths", [([1, 1], [200, 33]), ([50, 3, 1], [130, 90, 40]), ([33], [700])])
@pytest.mark.parametrize("what", ["window 1", "window 40", "prefix", "documents", "prefix window", "window huge"])
def test_masks(env, counts, lengths, what):
    rng = np.random.default_rng(len(what) + sum(counts))
    kw = {}
    if "window" in what:
        kw["window"] = 1 if what == "window 1" else 2 ** 31 - 1 if "huge" in what else 40
    if "prefix" in what:
        kw["prefix"] = [n - n // 4 if b % 2 == 0 else 0 for b, n in enumerate(lengths)]
    if what == "documents":
        kw["first"] = [(n - c + i) // 27 * 27 for c, n in zip(counts, lengths) for i in range(c)]
    run(env, rng, counts, lengths, 8, 2, 64, 32, **kw)


@pytest.mark.parametrize("counts,lengths", [([1, 1], [200, 33]), ([50, 3], [130, 90])])
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("kw", [dict(cap=5.0), dict(cap=0.01), dict(slopes=[0.5, 0.25, 0.1, 0.0]),
                                dict(cap=30.0, slopes=[2.0, 0.01, 0.0, 0.3], window=60), dict(scale=3.0),
                                dict(slopes=[0.1] * 4, prefix=[1000, 5])])
def test_scores(env, counts, lengths, dim, kw):
    rng = np.random.default_rng(dim)
    run(env, rng, counts, lengths, 4, 1, dim, 64, **kw)


@pytest.mark.parametrize("counts,lengths,words", [([1, 7], [50, 7], 1), ([64, 30], [300, 95], 1), ([100, 9], [101, 41], 2),
                                                  ([61], [1000], 1), ([70], [200], 1)])
@pytest.mark.parametrize("kw", [dict(), dict(cap=20.0), dict(window=5), dict(slopes=[0.3, 0.1, 0.0, 0.7], window=70),
                                dict(first=7)])
def test_trees(env, counts, lengths, words, kw):
    rng = np.random.default_rng(sum(lengths))
    masks = [m for c in counts for m in tree(rng, c)]
    if words * 64 < max(counts):  # bits beyond the words are 0
        masks = [m & ((1 << 64 * words) - 1) for m in masks]
    kw = dict(kw)
    if "first" in kw:
        kw["first"] = [(n - c + i) // 7 * 7 for c, n in zip(counts, lengths) for i in range(c)]
    run(env, rng, counts, lengths, 4, 2, 64, 32, masks=masks, words=words, **kw)


def test_pages_that_are_not_there(env):
    """Entries outside the cache and lengths beyond the table hide keys (both kernels)."""
    for counts in ([1, 1, 1], [40, 2, 3]):
        rng = np.random.default_rng(6)
        lengths = [300, 100, 90]
        c = Cache(rng, lengths, 2, 64, 32, garbage=False)
        c.tables[0, 2], c.tables[0, 5], c.tables[1, 0], c.tables[2, :] = -1, 10 ** 6, c.k.shape[0], -7
        run(env, rng, counts, lengths, 8, 2, 64, 32, cache=c)
        c = Cache(rng, lengths, 2, 64, 32, garbage=False)
        c.tables = np.ascontiguousarray(c.tables[:, :4])
        run(env, rng, counts, lengths, 8, 2, 64, 32, cache=c)


@pytest.mark.parametrize("counts,lengths,kw", [([1], [70], dict(window=20)), ([40], [70], {}), ([40], [300], dict(cap=9.0)),
                                               ([3], [50], dict(masks=[1, 3, 5]))])
@pytest.mark.parametrize("bits", [0x7F80, 0xFF80, 0x7FC0])
def test_infinities_reach_those_that_see_them(env, counts, lengths, kw, bits):
    """An infinity or NaN among the values: at a place that only some tokens see."""
    for place, e in ((lengths[0] - counts[0] // 2 - 1, 5), (5, 63), (lengths[0] - 1, 0)):
        rng = np.random.default_rng(bits)
        clean = Cache(rng, lengths, 1, 64, 32)
        q = bf16(rng, counts[0] + 1, 2 * 64)
        rng2 = np.random.default_rng(1)
        y0, l0 = run(env, rng2, counts, lengths, 2, 1, 64, 32, cache=clean, q=q, **kw)
        row = synth.f32_to_bf16_bits(np.ones(64, dtype=np.float32))
        row[e] = bits
        clean.set_row(0, place, 0, False, row)
        y1, l1 = run(env, rng2, counts, lengths, 2, 1, 64, 32, cache=clean, q=q, compare=False, **kw)
        assert np.array_equal(l0, l1)
        masks = kw.get("masks")
        for i in range(counts[0]):
            sees = place in att.visible(i, counts[0], lengths[0], kw.get("window", 0), masks=masks)[0]
            for h in range(2):
                if sees:
                    got = y1[i, h * 64 + e]
                    assert np.isnan(got) if bits == 0x7FC0 else got == (INF if bits == 0x7F80 else -INF), (place, i, h)
                    rest = np.delete(y1[i, h * 64:h * 64 + 64], e)
                    assert np.isfinite(rest).all()
                else:
                    assert np.array_equal(y0[i, h * 64:h * 64 + 64], y1[i, h * 64:h * 64 + 64]), (place, i, h)


def test_infinities_of_keys_and_queries(env):
    """A NaN key poisons those that see it and no others; so does a NaN query its own row."""
    for counts, lengths in (([40], [60]), ([2], [60])):
        rng = np.random.default_rng(9)
        c = Cache(rng, lengths, 1, 64, 32)
        q = bf16(rng, counts[0] + 1, 2 * 64)
        y0, _ = run(env, rng, counts, lengths, 2, 1, 64, 32, cache=c, q=q)
        place = lengths[0] - 1
        c.set_row(0, place, 0, True, np.full(64, 0x7FC0))
        q[0][0, 70] = 0x7FC0  # token 0, head 1
        y1, _ = run(env, rng, counts, lengths, 2, 1, 64, 32, cache=c, q=q, compare=False)
        last = counts[0] - 1
        assert np.isnan(y1[last]).all() and np.isnan(y1[0, 64:]).all()
        assert np.array_equal(y0[0, :64], y1[0, :64]) and np.array_equal(y0[1:last], y1[1:last])


def test_large_scores(env):
    """Scores of thousands: the running maximum moves far, one key takes it all."""
    rng = np.random.default_rng(10)
    for counts, lengths in (([1], [3000]), ([40], [200])):
        run(env, rng, counts, lengths, 2, 1, 64, 32, scale=100.0)


def test_strides_and_streams(env):
    """Rows cut out of wider ones, tables too, on a stream of its own; the same as contiguous."""
    torch, uw = env
    rng = np.random.default_rng(11)
    counts, lengths, heads, kv, dim, page = [3, 50], [90, 77], 4, 2, 64, 32
    c = Cache(rng, lengths, kv, dim, page)
    qb, _ = bf16(rng, 53, heads * dim)
    q = uw.bf16_tensor(qb)
    kc, vc, off, ln, tb = uw.bf16_tensor(c.k), uw.bf16_tensor(c.v), i32(env, [0, 3, 53]), i32(env, lengths), i32(env, c.tables)
    y, lse = torch.empty_like(q), torch.empty((53, heads), device="cuda")
    work = torch.empty(uw.attend_workspace_bytes(53, 2, heads, kv, dim, 50, 90), dtype=torch.uint8, device="cuda")
    uw.attend(q, kc, vc, off, ln, tb, y, work, max_tokens=50, max_length=90, lse=lse)
    wq = torch.zeros((53, heads * dim + 24), dtype=torch.bfloat16, device="cuda")
    wq[:, 8:8 + heads * dim] = q
    wt = torch.zeros((2, tb.shape[1] + 3), dtype=torch.int32, device="cuda")
    wt[:, 1:1 + tb.shape[1]] = tb
    wy = torch.full((53, heads * dim + 16), 3.0, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    uw.attend(wq[:, 8:8 + heads * dim], kc, vc, off, ln, wt[:, 1:1 + tb.shape[1]], wy[:, 16:], work, max_tokens=50,
              max_length=90, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(wy[:, 16:], y) and (wy[:, :16] == 3.0).all()


def test_far_pages(env):
    """Pages whose elements lie behind 2^32 in the cache."""
    torch, uw = env
    rng = np.random.default_rng(12)
    kv, dim, page, pages = 8, 128, 256, 17000  # 4.46 * 10^9 elements each of keys and values
    kc = torch.zeros((pages, kv, page, dim), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    small = Cache(rng, [300], kv, dim, page, extra=0)
    far = [pages - 1, pages - 2]
    for i, p in enumerate(far):
        kc[p] = uw.bf16_tensor(small.k[small.tables[0, i]])
        vc[p] = uw.bf16_tensor(small.v[small.tables[0, i]])
    for count in (1, 50):
        qb, _ = bf16(rng, count, 16 * dim)
        ys = []
        for k, v, table in ((kc, vc, [far]), (uw.bf16_tensor(small.k), uw.bf16_tensor(small.v), small.tables[:, :2])):
            y = torch.empty((count, 16 * dim), dtype=torch.bfloat16, device="cuda")
            work = torch.empty(uw.attend_workspace_bytes(count, 1, 16, kv, dim, count, 300), dtype=torch.uint8, device="cuda")
            uw.attend(uw.bf16_tensor(qb), k, v, i32(env, [0, count]), i32(env, [300]), i32(env, table), y, work,
                      max_tokens=count, max_length=300)
            ys.append(y)
        assert torch.equal(*ys)
    # written, copied and kept there, too
    rows = torch.randn((3, kv * dim), device="cuda")
    slots = i32(env, [(pages - 1) * page + 255, (pages - 1) * page + 254, 7])
    uw.cache_write(None, rows, rows, i32(env, [[0, 0, 0]]), torch.zeros(0, device="cuda"), slots, None, kc, vc)
    uw.cache_copy_pages(kc[None], vc[None], i32(env, [pages - 1]), i32(env, [pages - 3]))
    assert torch.equal(kc[pages - 3], kc[pages - 1]) and torch.equal(vc[pages - 3], vc[pages - 1])
    length = i32(env, [0])
    uw.cache_keep(kc[None], vc[None], i32(env, [[pages - 3]]), i32(env, [3]), i32(env, [[251, 252]]), length)
    page_k, page_v = uw.bits_of(kc[pages - 3]), uw.bits_of(vc[pages - 3])
    want = synth.f32_to_bf16_bits(rows[:2].cpu().numpy()).reshape(2, kv, dim)
    for at, row in ((3, want[1]), (4, want[0])):
        assert np.array_equal(att.read_cache(page_k[None], [0], 5, True)[at], row)
        assert np.array_equal(att.read_cache(page_v[None], [0], 5, False)[at], row)
    assert length.item() == 5


def test_two_calls_at_once(env):
    """Two streams over one cache, each with its workspace."""
    torch, uw = env
    rng = np.random.default_rng(13)
    c = Cache(rng, [5000], 2, 64, 64)
    kc, vc, tb = uw.bf16_tensor(c.k), uw.bf16_tensor(c.v), i32(env, c.tables)
    qs = [uw.bf16_tensor(bf16(rng, n, 4 * 64)[0]) for n in (1, 30)]

    def call(q, stream=None):
        n = q.shape[0]
        y = torch.empty_like(q)
        work = torch.empty(uw.attend_workspace_bytes(n, 1, 4, 2, 64, n, 5000), dtype=torch.uint8, device="cuda")
        args = (q, kc, vc, i32(env, [0, n]), i32(env, [5000]), tb, y, work)
        torch.cuda.synchronize()
        return lambda: uw.attend(*args, max_tokens=n, max_length=5000, stream=stream), y

    want = []
    for q in qs:
        f, y = call(q)
        f()
        torch.cuda.synchronize()
        want.append(y.clone())
    streams = [torch.cuda.Stream() for _ in qs]
    calls = [call(q, s) for q, s in zip(qs, streams)]
    for _ in range(5):
        for f, _ in calls:
            f()
    torch.cuda.synchronize()
    for (_, y), w in zip(calls, want):
        assert torch.equal(y, w)  # and no result depends on timing


# ---- rows of the cache ----

@pytest.mark.parametrize("tokens", [1, 3, 33, 300, 1100])
@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,dim,page,axes,pairs,adjacent", [
    (4, 2, 64, 32, 1, 32, False), (8, 2, 128, 64, 3, 64, True), (6, 6, 96, 32, 2, 17, False), (4, 1, 256, 128, 4, 128, False),
    (2, 1, 128, 256, 1, 0, False), (20, 5, 64, 32, 2, 13, True), (3, 3, 128, 64, 2, 32, False)])
def test_write(env, tokens, type, heads, kv, dim, page, axes, pairs, adjacent):
    torch, uw = env
    rng = np.random.default_rng(tokens + dim + pairs)
    pages = -(-(tokens + 40) // page) + 3
    kb, vb = bf16(rng, pages, kv, page, dim)[0], bf16(rng, pages, kv, page, dim)[0]
    x = {n: rng.standard_normal((tokens, c * dim), dtype=np.float32) for n, c in (("q", heads), ("k", kv), ("v", kv))}
    if type == "bf16":
        x = {n: synth.bf16_bits_to_f32(synth.f32_to_bf16_bits(a)) for n, a in x.items()}
    dev = {}
    for n, a in x.items():  # rows cut out of wider ones
        wide = torch.zeros((tokens, a.shape[1] + 8), dtype=torch.float32 if type == "f32" else torch.bfloat16, device="cuda")
        wide[:, 8:] = torch.from_numpy(a).cuda()
        dev[n] = wide[:, 8:]
    positions = rng.integers(-5, 2 ** 20, size=(axes, tokens)).astype(np.int32)
    positions[:, 0] = 2 ** 31 - 1
    freqs = (10000.0 ** -(np.arange(pairs) / max(1, pairs))).astype(np.float32)
    axis = rng.integers(-1, axes + 1, size=pairs).astype(np.int32)  # some of no axis
    # a run of places over pages in no order, with gaps and numbers outside; the run starts anywhere
    order = rng.permutation(pages)
    place = np.arange(tokens) + rng.integers(0, 37)
    place[tokens // 2:] += rng.integers(0, 3)
    slots = (order[place // page] * page + place % page).astype(np.int64)
    out = rng.random(tokens) < 0.02
    slots[out] = rng.choice([-1, pages * page, 2 ** 31 - 1, -2 ** 31], size=out.sum())
    if tokens % 2:  # and single places in no order
        some = rng.permutation(tokens)[:tokens // 3]
        slots[some] = slots[rng.permutation(some)]
    kc, vc = uw.bf16_tensor(kb), uw.bf16_tensor(vb)
    qr = torch.full((tokens, heads * dim + 8), 5.0, dtype=torch.bfloat16, device="cuda")
    print(f"write {tokens}, {heads}/{kv} of {dim}, page {page}, {axes} axes, {pairs} pairs", flush=True)
    uw.cache_write(dev["q"], dev["k"], dev["v"], torch.from_numpy(positions).cuda(), torch.from_numpy(freqs).cuda(),
                   i32(env, slots), qr[:, :heads * dim], kc, vc, axis=torch.from_numpy(axis).cuda(), adjacent=adjacent)
    torch.cuda.synchronize()
    assert (qr[:, heads * dim:] == 5.0).all()
    angles = np.zeros((tokens, pairs))
    for j in range(pairs):
        if 0 <= axis[j] < axes:
            angles[:, j] = positions[axis[j]].astype(np.float64) * np.float64(freqs[j])

    def check(got, a, c):
        """An angle below 2 pi in float32 is off by 2^-22, the functions by two of their steps,
        the sum by two of its own: 2^-20 (|a| + |b|) in all; then one rounding to bf16."""
        a = a.astype(np.float64).reshape(tokens, c, dim)
        want = att.turn(a, angles, adjacent)
        bound = att.turn(np.abs(a), np.zeros_like(angles), adjacent)
        other = np.array(bound)
        for j in range(pairs):
            p, s = (2 * j, 2 * j + 1) if adjacent else (j, j + pairs)
            other[:, :, p] = other[:, :, s] = bound[:, :, p] + bound[:, :, s]
        assert (np.abs(got - want) <= 2.0 ** -20 * other * 1.01 + att.BF16_HALF * np.abs(want)).all()

    f = lambda t: synth.bf16_bits_to_f32(t).astype(np.float64)  # noqa: E731
    check(qr[:, :heads * dim].float().cpu().numpy().astype(np.float64).reshape(tokens, heads, dim), x["q"], heads)
    gk, gv = uw.bits_of(kc), uw.bits_of(vc)
    there = (slots >= 0) & (slots < pages * page)
    live = np.nonzero(there)[0]
    rows_k, rows_v = np.zeros((tokens, kv, dim), np.uint16), np.zeros((tokens, kv, dim), np.uint16)
    d = np.arange(dim)
    for t in live:
        p, o = slots[t] // page, slots[t] % page
        fk, fv = gk[p].reshape(kv, -1), gv[p].reshape(kv, -1)
        rows_k[t], rows_v[t] = fk[:, att.key_index(o, d, dim)], fv[:, att.value_index(o, d, dim)]
        # what was there before goes back, so that the rest can be compared as a whole
        fk[:, att.key_index(o, d, dim)] = kb[p].reshape(kv, -1)[:, att.key_index(o, d, dim)]
        fv[:, att.value_index(o, d, dim)] = vb[p].reshape(kv, -1)[:, att.value_index(o, d, dim)]
    assert np.array_equal(gk, kb) and np.array_equal(gv, vb)
    if there.all():
        check(f(rows_k), x["k"], kv)
    want_v = synth.f32_to_bf16_bits(x["v"]).reshape(tokens, kv, dim)
    assert np.array_equal(rows_v[live], want_v[live])
    turned = att.turn(x["k"].astype(np.float64).reshape(tokens, kv, dim), angles, adjacent)
    assert (np.abs(f(rows_k) - turned)[live] <= 2.0 ** -18 * (1 + np.abs(x["k"]).max()) + att.BF16_HALF * np.abs(turned)[live]).all()


def test_write_without_queries_and_special_values(env):
    torch, uw = env
    kc = torch.zeros((2, 1, 32, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    k = torch.tensor([INF, -INF, NAN, 0.0, -0.0, 1e-40, 3.4e38, 1.00390625] * 8, device="cuda").reshape(1, 64)
    uw.cache_write(None, k, k, i32(env, [[7]]), torch.zeros(0, device="cuda"), i32(env, [33]), None, kc, vc)
    want = synth.f32_to_bf16_bits(k.cpu().numpy())[0]
    for c, key in ((kc, True), (vc, False)):
        got = att.read_cache(uw.bits_of(c), [1], 2, key)[1, 0]
        nan = np.isnan(synth.bf16_bits_to_f32(want))
        assert np.array_equal(got[~nan], want[~nan]) and np.isnan(synth.bf16_bits_to_f32(got[nan])).all()


@pytest.mark.parametrize("layers,pages,kv,page,dim,n", [(1, 2, 1, 32, 64, 1), (3, 40, 2, 64, 96, 17), (2, 20, 5, 32, 256, 10),
                                                         (32, 9, 8, 64, 128, 4)])
def test_copy_pages(env, layers, pages, kv, page, dim, n):
    torch, uw = env
    rng = np.random.default_rng(n)
    kb, vb = bf16(rng, layers, pages, kv, page, dim)[0], bf16(rng, layers, pages, kv, page, dim)[0]
    order = rng.permutation(pages)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    if n > 3:  # skipped: numbers outside, and a page onto itself
        src[0], dst[1], src[2], dst[2] = -1, pages, order[2], order[2]
    kc, vc = uw.bf16_tensor(kb), uw.bf16_tensor(vb)
    uw.cache_copy_pages(kc, vc, i32(env, src), i32(env, dst))
    torch.cuda.synchronize()
    for a, b in zip(src, dst):
        if 0 <= a < pages and 0 <= b < pages:
            kb[:, b], vb[:, b] = kb[:, a], vb[:, a]
    assert np.array_equal(uw.bits_of(kc), kb) and np.array_equal(uw.bits_of(vc), vb)


@pytest.mark.parametrize("layers,kv,page,dim,most", [(1, 1, 32, 64, 1), (2, 3, 32, 96, 40), (3, 2, 64, 128, 9),
                                                     (2, 1, 32, 256, 256)])
def test_keep(env, layers, kv, page, dim, most):
    torch, uw = env
    rng = np.random.default_rng(most)
    seqs = 5
    starts = np.array([0, 31, 64, 5, 90])
    drafts = max(most, 8)
    kept = np.full((seqs, most), -1, dtype=np.int32)
    for b in range(4):
        n = [most, most // 2 + 1, 1, most - most // 3][b]
        kept[b, :n] = np.sort(rng.permutation(drafts)[:n])
    if most > 4:
        kept[1, 3] = kept[1, 2]  # a list ends where it does not rise
    c = Cache(rng, [s + drafts for s in starts], kv, dim, page, garbage=False)
    c.tables[3, 0] = -1  # rows to or from here are not moved
    kb, vb = (np.stack([x, x[::-1], x ^ 1][:layers]).copy() for x in (c.k, c.v))
    kc, vc = uw.bf16_tensor(kb), uw.bf16_tensor(vb)
    lengths = i32(env, [9] * seqs)
    uw.cache_keep(kc, vc, i32(env, c.tables), i32(env, starts), i32(env, kept), lengths)
    torch.cuda.synchronize()
    d = np.arange(dim)
    want = []
    for b in range(seqs):
        old_k, old_v, n = kb.copy(), vb.copy(), 0
        while n < most and kept[b, n] >= 0 and (n == 0 or kept[b, n] > kept[b, n - 1]):
            f, t = starts[b] + kept[b, n], starts[b] + n
            pf, pt = c.tables[b, f // page], c.tables[b, t // page]
            if pf >= 0 and pt >= 0:
                for new, old, index in ((kb, old_k, att.key_index), (vb, old_v, att.value_index)):
                    rows = old[:, pf].reshape(layers, kv, -1)[:, :, index(f % page, d, dim)]
                    new[:, pt].reshape(layers, kv, -1)[:, :, index(t % page, d, dim)] = rows
            n += 1
        want.append(starts[b] + n)
    assert lengths.cpu().tolist() == want
    assert np.array_equal(uw.bits_of(kc), kb) and np.array_equal(uw.bits_of(vc), vb)
