"""Attention's masks, trees, infinities and missing pages on every instance of its kernels: all
sizes of heads, with few rows, with many and one part of the keys, with many and several parts;
keys long enough that the loops over whole blocks run, by turns of every length (GPU)."""
import numpy as np
import pytest

import synth
import test_gpu_attention as cases
from oracle import attention as att
from test_gpu_attention import INF, bf16, env, tree  # noqa: F401
from test_gpu_attention_ranges import LAID_OUT, laid_out, one_long

pytestmark = pytest.mark.gpu

DIMS = [64, 96, 128, 256]


def run(env, seed, how, dim, count, length, heads=4, page=32, cache=None, **kw):  # noqa: F811
    """One sequence of `count` tokens and one key head; y and lse of its tokens."""
    rng = np.random.default_rng(seed)
    counts, lengths, sizes = laid_out(how, count, length, heads, 1)
    if "prefix" in kw:
        kw["prefix"] = [kw["prefix"]] + [0] * (len(counts) - 1)
    return cases.run(env, rng, counts, lengths, heads, 1, dim, page, cache=cache or one_long(rng, lengths, 1, dim, page),
                     **kw, **sizes)


@pytest.mark.parametrize("how", LAID_OUT)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("kw", [dict(), dict(slopes=[0.1, 0.0, 0.02, 0.5]), dict(cap=15.0), dict(window=333),
                                dict(slopes=[0.1, 0.0, 0.02, 0.5], cap=200.0, window=450)])
@pytest.mark.parametrize("step", [97, 23])
def test_documents(env, how, dim, kw, step):  # noqa: F811
    """Each row hides another share of blocks that its neighbours see whole."""
    first = [i * step % 700 for i in range(50)]
    run(env, dim + step, how, dim, 50, 700, first=first, **kw)


@pytest.mark.parametrize("how", LAID_OUT)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("kw", [dict(), dict(cap=20.0), dict(cap=300.0), dict(window=200), dict(slopes=[0.3, 0.1, 0.0, 0.7]),
                                dict(slopes=[0.3, 0.01, 0.0, 0.7], cap=30.0, window=300), dict(first=True)])
def test_trees(env, how, dim, kw):  # noqa: F811
    kw = dict(kw)
    if "first" in kw:
        kw["first"] = [i * 61 % 500 for i in range(33)]
    run(env, dim, how, dim, 33, 515, masks=tree(np.random.default_rng(dim), 33), **kw)


@pytest.mark.parametrize("how", LAID_OUT)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("kw", [dict(prefix=420), dict(prefix=420, slopes=[0.1, 0.0, 0.02, 0.5]), dict(prefix=1000, cap=9.0),
                                dict(prefix=430, window=300), dict(window=70), dict(window=350, slopes=[0.1, 0.0, 0.02, 0.5])])
def test_prefixes_and_windows(env, how, dim, kw):  # noqa: F811
    run(env, dim, how, dim, 60, 460, **kw)


@pytest.mark.parametrize("how", LAID_OUT)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("kw", [dict(), dict(cap=15.0), dict(cap=150.0), dict(slopes=[0.01, 0.0, 0.002, 0.1]),
                                dict(slopes=[0.01, 0.0, 0.002, 0.1], cap=15.0)])
@pytest.mark.parametrize("length,page", [(1100, 32), (1187, 64), (1216, 128), (1313, 256)])
def test_long_keys(env, how, dim, kw, length, page):  # noqa: F811
    """More than 1000 keys in front of every row: the loop over whole tiles takes many turns (in
    one part), and ends after whole and half ones."""
    run(env, dim + length, how, dim, 12, length, page=page, **kw)


@pytest.mark.parametrize("how", LAID_OUT)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("kw", [dict(), dict(cap=9.0), dict(first=True)])
def test_pages_that_are_not_there(env, how, dim, kw):  # noqa: F811
    """Entries outside the cache, one after another and alone, in front of whole blocks and behind
    them, and a table that ends before the keys do."""
    rng = np.random.default_rng(dim)
    lengths = laid_out(how, 40, 900, 4, 1)[1]
    kw = dict(kw, first=[i * 53 % 600 for i in range(40)]) if "first" in kw else kw
    c = one_long(rng, lengths, 1, dim, 32)
    c.tables[0, [0, 8, 9, 17, 28]] = -1, 10 ** 6, -7, c.k.shape[0], 2 ** 31 - 1
    run(env, dim, how, dim, 40, 900, cache=c, **kw)
    c = one_long(rng, lengths, 1, dim, 32)
    c.tables = np.ascontiguousarray(c.tables[:, :21])
    run(env, dim, how, dim, 40, 900, cache=c, **kw)


@pytest.mark.parametrize("how", LAID_OUT)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("kw", [dict(), dict(cap=9.0), dict(cap=300.0), dict(window=200), dict(slopes=[0.01, 0.0, 0.002, 0.1]),
                                dict(masks=True), dict(first=True)])
@pytest.mark.parametrize("bits", [0x7F80, 0xFF80, 0x7FC0])
def test_infinities_reach_those_that_see_them(env, how, dim, kw, bits):  # noqa: F811
    """Infinities and NaN among the values, in several blocks, all but one of their elements
    alone in their column."""
    count, length, heads = 25, 460, 2
    kw = dict(kw)
    if kw.pop("masks", None):
        kw["masks"] = tree(np.random.default_rng(3), count)
    if kw.pop("first", None):
        kw["first"] = [i * 53 % 400 for i in range(count)]
    if "slopes" in kw:
        kw["slopes"] = kw["slopes"][:heads]
    rng = np.random.default_rng(bits + dim)
    lengths = laid_out(how, count, length, heads, 1)[1]
    c = one_long(rng, lengths, 1, dim, 32)
    q = bf16(rng, count + 1, heads * dim)
    y0, l0 = run(env, 1, how, dim, count, length, heads, cache=c, q=q, **kw)
    places = {5: 3, 300: dim - 1, 447: 40, 459: 7, 446: 40}
    for place, e in places.items():
        row = synth.f32_to_bf16_bits(np.ones(dim, dtype=np.float32))
        row[e] = bits
        c.set_row(0, place, 0, False, row)
    # what the rows see of them, with ones in their place
    ones = one_long(rng, lengths, 1, dim, 32)
    ones.k, ones.v, ones.tables = c.k, c.v.copy(), c.tables
    for place, e in places.items():
        ones.set_row(0, place, 0, False, synth.f32_to_bf16_bits(np.ones(dim, dtype=np.float32)))
    y1, l1 = run(env, 1, how, dim, count, length, heads, cache=ones, q=q, **kw)
    y2, l2 = run(env, 1, how, dim, count, length, heads, cache=c, q=q, compare=False, **kw)
    assert np.array_equal(l0, l1) and np.array_equal(l1, l2)
    masks = kw.get("masks")
    for i in range(count):
        sees = att.visible(i, count, length, kw.get("window", 0), first=kw["first"][i] if "first" in kw else 0, masks=masks)[0]
        odd = sorted({e for place, e in places.items() if place in sees})
        for h in range(heads):
            got, want = y2[i, h * dim:(h + 1) * dim], y1[i, h * dim:(h + 1) * dim]
            bad = got[odd]
            assert np.isnan(bad).all() if bits == 0x7FC0 else (bad == (INF if bits == 0x7F80 else -INF)).all(), (i, h)
            rest = np.delete(np.arange(dim), odd)
            assert np.array_equal(got[rest], want[rest]), (i, h)


@pytest.mark.parametrize("how", LAID_OUT)
@pytest.mark.parametrize("dim", DIMS)
@pytest.mark.parametrize("kw", [dict(), dict(cap=9.0), dict(cap=300.0), dict(first=True)])
def test_infinities_of_keys_and_queries(env, how, dim, kw):  # noqa: F811
    """A NaN key poisons those that see it and no others; so does a NaN query its own row."""
    count, length, heads = 25, 460, 2
    kw = dict(kw, first=[i * 53 % 400 for i in range(count)]) if "first" in kw else kw
    rng = np.random.default_rng(dim)
    lengths = laid_out(how, count, length, heads, 1)[1]
    c = one_long(rng, lengths, 1, dim, 32)
    q = bf16(rng, count + 1, heads * dim)
    y0, _ = run(env, 1, how, dim, count, length, heads, cache=c, q=q, **kw)
    for place in (450, 459):
        c.set_row(0, place, 0, True, np.full(dim, 0x7FC0))
    q[0][0, dim + 6] = 0x7FC0  # token 0, head 1
    y1, _ = run(env, 1, how, dim, count, length, heads, cache=c, q=q, compare=False, **kw)
    for i in range(count):
        sees = att.visible(i, count, length, first=kw["first"][i] if "first" in kw else 0)[0]
        for h in range(heads):
            got, want = y1[i, h * dim:(h + 1) * dim], y0[i, h * dim:(h + 1) * dim]
            if 450 in sees or 459 in sees or (i, h) == (0, 1):
                assert np.isnan(got).all(), (i, h)
            else:
                assert np.array_equal(got, want), (i, h)
