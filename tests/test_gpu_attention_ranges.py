"""Attention at the ends of its arguments' ranges (GPU): marks that hide everything, caps far
above and far below the scores, values near the largest bf16; each laid out so that the
kernel for few rows, the one for many with one part of the keys and with many take it."""
import numpy as np
import pytest

import synth
import test_gpu_attention as cases
from test_gpu_attention import Cache, bf16, env  # noqa: F401

pytestmark = pytest.mark.gpu

INT_MAX = 2 ** 31 - 1
LAID_OUT = ["few", "one part", "parts"]


def laid_out(how, count, length, heads, kv):
    """(counts, lengths, sizes for run) of one sequence of `count` tokens over `length` keys.

    "one part": with 520 / kv empty sequences beside it the call has workgroups enough (512)
    for every key to be in one part, and so many keys by its sizes that the kernel for many
    rows takes it; "parts": a call for 30000 keys divides them."""
    if how == "few":
        return [count], [length], dict(max_length=length)
    assert count * heads // kv > 32
    if how == "parts":
        return [count], [length], dict(max_length=30000)
    empty = -(-520 // kv)
    return [count] + [0] * empty, [length] + [0] * empty, dict(max_length=30000)


def one_long(rng, lengths, kv, dim, page):
    """A cache for the first sequence; the others, empty, have no pages."""
    c = Cache(rng, lengths[:1], kv, dim, page)
    c.tables = np.concatenate([c.tables, np.full((len(lengths) - 1, c.tables.shape[1]), -1, dtype=np.int32)])
    return c


@pytest.mark.parametrize("how", LAID_OUT)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("kw", [dict(cap=20.0), dict(), dict(cap=20.0, slopes=[0.5, 0.25, 0.1, 0.0]), dict(cap=20.0, window=150)])
@pytest.mark.parametrize("mark", [INT_MAX, 700])
def test_documents_and_marks_behind_the_keys(env, how, dim, kw, mark):  # noqa: F811
    """A token's first key far behind the keys hides all of them from it, and none from its
    neighbours, some of which see every key, others documents that begin among them."""
    rng = np.random.default_rng(dim)
    count, length = 90, 400
    counts, lengths, sizes = laid_out(how, count, length, 4, 1)
    first = [i * 37 % 300 for i in range(count)]
    first[45] = first[80] = mark
    y, lse = cases.run(env, rng, counts, lengths, 4, 1, dim, 32, first=first,
                       cache=one_long(rng, lengths, 1, dim, 32), **kw, **sizes)
    for i in (45, 80):
        assert (y[i] == 0).all() and (lse[i] == -np.inf).all()


@pytest.mark.parametrize("how", LAID_OUT)
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("cap", [1e-45, 1e-38, 1.0, 128.0, 129.0, 1e4, 1e8, 3e38])
@pytest.mark.parametrize("kw", [dict(), dict(slopes=[0.5, 0.02, 0.1, 0.0]), dict(scale=3.0)])
def test_caps(env, how, dim, cap, kw):  # noqa: F811
    """Far above the scores a cap leaves them as they are, far below it leaves nothing of them."""
    rng = np.random.default_rng(dim + 1)
    counts, lengths, sizes = laid_out(how, 20, 260, 4, 1)
    q = bf16(rng, 21, 4 * dim)
    for a in q:
        a[7] = 0  # (scores of zero)
    cases.run(env, rng, counts, lengths, 4, 1, dim, 32, cache=one_long(rng, lengths, 1, dim, 32), q=q, cap=cap, out="f32",
              **kw, **sizes)


@pytest.mark.parametrize("how", LAID_OUT)
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("kw", [dict(), dict(cap=20.0), dict(window=200), dict(slopes=[0.01, 0.0, 0.0, 0.1])])
def test_large_values(env, how, dim, kw):  # noqa: F811
    """Values of 2^127, whose unnormalised sums pass float32's range: their mean does not."""
    rng = np.random.default_rng(dim + 2)
    for count, length in ((40, 300), (8 if how == "few" else 10, 2500)):
        counts, lengths, sizes = laid_out(how, count, length, 4, 1)
        c = one_long(rng, lengths, 1, dim, 32)
        sign = rng.random(dim) < 0.5  # one sign an element: nothing cancels
        for p in range(length):
            row = np.where(sign, -1, 1) * np.float32(2.0 ** 127) * rng.uniform(0.9, 1.0, dim)
            c.set_row(0, p, 0, False, synth.f32_to_bf16_bits(row.astype(np.float32)))
        q = bf16(rng, count + 1, 4 * dim)
        for out in ("bf16", "f32"):
            y, _ = cases.run(env, rng, counts, lengths, 4, 1, dim, 32, cache=c, q=q, out=out, **kw, **sizes)
            assert np.isfinite(y).all()
    # a few of them, seen by some tokens only, beside ordinary ones
    counts, lengths, sizes = laid_out(how, 40, 300, 4, 1)
    c = one_long(rng, lengths, 1, dim, 32)
    for p in (5, 250, 280, 299):
        c.set_row(0, p, 0, False, synth.f32_to_bf16_bits(np.full(dim, 2.0 ** 127, dtype=np.float32)))
    y, _ = cases.run(env, rng, counts, lengths, 4, 1, dim, 32, cache=c, **kw, **sizes)
    assert np.isfinite(y).all()
