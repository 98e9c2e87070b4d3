"""Attention at the ends of its arguments' ranges (GPU): marks that hide everything;
each laid out so that the kernel for few rows, the one for many with one part of the keys and
with many take it."""
import numpy as np
import pytest

import test_gpu_attention as cases
from test_gpu_attention import env  # noqa: F401

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
    y, lse = cases.run(env, rng, counts, lengths, 4, 1, dim, 32, first=first, **kw, **sizes)
    for i in (45, 80):
        assert (y[i] == 0).all() and (lse[i] == -np.inf).all()
