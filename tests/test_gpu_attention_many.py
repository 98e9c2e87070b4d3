"""Attention's cases again, laid out for other lengths than they have, so that whatever the
sizes the kernel for many rows takes those of more than 32 rows: with one part of the keys
(laid out for one key) and with many (GPU)."""
import pytest

import test_gpu_attention as cases
from test_gpu_attention import env  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[1, 30000], autouse=True)
def laid_out(request, monkeypatch):
    plain = cases.run
    monkeypatch.setattr(cases, "run", lambda *a, **kw: plain(*a, **dict(kw, max_length=request.param)))


@pytest.mark.parametrize("heads,kv,dim,page", [(4, 2, 64, 32), (8, 2, 128, 64), (6, 2, 96, 32), (4, 1, 256, 128), (8, 1, 128, 32)])
@pytest.mark.parametrize("counts,lengths", [([40], [40]), ([37, 1, 0, 5], [101, 64, 17, 5]), ([150, 3], [400, 290])])
def test_sizes(env, heads, kv, dim, page, counts, lengths):  # noqa: F811
    cases.test_sizes(env, heads, kv, dim, page, counts, lengths)


@pytest.mark.parametrize("counts,lengths", [([50, 3, 1], [130, 90, 40]), ([33], [700]), ([300], [500])])
@pytest.mark.parametrize("what", ["window 1", "window 40", "prefix", "documents", "prefix window", "window huge"])
def test_masks(env, counts, lengths, what):  # noqa: F811
    cases.test_masks(env, counts, lengths, what)


@pytest.mark.parametrize("counts,lengths", [([50, 3], [130, 90]), ([200], [300])])
@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("kw", [dict(cap=5.0), dict(cap=0.01), dict(slopes=[0.5, 0.25, 0.1, 0.0]),
                                dict(cap=30.0, slopes=[2.0, 0.01, 0.0, 0.3], window=60), dict(scale=3.0),
                                dict(slopes=[0.1] * 4, prefix=[250, 5])])
def test_scores(env, counts, lengths, dim, kw):  # noqa: F811
    cases.test_scores(env, counts, lengths, dim, dict(kw, prefix=kw["prefix"][:len(counts)]) if "prefix" in kw else kw)


@pytest.mark.parametrize("counts,lengths,words", [([64, 30], [300, 95], 1), ([100, 9], [101, 41], 2), ([61], [1000], 1)])
@pytest.mark.parametrize("kw", [dict(), dict(cap=20.0), dict(window=5), dict(slopes=[0.3, 0.1, 0.0, 0.7], window=70),
                                dict(first=7)])
def test_trees(env, counts, lengths, words, kw):  # noqa: F811
    cases.test_trees(env, counts, lengths, words, kw)


def test_pages_that_are_not_there(env):  # noqa: F811
    cases.test_pages_that_are_not_there(env)


def test_nothing_to_see(env):  # noqa: F811
    cases.test_nothing_to_see(env)


@pytest.mark.parametrize("counts,lengths,kw", [([40], [70], {}), ([40], [300], dict(cap=9.0)), ([150], [300], dict(window=90))])
@pytest.mark.parametrize("bits", [0x7F80, 0xFF80, 0x7FC0])
def test_infinities_reach_those_that_see_them(env, counts, lengths, kw, bits):  # noqa: F811
    cases.test_infinities_reach_those_that_see_them(env, counts, lengths, kw, bits)


def test_infinities_of_keys_and_queries(env):  # noqa: F811
    cases.test_infinities_of_keys_and_queries(env)


def test_large_scores(env):  # noqa: F811
    cases.test_large_scores(env)
