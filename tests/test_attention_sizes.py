"""Workspace sizes of arguments out of range, and numbers that the C types cannot hold (CPU)."""
import ctypes as C

import numpy as np
import pytest
import torch

import decode_gemm_bf16_amd as uw

L = uw._lib


@pytest.mark.parametrize("kw", [dict(dim=100), dict(dim=0), dict(dim=32), dict(dim=-64), dict(heads=65, kv_heads=1),
                                dict(heads=1, kv_heads=2), dict(heads=264, kv_heads=8), dict(kv_heads=-1), dict(page=48),
                                dict(page=0), dict(pages=0), dict(pages=1 << 40), dict(tokens=0), dict(tokens=(1 << 20) + 1),
                                dict(seqs=65536), dict(max_tokens=7), dict(max_length=(1 << 30) + 1)])
def test_layer_workspace_out_of_range(kw):
    d = dict(heads=8, kv_heads=2, dim=64, page=32, pages=10, tokens=6, seqs=2, max_tokens=3, max_length=5000)
    sizes = lambda d: (C.byref(uw.CacheConfig(*[d[k] for k, _ in uw.CacheConfig._fields_])),  # noqa: E731
                       d["tokens"], d["seqs"], d["max_tokens"], d["max_length"])
    assert L.uw_attention_workspace_bytes(*sizes(d)) > 0
    d.update(kw)
    assert L.uw_attention_workspace_bytes(*sizes(d)) == 0
    if not {"page", "pages"} & kw.keys():
        for f in (uw.attention_workspace_bytes, uw.attend_workspace_bytes):
            assert f(d["tokens"], d["seqs"], d["heads"], d["kv_heads"], d["dim"], d["max_tokens"], d["max_length"]) == 0


FAR = 1 << 32  # (cut to 32 bits: 0)


@pytest.mark.parametrize("window", [FAR, FAR + 5, 2 ** 31, -2 ** 31 - 1, FAR - 1])
def test_a_window_is_not_cut(window):
    kc = torch.zeros((3, 2, 32, 64), dtype=torch.bfloat16)
    q, i, table = torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.zeros((3, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="window"):
        uw.attend(q, kc, kc, i, i[:3], table, q, window=window)


@pytest.mark.parametrize("cap", [1e-50, 5e-46])
def test_a_cap_is_not_cut(cap):
    """(a cap of 0 would be none)"""
    kc = torch.zeros((3, 2, 32, 64), dtype=torch.bfloat16)
    q, i, table = torch.zeros((4, 256), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32), torch.zeros((3, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="cap"):
        uw.attend(q, kc, kc, i, i[:3], table, q, cap=cap)


@pytest.mark.parametrize("kw", [dict(heads=FAR + 8), dict(kv_heads=FAR + 2), dict(dim=FAR + 64), dict(tokens=(1 << 64) + 6)])
def test_sizes_are_not_cut(kw):
    d = dict(tokens=6, seqs=2, heads=8, kv_heads=2, dim=64, max_tokens=3, max_length=5000)
    d.update(kw)
    for f in (uw.attention_workspace_bytes, uw.attend_workspace_bytes):
        assert f(**d) == 0


def test_pages_are_not_cut():
    p = uw.Pages(4)
    p.take(2)
    far = np.array([FAR + 1])
    for f, bad in ((p.share, far), (p.share, [FAR]), (p.drop, far), (p.drop, [FAR]), (p.share, [0.5]), (p.drop, np.array([1.0])),
                   (p.share, np.array([True])), (p.own, FAR), (p.own, 1 - FAR), (p.take, (1 << 64) + 1)):
        with pytest.raises((ValueError, TypeError)):
            f(bad)
    assert p.holders(FAR) == p.holders(FAR + 1) == p.holders(-FAR) == 0
    assert p.left == 2 and p.holders(0) == p.holders(1) == 1
    p.share([])
    p.drop(np.array([0, 1], dtype=np.uint8))
    assert p.left == 4
    with pytest.raises(ValueError):
        uw.Pages((1 << 64) + 4)


@pytest.mark.timeout(20)
@pytest.mark.parametrize("kind", [np.int32, np.int64, np.uint8])
def test_numbers_as_arrays_hold_them(kind):
    """Page numbers and sizes that come out of arrays."""
    p = uw.Pages(kind(6))
    pages = p.take(kind(4))
    assert p.holders(kind(3)) == 1 and p.own(kind(3)) == 3
    assert p.own(pages[2]) == 2 and p.holders(pages[2]) == 1
    sizes = [kind(v) for v in (6, 2, 8, 2, 64, 3, 100)]
    for f in (uw.attention_workspace_bytes, uw.attend_workspace_bytes):
        assert f(*sizes) == f(*[int(v) for v in sizes])
    for f in (p.own, p.holders, p.take):
        with pytest.raises(TypeError):
            f(1.0)
