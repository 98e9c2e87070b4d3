"""Workspace sizes of arguments out of range (CPU)."""
import ctypes as C

import pytest

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
