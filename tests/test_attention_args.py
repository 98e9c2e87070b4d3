"""Refused arguments of the cache and attention calls: the C entry points check them
on the host before any launch (CPU; addresses are never read), and the Python calls
check what only they see of a tensor."""
import ctypes as C

import pytest
import torch

import decode_gemm_bf16_amd as uw
import synth

L = uw._lib
INVALID, SHAPE, UNSUPPORTED = uw.ERR_INVALID_ARG, uw.ERR_SHAPE, uw.ERR_UNSUPPORTED
AT = [i << 32 for i in range(1, 20)]  # stand-ins for device addresses, 4 GiB apart


def cache(**kw):
    d = dict(heads=8, kv_heads=2, dim=64, page=32, pages=10)
    d.update(kw)
    return uw.CacheConfig(*[d[k] for k, _ in uw.CacheConfig._fields_])


CACHES = [(dict(kv_heads=0), SHAPE), (dict(kv_heads=129, heads=129), SHAPE), (dict(dim=80), SHAPE), (dict(dim=0), SHAPE),
          (dict(page=16), SHAPE), (dict(page=48), SHAPE), (dict(page=512), SHAPE), (dict(pages=0), INVALID),
          (dict(pages=1 << 26), INVALID)]
HEADS = [(dict(heads=0), SHAPE), (dict(heads=9), SHAPE), (dict(heads=130), SHAPE), (dict(heads=258, kv_heads=3), SHAPE)]


def write(config=None, axes=2, pairs=16, adjacent=0, q=AT[0], ldq=512, k=AT[1], ldk=128, v=AT[2], ldv=128, type=0,
          positions=AT[3], freqs=AT[4], axis=AT[5], slots=AT[6], tokens=100, out=AT[7], ldo=512, kc=AT[8], vc=AT[9],
          rotary=True):
    return L.uw_cache_write(C.byref(config or cache()), C.byref(uw.Rotary(axes, pairs, adjacent)) if rotary else None, q,
                            ldq, k, ldk, v, ldv, type, positions, freqs, axis, slots, tokens, out, ldo, kc, vc, None)


@pytest.mark.parametrize("kw,status", [(dict(config=cache(**c)), s) for c, s in CACHES + HEADS] + [
    (dict(rotary=False), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(slots=None), INVALID),
    (dict(out=None), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(positions=None), INVALID),
    (dict(freqs=None), INVALID), (dict(tokens=0), INVALID), (dict(tokens=(1 << 20) + 1), INVALID), (dict(type=2), INVALID),
    (dict(axes=0), INVALID), (dict(axes=5), INVALID), (dict(pairs=-1), SHAPE), (dict(pairs=33), SHAPE),
    (dict(ldq=504), SHAPE), (dict(ldq=516), SHAPE), (dict(ldk=120), SHAPE), (dict(ldv=132), SHAPE), (dict(ldo=500), SHAPE),
    (dict(q=AT[0] + 8), INVALID), (dict(k=AT[1] + 4), INVALID), (dict(out=AT[7] + 2), INVALID), (dict(kc=AT[8] + 8), INVALID),
    (dict(positions=AT[3] + 2), INVALID), (dict(slots=AT[6] + 1), INVALID), (dict(axis=AT[5] + 3), INVALID),
    (dict(out=AT[0]), INVALID), (dict(out=AT[1] + 16), INVALID), (dict(kc=AT[2]), INVALID), (dict(vc=AT[8] + 16), INVALID),
    (dict(vc=AT[7] + 1024), INVALID), (dict(out=AT[3] - 64), INVALID), (dict(kc=AT[6] - 64), INVALID),
    (dict(vc=AT[4]), INVALID), (dict(out=AT[5]), INVALID)])
def test_cache_write_refuses(kw, status):
    assert write(**kw) == status
    assert uw.last_error()


def attend(config=None, scale=0.1, cap=0.0, window=0, q=AT[0], ldq=512, kc=AT[1], vc=AT[2], offsets=AT[3],
           lengths=AT[4], tables=AT[5], ldt=20, max_pages=20, slopes=None, prefix=None, first=None, mask=None, words=0,
           tokens=100, seqs=4, max_tokens=100, max_length=100000, y=AT[6], ldy=512, type=1, lse=AT[7], work=AT[8],
           work_bytes=1 << 30, options=True):
    return L.uw_attend(C.byref(config or cache()), C.byref(uw.AttendConfig(scale, cap, window)) if options else None, q,
                       ldq, kc, vc, offsets, lengths, tables, ldt, max_pages, slopes, prefix, first, mask, words, tokens,
                       seqs, max_tokens, max_length, y, ldy, type, lse, work, work_bytes, None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("kw,status", [(dict(config=cache(**c)), s) for c, s in CACHES + HEADS] + [
    (dict(options=False), INVALID), (dict(q=None), INVALID), (dict(kc=None), INVALID), (dict(offsets=None), INVALID),
    (dict(lengths=None), INVALID), (dict(tables=None), INVALID), (dict(y=None), INVALID), (dict(tokens=0), INVALID),
    (dict(tokens=(1 << 20) + 1), INVALID), (dict(seqs=0), INVALID), (dict(seqs=65536), INVALID),
    (dict(max_pages=0), SHAPE), (dict(ldt=19), SHAPE), (dict(max_tokens=0), INVALID), (dict(max_tokens=101), INVALID),
    (dict(max_length=0), INVALID), (dict(max_length=(1 << 30) + 1), INVALID), (dict(type=2), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=NAN), INVALID), (dict(scale=INF), INVALID),
    (dict(cap=-1.0), INVALID), (dict(cap=NAN), INVALID), (dict(cap=INF), INVALID), (dict(window=-1), INVALID),
    (dict(mask=AT[9], words=0), SHAPE), (dict(mask=AT[9], words=1025), SHAPE),
    (dict(mask=AT[9], words=2, prefix=AT[10]), UNSUPPORTED), (dict(ldq=508), SHAPE), (dict(ldy=504), SHAPE),
    (dict(q=AT[0] + 8), INVALID), (dict(y=AT[6] + 8), INVALID), (dict(vc=AT[2] + 2), INVALID),
    (dict(offsets=AT[3] + 1), INVALID), (dict(mask=AT[9] + 4, words=2), INVALID), (dict(lse=AT[7] + 2), INVALID),
    (dict(slopes=AT[9] + 2), INVALID), (dict(work=None), INVALID), (dict(work_bytes=64), INVALID),
    (dict(work=AT[8] + 8), INVALID), (dict(y=AT[0]), INVALID), (dict(y=AT[1]), INVALID), (dict(lse=AT[6] + 64), INVALID),
    (dict(work=AT[0] + 16), INVALID), (dict(work=AT[2]), INVALID), (dict(work=AT[6] + 16), INVALID),
    (dict(lse=AT[4]), INVALID), (dict(y=AT[5] - 64), INVALID), (dict(slopes=AT[6] + 16), INVALID),
    (dict(first=AT[8]), INVALID), (dict(mask=AT[7], words=1), INVALID), (dict(prefix=AT[8] + 16), INVALID)])
def test_attend_refuses(kw, status):
    assert uw.attend_workspace_bytes(100, 4, 8, 2, 64, 100, 100000) > 64  # (the keys are split, the workspace is needed)
    assert attend(**kw) == status
    assert uw.last_error()


def test_attend_workspace_out_of_range():
    good = dict(tokens=100, seqs=4, heads=8, kv_heads=2, dim=64, max_tokens=1, max_length=100000)
    assert uw.attend_workspace_bytes(*good.values()) > 0
    for kw in (dict(tokens=0), dict(seqs=0), dict(heads=7), dict(kv_heads=0), dict(dim=100), dict(max_tokens=0),
               dict(max_tokens=101), dict(max_length=0)):
        assert uw.attend_workspace_bytes(*dict(good, **kw).values()) == 0, kw
    # few keys are not split
    assert uw.attend_workspace_bytes(*dict(good, max_length=100).values()) == 0


def test_cache_moves_refuse():
    def copy(config=None, layers=3, kc=AT[0], vc=AT[1], src=AT[2], dst=AT[3], n=10):
        return L.uw_cache_copy_pages(C.byref(config or cache(heads=0)), layers, kc, vc, src, dst, n, None)

    for kw, status in [(dict(config=cache(**c)), s) for c, s in CACHES] + [
            (dict(kc=None), INVALID), (dict(src=None), INVALID), (dict(dst=None), INVALID), (dict(layers=0), INVALID),
            (dict(layers=4097), INVALID), (dict(n=0), INVALID), (dict(n=11), INVALID), (dict(src=AT[2] + 2), INVALID),
            (dict(vc=AT[0] + 4096), INVALID), (dict(src=AT[0] + 64), INVALID), (dict(dst=AT[1] + 64), INVALID)]:
        assert copy(**kw) == status, kw

    def keep(config=None, layers=3, kc=AT[0], vc=AT[1], tables=AT[2], ldt=20, max_pages=20, starts=AT[3], kept=AT[4],
             most=8, seqs=4, lengths=AT[5]):
        return L.uw_cache_keep(C.byref(config or cache(heads=0)), layers, kc, vc, tables, ldt, max_pages, starts, kept,
                               most, seqs, lengths, None)

    for kw, status in [(dict(config=cache(**c)), s) for c, s in CACHES] + [
            (dict(vc=None), INVALID), (dict(tables=None), INVALID), (dict(starts=None), INVALID), (dict(kept=None), INVALID),
            (dict(lengths=None), INVALID), (dict(layers=0), INVALID), (dict(seqs=0), INVALID), (dict(seqs=65536), INVALID),
            (dict(max_pages=21), SHAPE), (dict(most=0), SHAPE), (dict(most=257), SHAPE), (dict(kept=AT[4] + 1), INVALID),
            (dict(lengths=AT[3]), INVALID), (dict(lengths=AT[4] + 8), INVALID), (dict(lengths=AT[0] + 16), INVALID),
            (dict(tables=AT[1] + 16), INVALID), (dict(vc=AT[0]), INVALID)]:
        assert keep(**kw) == status, kw


def test_python_refuses_tensors():
    kc = torch.zeros((3, 2, 32, 64), dtype=torch.bfloat16)
    q = torch.zeros((4, 256), dtype=torch.bfloat16)
    k = torch.zeros((4, 128), dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(8)
    pos = torch.zeros((1, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="current GPU"):
        uw.cache_write(q, k, k, pos, f, i, q, kc, kc)
    with pytest.raises(TypeError):
        uw.cache_write(q, k.half(), k, pos, f, i, q, kc, kc)
    with pytest.raises((TypeError, ValueError)):  # q of another type than k
        uw.cache_write(q.float(), k, k, pos, f, i, q, kc, kc)
    with pytest.raises(ValueError, match="dimensions"):
        uw.cache_write(q, k, k, pos, f, i, q, kc[0], kc[0])
    with pytest.raises(TypeError):
        uw.attend(q, None, kc, i, i, pos, q)
    with pytest.raises(ValueError, match="columns"):
        uw.attend(q[:, :100], kc, kc, i, i, pos, q)
    with pytest.raises(ValueError, match="current GPU"):
        uw.attend(q, kc, kc, i, i, pos, q)
    with pytest.raises(ValueError, match="dimensions"):
        uw.cache_copy_pages(kc, kc, i, i)
    with pytest.raises(ValueError, match="dimensions"):
        uw.cache_keep(kc, kc, pos, i, pos, i)


def test_layer_refuses():
    host = uw.FMT_PALETTE | uw.ENC_HOST_ONLY
    mk = lambda r, c, s: uw.Matrix(synth.weights(r, c, s, 0.0, 0), host)  # noqa: E731
    q, k, v, o = mk(128, 192, 1), mk(64, 192, 2), mk(64, 192, 3), mk(192, 128, 4)
    config = cache(heads=2, kv_heads=1, dim=64, page=32, pages=10)
    good = dict(positions=AT[3], freqs=AT[4], axis=None, slots=AT[5], offsets=AT[6], lengths=AT[7], tables=AT[8], slopes=None,
                prefix=None, first=None, mask=None, tokens=6, seqs=2, max_tokens=3, max_length=5000, ldt=20, max_pages=20,
                mask_words=0)
    need = L.uw_attention_workspace_bytes(C.byref(config), 6, 2, 3, 5000)
    assert need > 0

    def call(hs=(q, k, v, o), pipelines=(4, 4, 4, 4), config=config, rotary=uw.Rotary(1, 32, 0), options=uw.AttendConfig(0.1, 0, 0),
             x=AT[0], kc=AT[1], vc=AT[2], y=AT[9], work=AT[10], work_bytes=need, batch=True, **kw):
        b = uw.AttentionBatch(**dict(good, **kw))
        by = lambda p: None if p is None else C.byref(p)  # noqa: E731
        return L.uw_attention_forward(*[h and h._h for h in hs], pipelines and (C.c_int32 * 4)(*pipelines), by(config), by(rotary),
                                      by(options), C.byref(b) if batch else None, x, kc, vc, y, work, work_bytes)

    assert call() == UNSUPPORTED  # every check passed but the one for device copies
    for kw, status in [(dict(hs=(None, k, v, o)), INVALID), (dict(hs=(q, k, v, None)), INVALID), (dict(pipelines=None), INVALID),
                       (dict(config=None), INVALID), (dict(batch=False), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
                       (dict(work=None), INVALID), (dict(hs=(q, k, v, q)), SHAPE), (dict(hs=(k, k, v, o)), SHAPE),
                       (dict(hs=(q, q, v, o)), SHAPE), (dict(config=cache(heads=2, kv_heads=2, dim=64)), SHAPE),
                       (dict(tokens=0), INVALID), (dict(tokens=(1 << 20) + 1), INVALID), (dict(seqs=0), INVALID),
                       (dict(max_tokens=7), INVALID), (dict(max_length=0), INVALID), (dict(work_bytes=need - 1), INVALID),
                       (dict(work=AT[10] + 128), INVALID), (dict(x=AT[0] + 8), INVALID), (dict(y=AT[9] + 4), INVALID)]:
        assert call(**kw) == status, kw
        assert uw.last_error()
    side = mk(64, 192, 2)
    side.set_streams(main=0x1000)  # never used: the check fails first
    assert call(hs=(q, side, v, o)) == INVALID and "stream" in uw.last_error()
    for kw in (dict(tokens=0), dict(seqs=0), dict(max_tokens=0), dict(max_length=0), dict(max_tokens=7)):
        d = dict(tokens=6, seqs=2, max_tokens=3, max_length=5000)
        d.update(kw)
        assert L.uw_attention_workspace_bytes(C.byref(config), *d.values()) == 0, kw
    assert L.uw_attention_workspace_bytes(C.byref(cache(heads=3)), 6, 2, 3, 5000) == 0
    assert L.uw_attention_workspace_bytes(None, 6, 2, 3, 5000) == 0


def test_a_window_asks_for_no_more_workspace():
    """The workspace is sized without the window that the call has."""
    for heads, kv, dim in ((8, 2, 64), (32, 8, 128), (4, 1, 256)):
        for tokens, seqs in ((1, 1), (24, 1), (61, 4), (700, 3)):
            for length in (100, 3000, 40000, 200000):
                need = uw.attend_workspace_bytes(tokens * seqs, seqs, heads, kv, dim, tokens, length)
                for window in (0, 1, 500, 3000, 30000, 2 ** 31 - 1):
                    # (refused for its tables, the last of the checks before the workspace's that can be)
                    good = dict(config=cache(heads=heads, kv_heads=kv, dim=dim), ldq=heads * dim, ldy=heads * dim, window=window,
                                tokens=tokens * seqs, seqs=seqs, max_tokens=tokens, max_length=length, lse=AT[5])
                    assert attend(work=AT[8] if need else None, work_bytes=need, **good) == INVALID
                    assert "overlap" in uw.last_error(), (heads, tokens, seqs, length, window, uw.last_error())
