"""Rows of the cache whose values are not all finite, or not all turned (GPU)."""
import numpy as np
import pytest

import synth
import test_gpu_attention as cases
from oracle import attention as att
from test_gpu_attention import INF, NAN, env, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 600, 1100])
@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("pairs,adjacent", [(13, True), (1, True), (3, True), (30, True), (13, False), (31, False), (8, False)])
def test_what_is_not_turned_stays(env, tokens, type, pairs, adjacent):  # noqa: F811
    """Infinities, NaN and zeros of both signs behind the turned pairs."""
    torch, uw = env
    dim, kv, heads, page = 64, 2, 4, 32
    special = np.array([INF, 1.0, NAN, 2.0, -0.0, -INF, 3.0, -0.0, 0.0, INF, -1.5], dtype=np.float32)
    x = np.resize(special, (tokens, heads, dim)).copy()
    x[:, :, :2 * pairs] = 0.25
    at = np.arange(tokens)
    xt = torch.from_numpy(x.reshape(tokens, -1)).cuda()
    xt = xt if type == "f32" else xt.bfloat16()
    k = xt[:, :kv * dim].contiguous()
    pages = -(-tokens // page)
    kc = torch.zeros((pages, kv, page, dim), dtype=torch.bfloat16, device="cuda")
    vc, qr = torch.zeros_like(kc), torch.zeros((tokens, heads * dim), dtype=torch.bfloat16, device="cuda")
    freqs = torch.full((pairs,), 0.7, device="cuda")
    uw.cache_write(xt, k, k, i32(env, at[None]), freqs, i32(env, at), qr, kc, vc, adjacent=adjacent)
    want = synth.f32_to_bf16_bits(x)[:, :, 2 * pairs:]
    nan = np.isnan(x[:, :, 2 * pairs:])
    turned = 0.25 * np.cos(0.7 * at) - 0.25 * np.sin(0.7 * at)  # element 0 of each head

    def check(got, n):
        rest = got[:, :, 2 * pairs:]
        assert np.array_equal(rest[~nan[:, :n]], want[:, :n][~nan[:, :n]])
        assert np.isnan(synth.bf16_bits_to_f32(rest[nan[:, :n]])).all()
        assert np.allclose(synth.bf16_bits_to_f32(got[:, :, 0]), np.float32(turned)[:, None], atol=2.0 ** -8)

    check(uw.bits_of(qr).reshape(tokens, heads, dim), heads)
    check(att.read_cache(uw.bits_of(kc), np.arange(pages), tokens, True, absent=0), kv)


@pytest.mark.parametrize("tokens", [512, 777, 1023, 6001])
@pytest.mark.parametrize("type", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,dim,page,axes,pairs,adjacent", [(4, 2, 64, 32, 1, 32, False), (6, 6, 96, 32, 2, 17, False),
                                                                   (4, 1, 256, 128, 4, 128, True)])
def test_tiles_of_all_sizes(env, tokens, type, heads, kv, dim, page, axes, pairs, adjacent):  # noqa: F811
    """Tiles of 8 tokens and of 32 with many heads each, over slots in runs and in no order."""
    cases.test_write(env, tokens, type, heads, kv, dim, page, axes, pairs, adjacent)
