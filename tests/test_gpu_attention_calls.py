"""Attention's calls as batches come: many sequences, tokens in front of the first one, the same
call twice (GPU)."""
import numpy as np
import pytest

import test_gpu_attention as cases
from test_gpu_attention import Cache, bf16, env, i32  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_length", [1, 60, 30000])
@pytest.mark.parametrize("seqs,heads,kv,dim", [(64, 4, 1, 64), (65, 4, 2, 128), (200, 2, 1, 96), (130, 8, 1, 256)])
def test_many_sequences(env, seqs, heads, kv, dim, max_length):  # noqa: F811
    """More of them than a wave looks through at once, empty ones and those without keys among them."""
    rng = np.random.default_rng(seqs)
    counts = rng.integers(0, 4, seqs) * (rng.random(seqs) < 0.7)
    counts[rng.integers(0, seqs, 3)] = 45
    counts[-1] = 37
    lengths = counts + rng.integers(0, 60, seqs) * (rng.random(seqs) < 0.8)
    c = Cache(rng, lengths.tolist(), kv, dim, 32, garbage=False)
    cases.run(env, rng, counts.tolist(), lengths.tolist(), heads, kv, dim, 32, cache=c, max_length=max_length)


@pytest.mark.parametrize("count,length", [(1, 90), (3, 5000), (50, 90), (50, 700)])
@pytest.mark.parametrize("max_length", [None, 30000])
def test_tokens_in_front_and_the_same_call_twice(env, count, length, max_length):  # noqa: F811
    """Offsets that begin behind the first tokens, whose rows stay; every call gives the same bits."""
    torch, uw = env
    rng = np.random.default_rng(count)
    heads, kv, dim = 4, 1, 128
    c = Cache(rng, [length], kv, dim, 64)
    kc, vc, tables, lengths = uw.bf16_tensor(c.k), uw.bf16_tensor(c.v), i32(env, c.tables), i32(env, [length])
    q = uw.bf16_tensor(bf16(rng, count, heads * dim)[0])
    laid = max_length or length

    def call(front):
        n = count + 7
        rows = torch.zeros((n, heads * dim), dtype=torch.bfloat16, device="cuda")
        rows[front:front + count] = q
        y, lse = torch.full_like(rows, 7.0), torch.full((n, heads), 7.0, device="cuda")
        work = torch.full((uw.attend_workspace_bytes(n, 1, heads, kv, dim, n, laid),), 255, dtype=torch.uint8, device="cuda")
        uw.attend(rows, kc, vc, i32(env, [front, front + count]), lengths, tables, y, work, lse=lse, max_tokens=n,
                  max_length=laid)
        for t in (y, lse):
            assert (t[:front] == 7.0).all() and (t[front + count:] == 7.0).all()
        return y[front:front + count], lse[front:front + count]

    first = call(0)
    for front in (0, 5, 7):
        assert all(torch.equal(a, b) for a, b in zip(first, call(front)))
