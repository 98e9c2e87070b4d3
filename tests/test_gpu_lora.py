"""Low-rank adapters beside a projection on the GPU against the 64-bit oracle,
within the bound that the oracle derives from the float32 sums; and a layer of
compressed projections with adapters and routed experts together."""
import numpy as np
import pytest

import oracle
import synth
from oracle import routing

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import decode_gemm_bf16_amd as uw
    return torch, uw


def values(rng, *shape):
    """bf16 bit patterns of standard normal values, and the values."""
    bits = synth.f32_to_bf16_bits(rng.standard_normal(shape, dtype=np.float32))
    return bits, synth.bf16_bits_to_f32(bits).astype(np.float64)


class Setup:
    """A projection's adapters on the GPU and their values: {slot: (A, B, scale)}."""

    def __init__(self, env, rng, slots, rows, cols, max_rank, ranks):
        torch, uw = env
        self.h = uw.Adapters(slots, rows, cols, max_rank)
        self.values = {}
        for i, r in enumerate(ranks):
            if r == 0:
                continue
            ab, a = values(rng, r, cols)
            bb, b = values(rng, rows, r)
            scale = float(np.float32(rng.normal()))
            self.h.load(i, uw.bf16_tensor(ab), uw.bf16_tensor(bb), scale)
            self.values[i] = (a, b, scale)


def apply(env, setups, x, index, bases, work_fill=255, stream=None, xdev=None):
    """One call out of place; returns float64 outputs."""
    torch, uw = env
    t = len(index)
    d = torch.from_numpy(np.asarray(index, dtype=np.int32)).cuda()
    hs = [s.h for s in setups]
    plan = torch.full((uw.lora_plan_bytes(t, hs[0].slots),), 255, dtype=torch.uint8, device="cuda")
    work = torch.full((uw.lora_workspace_bytes(hs, t),), work_fill, dtype=torch.uint8, device="cuda")
    ys = [torch.full((t, h.rows), NAN, device="cuda") for h in hs]
    print(f"lora {t} tokens, {hs[0].slots} slots of {hs[0].max_rank}, {[h.rows for h in hs]} x {hs[0].cols}", flush=True)
    uw.lora_plan(d, hs[0].slots, plan, stream=stream)
    uw.lora_apply(hs, plan, uw.bf16_tensor(x) if xdev is None else xdev, ys, work,
                  bases=[None if b is None else torch.from_numpy(b).cuda() for b in bases], stream=stream)
    torch.cuda.synchronize()
    return [y.cpu().numpy().astype(np.float64) for y in ys]


def check(got, xv, index, adapters, base):
    want = routing.lora(xv, index, adapters, base)
    bound = routing.lora_error_bound(xv, index, adapters, base)
    assert (np.abs(got - want) <= bound).all(), np.max(np.abs(got - want) / np.maximum(bound, 1e-300))
    plain = [t for t, i in enumerate(index) if int(i) not in adapters]
    assert np.array_equal(got[plain], base[plain].astype(np.float64))  # no adapter: the base itself


@pytest.mark.parametrize("tokens", [1, 2, 15, 16, 17, 63, 64, 65, 130, 333])
@pytest.mark.parametrize("rows,cols,max_rank", [(16, 64, 1), (272, 576, 8), (256, 128, 16), (528, 64, 17),
                                                 (64, 2048, 64), (32, 192, 65), (48, 320, 256)])
def test_sizes(env, tokens, rows, cols, max_rank):
    rng = np.random.default_rng(tokens * 7 + rows + max_rank)
    slots = 5
    ranks = [max_rank, 0, max(1, max_rank // 2), 1, max(1, max_rank - 3)]
    s = Setup(env, rng, slots, rows, cols, max_rank, ranks)
    x, xv = values(rng, tokens, cols)
    index = rng.integers(-2, slots + 2, size=tokens)  # some outside the slots, some in the empty one
    base = rng.standard_normal((tokens, rows), dtype=np.float32)
    check(apply(env, [s], x, index, [base])[0], xv, index, s.values, base)


@pytest.mark.parametrize("pattern", ["one adapter", "none", "each its own", "runs", "one long"])
def test_batches(env, pattern):
    rng = np.random.default_rng(8)
    tokens, slots, rows, cols = 200, 40, 144, 256
    s = Setup(env, rng, slots, rows, cols, 12, rng.integers(0, 13, size=slots))
    index = {"one adapter": np.full(tokens, 3), "none": np.full(tokens, -1), "each its own": np.arange(tokens) % slots,
             "runs": np.sort(rng.integers(-1, slots, size=tokens)),
             "one long": np.where(np.arange(tokens) < 150, 2, rng.integers(0, slots, size=tokens))}[pattern]
    x, xv = values(rng, tokens, cols)
    base = rng.standard_normal((tokens, rows), dtype=np.float32)
    check(apply(env, [s], x, index, [base])[0], xv, index, s.values, base)


def test_many_slots_and_projections(env):
    """Several projections in one call, of other rows and ranks; more slots than a
    sort's smallest form; zeros as a base."""
    rng = np.random.default_rng(9)
    tokens, slots, cols = 150, 1100, 192
    ranks = np.zeros(slots, dtype=int)
    used = rng.permutation(slots)[:60]
    ranks[used] = 8
    setups = [Setup(env, rng, slots, rows, cols, m, np.minimum(ranks, m)) for rows, m in ((272, 8), (16, 4), (640, 70), (48, 8))]
    index = np.where(rng.random(tokens) < 0.2, -1, rng.choice(used, size=tokens))
    x, xv = values(rng, tokens, cols)
    bases = [rng.standard_normal((tokens, s.h.rows), dtype=np.float32) for s in setups]
    bases[2] = None
    for s, b, got in zip(setups, bases, apply(env, setups, x, index, bases)):
        check(got, xv, index, s.values, np.zeros(got.shape) if b is None else b)


def test_long_batch(env):
    """More tokens than one sort workgroup takes."""
    rng = np.random.default_rng(10)
    tokens, slots, rows, cols = 9000, 6, 32, 64
    s = Setup(env, rng, slots, rows, cols, 4, [4, 3, 0, 2, 1, 4])
    index = rng.integers(-1, slots, size=tokens)
    x, xv = values(rng, tokens, cols)
    base = rng.standard_normal((tokens, rows), dtype=np.float32)
    check(apply(env, [s], x, index, [base])[0], xv, index, s.values, base)


def test_wide_outputs_with_few_tokens_a_slot(env):
    """The form of the expansion for batches of few tokens per slot (1024 columns a
    workgroup), on tiles of 1, 4, 5, 6 and 64 tokens, with an end inside a workgroup
    and inside a wave's 64 columns."""
    rng = np.random.default_rng(20)
    tokens, slots, rows, cols = 130, 40, 12336, 64
    s = Setup(env, rng, slots, rows, cols, 20, rng.integers(0, 21, size=slots))
    index = np.concatenate([np.full(70, 3), np.full(5, 4), np.full(4, 5), np.full(4, -1), rng.integers(6, slots, size=47)])
    rng.shuffle(index)
    x, xv = values(rng, tokens, cols)
    base = rng.standard_normal((tokens, rows), dtype=np.float32)
    check(apply(env, [s], x, index, [base])[0], xv, index, s.values, base)


def test_output_larger_than_the_caches(env):
    """y of 128 MiB and more is stored past the caches."""
    rng = np.random.default_rng(21)
    tokens, slots, rows, cols = 2100, 3, 16384, 64
    s = Setup(env, rng, slots, rows, cols, 4, [4, 2, 0])
    index = np.sort(rng.integers(-1, slots, size=tokens))
    x, xv = values(rng, tokens, cols)
    base = rng.standard_normal((tokens, rows), dtype=np.float32)
    check(apply(env, [s], x, index, [base])[0], xv, index, s.values, base)


@pytest.mark.parametrize("tokens,rows,cols,max_rank,slots", [
    (40, 64, 4160, 40, 3),    # 65 batches of columns in uneven parts
    (3, 1040, 8192, 32, 2),   # few tokens, A too large for one launch
    (4, 1040, 8192, 16, 2),   # A of exactly the size that one launch takes
    (4, 1040, 8256, 16, 2),   # and past it
    (100, 64, 14336, 64, 50),
    (70, 2064, 1024, 256, 1),
])
def test_long_columns(env, tokens, rows, cols, max_rank, slots):
    rng = np.random.default_rng(tokens + cols)
    s = Setup(env, rng, slots, rows, cols, max_rank, [max(1, max_rank - i % 5) for i in range(slots)])
    x, xv = values(rng, tokens, cols)
    index = rng.integers(-1, slots, size=tokens)
    base = rng.standard_normal((tokens, rows), dtype=np.float32)
    check(apply(env, [s], x, index, [base])[0], xv, index, s.values, base)


@pytest.mark.parametrize("tokens", [1, 2, 3, 4])
@pytest.mark.parametrize("projections", [2, 3, 4])
def test_one_launch_of_several_projections(env, tokens, projections):
    """Few tokens on projections of other rows (within one workgroup's 512, past it, an
    end inside a wave's 64) and other ranks; some tokens share a slot."""
    rng = np.random.default_rng(40 + tokens + 10 * projections)
    slots, cols = 3, 320
    shapes = ((208, 16), (1040, 64), (16, 3), (528, 33))[:projections]
    setups = [Setup(env, rng, slots, n, cols, m, [m, max(1, m // 2), 0]) for n, m in shapes]
    x, xv = values(rng, tokens, cols)
    for index in (rng.integers(-1, slots, size=tokens), np.full(tokens, 1), np.full(tokens, 2)):
        bases = [rng.standard_normal((tokens, n), dtype=np.float32) for n, _ in shapes]
        for s, base, got in zip(setups, bases, apply(env, setups, x, index, bases)):
            check(got, xv, index, s.values, base)


@pytest.mark.parametrize("max_rank", [17, 64, 130])
@pytest.mark.parametrize("tokens,slots,cols,shapes", [
    (2000, 100, 192, (32,)),
    (1000, 112, 2048, (16,)),       # and two parts of the columns
    (700, 60, 192, (48, 16, 80)),
])
def test_half_tiles(env, max_rank, tokens, slots, cols, shapes):
    """So many tiles that the product with A takes 32 tokens a workgroup: tiles of one
    token to 64, ranks of one block of 16 to three of 64."""
    rng = np.random.default_rng(tokens + max_rank)
    ranks = np.zeros(slots, dtype=int)
    used = rng.permutation(slots)[:9]
    ranks[used] = [max_rank, max_rank, max_rank - 1, (max_rank + 1) // 2, 1, 16, 17, max_rank, max_rank - 13 if max_rank > 17 else 5]
    setups = [Setup(env, rng, slots, n, cols, max_rank, ranks) for n in shapes]
    index = np.concatenate([np.repeat(used[:6], [1, 31, 32, 33, 63, 64]), rng.choice(used, size=tokens - 274),
                            rng.integers(-1, slots, size=50)])
    rng.shuffle(index)
    x, xv = values(rng, tokens, cols)
    bases = [rng.standard_normal((tokens, n), dtype=np.float32) for n in shapes]
    for s, base, got in zip(setups, bases, apply(env, setups, x, index, bases)):
        check(got, xv, index, s.values, base)


@pytest.mark.parametrize("max_rank", [64, 70])
@pytest.mark.parametrize("slots", [3, 600])  # 256 columns a workgroup, and 1024
def test_ranks_of_an_output_larger_than_the_caches(env, max_rank, slots):
    rng = np.random.default_rng(max_rank + slots)
    tokens, rows, cols = 2100, 16384, 64
    ranks = np.zeros(slots, dtype=int)
    used = rng.permutation(slots)[:8]
    ranks[used] = [max_rank, max_rank - 3, 17, 64, 5, max_rank, 48, 1][:len(used)]
    s = Setup(env, rng, slots, rows, cols, max_rank, ranks)
    # a few tokens with adapters, in tiles of 1, 3, 4, 5 tokens and more; the others keep their base
    index = np.full(tokens, -1)
    index[:160] = np.concatenate([np.repeat(used[:3], [70, 33, 4]), rng.choice(used, size=53)])
    if slots > 8:
        index[:160] = np.concatenate([np.repeat(used, [1, 3, 4, 5, 40, 64, 33, 2]), rng.choice(used, size=8)])
    order = rng.permutation(tokens)
    index = index[order]
    x, xv = values(rng, tokens, cols)
    base = rng.standard_normal((tokens, rows), dtype=np.float32)
    check(apply(env, [s], x, index, [base])[0], xv, index, s.values, base)


@pytest.mark.parametrize("shapes", [((8208, 16), (2064, 130)), ((8208, 130), (272, 20)), ((4112, 70), (8208, 64), (1040, 5))])
def test_wide_outputs_of_several_projections(env, shapes):
    """1024 columns a workgroup on projections of other rows and ranks, on tiles of up
    to four tokens, up to 32 and more."""
    rng = np.random.default_rng(sum(n + m for n, m in shapes))
    tokens, slots, cols = 200, 50, 128
    ranks = rng.integers(0, 131, size=slots)
    ranks[:4] = 130
    setups = [Setup(env, rng, slots, n, cols, m, np.minimum(ranks, m)) for n, m in shapes]
    index = np.concatenate([np.repeat([0, 1, 2, 3], [64, 35, 7, 3]), rng.integers(-1, slots, size=91)])
    rng.shuffle(index)
    x, xv = values(rng, tokens, cols)
    bases = [rng.standard_normal((tokens, n), dtype=np.float32) for n, _ in shapes]
    for s, base, got in zip(setups, bases, apply(env, setups, x, index, bases)):
        check(got, xv, index, s.values, base)


def test_small_magnitudes(env):
    """Products with A near 2^-110, whose lower parts bf16 holds as denormals."""
    rng = np.random.default_rng(22)
    tokens, rows, cols = 20, 64, 64
    torch, uw = env
    h = uw.Adapters(1, rows, cols, 16)
    a = synth.f32_to_bf16_bits(rng.standard_normal((16, cols), dtype=np.float32) * np.float32(2.0 ** -57))
    b = synth.f32_to_bf16_bits(rng.standard_normal((rows, 16), dtype=np.float32) * np.float32(2.0 ** 60))
    x = synth.f32_to_bf16_bits(rng.standard_normal((tokens, cols), dtype=np.float32) * np.float32(2.0 ** -57))
    h.load(0, uw.bf16_tensor(a), uw.bf16_tensor(b), 1.0)
    s = Setup.__new__(Setup)
    s.h = h
    av, bv, xv = (synth.bf16_bits_to_f32(v).astype(np.float64) for v in (a, b, x))
    base = np.zeros((tokens, rows), dtype=np.float32)
    index = np.zeros(tokens, dtype=int)
    check(apply(env, [s], x, index, [base])[0], xv, index, {0: (av, bv, 1.0)}, base)


def test_far_offsets(env):
    """x, base and y whose rows lie past 2^31 elements."""
    torch, uw = env
    rng = np.random.default_rng(23)
    tokens, rows, cols, wide = 40000, 32, 64, 65536
    s = Setup(env, rng, 2, rows, cols, 4, [4, 3])
    far = np.sort(rng.choice(np.arange(33000, tokens), size=60, replace=False))
    index = np.full(tokens, -1)
    index[far] = rng.integers(0, 2, size=60)
    index[5] = 1
    at = np.concatenate([[5], far])
    xb, xv = values(rng, len(at), cols)
    base = rng.standard_normal((len(at), rows), dtype=np.float32)
    x = torch.zeros((tokens, wide), dtype=torch.bfloat16, device="cuda")[:, wide - cols:]
    y = torch.zeros((tokens, wide), device="cuda")[:, wide - rows:]
    where = torch.from_numpy(at).cuda()
    x[where] = uw.bf16_tensor(xb)
    y[where] = torch.from_numpy(base).cuda()
    plan = torch.empty(uw.lora_plan_bytes(tokens, 2), dtype=torch.uint8, device="cuda")
    work = torch.empty(uw.lora_workspace_bytes([s.h], tokens), dtype=torch.uint8, device="cuda")
    print("lora far offsets", flush=True)
    uw.lora_plan(torch.from_numpy(index.astype(np.int32)).cuda(), 2, plan)
    uw.lora_apply([s.h], plan, x, [y], work)
    torch.cuda.synchronize()
    check(y[where].cpu().numpy().astype(np.float64), xv, index[at], s.values, base)
    rest = torch.ones(tokens, dtype=torch.bool, device="cuda")
    rest[where] = False
    assert not y[rest].any()


def test_most_tokens_and_slots(env):
    """2^20 tokens over 4000 slots, most of them empty: every tile of the plan."""
    torch, uw = env
    rng = np.random.default_rng(25)
    tokens, slots, rows, cols = 1 << 20, 4000, 16, 64
    ranks = np.zeros(slots, dtype=int)
    ranks[::500] = 3
    s = Setup(env, rng, slots, rows, cols, 3, ranks)
    index = rng.integers(-1, slots, size=tokens)
    d = torch.from_numpy(index.astype(np.int32)).cuda()
    x = torch.randn((tokens, cols), device="cuda").to(torch.bfloat16)
    base = torch.randn((tokens, rows), device="cuda")
    y = torch.full_like(base, NAN)
    plan = torch.empty(uw.lora_plan_bytes(tokens, slots), dtype=torch.uint8, device="cuda")
    work = torch.empty(uw.lora_workspace_bytes([s.h], tokens), dtype=torch.uint8, device="cuda")
    print("lora 2^20 tokens, 4000 slots", flush=True)
    uw.lora_plan(d, slots, plan)
    uw.lora_apply([s.h], plan, x, [y], work, bases=[base])
    torch.cuda.synchronize()
    some = np.isin(index, list(s.values))
    none = torch.from_numpy(~some).cuda()
    assert torch.equal(y[none], base[none])
    at = np.nonzero(some)[0]
    assert len(at) > 1000
    where = torch.from_numpy(at).cuda()
    check(y[where].cpu().numpy().astype(np.float64), x[where].double().cpu().numpy(), index[at], s.values,
          base[where].cpu().numpy())


def test_no_bases_and_a_captured_load(env):
    """The C call without bases writes the adapters' part alone; a load that is
    captured takes what its sources hold at each replay."""
    import ctypes as C
    torch, uw = env
    rng = np.random.default_rng(26)
    tokens, rows, cols = 50, 80, 128
    s = Setup(env, rng, 2, rows, cols, 8, [0, 0])
    x, xv = values(rng, tokens, cols)
    xd = uw.bf16_tensor(x)
    index = rng.integers(-1, 2, size=tokens)
    d = torch.from_numpy(index.astype(np.int32)).cuda()
    plan = torch.empty(uw.lora_plan_bytes(tokens, 2), dtype=torch.uint8, device="cuda")
    work = torch.empty(uw.lora_workspace_bytes([s.h], tokens), dtype=torch.uint8, device="cuda")
    a, b = torch.zeros((5, cols), dtype=torch.bfloat16, device="cuda"), torch.zeros((rows, 5), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((tokens, rows), device="cuda")
    uw.lora_plan(d, 2, plan)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = torch.cuda.current_stream()
        s.h.load(1, a, b, 0.25, stream=st)
        uw._check(uw._lib.uw_lora_apply((C.c_void_p * 1)(s.h.handle), 1, plan.data_ptr(), plan.numel(), xd.data_ptr(), cols,
                                        None, None, (C.c_void_p * 1)(y.data_ptr()), (C.c_int64 * 1)(rows), tokens,
                                        work.data_ptr(), work.numel(), st.cuda_stream))
    for _ in range(3):
        ab, av = values(rng, 5, cols)
        bb, bv = values(rng, rows, 5)
        a.copy_(uw.bf16_tensor(ab))
        b.copy_(uw.bf16_tensor(bb))
        y.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        check(y.cpu().numpy().astype(np.float64), xv, index, {1: (av, bv, 0.25)}, np.zeros((tokens, rows), dtype=np.float32))


def test_two_streams_share_a_plan(env):
    torch, uw = env
    rng = np.random.default_rng(24)
    tokens, slots, cols = 300, 6, 512
    setups = [Setup(env, rng, slots, rows, cols, 16, rng.integers(0, 17, size=slots)) for rows in (512, 1024)]
    x, xv = values(rng, tokens, cols)
    index = rng.integers(-1, slots, size=tokens)
    bases = [rng.standard_normal((tokens, s.h.rows), dtype=np.float32) for s in setups]
    xd, bd = uw.bf16_tensor(x), [torch.from_numpy(b).cuda() for b in bases]
    ys = [torch.empty_like(b) for b in bd]
    plan = torch.empty(uw.lora_plan_bytes(tokens, slots), dtype=torch.uint8, device="cuda")
    works = [torch.empty(uw.lora_workspace_bytes([s.h], tokens), dtype=torch.uint8, device="cuda") for s in setups]
    uw.lora_plan(torch.from_numpy(index.astype(np.int32)).cuda(), slots, plan)
    streams = [torch.cuda.Stream() for _ in setups]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, st, y, b, w in zip(setups, streams, ys, bd, works):
            uw.lora_apply([s.h], plan, xd, [y], w, bases=[b], stream=st)
    torch.cuda.synchronize()
    for s, y, b in zip(setups, ys, bases):
        check(y.cpu().numpy().astype(np.float64), xv, index, s.values, b)


def test_in_place_strides_and_repeats(env):
    """In place, with x, base and y cut out of wider rows; columns beside stay as
    they were, and the same call gives the same bits."""
    torch, uw = env
    rng = np.random.default_rng(11)
    tokens, slots, rows, cols = 70, 3, 160, 128
    s, u = (Setup(env, rng, slots, rows, cols, 24, [24, 9, 16]) for _ in range(2))
    x, xv = values(rng, tokens, cols + 8)
    xd = uw.bf16_tensor(x)[:, 8:]
    index = rng.integers(-1, slots, size=tokens)
    d = torch.from_numpy(index.astype(np.int32)).cuda()
    plan = torch.empty(uw.lora_plan_bytes(tokens, slots), dtype=torch.uint8, device="cuda")
    uw.lora_plan(d, slots, plan)
    base = rng.standard_normal((tokens, 2 * rows + 12), dtype=np.float32)
    outs = []
    for _ in range(3):
        y = torch.from_numpy(base).cuda()
        work = torch.full((uw.lora_workspace_bytes([s.h, u.h], tokens),), 255, dtype=torch.uint8, device="cuda")
        # gate and up as two windows of one wider matrix
        uw.lora_apply([s.h, u.h], plan, xd, [y[:, :rows], y[:, rows + 4:2 * rows + 4]], work)
        torch.cuda.synchronize()
        outs.append(y.cpu().numpy())
    got = outs[0].astype(np.float64)
    check(got[:, :rows], xv[:, 8:], index, s.values, base[:, :rows])
    check(got[:, rows + 4:2 * rows + 4], xv[:, 8:], index, u.values, base[:, rows + 4:2 * rows + 4])
    assert np.array_equal(outs[0][:, rows:rows + 4], base[:, rows:rows + 4])
    assert np.array_equal(outs[0][:, 2 * rows + 4:], base[:, 2 * rows + 4:])
    assert np.array_equal(outs[0], outs[1]) and np.array_equal(outs[0], outs[2])


def test_replaced_adapters(env):
    """A slot loaded again with a smaller rank, and emptied."""
    torch, uw = env
    rng = np.random.default_rng(12)
    tokens, rows, cols = 20, 64, 128
    s = Setup(env, rng, 2, rows, cols, 40, [40, 40])
    x, xv = values(rng, tokens, cols)
    index = np.arange(tokens) % 2
    base = rng.standard_normal((tokens, rows), dtype=np.float32)
    for rank in (33, 17, 3, 40):
        ab, a = values(rng, rank, cols)
        bb, b = values(rng, rows, rank)
        s.h.load(1, uw.bf16_tensor(ab), uw.bf16_tensor(bb), -2.0)
        s.values[1] = (a, b, -2.0)
        check(apply(env, [s], x, index, [base])[0], xv, index, s.values, base)
    s.h.clear(1)
    del s.values[1]
    check(apply(env, [s], x, index, [base])[0], xv, index, s.values, base)


def test_infinities_stay_with_their_token(env):
    """An infinity or NaN in one token's x reaches that token only, and an
    infinity stays one where its products have one sign."""
    rng = np.random.default_rng(13)
    tokens, rows, cols = 18, 32, 64
    s = Setup(env, rng, 1, rows, cols, 3, [0])
    torch, uw = env
    ab, a = synth.f32_to_bf16_bits(np.abs(rng.standard_normal((3, cols), dtype=np.float32)) + 0.5), None
    bb = synth.f32_to_bf16_bits(np.abs(rng.standard_normal((rows, 3), dtype=np.float32)) + 0.5)
    s.h.load(0, uw.bf16_tensor(ab), uw.bf16_tensor(bb), 1.0)
    s.values[0] = (synth.bf16_bits_to_f32(ab).astype(np.float64), synth.bf16_bits_to_f32(bb).astype(np.float64), 1.0)
    x, xv = values(rng, tokens, cols)
    x[4, 7], x[9, 0] = 0x7F80, 0x7FC0  # +inf, NaN
    index = np.where(np.arange(tokens) == 9, -1, 0)
    index[9] = 0
    base = rng.standard_normal((tokens, rows), dtype=np.float32)
    got = apply(env, [s], x, index, [base])[0]
    assert (got[4] == INF).all() and np.isnan(got[9]).all()
    rest = [t for t in range(tokens) if t not in (4, 9)]
    check(got[rest], xv[rest], index[rest], s.values, base[rest])


@pytest.mark.parametrize("tokens,slots,rows,cols,max_rank", [
    (3, 2, (528, 1040), 64, 5),     # one launch
    (20, 1, (80,), 128, 3),
    (70, 2, (48, 272, 16), 64, 70),  # two stagings of the products with A
    (60, 40, (12336,), 64, 20),     # 1024 columns a workgroup, most tiles of one token
])
def test_infinities_in_b(env, tokens, slots, rows, cols, max_rank):
    """Infinities and NaN in B give what the formula gives: also where a product with A
    has few bits (here all are small whole numbers, zero among them) or is infinite itself."""
    torch, uw = env
    rng = np.random.default_rng(30 + tokens)
    setups = []
    for n in rows:
        s = Setup(env, rng, slots, n, cols, max_rank, [0] * slots)
        for i in range(slots):
            r = max(1, max_rank - i)
            a = rng.integers(-1, 2, size=(r, cols)).astype(np.float32) * (rng.random((r, cols)) < 0.1)
            a[:, 5] = 1.0
            b = values(rng, n, r)[1].astype(np.float32)
            b[:8] = np.abs(b[:8])
            if i != 1:  # slot 1's B is finite
                b[rng.random(b.shape) < 0.3 / r] = INF
                b[8:][rng.random(b[8:].shape) < 0.2 / r] = -INF
                b[rng.random(b.shape) < 0.05 / r] = NAN
            s.h.load(i, *(torch.from_numpy(v).to(torch.bfloat16).cuda() for v in (a, b)), 0.5)
            s.values[i] = (a.astype(np.float64), b.astype(np.float64), 0.5)
        setups.append(s)
    xv = rng.integers(-3, 4, size=(tokens, cols)).astype(np.float64)
    if tokens > 3:
        xv[tokens // 2, 5] = INF
    x = synth.f32_to_bf16_bits(xv.astype(np.float32))
    index = np.arange(tokens) % (slots + 1)
    bases = [rng.standard_normal((tokens, n), dtype=np.float32) for n in rows]

    def compare():
        for s, base, got in zip(setups, bases, apply(env, setups, x, index, bases)):
            with np.errstate(invalid="ignore"):
                want = routing.lora(xv, index, s.values, base)
                plain = {i: (a, np.where(np.isfinite(b), b, 0.0), c) for i, (a, b, c) in s.values.items()}
                bound = routing.lora_error_bound(xv, index, plain, base)
            finite = np.isfinite(want)
            assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got == INF, want == INF)
            assert np.array_equal(got == -INF, want == -INF)
            assert (np.abs(got[finite] - want[finite]) <= bound[finite]).all()

    compare()
    # finite again: over what was there, and in an emptied slot
    for s in setups:
        for i in range(slots):
            a, b, _ = s.values[i]
            b = np.where(np.isfinite(b), b, 1.0)
            if i % 2:
                s.h.clear(i)
            s.h.load(i, *(torch.from_numpy(v).to(torch.bfloat16).cuda() for v in (a, b)), -1.5)
            s.values[i] = (a, b, -1.5)
    compare()


def test_refusals(env):
    torch, uw = env
    rng = np.random.default_rng(14)
    s, other = Setup(env, rng, 2, 64, 128, 8, [8, 8]), Setup(env, rng, 2, 64, 192, 8, [8, 8])
    x = torch.zeros((4, 128), dtype=torch.bfloat16, device="cuda")
    y = torch.zeros((4, 64), device="cuda")
    plan = torch.zeros(uw.lora_plan_bytes(4, 2), dtype=torch.uint8, device="cuda")
    work = torch.zeros(uw.lora_workspace_bytes([s.h], 4), dtype=torch.uint8, device="cuda")

    def status(**kw):
        a = dict(adapters=[s.h], plan=plan, x=x, ys=[y], work=work)
        a.update(kw)
        with pytest.raises((uw.UwError, ValueError)) as e:
            uw.lora_apply(**a)
        return getattr(e.value, "status", "value")

    assert status(plan=plan[:-1]) == uw.ERR_INVALID_ARG
    assert status(work=work[:-1]) == uw.ERR_INVALID_ARG
    assert status(adapters=[s.h, other.h], ys=[y, y.clone()]) == uw.ERR_SHAPE
    assert status(adapters=[s.h, s.h], ys=[y, y], work=torch.zeros(1 << 16, dtype=torch.uint8, device="cuda")) == uw.ERR_INVALID_ARG
    assert status(adapters=[s.h] * 5, ys=[y] * 5) == "value"
    assert status(x=x[:, :64]) == "value"
    assert status(x=torch.zeros((4, 132), dtype=torch.bfloat16, device="cuda")[:, :128]) == uw.ERR_SHAPE
    wide = torch.zeros((5, 64), device="cuda")
    assert status(ys=[wide[1:]], bases=[wide[:4]]) == uw.ERR_INVALID_ARG
    for args in ((2, 8), (-1, 8), (0, 9)):
        with pytest.raises(uw.UwError) as e:
            s.h.load(args[0], torch.zeros((args[1], 128), dtype=torch.bfloat16, device="cuda"),
                     torch.zeros((64, args[1]), dtype=torch.bfloat16, device="cuda"))
        assert e.value.status == uw.ERR_INVALID_ARG
    # a plan that no uw_lora_plan made for these numbers: y stays as it is
    y.fill_(3.0)
    uw.lora_apply([s.h], plan, x, [y], work)
    torch.cuda.synchronize()
    assert (y == 3.0).all()


def test_streams_and_graph(env):
    """On another stream, and captured: replays follow new inputs and new adapters."""
    torch, uw = env
    rng = np.random.default_rng(15)
    tokens, slots, rows, cols = 90, 4, 192, 256
    s = Setup(env, rng, slots, rows, cols, 16, [16, 5, 0, 11])
    x, xv = values(rng, tokens, cols)
    index = rng.integers(-1, slots, size=tokens)
    base = rng.standard_normal((tokens, rows), dtype=np.float32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    check(apply(env, [s], x, index, [base], stream=side)[0], xv, index, s.values, base)
    d = torch.from_numpy(index.astype(np.int32)).cuda()
    xd, bd = uw.bf16_tensor(x), torch.from_numpy(base).cuda()
    y = torch.empty_like(bd)
    plan = torch.empty(uw.lora_plan_bytes(tokens, slots), dtype=torch.uint8, device="cuda")
    work = torch.empty(uw.lora_workspace_bytes([s.h], tokens), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        st = torch.cuda.current_stream()
        uw.lora_plan(d, slots, plan, stream=st)
        uw.lora_apply([s.h], plan, xd, [y], work, bases=[bd], stream=st)
    for rep in range(4):
        x, xv = values(rng, tokens, cols)
        index = rng.integers(-1, slots, size=tokens)
        xd.copy_(uw.bf16_tensor(x))
        d.copy_(torch.from_numpy(index.astype(np.int32)))
        if rep == 2:
            ab, a = values(rng, 9, cols)
            bb, b = values(rng, rows, 9)
            s.h.load(2, uw.bf16_tensor(ab), uw.bf16_tensor(bb), 0.5)
            s.values[2] = (a, b, 0.5)
        y.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        check(y.cpu().numpy().astype(np.float64), xv, index, s.values, base)


# ---- with the compressed projections ----


def test_layer_with_experts_and_adapters(env):
    """A layer as it is served: a shared SwiGLU branch of compressed projections
    with adapters on gate, up and down, plus routed experts combined onto it."""
    torch, uw = env
    rng = np.random.default_rng(16)
    tokens, hidden, inter, experts, k, slots = 45, 256, 512, 6, 2, 5
    shapes = ((inter, hidden), (inter, hidden), (hidden, inter))
    ws = [[synth.weights(r, c, 500 + 3 * e + j, 0.002, 10) for j, (r, c) in enumerate(shapes)] for e in range(experts + 1)]
    mats = [[uw.Matrix(w, uw.FMT_PALETTE) for w in three] for three in ws]
    ad = [Setup(env, rng, slots, r, c, 8, [8, 3, 0, 8, 5]) for r, c in shapes]
    for s in ad:  # factors as small as trained adapters', so that both parts matter
        for i, (a, b, _) in s.values.items():
            s.h.load(i, torch.from_numpy(a).to(torch.bfloat16).cuda(), torch.from_numpy(b).to(torch.bfloat16).cuda(), 0.002)
            s.values[i] = (a, b, float(np.float32(0.002)))
    xb, xv = values(rng, tokens, hidden)
    x = uw.bf16_tensor(xb)
    logits = rng.standard_normal((tokens, experts), dtype=np.float32)
    logits[7] = -INF  # a token without experts
    logits[8, 1:] = -INF  # and one with a single one
    index = rng.integers(-1, slots, size=tokens)
    d = torch.from_numpy(index.astype(np.int32)).cuda()
    ld = torch.from_numpy(logits).cuda()
    plan = torch.empty(uw.lora_plan_bytes(tokens, slots), dtype=torch.uint8, device="cuda")
    work = torch.empty(uw.lora_workspace_bytes([ad[0].h, ad[1].h], tokens), dtype=torch.uint8, device="cuda")
    gate, up = (torch.empty((tokens, inter), device="cuda") for _ in range(2))
    h = torch.empty((tokens, inter), dtype=torch.bfloat16, device="cuda")
    shared = torch.empty((tokens, hidden), device="cuda")
    y = torch.empty((tokens, hidden), device="cuda")
    moe_work = torch.empty(uw.moe_workspace_bytes(tokens, hidden, inter, experts, k), dtype=torch.uint8, device="cuda")
    print("layer with experts and adapters", flush=True)
    uw.lora_plan(d, slots, plan)
    mats[experts][0].matmul(x, gate)
    mats[experts][1].matmul(x, up)
    uw.lora_apply([ad[0].h, ad[1].h], plan, x, [gate, up], work)
    uw.silu_mul(gate, up, h)
    mats[experts][2].matmul(h, shared)
    uw.lora_apply([ad[2].h], plan, h, [shared], work)
    uw.moe_forward([m for three in mats[:experts] for m in three], [uw.P_AUTO] * 3, ld, x, y, moe_work, k, base=shared)
    torch.cuda.synchronize()
    w64 = [[oracle.bf16_to_f64(w) for w in three] for three in ws]
    g64 = routing.lora(xv, index, ad[0].values, xv @ w64[experts][0].T)
    u64 = routing.lora(xv, index, ad[1].values, xv @ w64[experts][1].T)
    assert oracle.rel_err(gate.cpu().numpy(), g64) <= 1e-3 and oracle.rel_err(up.cpu().numpy(), u64) <= 1e-3
    # the shared branch from the bf16 h that the GPU had
    h64 = h.double().cpu().numpy()
    # g and u within 1e-3 of their largest, and a bf16 rounding
    h_want = oracle.bf16_to_f64(oracle.silu_mul_bf16(g64, u64))
    slack = 1e-3 * 1.1 * (np.abs(g64).max() * np.abs(u64) + np.abs(u64).max() * np.abs(g64)) + 1e-6 * np.abs(g64).max() * np.abs(u64).max()
    assert (np.abs(h64 - h_want) <= slack * (1 + 2.0 ** -8) + 2.0 ** -7 * np.abs(h_want)).all()
    want = routing.lora(h64, index, ad[2].values, h64 @ w64[experts][2].T)
    assert oracle.rel_err(shared.cpu().numpy(), want) <= 1e-3
    chosen, weights = routing.route(logits, k)
    assert (chosen[7] == -1).all() and chosen[8].tolist() == [0, -1]
    for t in range(tokens):
        for e, w in zip(chosen[t], weights[t]):
            if e >= 0:
                want[t] += w * oracle.mlp_layer_fp64(xb[t:t + 1], *ws[e])[3][0]
    assert oracle.rel_err(y.cpu().numpy(), want) <= 1e-3
    # in place on the shared output, and the token without experts keeps it
    kept = shared[7].clone()
    uw.moe_forward([m for three in mats[:experts] for m in three], [uw.P_AUTO] * 3, ld, x, shared, moe_work, k, base=shared)
    torch.cuda.synchronize()
    # (not bit for bit: these short matrices split K over workgroups that add
    # atomically, and another order of those float32 sums can move h by a bf16 step)
    assert oracle.rel_err(shared.cpu().numpy(), want) <= 1e-3 and torch.equal(shared[7], kept)


@pytest.mark.parametrize("tokens,pipelines", [(1, (4, 4, 4)), (3, (3, 3, 4)), (130, (5, 4, 1)), (200, (0, 0, 0))])
def test_moe_layer(env, tokens, pipelines):
    torch, uw = env
    rng = np.random.default_rng(tokens)
    hidden, inter, experts, k = 256, 192, 5, 3
    shapes = ((inter, hidden), (inter, hidden), (hidden, inter))
    ws = [[synth.weights(r, c, 700 + 3 * e + j, 0.002, 10) for j, (r, c) in enumerate(shapes)] for e in range(experts)]
    mats = [uw.Matrix(w, uw.FMT_HUFFMAN | uw.FMT_PALETTE) for three in ws for w in three]
    xb, _ = values(rng, tokens, hidden)
    logits = rng.standard_normal((tokens, experts + 2), dtype=np.float32)
    bias = rng.standard_normal(experts).astype(np.float32) * 0.1
    ld = torch.from_numpy(logits).cuda()[:, :experts]
    y = torch.full((tokens, hidden), NAN, device="cuda")
    work = torch.full((uw.moe_workspace_bytes(tokens, hidden, inter, experts, k),), 255, dtype=torch.uint8, device="cuda")
    print(f"moe layer {tokens} tokens {pipelines}", flush=True)
    uw.moe_forward(mats, pipelines, ld, uw.bf16_tensor(xb), y, work, k, score=uw.SCORE_SIGMOID,
                   bias=torch.from_numpy(bias).cuda(), scale=1.5)
    torch.cuda.synchronize()
    chosen, weights = routing.route(logits[:, :experts], k, routing.SIGMOID, bias, scale=1.5)
    want = np.zeros((tokens, hidden))
    for e in range(experts):
        rows = np.nonzero((chosen == e).any(axis=1))[0]
        if len(rows):
            want[rows] += weights[rows, np.argmax(chosen[rows] == e, axis=1), None] * oracle.mlp_layer_fp64(xb[rows], *ws[e])[3]
    assert oracle.rel_err(y.cpu().numpy(), want) <= 1e-3
    # every expert off: zeros
    uw.moe_forward(mats, pipelines, torch.full((tokens, experts), -INF, device="cuda"), uw.bf16_tensor(xb), y, work, k)
    torch.cuda.synchronize()
    assert (y == 0).all()


def test_moe_layer_on_its_stream(env):
    """On the experts' own stream, behind work that is queued there."""
    torch, uw = env
    rng = np.random.default_rng(27)
    tokens, hidden, inter, experts = 24, 128, 128, 4
    ws = [[synth.weights(r, c, 900 + 3 * e + j, 0.002, 10) for j, (r, c) in
           enumerate(((inter, hidden), (inter, hidden), (hidden, inter)))] for e in range(experts)]
    mats = [uw.Matrix(w, uw.FMT_PALETTE) for three in ws for w in three]
    side = torch.cuda.Stream()
    for m in mats:
        m.set_streams(side)
    xb, _ = values(rng, tokens, hidden)
    xd, logits = uw.bf16_tensor(xb), torch.from_numpy(rng.standard_normal((tokens, experts), dtype=np.float32)).cuda()
    work = torch.empty(uw.moe_workspace_bytes(tokens, hidden, inter, experts, 2), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        x, l = torch.zeros_like(xd), torch.zeros_like(logits)
        big = torch.ones(1 << 26, device="cuda")
        for _ in range(10):
            big.mul_(1.0001)
        x.copy_(xd)
        l.copy_(logits)
        y = torch.zeros((tokens, hidden), device="cuda")
        uw.moe_forward(mats, [4, 4, 4], l, x, y, work, 2)
        y2 = y * 2  # and what is queued behind sees the result
    torch.cuda.synchronize()
    chosen, weights = routing.route(logits.cpu().numpy(), 2)
    want = np.zeros((tokens, hidden))
    for t in range(tokens):
        for e, w in zip(chosen[t], weights[t]):
            want[t] += w * oracle.mlp_layer_fp64(xb[t:t + 1], *ws[e])[3][0]
    assert oracle.rel_err(y2.cpu().numpy() / 2, want) <= 1e-3
    for m in mats:
        m.free()


def test_moe_layer_refuses_capture(env):
    torch, uw = env
    mats = [uw.Matrix(synth.weights(64, 64, i, 0.0, 1), uw.FMT_PALETTE) for i in range(3)]
    x = torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda")
    y, l = torch.zeros((2, 64), device="cuda"), torch.zeros((2, 1), device="cuda")
    work = torch.zeros(uw.moe_workspace_bytes(2, 64, 64, 1, 1), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, capture_error_mode="thread_local"):
        for m in mats:
            m.set_streams(torch.cuda.current_stream())
        with pytest.raises(uw.UwError) as e:
            uw.moe_forward(mats, [4, 4, 4], l, x, y, work, 1)
        y.add_(1.0)  # the capture goes on
    assert e.value.status == uw.ERR_UNSUPPORTED
    for m in mats:
        m.set_streams()
    graph.replay()
    torch.cuda.synchronize()
    assert (y == 1.0).all()
