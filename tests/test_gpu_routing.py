"""Routing, grouping, dispatch and combination of rows on the GPU against the
64-bit oracle: choices, positions and copies exactly, sums within bounds that
are derived here from their float32 roundings."""
import numpy as np
import pytest

from oracle import routing

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
# A weight is evaluated in 64 bits and rounded once (2^-24), but for the sum of
# a softmax that is not renormalised: at most 1024 float32 terms, added as <= 32
# in a lane and 6 times across lanes, each term within 2 ulp (2^-22) and the
# rounding of its argument (x exp(-x) <= 0.37 of 2^-24): (38 + 4 + 1 + 1) 2^-24.
WEIGHT_TOL = 44 * 2.0 ** -24


@pytest.fixture(scope="module")
def env():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a ROCm device"
    import decode_gemm_bf16_amd as uw
    return torch, uw


def bf16(torch, v):
    return torch.from_numpy(np.asarray(v, dtype=np.float32)).to(torch.bfloat16)


def within_64_bits(l, chosen, bias, kw):
    """A choice other than the oracle's, which has to be right up to the roundings of
    64-bit values, and its weights.  Both sides take a score from an exponential
    and a division (each within 1 ulp, 2^-52), the softmax's sum (the same factor on
    all scores of a token), a sum with the bias and one of two scores: merits or
    choices that the two sides order differently are at most 2 x 4 x 2^-52 of the
    largest apart.  Logits that decide have no rounding."""
    groups, top_groups = kw.get("groups", 1), kw.get("top_groups", 1)
    pairs = kw.get("group_score", 0)
    s = routing._scores(l, kw.get("score", 0))
    valued = s if bias is None else s + bias.astype(np.float64)
    assert np.isfinite(l).all() and np.isfinite(valued).all(), "only finite values can be this close"
    choice, tol = (l, 0.0) if bias is None else (valued, 2.0 ** -49 * np.abs(valued).max())
    per = len(l) // groups
    allowed = np.ones(len(l), dtype=bool)
    if groups > 1:
        merit = [sorted((valued if pairs else choice)[g * per:(g + 1) * per])[-1 - pairs:] for g in range(groups)]
        merit = np.array([sum(m) for m in merit])
        slack = 2.0 ** -49 * np.abs(merit).max() if pairs or bias is not None else 0.0
        kept = sorted(set(chosen // per) | set(np.argsort(-merit, kind="stable")[:top_groups]),
                      key=lambda g: (g not in chosen // per, -merit[g]))[:top_groups]
        dropped = [g for g in range(groups) if g not in kept]
        assert min(merit[kept]) >= max(merit[dropped]) - slack
        allowed = np.isin(np.arange(len(l)) // per, kept)
    assert len(set(chosen)) == len(chosen) and allowed[chosen].all()
    c = choice[chosen]
    assert (c[1:] <= c[:-1] + tol).all()
    rest = np.setdiff1d(np.nonzero(allowed)[0], chosen)
    assert not len(rest) or choice[rest].max() <= c[-1] + tol
    w = s[chosen]
    return (w / w.sum() if kw.get("renormalise", True) else w) * kw.get("scale", 1.0)


def run_route(env, logits, top_k, dtype="float32", pad=0, bias=None, **kw):
    """Routes numpy logits and compares with the oracle on the values the GPU saw."""
    torch, uw = env
    t, e = logits.shape
    wide = torch.zeros((t, e + pad), dtype=getattr(torch, dtype), device="cuda")
    wide[:, :e] = torch.from_numpy(logits.astype(np.float32)).to(wide.dtype)
    seen = wide[:, :e].float().cpu().numpy()
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    experts = torch.full((t, top_k), -7, dtype=torch.int32, device="cuda")
    weights = torch.full((t, top_k), NAN, device="cuda")
    print(f"route {t}x{e} k={top_k} {dtype} pad={pad} {kw}", flush=True)
    uw.route(wide[:, :e], experts, weights, bias=b, **kw)
    torch.cuda.synchronize()
    want_e, want_w = routing.route(seen, top_k, bias=None if bias is None else b.cpu().numpy(),
                                   largest=torch.finfo(wide.dtype).max, **kw)
    got_e, got = experts.cpu().numpy(), weights.cpu().numpy().astype(np.float64)
    for row in np.nonzero((got_e != want_e).any(axis=1))[0]:
        want_w[row] = within_64_bits(seen[row].astype(np.float64), got_e[row], None if b is None else b.cpu().numpy(), kw)
    # below the smallest normal float32 a rounding is absolute
    assert (np.abs(got - want_w) <= WEIGHT_TOL * np.abs(want_w) + 2.0 ** -149).all()
    return want_e, want_w


@pytest.mark.parametrize("tokens,experts,top_k", [
    (1, 1, 1), (1, 8, 2), (3, 5, 5), (7, 60, 4), (129, 64, 6), (65, 65, 3), (33, 127, 9), (17, 256, 8), (5, 300, 16),
    (3, 512, 17), (2, 1000, 64), (3, 1024, 33), (2000, 8, 2), (777, 96, 16)])
@pytest.mark.parametrize("score", [0, 1])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_sizes(env, tokens, experts, top_k, score, with_bias):
    rng = np.random.default_rng(tokens * 1000 + experts)
    bias = rng.normal(size=experts) * 0.1 if with_bias else None
    run_route(env, rng.normal(size=(tokens, experts)) * 2, top_k, score=score, bias=bias,
              renormalise=bool(tokens % 2), scale=1.0 if experts % 2 else 2.5)


@pytest.mark.parametrize("experts,groups,top_groups,top_k", [
    (8, 2, 1, 2), (8, 8, 3, 3), (60, 4, 2, 5), (96, 3, 2, 8), (256, 8, 4, 8), (256, 8, 8, 8), (160, 5, 1, 6),
    (1024, 64, 8, 16), (990, 33, 5, 12), (34, 17, 2, 4), (448, 7, 3, 10), (1023, 3, 1, 20), (64, 64, 5, 5),
    (512, 2, 1, 16), (512, 16, 3, 7)])
@pytest.mark.parametrize("pairs", [0, 1])
@pytest.mark.parametrize("score,with_bias", [(0, False), (0, True), (1, False), (1, True)])
def test_route_groups(env, experts, groups, top_groups, top_k, pairs, score, with_bias):
    rng = np.random.default_rng(experts + groups)
    bias = rng.normal(size=experts) * 0.2 if with_bias else None
    for tokens in (1, 37, 200):
        run_route(env, rng.normal(size=(tokens, experts)) * 1.5, top_k, score=score, bias=bias, groups=groups,
                  top_groups=top_groups, group_score=pairs, renormalise=top_k % 2 == 0)


@pytest.mark.parametrize("groups,pairs,with_bias", [(1, 0, False), (1, 0, True), (4, 0, False), (4, 1, True), (4, 1, False)])
@pytest.mark.parametrize("score", [0, 1])
def test_route_ties_and_masks(env, groups, pairs, with_bias, score):
    """bf16 logits on few values (ties everywhere), rows with masked experts, with
    the lowest finite value, with infinities and NaN, and with nothing left."""
    rng = np.random.default_rng(11)
    l = rng.integers(-3, 4, size=(90, 48)).astype(np.float64)
    l[10:20][rng.random((10, 48)) < 0.8] = -INF
    l[20:30][rng.random((10, 48)) < 0.3] = NAN
    l[30] = -INF
    l[31] = NAN
    l[32] = -3.3895313892515355e38  # bfloat16's lowest
    l[33, :40] = -3.3895313892515355e38
    l[34, 5] = l[34, 40] = INF
    l[35] = INF
    l[36] = 80.0
    l[37] = -120.0
    l[38, 1:] = -INF
    l[39, ::2] = -1000.0
    bias = rng.integers(-2, 3, size=48) * 0.25 if with_bias else None
    for dtype in ("bfloat16", "float32"):
        for renormalise in (False, True):
            run_route(env, l, 6, dtype=dtype, pad=3, score=score, bias=bias, groups=groups, top_groups=max(1, groups // 2),
                      group_score=pairs, renormalise=renormalise)


def test_route_bias_switches_off(env):
    rng = np.random.default_rng(12)
    bias = np.where(np.arange(32) % 3 == 0, -INF, 0.1)
    bias[7], bias[8] = NAN, INF
    for score in (0, 1):
        e, _ = run_route(env, rng.normal(size=(40, 32)), 24, score=score, bias=bias)
        assert (e[:, 0] == 8).all() and (e[:, 20:] == -1).all() and not np.isin(e, [0, 3, 7]).any()


def test_route_close_scores(env):
    """Scores that are equal in float32 but not in 64 bits: the larger one wins."""
    l = np.full((4, 16), -9.0)
    l[0, 3], l[0, 12] = 20.0, 21.0  # sigmoids 1 - 2.1e-9 and 1 - 7.6e-10
    l[1, 12], l[1, 3] = 20.0, 21.0
    l[2, :] = 19.0 + np.arange(16) / 64
    l[3, :] = 19.0 - np.arange(16) / 64
    for groups, pairs in ((1, 0), (4, 0), (4, 1)):
        run_route(env, l, 4, score=1, bias=np.full(16, 0.25), groups=groups, top_groups=min(2, groups), group_score=pairs)
        run_route(env, l, 4, score=1, groups=groups, top_groups=min(2, groups), group_score=pairs)


@pytest.mark.parametrize("tokens", [40, 2000])
@pytest.mark.parametrize("experts,top_k", [(64, 8), (256, 15), (256, 16)])
@pytest.mark.parametrize("score", [0, 1])
def test_route_near_ties(env, tokens, experts, top_k, score):
    """Choices that differ by less than a float32 rounding, by more and not at all,
    next to each other and in runs: logits in clusters of neighbouring floats, and
    biases that bring far logits' scores within a few 2^-24 of each other."""
    rng = np.random.default_rng(experts + top_k)
    l = rng.normal(size=(tokens, 6))[:, rng.integers(0, 6, size=experts)].astype(np.float32)
    l = l + rng.integers(-2, 3, size=l.shape).astype(np.float32) * np.spacing(np.abs(l))
    few = rng.random(tokens) < 0.5  # half of the tokens: spread out, with single close pairs
    l[few] = rng.normal(size=(int(few.sum()), experts)).astype(np.float32) * 2
    l[few, 3] = np.nextafter(l[few, 9], np.float32(9))
    l[0] = 0.0
    l[0, ::2] = -0.0
    level = np.full(experts, 0.75) + rng.integers(-3, 4, size=experts) * 2.0 ** -24
    for groups, top_groups, pairs in ((1, 1, 0), (8, 3, 1), (8, 3, 0), (4, 4, 1)):
        if top_k <= experts // groups * top_groups:
            for bias in (None, np.zeros(experts), level):
                run_route(env, l, top_k, score=score, bias=bias, groups=groups, top_groups=top_groups, group_score=pairs)
    # all scores + bias nearly equal: bias = 1 - score, rounded
    flat = rng.normal(size=experts).astype(np.float32)
    s = 1 / (1 + np.exp(-flat.astype(np.float64)))
    run_route(env, np.tile(flat, (tokens, 1)), top_k, score=1, bias=(1 - s))


def test_route_largest_values(env):
    """+inf is the type's largest finite value, equal to that value itself."""
    for dtype, largest in (("bfloat16", 3.3895313892515355e38), ("float32", float(np.finfo(np.float32).max))):
        l = np.full((3, 8), 1.0)
        l[0, 5], l[0, 2] = INF, largest
        l[1, 2], l[1, 5] = INF, largest
        l[2, 7] = -largest
        for score in (0, 1):
            for bias in (None, np.zeros(8)):
                run_route(env, l, 3, dtype=dtype, score=score, bias=bias, renormalise=False)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("experts,top_k,with_bias", [(8, 2, False), (60, 4, True), (256, 8, False), (256, 8, True),
                                                      (1000, 5, True), (1024, 16, False)])
def test_route_weights(env, experts, top_k, with_bias, dtype):
    """How exact a weight is.  It is evaluated in 64 bits and rounded once, by 2^-24 of
    itself; the terms of a softmax's sum alone are exponentials in float32, added in 64
    bits: each is off by 2 ulp (2^-22) and by the rounding of its argument d (|d| 2^-24),
    and the largest, exp(0), by nothing.  So the sum is off by at most the mean of 4 + |d|
    over the other terms, each by its share, times 2^-24: nearly nothing where one
    logit stands out (a float32 sum of such rows of 256 is off by up to 8 x 2^-24)."""
    torch, uw = env
    rng = np.random.default_rng(experts + top_k)
    l = rng.normal(size=(300, experts)) * 1.5
    l[:60] = -17.5 + rng.normal(size=(60, experts)) * 0.1  # about 2^-25 each
    l[np.arange(60), np.arange(60) * 7 % experts] = rng.integers(0, 2, size=60)
    l[60:80] *= 8
    bias = rng.normal(size=experts).astype(np.float32) * np.float32(0.1) if with_bias else None
    logits = torch.from_numpy(l.astype(np.float32)).to(getattr(torch, dtype)).cuda()
    seen = logits.double().cpu().numpy()
    p = np.exp(seen - seen.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    d = seen.max(axis=1, keepdims=True) - seen
    sums = (p * np.where(d > 0, 4 + d, 0.0)).sum(axis=1)[:, None]
    assert sums[:60].max() < 0.02 * experts / 1024 + 0.01
    for score in (0, 1):
        for renormalise in (False, True):
            e = torch.empty((300, top_k), dtype=torch.int32, device="cuda")
            w = torch.empty((300, top_k), device="cuda")
            print(f"weights 300x{experts} k={top_k} {dtype} score={score} renormalise={renormalise}", flush=True)
            uw.route(logits, e, w, score=score, bias=None if bias is None else torch.from_numpy(bias).cuda(),
                     renormalise=renormalise, scale=2.0)
            torch.cuda.synchronize()
            want_e, want = routing.route(seen, top_k, score, bias, renormalise=renormalise, scale=2.0)
            assert np.array_equal(e.cpu().numpy(), want_e)
            # (the oracle's own 64-bit roundings: 1200 of 2^-53 for the longest sum)
            tol = 1 + 2.0 ** -18 + (sums if score == 0 and not renormalise else 0.0)
            assert (np.abs(w.cpu().numpy() - want) <= tol * 2.0 ** -24 * want + 2.0 ** -150).all()


def test_route_merits_past_float32(env):
    """Biases so large that a group's merit, a sum of two, has no place in float32: it
    is compared in 64 bits, also against a group without candidates, which is behind."""
    l = np.zeros((3, 8))
    l[1, :4] = -INF  # group 0 has no candidates
    l[2, 4:7] = -INF  # group 1 a single one: its merit is no sum
    for bias, want in (((-3e38, -2e38), ([4, 5], [4, 5], [7, -1])), ((-2e38, -3e38), ([0, 1], [4, 5], [7, -1])),
                       ((3e38, 2e38), ([0, 1], [4, 5], [0, 1]))):
        for score in (0, 1):
            e, _ = run_route(env, l, 2, score=score, bias=np.repeat(bias, 4), groups=2, group_score=1)
            assert e.tolist() == list(want)
    rng = np.random.default_rng(14)
    for experts, groups, top_groups, top_k in ((8, 2, 1, 2), (60, 4, 2, 5), (256, 8, 3, 8), (512, 16, 5, 16), (990, 33, 5, 12)):
        per = experts // groups
        for size in (2e38, 3.4e38):
            level = rng.choice([-size, -0.9 * size, -0.5 * size, 0.0, size], size=groups)
            bias = np.repeat(level, per) * (1 - rng.integers(0, 3, size=experts) / 64)
            logits = rng.normal(size=(60, experts))
            logits[rng.random((60, groups)).repeat(per, axis=1) < 0.3] = -INF
            for score in (0, 1):
                for pairs in (0, 1):
                    run_route(env, logits, top_k, score=score, bias=bias, groups=groups, top_groups=top_groups,
                              group_score=pairs, renormalise=False)


def test_route_strides_and_alignment(env):
    torch, uw = env
    rng = np.random.default_rng(13)
    for dtype in ("float32", "bfloat16"):
        for pad in (1, 2, 5, 64):
            run_route(env, rng.normal(size=(50, 24)), 3, dtype=dtype, pad=pad)
    # a window that starts at an odd element
    wide = torch.randn((20, 41), device="cuda").to(torch.bfloat16)
    view = wide[:, 3:36]
    e, w = torch.empty((20, 5), dtype=torch.int32, device="cuda"), torch.empty((20, 5), device="cuda")
    uw.route(view, e, w)
    want, _ = routing.route(view.float().cpu().numpy(), 5)
    assert np.array_equal(e.cpu().numpy(), want)


# ---- grouping ----


def run_group(env, index, groups):
    torch, uw = env
    d = torch.from_numpy(np.ascontiguousarray(index, dtype=np.int32)).cuda()
    n = d.numel()
    offsets = torch.full((groups + 1,), -7, dtype=torch.int32, device="cuda")
    order = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    slot = torch.full_like(d, -7)
    work = torch.full((uw.group_rows_workspace_bytes(n, groups),), 255, dtype=torch.uint8, device="cuda")
    print(f"group {n} entries, {groups} groups", flush=True)
    uw.group_rows(d, groups, offsets, order, slot, work)
    torch.cuda.synchronize()
    flat = np.asarray(index).reshape(-1)
    label = np.where((flat >= 0) & (flat < groups), flat, groups)
    want_order = np.argsort(label, kind="stable")
    counts = np.bincount(label, minlength=groups + 1)[:groups]
    want_offsets = np.concatenate([[0], np.cumsum(counts)])
    want_slot = np.empty(n, dtype=np.int64)
    want_slot[want_order] = np.arange(n)
    want_slot[label == groups] = -1
    assert np.array_equal(offsets.cpu().numpy(), want_offsets)
    assert np.array_equal(order.cpu().numpy(), want_order)
    assert np.array_equal(slot.cpu().numpy().reshape(-1), want_slot)
    return offsets, order, slot


@pytest.mark.parametrize("n,groups", [(n, g) for n in (1, 2, 63, 64, 65, 1000, 1024, 4095, 4096, 4097, 8193, 40000, 131071)
                                      for g in (1, 2, 8, 60, 255, 256, 899, 900, 1699, 1700, 2999, 3000, 4000)]
                         + [(1100003, g) for g in (1, 60, 1000, 2000, 4000)])
def test_group_sizes(env, n, groups):
    rng = np.random.default_rng(n + groups)
    index = rng.integers(-1, groups + 1, size=n)  # -1 and groups are ungrouped
    run_group(env, index, groups)


@pytest.mark.parametrize("groups", [3, 256, 1200, 3500])
@pytest.mark.parametrize("n", [65535, 65537, 131073, 262144, 262145, 1048576, 1048577])
def test_group_section_limits(env, n, groups):
    """Where a lane's share grows from one entry to four, and past four; long runs and mixed labels."""
    index = np.random.default_rng(n).integers(-1, groups + 1, size=n)
    index[n // 3: n // 2] = groups - 1
    run_group(env, index, groups)


def test_group_values(env):
    for n in (100, 20000):
        run_group(env, np.full(n, 3), 8)
        run_group(env, np.full(n, -1), 8)
        run_group(env, np.arange(n)[::-1] % 8, 8)
        run_group(env, np.where(np.arange(n) % 2, 2 ** 31 - 1, -2 ** 31), 8)
        run_group(env, np.repeat([7, 0], n // 2), 8)
        i = (np.random.default_rng(n).pareto(0.5, size=(n // 4, 4)) * 2).clip(0, 40).astype(np.int64)
        run_group(env, i, 40)


def test_group_matches_the_oracle(env):
    rng = np.random.default_rng(4)
    index = rng.integers(-2, 13, size=(77, 3))
    offsets, order, slot = (v.cpu().numpy() for v in run_group(env, index, 11))
    for got, want in zip((offsets, order, slot), routing.group_rows(index, 11)):
        assert np.array_equal(got, want)


# ---- dispatch and combine ----


@pytest.mark.parametrize("tokens,top_k,cols,pad", [(1, 1, 8, 0), (1, 8, 2056, 8), (3, 2, 64, 0), (65, 3, 520, 16),
                                                    (130, 8, 4096, 0), (9, 5, 14336, 64), (700, 2, 24, 8)])
def test_dispatch(env, tokens, top_k, cols, pad):
    torch, uw = env
    rng = np.random.default_rng(tokens + cols)
    n = tokens * top_k
    rows = n + 3
    slot = rng.permutation(rows)[:n].reshape(tokens, top_k).astype(np.int32)
    gone = rng.random(slot.shape)
    slot[gone < 0.1] = -1
    slot[gone > 0.95] = rows  # outside: skipped
    bits = rng.integers(0, 65536, size=(tokens, cols + pad)).astype(np.uint16)  # every pattern, NaN too
    x = uw.bf16_tensor(bits)[:, :cols]
    before = rng.integers(0, 65536, size=(rows, cols)).astype(np.uint16)
    xs = uw.bf16_tensor(before)
    print(f"dispatch {tokens}x{top_k} {cols}+{pad}", flush=True)
    uw.dispatch_rows(x, torch.from_numpy(slot).cuda(), xs)
    torch.cuda.synchronize()
    assert np.array_equal(uw.bits_of(xs), routing.dispatch_rows(bits[:, :cols], slot, before))


@pytest.mark.parametrize("tokens,top_k,cols", [(1, 1, 8), (1, 8, 1032), (65, 3, 520), (130, 8, 4096), (9, 5, 14336),
                                                (700, 2, 24), (4, 64, 64), (33, 1, 2048)])
@pytest.mark.parametrize("with_base,out", [("none", "float32"), ("apart", "float32"), ("in place", "float32"),
                                           ("none", "bfloat16"), ("apart", "bfloat16")])
def test_combine(env, tokens, top_k, cols, with_base, out):
    torch, uw = env
    rng = np.random.default_rng(tokens + cols + top_k)
    rows = tokens * top_k + 5
    slot = rng.permutation(rows)[:tokens * top_k].reshape(tokens, top_k).astype(np.int32)
    gone = rng.random(slot.shape)
    slot[gone < 0.15] = -1
    slot[gone > 0.95] = rows
    if tokens > 3:
        slot[2] = -1  # a token without any row
        slot[3] = slot[0]  # the same row twice
    ys = rng.standard_normal((rows, cols), dtype=np.float32)
    named = np.zeros(rows, dtype=bool)
    named[slot[(slot >= 0) & (slot < rows)]] = True
    ys[~named] = NAN  # a row that no entry names is not read into a sum
    weights = rng.standard_normal((tokens, top_k)).astype(np.float32)
    weights[(slot < 0) | (slot >= rows)] = INF  # nor is the weight of an entry without a row
    base = rng.standard_normal((tokens, cols), dtype=np.float32)
    want, size = routing.combine_rows(ys, slot, weights, None if with_base == "none" else base)
    d = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    b = None if with_base == "none" else d(base)
    y = b if with_base == "in place" else torch.full((tokens, cols), NAN, device="cuda", dtype=getattr(torch, out))
    print(f"combine {tokens}x{top_k} {cols} {with_base} {out}", flush=True)
    uw.combine_rows(d(ys), d(slot), d(weights), y, base=b)
    torch.cuda.synchronize()
    got = y.float().cpu().numpy().astype(np.float64)
    # top_k products and sums and the base's, each rounded by 2^-24 of at most the terms' magnitudes
    tol = (2 * top_k + 1) * 2.0 ** -24 * size
    if out == "bfloat16":
        tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got - want) <= tol).all()


def test_combine_specials(env):
    """Infinities and NaN that an entry names arrive in the sum; bf16 keeps them."""
    torch, uw = env
    ys = torch.zeros((3, 8), device="cuda")
    ys[0, 0], ys[1, 0], ys[0, 1], ys[2, 2] = INF, -INF, NAN, INF
    slot = torch.tensor([[0, 1], [2, -1]], dtype=torch.int32, device="cuda")
    w = torch.ones((2, 2), device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        y = torch.empty((2, 8), device="cuda", dtype=dtype)
        uw.combine_rows(ys, slot, w, y)
        r = y.float().cpu().numpy()
        assert np.isnan(r[0, 0]) and np.isnan(r[0, 1]) and r[1, 2] == INF and (r[:, 3:] == 0).all()
    big = torch.full((1, 8), 3.4e38, device="cuda")  # rounds up to bf16's infinity
    y = torch.empty((1, 8), device="cuda", dtype=torch.bfloat16)
    uw.combine_rows(big, torch.zeros((1, 1), dtype=torch.int32, device="cuda"), torch.ones((1, 1), device="cuda"), y)
    assert torch.equal(y, big.to(torch.bfloat16))


def test_dispatch_larger_than_the_caches(env):
    """Copies of 128 MiB and more are stored past the caches."""
    torch, uw = env
    rng = np.random.default_rng(6)
    tokens, top_k, cols = 4100, 4, 4096
    slot = rng.permutation(tokens * top_k).reshape(tokens, top_k).astype(np.int32)
    slot[rng.random(slot.shape) < 0.1] = -1
    x = torch.randn((tokens, cols), device="cuda").to(torch.bfloat16)
    xs = torch.full((tokens * top_k, cols), 7.0, dtype=torch.bfloat16, device="cuda")
    s = torch.from_numpy(slot).cuda().long()
    want = xs.clone()
    for j in range(top_k):
        there = s[:, j] >= 0
        want[s[there, j]] = x[there]
    uw.dispatch_rows(x, torch.from_numpy(slot).cuda(), xs)
    torch.cuda.synchronize()
    assert torch.equal(xs, want)


def test_far_offsets(env):
    """Rows past 2^31 elements: logits, activations, their copies and the experts' rows."""
    torch, uw = env
    rows, cols = 70000, 32768
    wide = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([3, 65530, 65600, 69998, 69999], device="cuda")
    logits = torch.randn((5, 8), device="cuda").to(torch.bfloat16)
    wide[at, cols - 8:] = logits
    e, w = torch.empty((rows, 2), dtype=torch.int32, device="cuda"), torch.empty((rows, 2), device="cuda")
    print("far offsets: route", flush=True)
    uw.route(wide[:, cols - 8:], e, w)
    want, _ = routing.route(logits.float().cpu().numpy(), 2)
    assert np.array_equal(e[at].cpu().numpy(), want) and (e[10].cpu().numpy() == [0, 1]).all()
    # dispatch from far rows to far rows and back
    slot = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
    slot[at, 0] = torch.tensor([69999, 5, 69000, 66000, 0], dtype=torch.int32, device="cuda")
    wide[at] = torch.randn((5, cols), device="cuda").to(torch.bfloat16)
    xs = torch.zeros_like(wide)
    print("far offsets: dispatch", flush=True)
    uw.dispatch_rows(wide, slot, xs)
    torch.cuda.synchronize()
    assert torch.equal(xs[slot[at, 0].long()], wide[at]) and int((xs != 0).any(dim=1).sum()) == 5
    del xs
    ys = torch.full((rows, cols), float("nan"), device="cuda")
    ys[slot[at, 0].long()] = wide[at].float()
    weights = torch.full((rows, 1), 2.0, device="cuda")
    y = torch.empty((rows, cols), device="cuda", dtype=torch.bfloat16)
    print("far offsets: combine", flush=True)
    uw.combine_rows(ys, slot, weights, y)
    torch.cuda.synchronize()
    assert torch.equal(y[at].float(), wide[at].float() * 2) and int((y != 0).any(dim=1).sum()) == 5


def test_most_tokens(env):
    """The largest token counts: 2^24 routed, and more dispatched and combined than
    one grid has workgroups along the tokens."""
    torch, uw = env
    t = 1 << 24
    logits = torch.randn((t, 3), device="cuda")
    e, w = torch.empty((t, 1), dtype=torch.int32, device="cuda"), torch.empty((t, 1), device="cuda")
    print("route 2^24 tokens", flush=True)
    uw.route(logits, e, w, renormalise=False)
    top, at = torch.softmax(logits.double(), dim=1).max(dim=1)
    assert torch.equal(e[:, 0].long(), at)  # (float32 normals: no equal logits where the largest decides)
    assert float(((w[:, 0].double() - top).abs() / top).max()) <= WEIGHT_TOL
    del logits, top, at, e, w
    t = (1 << 20) + 1000
    x = torch.randn((t, 8), device="cuda").to(torch.bfloat16)
    slot = torch.randperm(t, device="cuda").to(torch.int32).reshape(t, 1)
    xs = torch.empty_like(x)
    print("dispatch and combine 2^20 + 1000 tokens", flush=True)
    uw.dispatch_rows(x, slot, xs)
    torch.cuda.synchronize()
    assert torch.equal(xs[slot[:, 0].long()], x)
    y = torch.empty((t, 8), device="cuda")
    uw.combine_rows(xs.float(), slot, torch.full((t, 1), 0.5, device="cuda"), y)
    torch.cuda.synchronize()
    assert torch.equal(y, x.float() * 0.5)


def test_group_in_a_graph(env):
    """Both forms of the sort captured, replayed over new labels."""
    torch, uw = env
    for n, groups in ((3000, 40), (30000, 300)):
        d = torch.zeros(n, dtype=torch.int32, device="cuda")
        offsets = torch.empty(groups + 1, dtype=torch.int32, device="cuda")
        order, slot = torch.empty_like(d), torch.empty_like(d)
        work = torch.empty(uw.group_rows_workspace_bytes(n, groups), dtype=torch.uint8, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            uw.group_rows(d, groups, offsets, order, slot, work, stream=torch.cuda.current_stream())
        for seed in range(4):
            index = np.random.default_rng(seed).integers(-1, groups, size=n)
            d.copy_(torch.from_numpy(index.astype(np.int32)))
            for b in (offsets, order, slot, work):
                b.fill_(7)
            graph.replay()
            torch.cuda.synchronize()
            label = np.where(index < 0, groups, index)
            want = np.argsort(label, kind="stable")
            assert np.array_equal(order.cpu().numpy(), want)
            assert np.array_equal(offsets.cpu().numpy(), np.searchsorted(label[want], np.arange(groups + 1)))


# ---- together, on another stream and in a graph ----


def test_routed_rows_together(env):
    """Route, group, dispatch and combine as a layer calls them, with the identity
    as every expert: each token gets the sum of its weights times itself."""
    torch, uw = env
    tokens, experts, k, cols = 300, 24, 4, 128
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    bias = torch.randn(experts, generator=g, device="cuda") * 0.1
    buf = dict(e=torch.empty((tokens, k), dtype=torch.int32, device="cuda"), w=torch.empty((tokens, k), device="cuda"),
               offsets=torch.empty(experts + 1, dtype=torch.int32, device="cuda"),
               order=torch.empty(tokens * k, dtype=torch.int32, device="cuda"),
               slot=torch.empty((tokens, k), dtype=torch.int32, device="cuda"),
               xs=torch.zeros((tokens * k, cols), dtype=torch.bfloat16, device="cuda"),
               y=torch.empty((tokens, cols), device="cuda"))
    logits = torch.randn((tokens, experts), generator=g, device="cuda")
    x = torch.randn((tokens, cols), generator=g, device="cuda").to(torch.bfloat16)
    rows = torch.empty((tokens * k, cols), device="cuda")

    def layer(stream=None):
        uw.route(logits, buf["e"], buf["w"], score=uw.SCORE_SIGMOID, bias=bias, groups=4, top_groups=2,
                 group_score=uw.GROUP_TOP2, scale=1.5, stream=stream)
        uw.group_rows(buf["e"], experts, buf["offsets"], buf["order"], buf["slot"], stream=stream)
        uw.dispatch_rows(x, buf["slot"], buf["xs"], stream=stream)
        rows.copy_(buf["xs"])
        uw.combine_rows(rows, buf["slot"], buf["w"], buf["y"], stream=stream)

    def check():
        torch.cuda.synchronize()
        want_e, want_w = routing.route(logits.cpu().numpy(), k, routing.SIGMOID, bias.cpu().numpy(), 4, 2,
                                       routing.GROUP_TOP2, True, 1.5)
        assert np.array_equal(buf["e"].cpu().numpy(), want_e)
        offsets, order, slot = routing.group_rows(want_e, experts)
        assert np.array_equal(buf["slot"].cpu().numpy(), slot) and np.array_equal(buf["order"].cpu().numpy(), order)
        # weights that sum to 1.5; k products and sums
        want = x.double().cpu().numpy() * 1.5
        assert (np.abs(buf["y"].cpu().numpy() - want) <= (3 * k + 4) * 2.0 ** -24 * np.abs(want)).all()
        assert int(buf["offsets"][-1]) == tokens * k

    layer()
    check()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        logits.normal_(generator=g)
        layer(stream=side)
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(stream=torch.cuda.current_stream())
    for _ in range(4):
        logits.normal_(generator=g)
        x.normal_(generator=g)
        for b in buf.values():
            b.zero_()
        graph.replay()
        check()
