"""Refused arguments of the routing and adapter calls: the C entry points check
them on the host before any launch (CPU; addresses are never read), and the
Python calls check what only they see of a tensor."""
import ctypes as C

import pytest
import torch

import decode_gemm_bf16_amd as uw

L = uw._lib
A, B, D, E, F = 0x10000000, 0x20000000, 0x30000000, 0x40000000, 0x50000000  # stand-ins for device addresses
HUGE = (1 << 24) + 1


def cfg(**kw):
    d = dict(experts=8, top_k=2, score=0, groups=1, top_groups=1, group_score=0, renormalise=1, scale=1.0)
    d.update(kw)
    return uw.RouteConfig(*[d[k] for k, _ in uw.RouteConfig._fields_])


def route(logits=A, type=0, ld=8, tokens=4, bias=None, config=None, experts=B, weights=D, **kw):
    return L.uw_route(logits, type, ld, tokens, bias, C.byref(config or cfg(**kw)), experts, weights, None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), uw.ERR_INVALID_ARG), (dict(experts=None), uw.ERR_INVALID_ARG),
    (dict(weights=None), uw.ERR_INVALID_ARG), (dict(tokens=0), uw.ERR_INVALID_ARG),
    (dict(tokens=-1), uw.ERR_INVALID_ARG), (dict(tokens=HUGE), uw.ERR_INVALID_ARG),
    (dict(type=2), uw.ERR_INVALID_ARG), (dict(ld=7), uw.ERR_SHAPE), (dict(logits=A + 2), uw.ERR_INVALID_ARG),
    (dict(bias=A + 1), uw.ERR_INVALID_ARG), (dict(experts=A + 16), uw.ERR_INVALID_ARG),
    (dict(weights=B + 4), uw.ERR_INVALID_ARG), (dict(bias=D + 8), uw.ERR_INVALID_ARG),
    (dict(config=cfg(experts=0)), uw.ERR_SHAPE), (dict(config=cfg(experts=1025), ld=2000), uw.ERR_SHAPE),
    (dict(config=cfg(top_k=0)), uw.ERR_INVALID_ARG), (dict(config=cfg(top_k=9)), uw.ERR_INVALID_ARG),
    (dict(config=cfg(experts=128, top_k=65), ld=128), uw.ERR_INVALID_ARG),
    (dict(config=cfg(groups=0)), uw.ERR_SHAPE), (dict(config=cfg(groups=3)), uw.ERR_SHAPE),
    (dict(config=cfg(experts=130, groups=65), ld=130), uw.ERR_SHAPE),
    (dict(config=cfg(groups=2, top_groups=3)), uw.ERR_INVALID_ARG),
    (dict(config=cfg(groups=2, top_groups=0)), uw.ERR_INVALID_ARG),
    (dict(config=cfg(score=2)), uw.ERR_INVALID_ARG), (dict(config=cfg(group_score=-1)), uw.ERR_INVALID_ARG),
    (dict(config=cfg(scale=float("nan"))), uw.ERR_INVALID_ARG),
    (dict(config=cfg(scale=float("inf"))), uw.ERR_INVALID_ARG),
])
def test_route_refuses(kw, status):
    assert route(**kw) == status
    assert uw.last_error()


def group(index=A, n=100, groups=8, offsets=B, order=D, slot=E, work=None, work_bytes=0):
    return L.uw_group_rows(index, n, groups, offsets, order, slot, work, work_bytes, None)


def test_group_rows_refuses():
    for kw in (dict(index=None), dict(offsets=None), dict(order=None), dict(slot=None), dict(n=0), dict(n=-5),
               dict(n=(1 << 30) + 1), dict(groups=0), dict(groups=4001), dict(index=A + 2), dict(slot=A),
               dict(order=A + 396), dict(offsets=E + 4), dict(n=100000), dict(n=100000, work=F, work_bytes=64)):
        assert group(**kw) == uw.ERR_INVALID_ARG, kw
    assert uw.group_rows_workspace_bytes(100, 8) == 0
    assert uw.group_rows_workspace_bytes(100000, 8) > 0
    assert uw.group_rows_workspace_bytes(0, 8) == uw.group_rows_workspace_bytes(5, 4001) == 0


def test_dispatch_and_combine_refuse():
    def dispatch(x=A, ldx=64, slot=B, tokens=4, top_k=2, cols=64, xs=D, rows=8):
        return L.uw_dispatch_rows(x, ldx, slot, tokens, top_k, cols, xs, rows, None)

    for kw, status in ((dict(x=None), 1), (dict(slot=None), 1), (dict(xs=None), 1), (dict(tokens=0), 1),
                       (dict(tokens=HUGE), 1), (dict(top_k=0), 1), (dict(tokens=1 << 24, top_k=65), 1),
                       (dict(rows=0), 1), (dict(cols=60), 2), (dict(cols=0), 2), (dict(ldx=56), 2), (dict(ldx=68), 2),
                       (dict(x=A + 8), 1), (dict(xs=D + 2), 1), (dict(xs=A + 16), 1), (dict(xs=B - 512), 1)):
        assert dispatch(**kw) == status, kw

    def combine(ys=A, rows=8, slot=B, weights=D, tokens=4, top_k=2, cols=64, base=None, y=E, type=0):
        return L.uw_combine_rows(ys, rows, slot, weights, tokens, top_k, cols, base, y, type, None)

    for kw, status in ((dict(ys=None), 1), (dict(slot=None), 1), (dict(weights=None), 1), (dict(y=None), 1),
                       (dict(type=3), 1), (dict(tokens=0), 1), (dict(cols=4), 2), (dict(rows=-1), 1),
                       (dict(ys=A + 4), 1), (dict(y=A), 1), (dict(base=E + 16), 1), (dict(base=E, type=1), 1),
                       (dict(y=D - 16), 1), (dict(base=F + 8), 1)):
        assert combine(**kw) == status, kw


def test_lora_refuses_without_a_device_handle():
    h = C.c_void_p()
    for args, status in (((0, 64, 4, 8), 2), ((24, 64, 4, 8), 2), ((16, 32, 4, 8), 2), ((16, 96, 4, 8), 2),
                         ((1 << 24, 64, 4, 8), 2), ((16, 64, 0, 8), 1), ((16, 64, 4001, 8), 1), ((16, 64, 4, 0), 1),
                         ((16, 64, 4, 257), 1)):
        assert L.uw_lora_create(*args, C.byref(h)) == status, args
        assert not h.value
    assert L.uw_lora_create(16, 64, 4, 8, None) == uw.ERR_INVALID_ARG
    assert L.uw_lora_load(None, 0, A, B, 1, 1.0, None) == uw.ERR_INVALID_ARG
    L.uw_lora_free(None)
    assert uw.lora_plan_bytes(0, 4) == uw.lora_plan_bytes(4, 0) == uw.lora_plan_bytes(HUGE, 4) == 0
    need = uw.lora_plan_bytes(100, 4)
    assert need > 0
    for args in ((None, 100, 4, B, need), (A, 0, 4, B, need), (A, 100, 0, B, need), (A, 100, 4, None, need),
                 (A, 100, 4, B, need - 1), (A, 100, 4, B + 8, need), (A, 100, 4, A, need), (A + 2, 100, 4, B, need)):
        assert L.uw_lora_plan(*args, None) == uw.ERR_INVALID_ARG, args
    one, none = (C.c_void_p * 1)(A), (C.c_void_p * 1)(None)
    ld = (C.c_int64 * 1)(64)
    assert L.uw_lora_workspace_bytes(none, 1, 4) == L.uw_lora_workspace_bytes(one, 0, 4) == 0
    for n, handles in ((1, none), (0, none), (5, none)):
        assert L.uw_lora_apply(handles, n, A, 1 << 20, B, 64, None, None, one, ld, 4, D, 1 << 20, None) == uw.ERR_INVALID_ARG
    assert L.uw_lora_apply(none, 1, A, 1 << 20, B, 64, one, None, one, ld, 4, D, 1 << 20, None) == uw.ERR_INVALID_ARG


class AdaptersRecord(C.Structure):
    """The host side of a uw_lora, as routing.cpp lays it out: without a device no call makes one."""
    _fields_ = ([(k, C.c_int64) for k in ("rows", "cols", "rows64")] +
                [(k, C.c_int32) for k in ("slots", "max_rank", "rank16", "device")] +
                [(k, C.c_void_p) for k in ("mem", "a", "b", "table")])


def test_lora_apply_refuses_overlaps():
    """Each buffer that the call writes, against each other buffer of the call."""
    tokens, rows, cols, slots = 100, 64, 128, 4
    records = [AdaptersRecord(rows, cols, rows, slots, 16, 16, 0, None, None, None, None) for _ in range(2)]
    hs = (C.c_void_p * 2)(*[C.addressof(r) for r in records])
    plan_bytes = uw.lora_plan_bytes(tokens, slots)
    need = L.uw_lora_workspace_bytes(hs, 2, tokens)
    assert need > 0
    xbytes, ybytes = tokens * cols * 2, tokens * rows * 4
    plan, x, work, y0, y1, b0, b1 = (i << 28 for i in range(1, 8))

    def call(plan=plan, x=x, work=work, ys=(y0, y1), bases=(b0, b1)):
        ld = (C.c_int64 * 2)(rows, rows)
        return L.uw_lora_apply(hs, 2, plan, plan_bytes, x, cols, (C.c_void_p * 2)(*bases), ld, (C.c_void_p * 2)(*ys), ld,
                               tokens, work, need, None)

    down, up = (lambda n: n - n % 256), (lambda n: n + -n % 256)
    for kw in (dict(work=plan), dict(work=plan + down(plan_bytes - 1)), dict(work=plan - down(need - 1)),
               dict(work=x), dict(work=x + down(xbytes - 1)), dict(work=x - down(need - 1)),
               dict(work=b0), dict(work=b0 + down(ybytes - 1)), dict(work=b1 - down(need - 1)),
               dict(work=y0), dict(work=y1 + down(ybytes - 1)), dict(ys=(y0, y0 + 16)), dict(ys=(x, y1)),
               dict(ys=(y0, plan + 16)), dict(ys=(b1, y1)), dict(ys=(y0, b1 + 16))):
        assert call(**kw) == uw.ERR_INVALID_ARG, kw
        assert "overlap" in uw.last_error(), kw
    if not torch.cuda.is_available():  # side by side, and in place, they go on to ask for the device
        for kw in (dict(), dict(work=plan + up(plan_bytes)), dict(work=x - up(need)), dict(work=b1 + up(ybytes)),
                   dict(bases=(y0, y1)), dict(bases=(None, b1))):
            assert call(**kw) == uw.ERR_HIP, kw


def test_moe_forward_refuses():
    assert uw.moe_workspace_bytes(0, 64, 64, 8, 2) == uw.moe_workspace_bytes(4, 64, 64, 8, 9) == 0
    assert uw.moe_workspace_bytes(4, 64, 64, 1025, 2) == 0
    w = torch.zeros((64, 64), dtype=torch.int16).numpy().view("uint16")
    mats = [uw.Matrix(w, uw.FMT_PALETTE | uw.ENC_HOST_ONLY) for _ in range(6)]
    hs = (C.c_void_p * 6)(*[m.handle for m in mats])
    ps = (C.c_int32 * 3)(4, 4, 4)

    def call(handles=hs, pipelines=ps, logits=A, config=None, x=B, base=None, y=D, tokens=4, work=E, size=1 << 20):
        return L.uw_moe_forward(handles, pipelines, logits, 0, 2, None, C.byref(config or cfg(experts=2)), x, base, y,
                                tokens, work, size)

    for kw in (dict(handles=None), dict(pipelines=None), dict(logits=None), dict(x=None), dict(y=None),
               dict(work=None), dict(work=E + 64), dict(tokens=0), dict(config=cfg(experts=0)),
               dict(config=cfg(experts=2000)), dict(config=cfg(experts=2, top_k=3)),
               dict(handles=(C.c_void_p * 6)(hs[0], hs[1], hs[2], hs[3], None, hs[5]))):
        assert call(**kw) == uw.ERR_INVALID_ARG, kw
    assert call() == uw.ERR_UNSUPPORTED  # host-only experts
    with pytest.raises(ValueError):
        uw.moe_forward(mats[:2], [4, 4, 4], None, None, None, None, 1)


def test_python_refuses_tensors():
    f, i = torch.zeros(4, 8), torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="current GPU"):  # a CPU tensor
        uw.route(f, i, torch.zeros(4, 2))
    with pytest.raises(TypeError):
        uw.route(f.double(), i, torch.zeros(4, 2))
    with pytest.raises(TypeError):
        uw.route(f.numpy(), i, torch.zeros(4, 2))
    with pytest.raises(ValueError):
        uw.route(f[0], i, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="contiguous"):
        uw.route(f.t(), i, torch.zeros(4, 2))
    with pytest.raises(ValueError, match="contiguous"):
        uw.route(f[:1].expand(4, 8), i, torch.zeros(4, 2))
    with pytest.raises(TypeError):
        uw.group_rows(i.long(), 8, i, i, i)
    with pytest.raises(TypeError):
        uw.dispatch_rows(f, i, f)
    with pytest.raises(ValueError):
        uw.lora_apply([], None, torch.zeros(4, 8, dtype=torch.bfloat16), [f], None)
