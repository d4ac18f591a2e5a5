"""Refusals of the gate, routed side path and 4-bit entry points that need no GPU: argument
errors are found on the host before any CUDA call, through the C ABI and in the binding."""
import ctypes
import weakref

import numpy as np
import pytest
import torch

from post_hoc_rank_b200 import api, build
from post_hoc_rank_b200 import loraforge as lf

INVALID, SHAPE, WORKSPACE, ALIGNMENT = 1, 2, 4, 8


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def test_structures_match_the_header():
    assert ctypes.sizeof(lf.lf_router) == 32
    assert ctypes.sizeof(lf.lf_mixture_projection) == 3 * 8 + 8 + 16 + ctypes.sizeof(lf.lf_slice)
    assert ctypes.sizeof(lf.lf_mixture_grad) == 4 * 8 + 8 + 24 + ctypes.sizeof(lf.lf_slice)
    assert ctypes.sizeof(lf.lf_w4_projection) == 80


def route(T=4, logits=16, type=0, ld=8, bias=None, ids=16, w=16, counts=None, backward=False, grad=16, grad_ld=8, **kw):
    r = lf.make_router(kw.pop("E", 8), kw.pop("K", 2))
    for k, v in kw.items():
        setattr(r, k, v)
    if backward:
        return lf.lib().lf_route_experts_backward(T, ctypes.byref(r), logits, type, ld, ids, w, grad, grad_ld, None)
    return lf.lib().lf_route_experts(T, ctypes.byref(r), logits, type, ld, bias, ids, w, counts, None)


@pytest.mark.parametrize("backward", [False, True])
def test_router_refusals(backward):
    for bad in (dict(T=-1), dict(logits=0), dict(ids=0), dict(w=0), dict(type=3), dict(type=-1), dict(score=2), dict(score=-1),
                dict(renorm=2), dict(ld=7), dict(weight_scale=float("inf")), dict(weight_scale=float("nan"))):
        assert route(backward=backward, **bad) == INVALID, bad
    for bad in (dict(E=0, K=1), dict(E=1025, ld=2000), dict(K=0), dict(K=9), dict(E=40, K=17, ld=40), dict(n_groups=0),
                dict(n_groups=3), dict(E=64, ld=64, n_groups=64), dict(n_groups=4, top_groups=5), dict(top_groups=0),
                dict(group_top=0), dict(group_top=3)):
        assert route(backward=backward, **bad) == SHAPE, bad
    for bad in (dict(logits=18), dict(ids=18), dict(w=18), dict(logits=17, type=1)):
        assert route(backward=backward, **bad) == ALIGNMENT, bad
    assert lf.lib().lf_route_experts(4, None, 16, 0, 8, None, 16, 16, None, None) == INVALID
    if backward:
        assert route(backward=True, grad=0) == INVALID and route(backward=True, grad_ld=7) == INVALID
        assert route(backward=True, grad=18) == ALIGNMENT
        assert route(backward=True, T=0) == 0
    else:
        assert route(bias=18) == ALIGNMENT and route(counts=18) == ALIGNMENT
        assert route(T=0) == 0


def a_slice(**kw):
    d = dict(d_out=64, max_rank=8, y_offset=0, ranks=16, off_A=16, off_Bt=16, A_pool=16, Bt_pool=16, pool_elems_A=1 << 20,
             pool_elems_Bt=1 << 20)
    d.update({k: v for k, v in kw.items() if k in d})
    return lf.lf_slice(*d.values())


def mix(backward=False, T=4, K=2, ids=16, n=4, n_proj=1, projs=True, ws=16, wsb=1 << 30, gw=16, x=16, base=16, y=16, d_in=64,
        reserved=0, x_ld=64, y_ld=64, dx=16, dx_ld=64, **kw):
    sl = a_slice(**kw)
    if backward:
        arr = (lf.lf_mixture_grad * max(n_proj, 1))(*[lf.lf_mixture_grad(x, y, base, dx, d_in, reserved, x_ld, y_ld, dx_ld, sl)
                                                      for _ in range(max(n_proj, 1))])
        return lf.lib().lf_lora_mixture_backward(T, K, ids, 16, n, arr if projs else None, n_proj, 1.0, None, gw, ws, wsb, None)
    arr = (lf.lf_mixture_projection * max(n_proj, 1))(*[lf.lf_mixture_projection(x, base, y, d_in, reserved, x_ld, y_ld, sl)
                                                        for _ in range(max(n_proj, 1))])
    return lf.lib().lf_lora_mixture(T, K, ids, 16, n, arr if projs else None, n_proj, 1.0, None, ws, wsb, None)


@pytest.mark.parametrize("backward", [False, True])
def test_mixture_refusals(backward):
    assert mix(backward, T=0) == 0
    for bad in (dict(T=-1), dict(n=0), dict(n=20000), dict(n_proj=0), dict(n_proj=9), dict(projs=False), dict(ids=0), dict(x=0),
                dict(y=0), dict(d_in=0), dict(reserved=1), dict(x_ld=56), dict(y_ld=56), dict(d_out=0), dict(max_rank=65),
                dict(max_rank=-1), dict(y_offset=-8), dict(y_offset=8), dict(ranks=0), dict(off_A=0), dict(A_pool=0),
                dict(pool_elems_A=-1)):
        assert mix(backward, **bad) == INVALID, bad
    for bad in (dict(K=0), dict(K=17), dict(T=1 << 30)):
        assert mix(backward, **bad) == SHAPE, bad
    for bad in (dict(x=24), dict(y=24), dict(base=24), dict(d_in=60), dict(x_ld=68), dict(y_ld=68), dict(d_out=60),
                dict(A_pool=24)):
        assert mix(backward, **bad) == ALIGNMENT, bad
    # the dense path needs its workspace
    big = dict(T=8192, n=16, max_rank=64, d_in=2048, x_ld=2048, d_out=2048, y_ld=2048, dx_ld=2048, K=4)
    assert mix(backward, ws=0, **big) == INVALID
    assert mix(backward, wsb=1024, **big) == WORKSPACE
    if backward:
        assert mix(True, dx_ld=56) == INVALID and mix(True, dx=24) == ALIGNMENT and mix(True, dx_ld=68) == ALIGNMENT
        assert mix(True, dx=0) == INVALID              # a base without its gradient
        assert mix(True, dx=0, base=0, gw=0) == 0      # nothing asked for
        assert mix(True, n_proj=2, ws=0) == INVALID    # the sum over projections goes through the workspace
        assert mix(True, n_proj=2, wsb=16) == WORKSPACE


@pytest.mark.parametrize("backward", [False, True])
def test_mixture_refuses_misaligned_tables_and_far_slices(backward):
    for bad in (dict(ids=18), dict(ranks=18), dict(off_A=20), dict(off_Bt=20)):
        assert mix(backward, **bad) == ALIGNMENT, bad
    if backward:
        assert mix(True, gw=18) == ALIGNMENT
    # y_offset + d_out past 63 bits
    assert mix(backward, y_offset=(1 << 63) - 8) == INVALID


def test_mixture_workspace_sizes():
    sl = a_slice(d_out=2048, max_rank=64)
    p = lf.lf_mixture_projection(16, None, 16, 2048, 0, 2048, 2048, sl)
    g = lf.lf_mixture_grad(16, 16, None, 16, 2048, 0, 2048, 2048, 2048, sl)
    fwd = lf.lf_lora_mixture_workspace_size(8192, 4, 16, [p])
    assert fwd >= 1024 * 4096 * 2 + 2 * 8192 * 1024 * 2
    assert lf.lf_lora_mixture_backward_workspace_size(8192, 4, 16, [g]) >= fwd + 2 * 8192 * 1024 * 4
    assert lf.lf_lora_mixture_workspace_size(4, 4, 16, [p]) == 0        # token by token
    assert lf.lf_lora_mixture_workspace_size(8192, 4, 64, [p]) == 0     # a pool of 4096 rows
    assert lf.lf_lora_mixture_backward_workspace_size(4, 2, 16, [g, g]) >= 2 * 4 * 2 * 4
    for bad in ((-1, 2, 4), (4, 0, 4), (4, 17, 4), (4, 2, 0)):
        assert lf.lf_lora_mixture_workspace_size(*bad, [p]) == 0


def w4(T=4, n_proj=1, projs=True, **kw):
    d = dict(x=16, y=16, q=16, scales=16, zeros=16, bias=16, d_in=64, d_out=64, group=32, reserved=0, x_ld=64, y_ld=64)
    d.update(kw)
    arr = (lf.lf_w4_projection * max(n_proj, 1))(*[lf.lf_w4_projection(*d.values()) for _ in range(max(n_proj, 1))])
    return lf.lib().lf_w4_projections(T, arr if projs else None, n_proj, None)


def test_w4_refusals():
    assert w4(T=0) == 0
    for bad in (dict(T=-1), dict(n_proj=0), dict(n_proj=9), dict(projs=False), dict(x=0), dict(y=0), dict(q=0), dict(scales=0),
                dict(x_ld=32), dict(y_ld=56), dict(reserved=1)):
        assert w4(**bad) == INVALID, bad
    for bad in (dict(d_in=0), dict(d_in=48), dict(d_out=0), dict(group=16), dict(group=96), dict(group=0), dict(group=512)):
        assert w4(**bad) == SHAPE, bad
    for bad in (dict(x=24), dict(y=24), dict(q=24), dict(scales=17), dict(bias=17), dict(d_out=60), dict(x_ld=68), dict(y_ld=68)):
        assert w4(**bad) == ALIGNMENT, bad
    L = lf.lib()
    ok = dict(W=16, t=1, d_out=64, d_in=64, g=32, q=16, s=16, z=16)

    def quant(**kw):
        a = dict(ok, **kw)
        return L.lf_w4_quantize(a["W"], a["t"], a["d_out"], a["d_in"], a["g"], a["q"], a["s"], a["z"], None)

    def dequant(**kw):
        a = dict(ok, **kw)
        return L.lf_w4_dequantize(a["q"], a["s"], a["z"], a["d_out"], a["d_in"], a["g"], a["W"], a["t"], None)
    for f in (quant, dequant):
        for bad in (dict(W=0), dict(q=0), dict(s=0), dict(t=3), dict(t=-1)):
            assert f(**bad) == INVALID, bad
        for bad in (dict(d_in=40), dict(d_in=-32), dict(d_out=0), dict(g=100)):
            assert f(**bad) == SHAPE, bad
        for bad in (dict(W=24), dict(q=24), dict(s=17), dict(d_out=12)):
            assert f(**bad) == ALIGNMENT, bad


def test_binding_refusals():
    b = torch.bfloat16
    x, y = torch.zeros(4, 64, dtype=b), torch.zeros(4, 96, dtype=b)
    sl = lf.make_slice(64, 0, None, None, None, x, x)
    lf.make_mixture_projection(x, y, sl, base=y)
    wide = torch.zeros(4, 200, dtype=b)
    p = lf.make_mixture_projection(wide[:, 8:72], wide[:, 80:176], sl)
    assert (p.d_in, p.x_ld, p.y_ld, p.rows) == (64, 200, 200, 4)
    one = torch.zeros(64, dtype=b).expand(1, 64)
    assert lf.make_mixture_projection(one, y[:1], sl).x_ld >= 64
    for bad in (lambda: lf.make_mixture_projection(x.float(), y, sl), lambda: lf.make_mixture_projection(x, y[:3], sl),
                lambda: lf.make_mixture_projection(x, y, sl, base=x), lambda: lf.make_mixture_projection(x.t(), y, sl),
                lambda: lf.make_mixture_projection(x[0], y, sl), lambda: lf.make_mixture_projection(x, y, sl, base=wide[:, :96]),
                lambda: lf.make_mixture_grad(x, y[:2], None, sl), lambda: lf.make_mixture_grad(x, y, y, sl),
                lambda: lf.make_mixture_grad(x, y, None, sl, dx_base=x),
                lambda: lf.make_router(8, 2, "tanh"), lambda: lf.type_code(torch.float64)):
        with pytest.raises(ValueError):
            bad()
    q, s = torch.zeros(96, 32, dtype=torch.uint8), torch.zeros(96, 2, dtype=b)
    lf.make_w4_projection(x, y, q, s, 32, zeros=torch.zeros(96, 2, dtype=torch.uint8), bias=torch.zeros(96, dtype=b))
    for bad in (lambda: lf.make_w4_projection(x, y, q, s, 64), lambda: lf.make_w4_projection(x, y, q, s.float(), 32),
                lambda: lf.make_w4_projection(x, y[:, :88], q, s, 32), lambda: lf.make_w4_projection(y, y, q, s, 32),
                lambda: lf.make_w4_projection(x, y, q[:, ::2], s, 32), lambda: lf.make_w4_projection(x, y, q, s, 32, bias=s),
                lambda: lf.make_w4_projection(x, y, q, s, 32, zeros=q), lambda: lf.make_w4_projection(x, y, q.int(), s, 32)):
        with pytest.raises(ValueError):
            bad()
    logits = torch.zeros(4, 8)
    r = lf.make_router(8, 2)
    for bad in (lambda: api.route_experts(logits, r), lambda: api.route_experts(logits[:, :4], r),
                lambda: api.route_experts(logits.t(), lf.make_router(4, 2)),
                lambda: api.route_experts(logits[:1].expand(4, 8), r),
                lambda: api.route_experts(logits, r, bias=torch.zeros(7)),
                lambda: api.route_experts_backward(logits, r, torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)),
                lambda: api.lora_mixture(torch.zeros(4, 2, dtype=torch.int64), None, 4, [p], 1.0),
                lambda: api.lora_mixture(torch.zeros(5, 2, dtype=torch.int32), None, 4, [p], 1.0),
                lambda: api.w4_quantize(torch.zeros(8, 64), 32)):
        with pytest.raises(ValueError):
            bad()


def test_binding_refuses_slices_past_the_columns_and_mixed_devices():
    b = torch.bfloat16
    x, wide = torch.zeros(4, 64, dtype=b), torch.zeros(4, 200, dtype=b)
    y = wide[:, :96]                      # rows of 200, of which 96 columns are y's
    pool = torch.zeros(1024, dtype=b)
    at = lambda off: lf.make_slice(64, off, None, None, None, pool, pool)  # noqa: E731
    lf.make_mixture_projection(x, y, at(32), base=y)
    lf.make_mixture_grad(x, y, None, at(32))
    m = torch.zeros(4, 64, dtype=b, device="meta")
    there = lf.make_slice(64, 0, None, None, None, pool.to("meta"), pool)
    q, s = torch.zeros(96, 32, dtype=torch.uint8), torch.zeros(96, 2, dtype=b)
    for bad in (lambda: lf.make_mixture_projection(x, y, at(40)), lambda: lf.make_mixture_grad(x, y, None, at(40)),
                lambda: lf.make_mixture_projection(x, m, at(0)), lambda: lf.make_mixture_projection(x, y, there),
                lambda: lf.make_mixture_grad(x, m, None, at(0)), lambda: lf.make_mixture_grad(x, y, m, at(0)),
                lambda: lf.make_mixture_grad(x, y, None, there), lambda: lf.make_w4_projection(x, y, q.to("meta"), s, 32),
                lambda: lf.make_w4_projection(x, y, q, s, 32, bias=torch.zeros(96, dtype=b, device="meta"))):
        with pytest.raises(ValueError):
            bad()


def test_flags_and_names_reach_the_structure():
    r = lf.make_router(64, 4, "sigmoid", n_groups=8, top_groups=3, group_top=2, renorm=False, weight_scale=2.5)
    assert (r.n_experts, r.top_k, r.score, r.n_groups, r.top_groups, r.group_top, r.renorm) == (64, 4, 1, 8, 3, 2, 0)
    assert np.float32(r.weight_scale) == np.float32(2.5)


def test_descriptions_hold_their_tensors():
    """Tensors made in place (a cast input, a slice's tables) live as long as the description
    that carries their addresses, and as the array that is made of descriptions."""
    b = torch.bfloat16
    new = lambda *shape, **kw: torch.zeros(*shape, dtype=kw.get("dtype", b))  # noqa: E731

    def a_slice(seen):
        t = [new(4, dtype=torch.int32), new(4, dtype=torch.int64), new(4, dtype=torch.int64), new(1024), new(1024)]
        seen += [weakref.ref(v) for v in t]
        return lf.make_slice(64, 0, *t)

    def mixture(seen):
        t = [new(4, 64), new(4, 96), new(4, 96)]
        seen += [weakref.ref(v) for v in t]
        return lf.make_mixture_projection(t[0], t[1], a_slice(seen), base=t[2])

    def gradient(seen):
        t = [new(4, 64), new(4, 96), new(4, 64), new(4, 64)]
        seen += [weakref.ref(v) for v in t]
        return lf.make_mixture_grad(t[0], t[1], t[2], a_slice(seen), dx_base=t[3])

    def w4_one(seen):
        t = [new(4, 64), new(4, 96), new(96, 32, dtype=torch.uint8), new(96, 2), new(96, 2, dtype=torch.uint8), new(96)]
        seen += [weakref.ref(v) for v in t]
        return lf.make_w4_projection(*t[:4], 32, zeros=t[4], bias=t[5])

    for make, kind in ((mixture, lf.lf_mixture_projection), (gradient, lf.lf_mixture_grad), (w4_one, lf.lf_w4_projection)):
        seen = []
        p = make(seen)
        assert all(r() is not None for r in seen), make
        arr = lf._array(kind, [p])
        del p
        assert all(r() is not None for r in seen), make
        del arr
        assert all(r() is None for r in seen), make


def test_arrays_made_once_are_taken_and_bare_ones_refused():
    """The entry points take what make_* returns, as a list, a tuple or an array made of it; an
    array of bare structures says neither rows nor device and is refused, as is an empty one."""
    b = torch.bfloat16
    x, y = torch.zeros(4, 64, dtype=b), torch.zeros(4, 96, dtype=b)
    pool = torch.zeros(1024, dtype=b)
    sl = lf.make_slice(64, 0, None, None, None, pool, pool)
    q, s = torch.zeros(96, 32, dtype=torch.uint8), torch.zeros(96, 2, dtype=b)
    made = {lf.lf_mixture_projection: lf.make_mixture_projection(x, y, sl), lf.lf_mixture_grad: lf.make_mixture_grad(x, y, None, sl),
            lf.lf_w4_projection: lf.make_w4_projection(x, y, q, s, 32)}
    for kind, p in made.items():
        for ok in ([p, p], (p, p), lf._array(kind, [p, p])):
            assert lf._rows_device(ok) == (4, x.device)
        other = type(p).from_buffer_copy(p)
        for bad in ([], (kind * 2)(p, p), [p, other], lf._array(kind, [other])):
            with pytest.raises(ValueError):
                lf._rows_device(bad)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    bare = {k: (k * 1)(p) for k, p in made.items()}
    for bad in (lambda: api.lora_mixture(ids, None, 4, bare[lf.lf_mixture_projection], 1.0),
                lambda: api.lora_mixture_backward(ids, None, 4, bare[lf.lf_mixture_grad], 1.0),
                lambda: api.w4_project(bare[lf.lf_w4_projection]), lambda: api.w4_project([]),
                lambda: api.lora_mixture(ids, None, 4, [], 1.0)):
        with pytest.raises(ValueError):
            bad()


def test_factor_tables_that_do_not_fit_are_refused():
    """The device reads entries 0 .. n_adapters of ranks and offsets whatever the ids name, as
    32- and 64-bit integers, and the pools as bf16 values side by side."""
    b = torch.bfloat16
    x, y = torch.zeros(4, 64, dtype=b), torch.zeros(4, 96, dtype=b)
    pool, ids = torch.zeros(2048, dtype=b), torch.zeros(4, 2, dtype=torch.int32)
    good = dict(ranks=torch.zeros(5, dtype=torch.int32), off_A=torch.zeros(6, dtype=torch.int64),
                off_Bt=torch.zeros(6, dtype=torch.int64)[:5], A_pool=pool, Bt_pool=pool.view(32, 64))
    both = (lambda sl: lf.make_mixture_projection(x, y, sl), lambda sl: lf.make_mixture_grad(x, y, None, sl))
    for make in both:
        make(lf.make_slice(64, 0, *good.values()))
        for bad in (dict(ranks=good["ranks"].long()), dict(off_A=good["off_A"].int()), dict(off_Bt=good["off_Bt"].int()),
                    dict(ranks=torch.zeros(10, dtype=torch.int32)[::2]), dict(off_A=torch.zeros(10, dtype=torch.int64)[::2]),
                    dict(A_pool=pool.float()), dict(Bt_pool=pool.half()), dict(A_pool=pool[::2])):
            with pytest.raises(ValueError):
                make(lf.make_slice(64, 0, *dict(good, **bad).values()))
    for short in (dict(), dict(ranks=good["ranks"][:3]), dict(off_A=good["off_A"][:3]), dict(off_Bt=good["off_Bt"][:3])):
        sl = lf.make_slice(64, 0, *dict(good, **short).values())
        n = 6 if not short else 4
        p, g = lf.make_mixture_projection(x, y, sl), lf.make_mixture_grad(x, y, None, sl)
        for call in (lambda: lf.lf_lora_mixture(ids, None, n, [p], 1.0, stream=0),
                     lambda: lf.lf_lora_mixture_backward(ids, None, n, [g], 1.0, stream=0),
                     lambda: lf.lf_lora_mixture(ids, None, n, lf._array(lf.lf_mixture_projection, [p]), 1.0, stream=0)):
            with pytest.raises(ValueError, match="adapters"):
                call()


def test_the_row_stride_of_a_single_row_does_not_matter():
    b = torch.bfloat16
    pool = torch.zeros(1024, dtype=b)
    sl = lf.make_slice(64, 0, None, None, None, pool, pool)
    odd, wide = torch.zeros(3, 201, dtype=b), torch.zeros(3, 200, dtype=b)
    x, y = odd[:1, :64], wide[1:2, :96]
    p = lf.make_mixture_projection(x, y, sl, base=torch.zeros(1, 96, dtype=b))
    assert p.x_ld % 8 == 0 and p.x_ld >= 64 and p.y_ld % 8 == 0 and p.y_ld >= 96
    g = lf.make_mixture_grad(x, y, wide[2:, :64], sl, dx_base=odd[:1, :64])
    assert g.x_ld % 8 == g.dy_ld % 8 == g.dx_ld % 8 == 0
    q, s = torch.zeros(96, 32, dtype=torch.uint8), torch.zeros(96, 2, dtype=b)
    w = lf.make_w4_projection(x, odd[2:, :97], q, s, 32)
    assert w.x_ld % 8 == w.y_ld % 8 == 0 and w.x_ld >= 64 and w.y_ld >= 96
    for bad in (lambda: lf.make_mixture_projection(x, y, sl, base=torch.zeros(1, 88, dtype=b)),
                lambda: lf.make_mixture_projection(odd[:2, :64], wide[:2, :96], sl, base=torch.zeros(2, 96, dtype=b))):
        with pytest.raises(ValueError):
            bad()


def test_the_current_stream_without_torchs_own_calls(monkeypatch):
    class Stream:
        def __init__(self, index):
            self.cuda_stream = 1000 + index
    monkeypatch.setattr(lf, "_CUDA_NOW", [])
    for name in ("_cuda_getDevice", "_cuda_getCurrentRawStream"):
        monkeypatch.delattr(torch._C, name, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index=None: Stream(index))
    assert lf.current_device() == 3 and lf._stream(None) == 1003 and lf._stream(7) == 7


def test_arrays_of_other_structures_are_refused():
    """An array's bytes are read as the entry point's own structure."""
    made = {k: (k * 2)() for k in (lf.lf_projection, lf.lf_mixture_projection, lf.lf_mixture_grad, lf.lf_w4_projection)}
    ids = torch.zeros(4, 2, dtype=torch.int32)
    calls = {lf.lf_projection: lambda a: lf.lf_lora_shrink_expand_projections(4, ids, 4, a, 1.0, stream=0),
             lf.lf_mixture_projection: lambda a: lf.lf_lora_mixture(ids, None, 4, a, 1.0, stream=0),
             lf.lf_mixture_grad: lambda a: lf.lf_lora_mixture_backward(ids, None, 4, a, 1.0, stream=0),
             lf.lf_w4_projection: lambda a: lf.lf_w4_projections(4, a, stream=0)}
    for kind, call in calls.items():
        for other, arr in made.items():
            with pytest.raises(TypeError if other is not kind else lf.LFError):
                call(arr)
