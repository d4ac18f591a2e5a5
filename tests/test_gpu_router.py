"""GPU parity of lf_route_experts and its gradient against the float64 oracle on the same
logits.  Chosen ids must be equal; weights and gradients are held to the arithmetic's bound:
expf is within 2 ulp (2^-22), its argument l - m is rounded once (|l - m| 2^-24 relative in
the result), a sum of E terms over 32 lanes adds E / 32 + 8 roundings, and numerator and
denominator each carry that."""
import numpy as np
import pytest
import torch

from oracle import routed as R
from post_hoc_rank_b200 import api, build
from post_hoc_rank_b200 import loraforge as lf

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}   # half a step, relative


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    assert torch.cuda.is_available()


def bound(l, E):
    spread = float(np.nanmax(np.where(np.isfinite(l), np.abs(l), 0.0), initial=0.0)) * 2
    return 2 * (2.0 ** -22 + min(spread, 104.0) * 2.0 ** -24 + (E / 32 + 8) * 2.0 ** -24) + 4 * 2.0 ** -24


def run(l, K, dtype="f32", bias=None, counts=False, gw=None, scale=1.0, **kw):
    """(ids, weights, grad, counts) on the GPU, and the logits as float64."""
    ld = torch.from_numpy(l).to(DT[dtype]).cuda()
    r = lf.make_router(l.shape[1], K, weight_scale=scale, **kw)
    b = None if bias is None else torch.from_numpy(bias.astype(np.float32)).cuda()
    cnt = torch.full((l.shape[1],), 77, dtype=torch.int32, device="cuda") if counts else None
    ids, w = api.route_experts(ld, r, bias=b, counts=cnt)
    grad = None
    if gw is not None:
        grad = api.route_experts_backward(ld, r, ids, torch.from_numpy(gw).cuda())
    assert lf.lf_get_device_status() == 0
    return (ids.cpu().numpy(), w.cpu().numpy(), None if grad is None else grad.double().cpu().numpy(),
            None if cnt is None else cnt.cpu().numpy(), ld.double().cpu().numpy())


CASES = [
    # T, E, K, groups, top_groups, group_top
    (1, 1, 1, 1, 1, 1), (1, 8, 2, 1, 1, 1), (37, 17, 6, 1, 1, 1), (9, 33, 8, 1, 1, 1), (70, 64, 3, 4, 2, 2),
    (65, 256, 8, 8, 4, 2), (33, 96, 5, 3, 2, 1), (20, 130, 4, 13, 5, 2), (12, 1000, 16, 1, 1, 1),
    (11, 512, 7, 32, 3, 2), (8, 1024, 2, 4, 1, 1), (5, 40, 16, 8, 2, 2), (300, 5, 5, 5, 2, 2),
]


@pytest.mark.parametrize("T,E,K,G,tg,gt", CASES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_route_and_gradient(T, E, K, G, tg, gt, score, with_bias):
    g = np.random.default_rng(T * 1000 + E + K)
    l = (2 * g.normal(size=(T, E))).astype(np.float32)
    l[g.random((T, E)) < 0.1] = -np.inf
    if T > 2:
        l[T // 2] = -np.inf                      # nothing to route
        l[T - 1] = np.float32(-3.4028234e38)     # the type's lowest value shuts nothing out
    bias = (0.1 * g.normal(size=E)).astype(np.float32) if with_bias else None
    if with_bias and E > 4:
        bias[2] = -np.inf
    gw = g.normal(size=(T, K)).astype(np.float32)
    for renorm in (True, False):
        for dtype in ("f32", "bf16"):
            ls = l
            if dtype == "bf16" and T > 2:        # its own lowest value
                ls = l.copy()
                ls[T - 1] = torch.finfo(torch.bfloat16).min
            ids, w, grad, cnt, l64 = run(ls, K, dtype, bias, counts=True, gw=gw, scale=1.5, score=score, n_groups=G,
                                         top_groups=tg, group_top=gt, renorm=renorm)
            want = R.choose(l64, K, score, bias, G, tg, gt)
            assert (ids == want).all()
            assert (cnt == np.bincount(want[want >= 0], minlength=E)).all()
            wr = R.weights(l64, want, score, renorm, 1.5)
            tol = bound(np.where(np.abs(l64) > 1e30, 0, l64), E)
            assert (np.abs(w - wr) <= tol * np.abs(wr) + 1e-37).all()
            assert (w[want < 0] == 0).all()
            dr = R.route_grad(l64, want, gw, score, renorm, 1.5)
            # each entry is a few products of factors within tol; the subtracted mean is
            # bounded by the row's largest |gw|
            mag = 1.5 * (np.abs(gw).max(axis=1, keepdims=True) * np.maximum(R.scores(l64, score), 0))
            if renorm:
                mag = np.zeros_like(dr)
                rows = np.arange(T)[:, None].repeat(K, 1)
                np.add.at(mag, (rows[want >= 0], want[want >= 0]),
                          (np.abs(wr) * np.abs(gw).max(axis=1, keepdims=True) * 2)[want >= 0])
            assert (np.abs(grad - dr) <= (8 * tol) * mag + HALF[dtype] * np.abs(dr) + 1e-37).all()


def test_ties_go_to_the_lowest_index():
    l = np.zeros((40, 64), np.float32)
    l[1:, 1::2] = -0.0                            # equal to +0
    l[2, [60, 5, 33]] = 2.0
    for kw in (dict(), dict(bias=np.zeros(64)), dict(bias=np.full(64, 0.25), n_groups=8, top_groups=3, group_top=2)):
        for score in ("softmax", "sigmoid"):
            ids, *_ , l64 = run(l, 4, score=score, **kw)
            kw2 = dict(kw)
            b = kw2.pop("bias", None)
            assert (ids == R.choose(l64, 4, score, b, **kw2)).all()


def test_close_scores_are_settled_as_exact_arithmetic_does():
    """Scores whose order fp32 cannot tell: neighbouring logits, and biases that nearly make
    up for a difference of scores."""
    g = np.random.default_rng(9)
    T, E = 400, 48
    l = g.normal(size=(T, E)).astype(np.float32)
    l[:, 1::2] = np.nextafter(l[:, 0::2], np.float32(10))
    s = R.scores(l, "sigmoid")
    bias = (np.float32(0.7) - s[0]).astype(np.float32)     # row 0: all sums within one rounding
    for score in ("sigmoid", "softmax"):
        for kw in (dict(), dict(n_groups=4, top_groups=2, group_top=2)):
            ids, *_, l64 = run(l, 8, score=score, bias=bias, **kw)
            assert (ids == R.choose(l64, 8, score, bias, **kw)).all()
        tiny = np.zeros(E, np.float32)
        ids, *_, l64 = run(l, 8, score=score, bias=tiny)
        assert (ids == R.choose(l64, 8, score, tiny)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_logits(score):
    """Chosen scores that underflow keep their ratios; saturated sigmoids keep their order."""
    l = np.full((3, 6), -1e30, np.float32)
    l[0] = [-300, -301, -302, 0, 1, 2]
    l[1] = [40, 50, 60, 70, 30, -300]
    bias = np.array([9, 9, 0, 0, 0, 0], np.float32)
    ids, w, _, _, l64 = run(l[:1], 2, score=score, bias=bias)
    assert ids.tolist() == [[0, 1]]
    assert np.allclose(w, R.weights(l64, ids, score, True), rtol=2.0 ** -18)
    ids, w, _, _, l64 = run(l[1:2], 3, score=score)
    assert ids.tolist() == [[3, 2, 1]]


def test_strided_rows_half_types_and_empty_batch():
    g = np.random.default_rng(2)
    wide = torch.from_numpy(g.normal(size=(21, 50)).astype(np.float32)).cuda()
    r = lf.make_router(17, 3)
    for dt in DT.values():
        v = wide.to(dt)[:, 5:22]
        ids, w = api.route_experts(v, r)
        want = R.choose(v.double().cpu().numpy(), 3, "softmax")
        assert (ids.cpu().numpy() == want).all()
    ids, w = api.route_experts(wide[:0, :17], r)
    assert ids.shape == (0, 3) and w.shape == (0, 3)
    cnt = torch.full((17,), 5, dtype=torch.int32, device="cuda")
    api.route_experts(wide[:0, :17].contiguous(), r, counts=cnt)
    assert (cnt == 0).all() and lf.lf_get_device_status() == 0


def test_not_finite_rows_are_left_without_experts_and_latched():
    l = torch.randn(9, 20, device="cuda")
    l[3, 7] = float("nan")
    l[5, 0] = float("inf")
    r = lf.make_router(20, 4)
    ids, w = api.route_experts(l, r)
    assert lf.lf_get_device_status() == 5
    bad = torch.zeros(9, dtype=torch.bool, device="cuda")
    bad[[3, 5]] = True
    assert (ids[bad] == -1).all() and (w[bad] == 0).all() and (ids[~bad] >= 0).all()
    bias = torch.zeros(20, device="cuda")
    bias[1] = float("nan")
    ids, w = api.route_experts(torch.randn(3, 20, device="cuda"), r, bias=bias)
    assert lf.lf_get_device_status() == 5 and (ids == -1).all()


def test_backward_skips_bad_ids_and_adds_equal_ones():
    l = torch.randn(2, 10, device="cuda")
    r = lf.make_router(10, 3, renorm=False, score="sigmoid")
    ids = torch.tensor([[4, 4, 10], [-1, -2, 0]], dtype=torch.int32, device="cuda")
    gw = torch.ones(2, 3, device="cuda")
    d = api.route_experts_backward(l, r, ids, gw)
    assert lf.lf_get_device_status() == 3
    s = torch.sigmoid(l.double())
    want = torch.zeros(2, 10, dtype=torch.float64, device="cuda")
    want[0, 4] = 2 * s[0, 4] * (1 - s[0, 4])
    want[1, 0] = s[1, 0] * (1 - s[1, 0])
    assert (d.double() - want).abs().max() <= 2.0 ** -20


def test_captured_and_on_another_stream():
    T, E = 64, 32
    l = torch.randn(T, E, device="cuda")
    r = lf.make_router(E, 2)
    ids, w = torch.empty(T, 2, dtype=torch.int32, device="cuda"), torch.empty(T, 2, device="cuda")
    cnt = torch.zeros(E, dtype=torch.int32, device="cuda")
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        lf.lf_route_experts(l, r, None, ids, w, cnt)
    torch.cuda.current_stream().wait_stream(st)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        lf.lf_route_experts(l, r, None, ids, w, cnt)
    for seed in range(3):
        torch.manual_seed(seed)
        l.copy_(torch.randn(T, E, device="cuda"))
        gr.replay()
        torch.cuda.synchronize()
        want = R.choose(l.double().cpu().numpy(), 2, "softmax")
        assert (ids.cpu().numpy() == want).all()
        assert (cnt.cpu().numpy() == np.bincount(want.reshape(-1), minlength=E)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kw", [dict(renorm=False), dict(), dict(score="sigmoid", renorm=False), dict(score="sigmoid")])
def test_rows_without_slots_have_no_gradient(dtype, kw):
    l = np.random.default_rng(4).normal(size=(40, 70)).astype(np.float32)
    l[3, 5], l[7, 69], l[9] = np.nan, np.inf, -np.inf
    ld = torch.from_numpy(l).to(DT[dtype]).cuda()
    r = lf.make_router(70, 4, **kw)
    ids, w = api.route_experts(ld, r)
    assert lf.lf_get_device_status() == 5
    empty = (ids == -1).all(dim=1)
    assert empty.nonzero().flatten().tolist() == [3, 7, 9] and not w[empty].any()
    gw = torch.randn(40, 4, device="cuda")
    gw[3] = float("nan")                  # slots that name no expert are not read
    d = api.route_experts_backward(ld, r, ids, gw)
    assert torch.isfinite(d).all() and not d[empty].any() and d[~empty].any(dim=1).all()
    assert lf.lf_get_device_status() == 0


def place(E, at, logits, biases, low, rest):
    """A row of `low` logits (bias `rest`) with the given logits and biases at the experts `at`."""
    l, b = np.full((1, E), low, np.float32), np.full(E, rest, np.float32)
    l[0, at], b[at] = logits, biases
    return l, b


ONE = float(np.nextafter(np.float32(1), np.float32(2)))
CUT = [
    # an exact tie at the cut, and one expert a step above both that fp32 sums do not tell apart
    (place(96, [0, 33, 66], [1, 1, ONE], 0.25, -5, 0), 1, 66),
    (place(96, [0, 33, 66], [17, 17, 17.125], 0, -5, 0), 1, 66),
    (place(96, [0, 33, 66], [0, 0, 0.0078125], 1e5, -5, 0), 1, 66),
    (place(256, [3, 35, 67, 99], [1, 1, 1, ONE], 0.25, -5, 0), 2, 99),
    # an expert whose bias takes nearly all of its score away, behind two that are small to begin with
    (place(3, [0, 1, 2], [-17.8, -18.5, 1.1744667], [0, 0, -0.76395142], 0, 0), 1, 2),
    (place(64, [0, 1, 2], [-13.629779, -13.630779, 4.8179813e-6], [0, 0, -0.5], -30, 0), 1, 2),
]


@pytest.mark.parametrize("i", range(len(CUT)))
def test_the_last_choice_looks_past_the_first_one_left_out(i):
    (l, b), K, first = CUT[i]
    want = R.choose(l, K, "sigmoid", b)
    assert want[0, 0] == first
    ids, *_ = run(l, K, bias=b, score="sigmoid")
    assert (ids == want).all()
    for E in (128, 512, 1024):           # the same among more experts that are far below
        if l.shape[1] < E:
            wide, wb = np.full((1, E), -40, np.float32), np.full(E, -3, np.float32)
            wide[:, :l.shape[1]], wb[:l.shape[1]] = l, b
            ids, *_ = run(wide, K, bias=wb, score="sigmoid")
            assert (ids == R.choose(wide, K, "sigmoid", wb)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,tg", [(6, 1, 1), (64, 1, 1), (96, 3, 2), (250, 1, 1)])
def test_biases_of_mixed_size_choose_exactly(score, E, G, tg):
    """Biases that take away nearly all of a score, next to scores that are as small as what is
    left; then far larger ones, which leave only some bits of the score."""
    g = np.random.default_rng(E)
    T = 500
    l0 = (2 * g.normal(size=E)).astype(np.float32)
    small = g.random(E) < 0.5
    l0[small] -= 16
    if score == "softmax":               # all scores but the first one's are small
        l0[0] = 12
    l = (l0 * (1 + g.integers(-4, 5, size=(T, E)) * 2.0 ** -22)).astype(np.float32)
    near = np.where(small, 0, -R.scores(l0[None], score)[0]).astype(np.float32)
    if score == "softmax":
        near[0] = -np.inf
    large = (near + g.choice([0.0, 1.0, 1e5, -1e9], size=E)).astype(np.float32)
    for bias in (near, large):
        for K in (1, 2, 5):
            ids, *_ = run(l, K, bias=bias, score=score, n_groups=G, top_groups=tg, group_top=2 if G > 1 else 1)
            assert (ids == R.choose(l, K, score, bias, G, tg, 2 if G > 1 else 1)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G,tg", [(40, 1, 1), (256, 8, 3), (900, 1, 1)])
def test_ties_at_the_cut_with_biases(score, E, G, tg):
    """Logits on a coarse grid and few biases: equal inputs at the cut in most rows, some of
    them saturated, and sums that only nearly meet."""
    g = np.random.default_rng(E + 1)
    l = (np.round(g.normal(size=(300, E)) * 4) / 4).astype(np.float32)
    l[:40] += 16                          # sigmoids next to 1
    l[200:240] -= 30
    for bias in (np.zeros(E), 0.25 * (np.arange(E) % 2), g.choice([0.0, 0.1, 0.1 + 2.0 ** -26], size=E)):
        bias = bias.astype(np.float32)
        for K in (1, 3, 8):
            ids, *_ = run(l, K, bias=bias, score=score, n_groups=G, top_groups=tg, group_top=2 if G > 1 else 1)
            assert (ids == R.choose(l, K, score, bias, G, tg, 2 if G > 1 else 1)).all()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_scores_far_below_fp32_are_ordered(score):
    """With a bias of zero the scores decide, and fp64 holds them down to logits of -740; equal
    ones go to the lower index."""
    l = np.full((4, 40), -np.inf, np.float32)
    l[0, [1, 5, 33]] = [-100, -99, -101]
    l[1, [1, 5, 33]] = [-650, -649, -651]
    l[2, [1, 5, 33]] = [-700, -700, -690]
    l[3, [1, 5, 33]] = [-720, -719, -717]
    if score == "softmax":
        l[:, 0] = 0
    b = np.zeros(40, np.float32)
    b[0] = -np.inf
    ids, *_ = run(l, 3, bias=b, score=score)
    assert (ids == R.choose(l, 3, score, b)).all()
    assert ids[:, 0].tolist() == [5, 5, 33, 33]
