"""GPU parity of the routed side path and its gradients against the float64 oracle on the
same bf16 bytes.  Bounds: a sum of n fp32 products in any order is within n 2^-24 of the sum
of their absolute values, taken over the two chained sums (d + R terms, and the scaling);
outputs are rounded once to bf16 (2^-8 relative)."""
import numpy as np
import pytest
import torch

from oracle import routed as OR
from post_hoc_rank_b200 import api, build
from post_hoc_rank_b200 import loraforge as lf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    assert torch.cuda.is_available()


def bf(g, *shape, std=1.0):
    return torch.from_numpy((std * g.normal(size=shape)).astype(np.float32)).bfloat16()


class Batch:
    """One projection's data: pools with the adapters in shuffled places (gaps between them)."""

    def __init__(self, T, E, K, d_in, d_out, max_rank, seed, empty=0.1, ranks=None, pad=0):
        g = np.random.default_rng(seed)
        self.T, self.E, self.K, self.d_in, self.d_out = T, E, K, d_in, d_out
        self.ranks = np.asarray(ranks if ranks is not None else g.integers(0, max_rank + 1, size=E), dtype=np.int32)
        order = g.permutation(E)
        self.offA, self.offB = np.zeros(E, np.int64), np.zeros(E, np.int64)
        a = b = 8
        for e in order:
            self.offA[e], self.offB[e] = a, b
            a += int(self.ranks[e]) * d_in + 8
            b += int(self.ranks[e]) * d_out + 16
        self.A, self.Bt = bf(g, a, std=d_in ** -0.5), bf(g, b, std=0.25)
        self.ids = np.stack([g.permutation(E)[:K] if E >= K else g.integers(0, E, K) for _ in range(T)]).astype(np.int32) \
            if T else np.zeros((0, K), np.int32)
        self.ids[g.random((T, K)) < empty] = -1
        if T > 3:
            self.ids[T // 2] = -1
            self.ids[1] = self.ids[1, 0]          # one adapter in every slot
        self.w = g.normal(size=(T, K)).astype(np.float32)
        self.x, self.base, self.dy = bf(g, T, d_in + pad), bf(g, T, d_out + pad), bf(g, T, d_out + pad)
        self.dxb = bf(g, T, d_in + pad)

    def dev(self):
        c = lambda v: torch.from_numpy(v).cuda() if isinstance(v, np.ndarray) else v.cuda()  # noqa: E731
        return {k: c(getattr(self, k)) for k in ("ranks", "offA", "offB", "A", "Bt", "ids", "w", "x", "base", "dy", "dxb")}

    def slice(self, D, y_off=0, max_rank=0):
        return lf.make_slice(self.d_out, y_off, D["ranks"], D["offA"], D["offB"], D["A"], D["Bt"], max_rank)

    def pools(self):
        return (self.ranks, self.offA, self.offB, self.A.float().numpy(), self.Bt.float().numpy())

    @property
    def R(self):
        return self.K * int(self.ranks.max(initial=0))


def check(got, want, mag, n, half=2.0 ** -8):
    got = got.double().cpu().numpy() if torch.is_tensor(got) else got
    tol = half * np.abs(want) + (1 + half) * n * 2.0 ** -24 * mag + 1e-37
    assert (np.abs(got - want) <= tol).all(), np.max((np.abs(got - want) - tol))
    # the rounding alone over the whole output (bounds on sums are far above what they lose)
    norm = np.linalg.norm(want)
    assert np.linalg.norm(got - want) <= (half + 2.0 ** -14) * norm + 1e-30


SHAPES = [
    # T, E, K, d_in, d_out, max_rank
    (1, 1, 1, 8, 8, 1), (1, 17, 6, 3584, 512, 16), (2, 3, 2, 136, 1032, 64), (5, 4, 3, 1032, 8, 20),
    (37, 8, 2, 520, 264, 33), (64, 16, 2, 512, 1024, 16), (150, 40, 4, 256, 248, 9), (333, 5, 2, 264, 520, 64),
    (700, 12, 2, 1024, 384, 16), (1025, 9, 3, 200, 136, 7), (40, 2, 16, 64, 64, 64), (600, 64, 2, 320, 512, 16),
    (300, 3, 1, 4096, 128, 8),
    # long batches over small pools (dense products over the stacked rows: up to 256, 512, 768, 1024)
    (1111, 16, 6, 1544, 2056, 16), (700, 12, 2, 2048, 1992, 64), (2000, 16, 4, 1032, 1304, 64), (300, 3, 16, 4096, 1024, 64),
    (513, 130, 8, 4096, 2048, 7), (640, 8, 3, 5000, 40, 32), (257, 4, 8, 64, 6008, 64),
]


@pytest.mark.parametrize("T,E,K,d_in,d_out,mr", SHAPES)
def test_forward_and_backward(T, E, K, d_in, d_out, mr):
    for bounded in (False, True):
        b = Batch(T, E, K, d_in, d_out, mr, seed=T + 7 * E + d_in)
        D = b.dev()
        sl = b.slice(D, max_rank=mr if bounded else 0)
        for w in (D["w"], None):
            wn = b.w if w is not None else None
            y = torch.empty_like(D["base"])
            api.lora_mixture(D["ids"], w, E, [lf.make_mixture_projection(D["x"], y, sl, base=D["base"])], 0.75)
            want, mag = OR.mixture(b.x.float().numpy(), b.base.float().numpy(), b.ids, wn, *b.pools(), 0.75)
            check(y, want, mag, d_in + b.R + 8)
            dx = torch.empty_like(D["x"])
            gw = api.lora_mixture_backward(D["ids"], w, E, [lf.make_mixture_grad(D["x"], D["dy"], dx, sl)], 0.75)
            dxr, dxm, dwr, dwm = OR.mixture_grad(b.x.float().numpy(), b.dy.float().numpy(), b.ids, wn, *b.pools(), 0.75)
            check(dx, dxr, dxm, d_out + b.R + 8)
            gwn = gw.double().cpu().numpy()
            assert (np.abs(gwn - dwr) <= (d_in + d_out + mr + 8) * 2.0 ** -24 * dwm + 1e-37).all()
            assert (gwn[b.ids < 0] == 0).all()
        assert lf.lf_get_device_status() == 0


# token by token, and long enough over a small pool for the dense products
@pytest.mark.parametrize("T,K,d_in,d_out,mr", [(3, 2, 264, 392, 24), (260, 2, 264, 392, 24), (260, 8, 1288, 1544, 64)])
def test_strides_offsets_scales_in_place(T, K, d_in, d_out, mr):
    """x, y and dx as column windows of wider tensors, a slice inside y, per-adapter scales, y
    and dx updated in place; everything outside the window keeps its bits."""
    b = Batch(T, 6, K, d_in, d_out, mr, seed=5, pad=40)
    D = b.dev()
    sc = np.array([0.5, 2.0, -1.0, 0.0, 3.0, 1.5], np.float32)
    scd = torch.from_numpy(sc).cuda()
    x = D["x"][:, 16:16 + d_in]
    y = D["base"].clone()
    sl = b.slice(D, y_off=24)
    api.lora_mixture(D["ids"], D["w"], 6, [lf.make_mixture_projection(x, y, sl, base=y)], 9.0, adapter_scale=scd)
    xn = b.x.float().numpy()[:, 16:16 + d_in]
    bn = b.base.float().numpy()
    want, mag = OR.mixture(xn, bn[:, 24:24 + d_out], b.ids, b.w, *b.pools(), 9.0, sc)
    check(y[:, 24:24 + d_out], want, mag, d_in + b.R + 8)
    assert torch.equal(y[:, :24], D["base"][:, :24]) and torch.equal(y[:, 24 + d_out:], D["base"][:, 24 + d_out:])
    idle = torch.from_numpy((b.ids < 0).all(axis=1)).cuda()
    assert torch.equal(y[idle], D["base"][idle])
    dx_all = D["dxb"].clone()
    dx = dx_all[:, 8:8 + d_in]
    gw = api.lora_mixture_backward(D["ids"], D["w"], 6, [lf.make_mixture_grad(x, D["dy"], dx, sl, dx_base=dx)], 9.0,
                                   adapter_scale=scd)
    dxr, dxm, dwr, dwm = OR.mixture_grad(xn, b.dy.float().numpy()[:, 24:24 + d_out], b.ids, b.w, *b.pools(), 9.0, sc)
    base = b.dxb.float().numpy()[:, 8:8 + d_in].astype(np.float64)
    check(dx, dxr + base, dxm + np.abs(base), d_out + b.R + 8)
    assert torch.equal(dx_all[:, :8], D["dxb"][:, :8]) and torch.equal(dx_all[:, 8 + d_in:], D["dxb"][:, 8 + d_in:])
    assert (np.abs(gw.double().cpu().numpy() - dwr) <= (d_in + d_out + mr + 8) * 2.0 ** -24 * dwm + 1e-37).all()
    assert lf.lf_get_device_status() == 0


@pytest.mark.parametrize("T,big", [(2, False), (300, False), (700, True)])
def test_several_projections_share_the_weights_gradient(T, big):
    """big: the second projection is wide enough for the dense products, the others are not."""
    d1, d2, r = (2048, 2056, 64) if big else (256, 520, 5)
    bs = [Batch(T, 7, 2, 128, 64, 16, seed=1), Batch(T, 7, 2, d1, d2, r, seed=2), Batch(T, 7, 2, 8, 128, 8, seed=3)]
    Ds = [b.dev() for b in bs]
    for b in bs:
        b.ids, b.w = bs[0].ids, bs[0].w
    ids, w = Ds[0]["ids"], Ds[0]["w"]
    ys = [torch.empty_like(D["base"]) for D in Ds]
    api.lora_mixture(ids, w, 7, [lf.make_mixture_projection(D["x"], y, b.slice(D)) for b, D, y in zip(bs, Ds, ys)], 1.0)
    dxs = [torch.empty_like(Ds[0]["x"]), None, torch.empty_like(Ds[2]["x"])]
    gw = api.lora_mixture_backward(ids, w, 7, [lf.make_mixture_grad(D["x"], D["dy"], dx, b.slice(D))
                                               for b, D, dx in zip(bs, Ds, dxs)], 1.0)
    tot, totm = 0.0, 0.0
    for b, y, dx in zip(bs, ys, dxs):
        xn = b.x.float().numpy()
        want, mag = OR.mixture(xn, np.zeros((T, b.d_out)), b.ids, b.w, *b.pools(), 1.0)
        check(y, want, mag, b.d_in + b.R + 8)
        dxr, dxm, dwr, dwm = OR.mixture_grad(xn, b.dy.float().numpy(), b.ids, b.w, *b.pools(), 1.0)
        if dx is not None:
            check(dx, dxr, dxm, b.d_out + b.R + 8)
        tot, totm = tot + dwr, totm + dwm
    assert (np.abs(gw.double().cpu().numpy() - tot) <= (d1 + d2 + r + 32) * 2.0 ** -24 * totm + 1e-37).all()
    # the weights' gradient alone, and dx alone
    g2 = api.lora_mixture_backward(ids, w, 7, [lf.make_mixture_grad(D["x"], D["dy"], None, b.slice(D))
                                               for b, D in zip(bs, Ds)], 1.0)
    assert torch.equal(gw, g2)
    dx0 = torch.empty_like(dxs[0])
    assert api.lora_mixture_backward(ids, w, 7, [lf.make_mixture_grad(Ds[0]["x"], Ds[0]["dy"], dx0, bs[0].slice(Ds[0]))],
                                     1.0, grad_weights=False) is None
    assert torch.equal(dx0, dxs[0])
    assert lf.lf_get_device_status() == 0


@pytest.mark.parametrize("T,d_in,d_out", [(4, 64, 128), (400, 64, 128), (900, 2048, 1096)])
def test_bad_ids_and_factors_leave_only_their_slots_out(T, d_in, d_out):
    b = Batch(T, 6, 3, d_in, d_out, 12, seed=8, empty=0.0, ranks=[4, 70, 3, 5, 6, 7])
    b.ids = np.tile(np.array([0, 2, 3], np.int32), (T, 1))
    b.ids[0] = [0, 6, 3]                # out of range
    ref = b.ids.copy()
    ref[0, 1] = -1
    D = b.dev()

    def y_of(D):
        y = torch.empty_like(D["base"])
        api.lora_mixture(D["ids"], D["w"], 6, [lf.make_mixture_projection(D["x"], y, b.slice(D), base=D["base"])], 1.0)
        return y
    y = y_of(D)
    assert lf.lf_get_device_status() == 3
    xn, bn = b.x.float().numpy(), b.base.float().numpy()
    want, mag = OR.mixture(xn, bn, ref, b.w, *b.pools(), 1.0)
    check(y, want, mag, d_in + 64 + 8)
    gw = api.lora_mixture_backward(D["ids"], D["w"], 6, [lf.make_mixture_grad(D["x"], D["dy"], None, b.slice(D))], 1.0)
    assert lf.lf_get_device_status() == 3 and float(gw[0, 1]) == 0.0
    # a rank above 64 (adapter 1) and an offset past the pool (adapter 2)
    b.ids = np.tile(np.array([0, 1, 3], np.int32), (T, 1))
    D = b.dev()
    y = y_of(D)
    assert lf.lf_get_device_status() == 2
    ref = b.ids.copy()
    ref[:, 1] = -1
    want, mag = OR.mixture(xn, bn, ref, b.w, *b.pools(), 1.0)
    check(y, want, mag, d_in + 64 + 8)
    b.ids = np.tile(np.array([0, 2, 3], np.int32), (T, 1))
    keep = b.offA[2]
    b.offA[2] = b.A.numel() - d_in
    D = b.dev()
    y = y_of(D)
    assert lf.lf_get_device_status() == 4
    b.offA[2] = keep
    ref = b.ids.copy()
    ref[:, 1] = -1
    want, mag = OR.mixture(xn, bn, ref, b.w, *b.pools(), 1.0)
    check(y, want, mag, d_in + 64 + 8)


@pytest.mark.parametrize("T,K,d_in,d_out", [(260, 2, 64, 64), (800, 4, 2048, 1544)])
def test_values_that_are_not_finite_stay_in_their_tokens(T, K, d_in, d_out):
    """An infinite weight of an empty slot is not read; NaN in one token's x stays there; factors
    that are not finite reach only the tokens that use them."""
    b = Batch(T, 8, K, d_in, d_out, 64, seed=4, ranks=[64, 8, 8, 64, 64, 8, 8, 8])
    b.ids[b.ids == 7] = -1               # adapter 7 is used by no token
    b.ids[(b.ids == 6) & (np.arange(T)[:, None] % 50 != 0)] = 5
    b.w[b.ids < 0] = np.inf
    b.A[b.offA[7]:b.offA[7] + 100] = float("nan")
    b.Bt[b.offB[7] + 3] = float("inf")
    b.Bt[b.offB[6] + d_out + 5] = float("nan")
    D = b.dev()
    D["x"][7] = float("nan")
    y, dx = torch.empty_like(D["base"]), torch.empty_like(D["x"])
    sl = b.slice(D)
    api.lora_mixture(D["ids"], D["w"], 8, [lf.make_mixture_projection(D["x"], y, sl, base=D["base"])], 1.0)
    gw = api.lora_mixture_backward(D["ids"], D["w"], 8, [lf.make_mixture_grad(D["x"], D["dy"], dx, sl)], 1.0)
    uses6 = torch.from_numpy((b.ids == 6).any(axis=1)).cuda()
    clean = ~uses6
    clean[7] = False
    assert torch.isfinite(y[clean]).all() and torch.isfinite(dx[clean]).all() and torch.isfinite(gw[clean]).all()
    assert torch.isnan(y[uses6]).any(dim=1).all() and torch.isnan(dx[uses6]).any(dim=1).all()
    assert torch.isnan(gw[torch.from_numpy(b.ids == 6).cuda()]).all()
    assert not torch.isfinite(y[7]).all() or (b.ids[7] < 0).all()
    assert lf.lf_get_device_status() == 0


@pytest.mark.parametrize("T", [4, 900])
@pytest.mark.parametrize("side", ["offA", "offB"])
def test_offsets_whose_end_passes_63_bits_are_refused(T, side):
    b = Batch(T, 6, 3, 2048, 1096, 12, seed=9, empty=0.0, ranks=[4, 2, 3, 5, 6, 7])
    b.ids[0] = [5, 2, 0]
    keep = getattr(b, side)[2]
    getattr(b, side)[2] = (1 << 63) - 8
    D = b.dev()
    y, dx = torch.empty_like(D["base"]), torch.empty_like(D["x"])
    api.lora_mixture(D["ids"], D["w"], 6, [lf.make_mixture_projection(D["x"], y, b.slice(D), base=D["base"])], 1.0)
    assert lf.lf_get_device_status() == 4
    gw = api.lora_mixture_backward(D["ids"], D["w"], 6, [lf.make_mixture_grad(D["x"], D["dy"], dx, b.slice(D))], 1.0)
    assert lf.lf_get_device_status() == 4 and not gw[D["ids"] == 2].any()
    getattr(b, side)[2] = keep
    ref = np.where(b.ids == 2, -1, b.ids)
    want, mag = OR.mixture(b.x.float().numpy(), b.base.float().numpy(), ref, b.w, *b.pools(), 1.0)
    check(y, want, mag, 2048 + 64 + 8)


@pytest.mark.parametrize("K,d_in,d_out", [(2, 512, 512), (4, 2048, 2048)])
def test_same_results_from_run_to_run_and_captured(K, d_in, d_out):
    b = Batch(512, 16, K, d_in, d_out, 64, seed=6)
    D = b.dev()
    sl = b.slice(D)
    y, dx = torch.empty_like(D["base"]), torch.empty_like(D["x"])
    gw = torch.empty(512, K, device="cuda")
    ws = api.workspace(max(lf.lf_lora_mixture_workspace_size(512, K, 16, [lf.make_mixture_projection(D["x"], y, sl, base=D["base"])]),
                           lf.lf_lora_mixture_backward_workspace_size(512, K, 16, [lf.make_mixture_grad(D["x"], D["dy"], dx, sl)])),
                       "cuda")

    def call():
        lf.lf_lora_mixture(D["ids"], D["w"], 16, [lf.make_mixture_projection(D["x"], y, sl, base=D["base"])], 1.0, ws)
        lf.lf_lora_mixture_backward(D["ids"], D["w"], 16, [lf.make_mixture_grad(D["x"], D["dy"], dx, sl)], 1.0, gw, ws)
    call()
    first = [t.clone() for t in (y, dx, gw)]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        for t in (y, dx, gw):
            t.zero_()
        call()
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(a, c) for a, c in zip(first, (y, dx, gw)))
    # the workspace of a call on a named stream belongs to that stream
    st.wait_stream(torch.cuda.current_stream())
    for t in (y, dx):
        t.zero_()
    st.wait_stream(torch.cuda.current_stream())
    api.lora_mixture(D["ids"], D["w"], 16, [lf.make_mixture_projection(D["x"], y, sl, base=D["base"])], 1.0, stream=st)
    g2 = api.lora_mixture_backward(D["ids"], D["w"], 16, [lf.make_mixture_grad(D["x"], D["dy"], dx, sl)], 1.0,
                                   stream=st.cuda_stream)
    junk = [torch.full((1 << 22,), 7.0, device="cuda") for _ in range(4)]
    torch.cuda.current_stream().wait_stream(st)
    assert all(torch.equal(a, c) for a, c in zip(first, (y, dx, g2))) and len(junk) == 4
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        call()
    for t in (y, dx, gw):
        t.zero_()
    gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, c) for a, c in zip(first, (y, dx, gw)))
    # new ids through the same graph
    b2 = Batch(512, 16, K, d_in, d_out, 64, seed=60)
    D["ids"].copy_(torch.from_numpy(b2.ids))
    gr.replay()
    want, mag = OR.mixture(b.x.float().numpy(), b.base.float().numpy(), b2.ids, b.w, *b.pools(), 1.0)
    check(y, want, mag, d_in + b.R + 8)
    assert lf.lf_get_device_status() == 0


def test_empty_batch_and_module_of_zero_ranks():
    b = Batch(0, 3, 2, 64, 64, 4, seed=1)
    D = b.dev()
    y = torch.empty_like(D["base"])
    api.lora_mixture(D["ids"], D["w"], 3, [lf.make_mixture_projection(D["x"], y, b.slice(D))], 1.0)
    for T, d in ((3, 64), (300, 64), (1500, 2048)):
        b = Batch(T, 3, 8, d, d, 4, seed=1, ranks=[0, 0, 0])
        D = b.dev()
        y = torch.empty_like(D["base"])
        api.lora_mixture(D["ids"], D["w"], 3, [lf.make_mixture_projection(D["x"], y, b.slice(D), base=D["base"])], 1.0)
        assert torch.equal(y, D["base"])
        y.fill_(3.0)
        api.lora_mixture(D["ids"], D["w"], 3, [lf.make_mixture_projection(D["x"], y, b.slice(D))], 1.0)
        assert (y == 0).all()
    assert lf.lf_get_device_status() == 0


@pytest.mark.parametrize("T", [3, 700])
def test_descriptions_of_temporaries(T):
    """Inputs cast and tables made where the call describes them: their memory is not handed out
    again (to the next one, to the workspace, to the gradient) before the call has read it."""
    b = Batch(T, 8, 2, 2048, 1032, 32, seed=12)
    D = b.dev()
    n = 5
    xs = [torch.randn(T, 2048, device="cuda") for _ in range(n)]
    wide = {k: D[k].double() for k in ("ranks", "offA", "offB")}

    def sl():
        return lf.make_slice(1032, 0, wide["ranks"].int(), wide["offA"].long(), wide["offB"].long(), D["A"].clone(),
                             D["Bt"].clone(), 32)
    held = [(x.bfloat16(), torch.empty_like(D["base"])) for x in xs]
    api.lora_mixture(D["ids"], D["w"], 8, [lf.make_mixture_projection(x, y, b.slice(D, max_rank=32), base=D["base"])
                                           for x, y in held], 1.0)
    ys = [torch.empty_like(D["base"]) for _ in range(n)]
    api.lora_mixture(D["ids"], D["w"], 8, [lf.make_mixture_projection(x.bfloat16(), y, sl(), base=D["base"].clone())
                                           for x, y in zip(xs, ys)], 1.0)
    assert all(torch.equal(y, h[1]) for y, h in zip(ys, held))
    dxs = [torch.empty_like(h[0]) for h in held]
    gw = api.lora_mixture_backward(D["ids"], D["w"], 8, [lf.make_mixture_grad(h[0], D["dy"], dx, b.slice(D, max_rank=32))
                                                         for h, dx in zip(held, dxs)], 1.0)
    dx2 = [torch.empty_like(h[0]) for h in held]
    g2 = api.lora_mixture_backward(D["ids"], D["w"], 8, [lf.make_mixture_grad(x.bfloat16(), D["dy"].clone(), dx, sl())
                                                         for x, dx in zip(xs, dx2)], 1.0)
    assert torch.equal(gw, g2) and all(torch.equal(a, c) for a, c in zip(dxs, dx2))
    assert lf.lf_get_device_status() == 0


def test_arrays_made_once_and_refused_tables():
    b = Batch(5, 4, 2, 64, 64, 8, seed=3)
    D = b.dev()
    y, y2 = torch.empty_like(D["base"]), torch.empty_like(D["base"])
    sl = b.slice(D)
    arr = lf._array(lf.lf_mixture_projection, [lf.make_mixture_projection(D["x"], y, sl, base=D["base"])])
    api.lora_mixture(D["ids"], D["w"], 4, arr, 1.0)
    api.lora_mixture(D["ids"], D["w"], 4, [lf.make_mixture_projection(D["x"], y2, sl, base=D["base"])], 1.0)
    assert torch.equal(y, y2)
    for call in (lambda: api.lora_mixture(D["ids"], D["w"], 5, arr, 1.0),
                 lambda: api.lora_mixture_backward(D["ids"], D["w"], 5, [lf.make_mixture_grad(D["x"], D["dy"], None, sl)], 1.0)):
        with pytest.raises(ValueError, match="adapters"):
            call()
    assert lf.lf_get_device_status() == 0


@pytest.mark.parametrize("T", [3, 700])
def test_projections_of_which_nothing_is_wanted_launch_nothing(T):
    bs = [Batch(T, 8, 4, 2048, 2056, 64, seed=s) for s in (1, 2)]
    Ds = [b.dev() for b in bs]
    ids, w = Ds[0]["ids"], Ds[0]["w"]

    def grads(dxs, ps):
        n = lf.lf_launch_count()
        api.lora_mixture_backward(ids, w, 8, [lf.make_mixture_grad(Ds[p]["x"], Ds[p]["dy"], dx, bs[p].slice(Ds[p]))
                                              for p, dx in zip(ps, dxs)], 1.0, grad_weights=False)
        return lf.lf_launch_count() - n
    one, two = torch.empty_like(Ds[1]["x"]), torch.empty_like(Ds[1]["x"])
    alone = grads([one], [1])
    assert grads([None, two], [0, 1]) == alone and torch.equal(one, two)
    assert grads([two, None], [1, 0]) == alone and torch.equal(one, two)
    assert grads([None, None], [0, 1]) == 0
    assert lf.lf_get_device_status() == 0


def test_one_row_of_a_tensor_of_odd_width():
    b = Batch(1, 4, 2, 64, 96, 8, seed=2, empty=0.0)
    D = b.dev()
    odd = torch.zeros(3, 201, dtype=torch.bfloat16, device="cuda")
    odd[0, :64] = D["x"][0]
    wide = torch.zeros(3, 208, dtype=torch.bfloat16, device="cuda")
    y, want = wide[1:2, :96], torch.empty_like(D["base"])
    api.lora_mixture(D["ids"], D["w"], 4, [lf.make_mixture_projection(odd[:1, :64], y, b.slice(D), base=D["base"])], 1.0)
    api.lora_mixture(D["ids"], D["w"], 4, [lf.make_mixture_projection(D["x"], want, b.slice(D), base=D["base"])], 1.0)
    assert torch.equal(y, want) and not wide[0].any() and not wide[2].any() and not wide[1, 96:].any()
    assert lf.lf_get_device_status() == 0
