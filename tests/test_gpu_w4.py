"""GPU parity of the 4-bit base weights against the float64 oracle: quantisation (codes,
scales and zero points equal), its inverse, and the products.  Product bounds: a sum of n
fp32 products in any order is within n 2^-24 of the sum of absolute values, and a group may
be formed as s (sum (128 + q) x - (128 + z) sum x), whose terms' absolute values are
s (256 + q + z) |x|; the output is rounded once to bf16 (2^-8 relative).  The norm of the
error over a whole output is held to the rounding alone."""
import numpy as np
import pytest
import torch

from oracle import routed as OR
from post_hoc_rank_b200 import api, build
from post_hoc_rank_b200 import loraforge as lf

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    assert torch.cuda.is_available()


@pytest.mark.parametrize("group", [32, 64, 128, 256])
@pytest.mark.parametrize("zp", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_quantize_and_back(group, zp, dtype):
    for d_out, d_in in ((8, 32), (24, 96), (16, 3584), (72, 288)):
        g = np.random.default_rng(group + d_in)
        W = torch.from_numpy(g.normal(size=(d_out, d_in)).astype(np.float32) * 0.02).to(DT[dtype]).cuda()
        W[1] = 0
        W[2] = W[2].abs()                         # one-sided
        W[3, :4] = torch.tensor([7.0, 3.5, -2.5, 0.5]) * 4       # halves of a power-of-two scale
        W[3, 4:] = 0
        w4 = api.w4_quantize(W, group, zero_points=zp)
        assert lf.lf_get_device_status() == 0
        c, s, z = OR.w4_quantize(W.double().cpu().numpy(), group, zp)
        assert (w4.scales.double().cpu().numpy() == s).all()
        assert (OR.w4_unpack(w4.q.cpu().numpy()) == c).all()
        if zp:
            assert (w4.zeros.cpu().numpy() == z).all()
        M = OR.w4_matrix(w4.q.cpu().numpy(), s, w4.zeros.cpu().numpy() if zp else None, group)
        assert (api.w4_dequantize(w4, torch.float32).double().cpu().numpy() == M).all()
        for dt, half in ((torch.bfloat16, 2.0 ** -8), (torch.float16, 2.0 ** -11)):
            back = api.w4_dequantize(w4, dt).double().cpu().numpy()
            assert (np.abs(back - M) <= half * np.abs(M) + 2.0 ** -25).all()


def test_quantize_extremes():
    """Huge, tiny and not finite weights: the last count as 0 and are latched."""
    W = torch.zeros(8, 64, device="cuda")
    W[0] = torch.from_numpy(np.linspace(-3e38, 3e38, 64).astype(np.float32))   # finite (fp32 linspace overflows)
    W[1] = torch.linspace(-1e-39, 1e-39, 64)
    W[2] = torch.linspace(1e-30, 2e-30, 64)
    for zp in (False, True):
        w4 = api.w4_quantize(W, 32, zero_points=zp)
        assert lf.lf_get_device_status() == 0
        c, s, z = OR.w4_quantize(W.double().cpu().numpy(), 32, zp)
        got = w4.scales.double().cpu().numpy()
        assert (got[[0, 2, 3]] == s[[0, 2, 3]]).all()
        q = OR.w4_unpack(w4.q.cpu().numpy())
        assert (q[[0, 2, 3]] == c[[0, 2, 3]]).all()
    W[4, 3] = float("nan")
    W[5, 40] = float("-inf")
    w4 = api.w4_quantize(W, 32)
    assert lf.lf_get_device_status() == 5
    W[4, 3] = W[5, 40] = 0
    assert torch.equal(w4.q, api.w4_quantize(W, 32).q)


def make(g, d_in, d_out, group, zp):
    ng = -(-d_in // group)
    q = torch.from_numpy(g.integers(0, 256, size=(d_out, d_in // 2), dtype=np.uint8)).cuda()
    s = torch.from_numpy((0.01 * (0.5 + g.random((d_out, ng)))).astype(np.float32)).bfloat16().cuda()
    z = torch.from_numpy(g.integers(0, 16, size=(d_out, ng), dtype=np.uint8)).cuda() if zp else None
    return api.W4(q, s, z, group)


def reference(x, w4, bias=None):
    M = OR.w4_matrix(w4.q.cpu().numpy(), w4.scales.double().cpu().numpy(),
                     None if w4.zeros is None else w4.zeros.cpu().numpy(), w4.group)
    xn = x.double().cpu().numpy()
    c, sc = OR.w4_unpack(w4.q.cpu().numpy()).astype(np.float64), w4.scales.double().cpu().numpy()
    at = np.arange(c.shape[1]) // w4.group
    z = 8.0 if w4.zeros is None else (w4.zeros.cpu().numpy() & 15).astype(np.float64)[:, at]
    y, mag = xn @ M.T, np.abs(xn) @ ((256 + c + z) * np.abs(sc)[:, at]).T
    if bias is not None:
        y, mag = y + bias.double().cpu().numpy(), mag + np.abs(bias.double().cpu().numpy())
    return y, mag


def check(y, want, mag, n):
    got = y.double().cpu().numpy()
    tol = 2.0 ** -8 * np.abs(want) + 1.01 * n * 2.0 ** -24 * mag
    assert (np.abs(got - want) <= tol).all(), np.max(np.abs(got - want) - tol)
    assert np.linalg.norm(got - want) <= (2.0 ** -8 + 2.0 ** -14) * np.linalg.norm(want) + 1e-30


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 16, 17, 33, 64, 100, 129, 257])
@pytest.mark.parametrize("d_in,d_out,group,zp", [(32, 8, 32, True), (96, 264, 64, False), (3584, 512, 128, True),
                                                 (1056, 136, 256, True), (4096, 1024, 64, False), (288, 1000, 32, True),
                                                 (18944, 56, 128, False)])
def test_products(T, d_in, d_out, group, zp):
    g = np.random.default_rng(T + d_in)
    w4 = make(g, d_in, d_out, group, zp)
    x = torch.from_numpy(g.normal(size=(T, d_in)).astype(np.float32)).cuda()
    x[:, ::16] *= 30
    x = x.bfloat16()
    bias = torch.from_numpy(g.normal(size=d_out).astype(np.float32)).bfloat16().cuda() if T % 2 else None
    y = api.w4_linear(x, w4, bias)
    check(y, *reference(x, w4, bias), d_in + 16)
    assert lf.lf_get_device_status() == 0


@pytest.mark.parametrize("T", [1, 5, 40, 200])
def test_several_projections_strided(T):
    """q, k, v sharing a strided x and a projection of its own, in one call; y as column windows
    whose surroundings keep their bits."""
    g = np.random.default_rng(T)
    wide = torch.from_numpy(g.normal(size=(T, 640)).astype(np.float32)).bfloat16().cuda()
    x, x2 = wide[:, 64:64 + 512], torch.from_numpy(g.normal(size=(T, 1184)).astype(np.float32)).bfloat16().cuda()
    ws = [make(g, 512, 512, 128, True), make(g, 512, 64, 64, False), make(g, 512, 64, 32, True), make(g, 1184, 264, 256, True)]
    xs = [x, x, x, x2]
    out = torch.full((T, 1000), 5.0, dtype=torch.bfloat16, device="cuda")
    ys = [out[:, 8:520], out[:, 528:592], out[:, 600:664], out[:, 672:936]]
    api.w4_project([lf.make_w4_projection(xi, yi, w.q, w.scales, w.group, w.zeros) for xi, yi, w in zip(xs, ys, ws)])
    for xi, yi, w in zip(xs, ys, ws):
        check(yi, *reference(xi, w), xi.shape[1] + 16)
    rest = torch.ones(1000, dtype=torch.bool, device="cuda")
    for a, b in ((8, 520), (528, 592), (600, 664), (672, 936)):
        rest[a:b] = False
    assert (out[:, rest] == 5.0).all()
    assert lf.lf_get_device_status() == 0


def test_high_bits_of_zero_points_are_ignored_and_rows_stay_apart():
    g = np.random.default_rng(1)
    w4 = make(g, 256, 64, 64, True)
    x = torch.from_numpy(g.normal(size=(20, 256)).astype(np.float32)).bfloat16().cuda()
    y = api.w4_linear(x, w4)
    w5 = api.W4(w4.q, w4.scales, w4.zeros | 0xA0, 64)
    assert torch.equal(api.w4_linear(x, w5), y)
    assert torch.equal(api.w4_dequantize(w5), api.w4_dequantize(w4))
    for T in (20, 200):
        x = torch.from_numpy(g.normal(size=(T, 256)).astype(np.float32)).bfloat16().cuda()
        y = api.w4_linear(x, w4)
        x2 = x.clone()
        x2[3] = float("nan")
        y2 = api.w4_linear(x2, w4)
        keep = torch.arange(T, device="cuda") != 3
        assert torch.equal(y2[keep], y[keep]) and torch.isnan(y2[3]).all()
    assert api.w4_linear(x[:0], w4).shape == (0, 64)


def test_captured_and_on_another_stream():
    g = np.random.default_rng(2)
    w4 = make(g, 1024, 256, 128, True)
    for T in (1, 96):
        x = torch.from_numpy(g.normal(size=(T, 1024)).astype(np.float32)).bfloat16().cuda()
        want = api.w4_linear(x, w4)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            got = api.w4_linear(x, w4)
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(got, want)
        for arg in (st, st.cuda_stream):          # named, as a stream and as a raw handle
            got = api.w4_linear(x, w4, stream=arg)
            torch.cuda.current_stream().wait_stream(st)
            assert torch.equal(got, want)
        out = torch.zeros_like(want)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            api.w4_linear(x, w4, out=out)
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_refusals_of_the_python_layer():
    W = torch.zeros(8, 64, device="cuda")
    with pytest.raises(ValueError):
        api.w4_quantize(W, 48)
    with pytest.raises(ValueError):
        api.w4_quantize(W.t(), 32)
    with pytest.raises(ValueError):
        api.w4_quantize(W.double(), 32)
    w4 = api.w4_quantize(W, 32)
    with pytest.raises(ValueError):
        api.w4_linear(torch.zeros(2, 32, dtype=torch.bfloat16, device="cuda"), w4)
    with pytest.raises(ValueError):
        api.w4_linear(torch.zeros(2, 64, device="cuda"), w4)


def test_a_layer_step_routed_over_4_bit_weights():
    """The operators as a decode step uses them: gate, base products, routed side path in
    place on their output; against the whole chain in float64 from the same bytes."""
    g = np.random.default_rng(11)
    for T in (1, 24, 300):
        d, E, K = 512, 12, 2
        dims = [(512, 512), (512, 128), (512, 1024)]
        x = torch.from_numpy(g.normal(size=(T, d)).astype(np.float32)).bfloat16().cuda()
        logits = torch.from_numpy(g.normal(size=(T, E)).astype(np.float32)).bfloat16().cuda()
        ids, w = api.route_experts(logits, lf.make_router(E, K))
        ws, ys, projs, pools = [], [], [], []
        for d_in, d_out in dims:
            W = torch.from_numpy(g.normal(size=(d_out, d_in)).astype(np.float32) * d_in ** -0.5).bfloat16().cuda()
            ws.append(api.w4_quantize(W, 128, zero_points=True))
            ranks = g.integers(1, 9, size=E).astype(np.int32)
            oA = np.concatenate([[0], np.cumsum(ranks * d_in)[:-1]]).astype(np.int64)
            oB = np.concatenate([[0], np.cumsum(ranks * d_out)[:-1]]).astype(np.int64)
            A = torch.from_numpy(g.normal(size=int(ranks.sum()) * d_in).astype(np.float32) * d_in ** -0.5).bfloat16().cuda()
            B = torch.from_numpy(g.normal(size=int(ranks.sum()) * d_out).astype(np.float32) * 0.2).bfloat16().cuda()
            dv = [torch.from_numpy(v).cuda() for v in (ranks, oA, oB)]
            y = torch.empty(T, d_out, dtype=torch.bfloat16, device="cuda")
            projs.append(lf.make_mixture_projection(x, y, lf.make_slice(d_out, 0, *dv, A, B), base=y))
            ys.append(y)
            pools.append((ranks, oA, oB, A.float().cpu().numpy(), B.float().cpu().numpy(), dv, A, B))
        api.w4_project([lf.make_w4_projection(x, y, q.q, q.scales, q.group, q.zeros) for y, q in zip(ys, ws)])
        api.lora_mixture(ids, w, E, projs, 2.0)
        assert lf.lf_get_device_status() == 0
        idn = OR.choose(logits.double().cpu().numpy(), K, "softmax")
        assert (ids.cpu().numpy() == idn).all()
        wn = OR.weights(logits.double().cpu().numpy(), idn, "softmax", True)
        for (d_in, d_out), y, q, pl in zip(dims, ys, ws, pools):
            y0, m0 = reference(x, q)
            want, mag = OR.mixture(x.double().cpu().numpy(), y0, idn, wn, *pl[:5], 2.0)
            # two roundings to bf16: the base product's and the sum's; weights within 2^-18
            tol = 2.0 ** -8 * (np.abs(want) + np.abs(y0) * (1 + 2.0 ** -8)) + \
                (d_in * 2.0 ** -24 * 1.1) * m0 + (2.0 ** -18 + (d_in + 64) * 2.0 ** -24) * mag * 1.1
            assert (np.abs(y.double().cpu().numpy() - want) <= tol).all()


def few(g, T, d_in, d_out, group, zp):
    """(w4, codes less zero points, scales per column): codes equal the zero point but for some
    columns, whose difference is -1 or 1."""
    w4 = make(g, d_in, d_out, group, zp)
    at = np.arange(d_in) // group
    z = (w4.zeros.cpu().numpy().astype(np.int64) if zp else np.full((d_out, -(-d_in // group)), 8))[:, at]
    step = np.where(z < 8, 1, -1) * (g.random((d_out, d_in)) < 0.03)
    w4.q = torch.from_numpy(np.ascontiguousarray(OR.w4_pack((z + step).astype(np.uint8)))).cuda()
    return w4, step.astype(np.float64), w4.scales.double().cpu().numpy()[:, at]


@pytest.mark.parametrize("T", [1, 5, 8, 9, 16, 17, 40])
@pytest.mark.parametrize("d_in,d_out,group,zp", [(96, 24, 32, True), (3584, 64, 128, True), (1056, 40, 256, False),
                                                 (4096, 32, 64, True)])
def test_columns_at_the_zero_point_add_nothing(T, d_in, d_out, group, zp):
    """Large activations where the codes are the zero point leave no trace of 128 + q: the error
    is within n 2^-24 (twice that, for sums that truncate) of the sum of |q - z| |s| |x| alone."""
    g = np.random.default_rng(T + d_in)
    w4, step, s = few(g, T, d_in, d_out, group, zp)
    x = g.normal(size=(T, d_in))
    x[:, (step == 0).all(axis=0) | (g.random(d_in) < 0.1)] *= 1000
    x = torch.from_numpy(x.astype(np.float32)).bfloat16().cuda()
    y = api.w4_linear(x, w4).double().cpu().numpy()
    xn = x.double().cpu().numpy()
    want, mag = xn @ (step * s).T, np.abs(xn) @ np.abs(step * s).T
    assert (np.abs(y - want) <= 2.0 ** -8 * np.abs(want) + 1.01 * (d_in + 16) * 2.0 ** -23 * mag).all()
    x = torch.where(torch.from_numpy((step == 0).all(axis=0)).cuda(), x, torch.zeros_like(x))
    assert (api.w4_linear(x, w4) == 0).all()     # nothing but zero points


@pytest.mark.parametrize("T", [1, 9, 16, 17])
@pytest.mark.parametrize("group", [32, 128])
def test_large_and_infinite_activations(T, group):
    """A finite x of 2^123 (16 x, at most, is finite) gives finite products; an infinite one gives
    an infinity of its weight's sign, NaN where that weight is 0."""
    g = np.random.default_rng(group)
    w4 = make(g, 256, 64, group, True)
    M = OR.w4_matrix(w4.q.cpu().numpy(), w4.scales.double().cpu().numpy(), w4.zeros.cpu().numpy(), group)
    x = torch.zeros(T, 256, dtype=torch.bfloat16, device="cuda")
    x[:, 77] = 2.0 ** 123
    y = api.w4_linear(x, w4).double().cpu().numpy()
    want = np.broadcast_to(2.0 ** 123 * M[:, 77], y.shape)
    assert (np.abs(y - want) <= 2.0 ** -8 * np.abs(want)).all()
    x[T - 1, 77] = float("inf")
    y = api.w4_linear(x, w4).double().cpu().numpy()
    assert (np.abs(y - want)[:T - 1] <= 2.0 ** -8 * np.abs(want)[:T - 1]).all()
    assert np.isnan(y[T - 1, M[:, 77] == 0]).all() and (M[:, 77] == 0).any()
    assert (y[T - 1, M[:, 77] > 0] == np.inf).all() and (y[T - 1, M[:, 77] < 0] == -np.inf).all()


def test_scales_are_bf16_values_of_fp32_quotients():
    """Quotients next to the middle of two bf16 values: fp32 makes the middle of them, which goes
    to even; those that fp32 holds apart from it go to their side."""
    W = torch.zeros(8, 32, device="cuda")
    mid = 1 + 2.0 ** -8                                  # between 1 and 1 + 2^-7
    W[0, 0], W[0, 1] = 15 * mid, -1e-9                   # above the middle by less than fp32 holds
    W[1, 0] = 15 * mid
    W[2, 0], W[2, 1] = 15 * mid, -2.0 ** -18             # by more
    W[3, 0] = float(np.nextafter(np.float32(15 * mid), np.float32(0)))
    W[4, 0], W[4, 1] = 15 * (1 + 3 * 2.0 ** -8), -1e-9   # between 1 + 2^-7 and 1 + 2^-6: up is even
    W[5, 0] = float(np.nextafter(np.float32(15 * (1 + 3 * 2.0 ** -8)), np.float32(0)))
    w4 = api.w4_quantize(W, 32, zero_points=True)
    want = [1, 1, 1 + 2.0 ** -7, 1, 1 + 2.0 ** -6, 1 + 2.0 ** -7, 0, 0]
    assert w4.scales[:, 0].tolist() == want
    c, s, z = OR.w4_quantize(W.double().cpu().numpy(), 32, True)
    assert s[:, 0].tolist() == want and (OR.w4_unpack(w4.q.cpu().numpy()) == c).all() and (w4.zeros.cpu().numpy() == z).all()
    W /= 15
    W *= 7
    w4 = api.w4_quantize(W, 32)
    c, s, z = OR.w4_quantize(W.double().cpu().numpy(), 32, False)
    assert (w4.scales.double().cpu().numpy() == s).all() and (OR.w4_unpack(w4.q.cpu().numpy()) == c).all()
    assert lf.lf_get_device_status() == 0
