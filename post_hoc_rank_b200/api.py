"""Convenience layer over the C ABI: allocates outputs/workspaces as torch CUDA
tensors and calls the binding.  No arithmetic of the method happens here."""
from __future__ import annotations

import contextlib
import dataclasses

import numpy as np
import torch

from . import loraforge as lf


def modules_from_layout(layout) -> np.ndarray:
    """lf_module array from a synth.FleetLayout (or any object with the same fields)."""
    m = np.zeros(layout.n, dtype=lf.MODULE_DTYPE)
    m["d_out"], m["d_in"], m["r"], m["group"] = layout.d_out, layout.d_in, layout.r, layout.group
    m["B_off"], m["A_off"] = layout.B_off, layout.A_off
    return m


@dataclasses.dataclass
class Factors:
    R_B: torch.Tensor
    R_A: torch.Tensor
    sigma: torch.Tensor
    U: torch.Tensor
    V: torch.Tensor
    rs: int


@dataclasses.dataclass
class Export:
    ranks: torch.Tensor
    off_A: torch.Tensor
    off_Bt: torch.Tensor
    A_pool: torch.Tensor
    Bt_pool: torch.Tensor
    A_pool16: torch.Tensor | None
    Bt_pool16: torch.Tensor | None


def workspace(nbytes: int, device) -> torch.Tensor:
    return torch.empty(max(int(nbytes), 1), dtype=torch.uint8, device=device)


def alloc_factors(mods: np.ndarray, device) -> Factors:
    n = mods.shape[0]
    rs = lf.lf_rank_stride(mods)
    f32 = dict(dtype=torch.float32, device=device)
    f64 = dict(dtype=torch.float64, device=device)
    return Factors(torch.empty((n, rs, rs), **f32), torch.empty((n, rs, rs), **f32),
                   torch.empty((n, rs), **f64), torch.empty((n, rs, rs), **f64),
                   torch.empty((n, rs, rs), **f64), rs)


def tsqr(mods, B_base, A_base, out: Factors | None = None, ws=None, stream=None) -> Factors:
    dev = B_base.device
    out = out or alloc_factors(mods, dev)
    ws = ws if ws is not None else workspace(lf.lf_tsqr_workspace_size(mods), dev)
    lf.lf_tsqr_batched(mods, B_base, A_base, out.R_B, out.R_A, out.sigma, out.U, out.V, ws, stream)
    return out


def alloc_export(mods, pol, device, bf16: bool = True) -> Export:
    n = mods.shape[0]
    capA, capB = lf.lf_export_pool_bound(mods, pol)
    i64 = dict(dtype=torch.int64, device=device)
    return Export(torch.empty(n, dtype=torch.int32, device=device), torch.empty(n + 1, **i64),
                  torch.empty(n + 1, **i64),
                  torch.empty(max(capA, 8), dtype=torch.float32, device=device),
                  torch.empty(max(capB, 8), dtype=torch.float32, device=device),
                  torch.empty(max(capA, 8), dtype=torch.bfloat16, device=device) if bf16 else None,
                  torch.empty(max(capB, 8), dtype=torch.bfloat16, device=device) if bf16 else None)


def truncate_export(mods, pol, B_base, A_base, F: Factors, out: Export | None = None, ws=None,
                    stream=None, bf16: bool = True) -> Export:
    dev = B_base.device
    out = out or alloc_export(mods, pol, dev, bf16)
    ws = ws if ws is not None else workspace(lf.lf_export_workspace_size(mods), dev)
    lf.lf_truncate_export(mods, pol, B_base, A_base, F.R_B, F.R_A, F.sigma, F.U, F.V, out.ranks,
                          out.off_A, out.off_Bt, out.A_pool, out.Bt_pool, out.A_pool16, out.Bt_pool16,
                          ws, stream)
    return out


def select_ranks(mods, pol, sigma, stream=None):
    dev = sigma.device
    n = mods.shape[0]
    ranks = torch.empty(n, dtype=torch.int32, device=dev)
    offA = torch.empty(n + 1, dtype=torch.int64, device=dev)
    offB = torch.empty(n + 1, dtype=torch.int64, device=dev)
    ws = workspace(lf.lf_select_workspace_size(mods), dev)
    lf.lf_select_ranks(mods, pol, sigma, ranks, offA, offB, ws, stream)
    return ranks, offA, offB


def pool_module(A_offs, ranks, d_in: int) -> np.ndarray:
    """lf_module of a pool's stacked row factors (LoRASpace's pool-wide subspace, the
    arXiv listing abstract): the A_i (r_i x d_in) of one module position stored back to
    back from element A_offs[0] of a pool form one contiguous (sum r_i) x d_in matrix,
    entered as the A factor of one module whose B factor is the identity of order
    sum r_i, so the module's singular values are those of the stack.  Host checks only:
    sum r_i <= 64 (the kernels' rank limit) and <= d_in, and the factors contiguous."""
    A_offs = [int(o) for o in A_offs]
    ranks = [int(r) for r in ranks]
    if not ranks or len(A_offs) != len(ranks) or min(ranks) < 1:
        raise ValueError("one offset and a positive rank per LoRA")
    R = sum(ranks)
    if R > 64 or R > d_in:
        raise ValueError("the stacked rank must be at most 64 and at most d_in")
    for i in range(len(ranks) - 1):
        if A_offs[i + 1] != A_offs[i] + ranks[i] * d_in:
            raise ValueError("the pool's row factors must be stored back to back")
    m = np.zeros(1, dtype=lf.MODULE_DTYPE)
    m["d_out"], m["d_in"], m["r"], m["group"], m["B_off"], m["A_off"] = R, d_in, R, 0, 0, A_offs[0]
    return m


def pool_subspace_rows(A_base, A_offs, ranks, d_in: int, num: int = 99, den: int = 100, stream=None):
    """Pool-wide subspace of stacked row factors on the GPU: lf_tsqr_batched on
    pool_module (singular values of the stack), then lf_select_ranks with the
    energy-fraction policy (floor 1).  Returns (k, sigma[sum r_i] fp64, Factors)."""
    mods = pool_module(A_offs, ranks, d_in)
    R = int(mods["r"][0])
    eye = torch.eye(R, dtype=torch.float32, device=A_base.device)
    F = tsqr(mods, eye.reshape(-1), A_base, stream=stream)
    k, _, _ = select_ranks(mods, lf.policy_E(num, den, 1), F.sigma, stream=stream)
    return int(k[0].item()), F.sigma[0, :R], F


@dataclasses.dataclass
class PoolSubspace:
    k: torch.Tensor        # int32 [1]
    sigma: torch.Tensor    # fp64 [R], descending
    basis: torch.Tensor    # fp32 [R, d], row j = direction j
    coef: torch.Tensor     # fp32 [R, R], coef[a, j] = stack vector a . direction j
    resid: torch.Tensor    # fp64 [1]


def pool_subspace(base, offs, ranks, d: int, side: str = "row", num: int = 99, den: int = 100, stream=None):
    """LoRASpace's pool-wide subspace of a pool's stacked factors on the GPU
    (lf_pool_subspace): side "row" stacks the A_i (r_i x d) stored at element offsets
    offs of `base`, side "col" puts the B_i (d x r_i) side by side.  Allocates the
    outputs and the workspace as torch tensors."""
    sd = {"row": 0, "col": 1}[side]
    R = int(sum(int(r) for r in ranks))
    dev = base.device
    ws = workspace(lf.lf_pool_workspace_size(sd, ranks, offs, d), dev)
    out = PoolSubspace(torch.zeros(1, dtype=torch.int32, device=dev), torch.zeros(R, dtype=torch.float64, device=dev),
                       torch.zeros(R, d, dtype=torch.float32, device=dev),
                       torch.zeros(R, R, dtype=torch.float32, device=dev),
                       torch.zeros(1, dtype=torch.float64, device=dev))
    lf.lf_pool_subspace(sd, ranks, offs, d, base, num, den, out.k, out.sigma, out.basis, out.coef, out.resid, ws,
                        stream)
    return out


def shrink_expand(x, y, ids, ranks, off_A, off_Bt, A_pool, Bt_pool, scale, ws=None, seg_out=None,
                  stream=None):
    n_adapters = ranks.numel()
    ws = ws if ws is not None else workspace(lf.lf_apply_workspace_size(x.shape[0], n_adapters), x.device)
    lf.lf_lora_shrink_expand(x, y, ids, n_adapters, ranks, off_A, off_Bt, A_pool, Bt_pool, scale, ws,
                             seg_out, stream)
    return y


def shrink_expand_slices(x, y, ids, slices, scale, adapter_scale=None, ws=None, seg_out=None, stream=None):
    """Side path of several output slices sharing x.  slices: list of tuples
    (d_out, y_offset, ranks, off_A, off_Bt, A_pool, Bt_pool) with device tensors
    (ranks int32 and offsets int64 per adapter, bf16 pools); y is T x y_ld."""
    n_adapters = slices[0][2].numel()
    ns = len(slices)
    ws = ws if ws is not None else workspace(lf.lf_apply_slices_workspace_size(x.shape[0], n_adapters, ns), x.device)
    sl = [lf.make_slice(*t) for t in slices]
    lf.lf_lora_shrink_expand_slices(x, y, ids, n_adapters, sl, scale, ws, adapter_scale, seg_out, stream)
    return y


@dataclasses.dataclass
class JdTables:
    members: np.ndarray    # int32 module indices, problem by problem
    probs: np.ndarray      # lf_jd_problem records
    U_total: int           # fp32 elements of the U buffer
    Vt_total: int          # fp32 elements of the V^T buffer
    sigma_total: int       # fp32 elements of the Sigma buffer


def jd_tables(mods: np.ndarray, positions, rank: int) -> JdTables:
    """Problem table for JD-Full over module positions.  positions: one list of module
    indices per problem (the LoRAs sharing that position, all of one shape).  U, V^T and
    Sigma of consecutive problems are laid out back to back (offsets multiples of 4)."""
    members, rows = [], []
    u = v = sg = 0
    for pos in positions:
        pos = [int(m) for m in pos]
        d_out, d_in = int(mods["d_out"][pos[0]]), int(mods["d_in"][pos[0]])
        rows.append((d_out, d_in, rank, len(members), len(pos), u, v, sg))
        members += pos
        u += (d_out * rank + 3) // 4 * 4
        v += (rank * d_in + 3) // 4 * 4
        sg += len(pos) * rank * rank
    probs = np.zeros(len(rows), dtype=lf.JD_PROBLEM_DTYPE)
    for i, r in enumerate(rows):
        probs[i] = r
    return JdTables(np.asarray(members, dtype=np.int32), probs, u, v, sg)


def jd_full(mods, tabs: JdTables, B_base, A_base, U, Vt, iters: int, weights=None, sigma=None, ws=None,
            stream=None):
    """JD-Full eigenvalue iteration in place on U / Vt (fp32 device buffers laid out by
    jd_tables); writes Sigma_i into `sigma` when given."""
    ws = ws if ws is not None else workspace(lf.lf_jd_workspace_size(mods, tabs.members, tabs.probs), U.device)
    lf.lf_jd_full(mods, tabs.members, tabs.probs, B_base, A_base, weights, iters, U, Vt, sigma, ws, stream)
    return U, Vt, sigma


# ---- routed side path and 4-bit base weights ------------------------------------------------

_HERE = contextlib.nullcontext()


def _on(device, stream=None):
    """Context in which `device` and `stream` (a torch stream or a raw handle; None = the device's
    current one) are the current ones: what is allocated inside belongs to the stream that the
    kernels run on, so its memory is not handed out again while they use it."""
    if device.type != "cuda":
        raise ValueError(f"tensors must live on a CUDA device, got {device}")
    if stream is not None:
        return torch.cuda.stream(torch.cuda.ExternalStream(stream, device) if isinstance(stream, int) else stream)
    return _HERE if device.index == lf.current_device() else torch.cuda.device(device)


def _expect(t, name: str, device, dtype, shape):
    if t is not None and (t.dtype != dtype or t.shape != shape or t.device != device or not t.is_contiguous()):
        raise ValueError(f"{name}: contiguous {dtype} tensor of shape {tuple(shape)} on {device} expected")


def _check_logits(logits, router: lf.lf_router):
    if logits.dim() != 2 or logits.shape[1] != router.n_experts or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError(f"logits must be T x {router.n_experts} with unit column stride, got {tuple(logits.shape)}")
    if logits.shape[0] > 1 and logits.stride(0) < logits.shape[1]:
        raise ValueError("logits rows must not overlap")


def route_experts(logits, router: lf.lf_router, bias=None, counts=None, stream=None):
    """Experts and weights of every token (lf_route_experts; lf.make_router): ids T x top_k int32
    (-1 = empty slot) and weights T x top_k fp32.  bias: fp32 per expert, steers the choice only;
    counts: int32 per expert, overwritten with the number of slots that chose it."""
    _check_logits(logits, router)
    T, dev = logits.shape[0], logits.device
    _expect(bias, "bias", dev, torch.float32, (router.n_experts,))
    _expect(counts, "counts", dev, torch.int32, (router.n_experts,))
    with _on(dev, stream):
        ids = torch.empty((T, router.top_k), dtype=torch.int32, device=dev)
        weights = torch.empty((T, router.top_k), dtype=torch.float32, device=dev)
        lf.lf_route_experts(logits, router, bias, ids, weights, counts)
    return ids, weights


def route_experts_backward(logits, router: lf.lf_router, ids, grad_weights, stream=None):
    """Gradient of route_experts' weights for the logits (same type), at its ids."""
    _check_logits(logits, router)
    T, dev = logits.shape[0], logits.device
    _expect(ids, "ids", dev, torch.int32, (T, router.top_k))
    _expect(grad_weights, "grad_weights", dev, torch.float32, (T, router.top_k))
    with _on(dev, stream):
        grad = torch.empty((T, router.n_experts), dtype=logits.dtype, device=dev)
        lf.lf_route_experts_backward(logits, router, ids, grad_weights, grad)
    return grad


def _same_rows(projections, T: int, device):
    have = lf._rows_device(projections)
    if have != (T, device):
        raise ValueError(f"every projection must have {T} rows on {device}, got {have[0]} on {have[1]}")


def lora_mixture(ids, weights, n_adapters: int, projections, scale: float, adapter_scale=None, ws=None, stream=None):
    """Routed side path (lf_lora_mixture) of lf.make_mixture_projection projections, whose y it
    writes: y = base + scale * sum_j weights_j B'_j (A'_j x).  ids T x top_k int32 (-1 = empty
    slot), weights T x top_k fp32 or None (all 1), as route_experts returns them."""
    dev = ids.device
    _expect(ids, "ids", dev, torch.int32, ids.shape)
    _expect(weights, "weights", dev, torch.float32, ids.shape)
    _expect(adapter_scale, "adapter_scale", dev, torch.float32, (n_adapters,))
    _same_rows(projections, ids.shape[0], dev)
    with _on(dev, stream):
        projections = lf._array(lf.lf_mixture_projection, projections)
        if ws is None:
            n = lf.lf_lora_mixture_workspace_size(ids.shape[0], ids.shape[1], n_adapters, projections)
            ws = workspace(n, dev) if n else None
        lf.lf_lora_mixture(ids, weights, n_adapters, projections, scale, ws, adapter_scale)


def lora_mixture_backward(ids, weights, n_adapters: int, grads, scale: float, adapter_scale=None, grad_weights=True,
                          ws=None, stream=None):
    """Gradients of lora_mixture (lf_lora_mixture_backward): writes the dx of every
    lf.make_mixture_grad entry and returns the weights' gradient (T x top_k fp32, summed over the
    entries), or None with grad_weights=False."""
    dev = ids.device
    _expect(ids, "ids", dev, torch.int32, ids.shape)
    _expect(weights, "weights", dev, torch.float32, ids.shape)
    _expect(adapter_scale, "adapter_scale", dev, torch.float32, (n_adapters,))
    _same_rows(grads, ids.shape[0], dev)
    with _on(dev, stream):
        gw = torch.empty(ids.shape, dtype=torch.float32, device=dev) if grad_weights else None
        grads = lf._array(lf.lf_mixture_grad, grads)
        if ws is None:
            n = lf.lf_lora_mixture_backward_workspace_size(ids.shape[0], ids.shape[1], n_adapters, grads)
            ws = workspace(n, dev) if n else None
        lf.lf_lora_mixture_backward(ids, weights, n_adapters, grads, scale, gw, ws, adapter_scale)
    return gw


@dataclasses.dataclass
class W4:
    """A base weight matrix in 4 bits: (q - zeros) * scales per group of columns."""
    q: torch.Tensor               # uint8 [d_out, d_in / 2], even columns in the low nibbles
    scales: torch.Tensor          # bf16 [d_out, ng]
    zeros: torch.Tensor | None    # uint8 [d_out, ng], None = 8
    group: int

    @property
    def shape(self):
        return self.q.shape[0], 2 * self.q.shape[1]


def w4_quantize(W, group: int = 128, zero_points: bool = False, stream=None) -> W4:
    """Quantises W (d_out x d_in fp32, bf16 or fp16) to 4 bits with a scale, and with
    zero_points a zero point, per `group` columns (lf_w4_quantize)."""
    if W.dim() != 2 or not W.is_contiguous():
        raise ValueError("W must be a contiguous matrix")
    if group not in (32, 64, 128, 256):
        raise ValueError(f"group must be 32, 64, 128 or 256, got {group}")
    d_out, d_in = W.shape
    dev, ng = W.device, (d_in + group - 1) // group
    with _on(dev, stream):
        out = W4(torch.empty((d_out, d_in // 2), dtype=torch.uint8, device=dev),
                 torch.empty((d_out, ng), dtype=torch.bfloat16, device=dev),
                 torch.empty((d_out, ng), dtype=torch.uint8, device=dev) if zero_points else None, group)
        lf.lf_w4_quantize(W, group, out.q, out.scales, out.zeros)
    return out


def w4_dequantize(w4: W4, dtype=torch.bfloat16, stream=None):
    """The matrix a W4 stands for (lf_w4_dequantize), fp32 (exact), bf16 or fp16."""
    dev = w4.q.device
    with _on(dev, stream):
        W = torch.empty(w4.shape, dtype=dtype, device=dev)
        lf.lf_w4_dequantize(w4.q, w4.scales, w4.zeros, w4.group, W)
    return W


def w4_project(projections, stream=None):
    """y = x W0^T + bias for lf.make_w4_projection projections of one token batch
    (lf_w4_projections): all have the same number of rows of x."""
    T, dev = lf._rows_device(projections)
    with _on(dev, stream):
        lf.lf_w4_projections(T, projections)


def w4_linear(x, w4: W4, bias=None, out=None, stream=None):
    """x (T x d_in bf16) times a 4-bit matrix: T x d_out bf16 (lf_w4_projections, one projection)."""
    if x.shape[1] != w4.shape[1]:
        raise ValueError(f"x has {x.shape[1]} columns, the matrix {w4.shape[1]}")
    with _on(x.device, stream):
        y = out if out is not None else torch.empty((x.shape[0], w4.shape[0]), dtype=torch.bfloat16, device=x.device)
        w4_project([lf.make_w4_projection(x, y, w4.q, w4.scales, w4.group, w4.zeros, bias)])
    return y


def device_status(stream=None) -> int:
    return lf.lf_get_device_status(stream)
