"""Operators beside the multi-LoRA side path, their plain forms and the sizes they are measured at:

  route  routing of tokens to experts (softmax or sigmoid gate, balance bias, groups, top-k,
         renormalised weights) and its gradient;
  mix    the routed side path: every token adds up the weighted LoRA updates of its experts,
         y = base + s sum_j w_j B'_j (A'_j x), and its gradients for x and the weights;
  w4     products with 4-bit base weights with group scales (and zero points);
  quant  quantisation of base weights to that form and back.

`own` picks between the framework's entry points and the plain forms in torch operations."""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# d_in x d_out of the adapted projections: q, k, v, o, gate, up, down
QWEN = "3584x3584 3584x512 3584x512 3584x3584 3584x18944 3584x18944 18944x3584"
LLAMA = "4096x4096 4096x1024 4096x1024 4096x4096 4096x14336 4096x14336 14336x4096"


def _shapes(text):
    return [tuple(int(n) for n in one.split("x")) for one in text.split()]


def listed():
    return [
        # a decode batch picks 2 of 128 resident adapters per token, from a bf16 gate; some adapters are not resident
        dict(name="route_decode", op="route", T=256, E=128, K=2, dtype="bf16", score="softmax", renorm=True, bias=False,
             groups=1, top_groups=1, group_top=1, masked=0.1, train=False),
        # training a gate of 256 experts on a long batch: sigmoid scores, balance bias, 4 of 8 groups
        dict(name="route_train_groups", op="route", T=16384, E=256, K=8, dtype="f32", score="sigmoid", renorm=True,
             bias=True, groups=8, top_groups=4, group_top=2, masked=0.0, train=True),
        # training a gate over a pool of 17 LoRAs with 6 active, an odd number of tokens, plain softmax weights
        dict(name="route_train_pool", op="route", T=1003, E=17, K=6, dtype="bf16", score="softmax", renorm=False,
             bias=False, groups=1, top_groups=1, group_top=1, masked=0.0, train=True),
        # one token of a request composed of 6 LoRAs out of 17, smallest projection
        dict(name="mix_token", op="mix", T=1, E=17, K=6, max_rank=16, shapes="3584x512", train=False),
        # a decode step: 256 tokens, 128 resident compressed adapters, all projections of a layer
        dict(name="mix_decode", op="mix", T=256, E=128, K=2, max_rank=10, shapes=LLAMA, train=False),
        # a short training batch over 8 uncompressed rank-64 adapters, an odd number of tokens
        dict(name="mix_train_short", op="mix", T=333, E=8, K=2, max_rank=64, shapes="3584x18944", train=True),
        # a training batch (or long prompts, with gradients) over 16 rank-16 adapters
        dict(name="mix_train", op="mix", T=8192, E=16, K=2, max_rank=16, shapes="3584x3584", train=True),
        # one decoded token through all projections of a layer
        dict(name="w4_token", op="w4", T=1, shapes=QWEN, group=128, zeros=True, bias=True),
        # a small decode batch through one up projection
        dict(name="w4_batch", op="w4", T=37, shapes="4096x14336", group=64, zeros=False, bias=False),
        # a prompt chunk
        dict(name="w4_prompt", op="w4", T=512, shapes="3584x18944", group=128, zeros=True, bias=False),
        # one small projection's weights, laid out for serving
        dict(name="quant_small", op="quant", d_in=3584, d_out=512, group=128, zeros=False, dtype="bf16"),
        # one large projection's weights
        dict(name="quant_large", op="quant", d_in=3584, d_out=18944, group=64, zeros=True, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "mix", "w4", "quant"])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, max(2, 8 // groups), 512 // groups)
        top_groups = rng.randint(1, groups)
        return dict(op=op, T=_log(rng, 1, 16384 * 256 // max(E, 256)), E=E, K=rng.randint(1, min(8, E)),
                    dtype=rng.choice(["f32", "bf16", "f16"]), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.5, bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                    group_top=rng.choice([1, 2]), masked=rng.choice([0.0, 0.1, 0.5]), train=rng.random() < 0.5)
    if op == "mix":
        d_in, d_out = rng.choice(_shapes(QWEN) + _shapes(LLAMA) + [(8 * rng.randint(16, 1000), 8 * rng.randint(16, 1000))])
        max_rank = rng.randint(1, 64)
        E = min(_log(rng, 2, 128), 1024 // max_rank + 2)
        return dict(op=op, T=_log(rng, 1, min(8192, 8192 * 7168 // (d_in + d_out), 8192 * 256 // (E * max_rank) + 1)),
                    E=E, K=rng.randint(1, min(6, E)), max_rank=max_rank, shapes=f"{d_in}x{d_out}",
                    train=rng.random() < 0.5)
    if op == "w4":
        d_in, d_out = rng.choice(_shapes(QWEN) + _shapes(LLAMA) + [(32 * rng.randint(4, 592), 8 * rng.randint(8, 1024))])
        return dict(op=op, T=_log(rng, 1, 512), shapes=f"{d_in}x{d_out}", group=rng.choice([32, 64, 128]),
                    zeros=rng.random() < 0.5, bias=rng.random() < 0.5)
    d_in, d_out = rng.choice(_shapes(QWEN) + [(32 * rng.randint(4, 592), 8 * rng.randint(8, 1024))])
    return dict(op=op, d_in=d_in, d_out=d_out, group=rng.choice([32, 64, 128]), zeros=rng.random() < 0.5,
                dtype=rng.choice(["f32", "bf16", "f16"]))


# ---- inputs ---------------------------------------------------------------------------------

def _ragged(E, max_rank, device, gen):
    """Retained ranks 1 .. max_rank, one of them max_rank."""
    r = torch.randint(1, max_rank + 1, (E,), device=device, generator=gen)
    r[0] = max_rank
    return r


def _groups_of(d_in, group):
    return (d_in + group - 1) // group


def _pack4(codes):
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).to(torch.uint8).contiguous()


def _base_weights(d_in, d_out, group, zeros, device, gen):
    """4-bit codes, scales and zero points as a quantiser of Gaussian weights leaves them."""
    ng = _groups_of(d_in, group)
    w = torch.randn(d_out, d_in, device=device, generator=gen) * d_in ** -0.5
    w = torch.nn.functional.pad(w, (0, ng * group - d_in)).view(d_out, ng, group)
    if zeros:
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        scale = ((hi - lo) / 15).bfloat16()
        zp = (-lo / scale.float()).round().clamp(0, 15)
    else:
        scale = (w.abs().amax(2) / 7).bfloat16()
        zp = torch.full_like(scale, 8, dtype=torch.float32)
    codes = ((w / scale.float().unsqueeze(2)).round() + zp.unsqueeze(2)).clamp(0, 15).to(torch.uint8)
    q = _pack4(codes.view(d_out, ng * group)[:, :d_in])
    return q, scale.contiguous(), zp.to(torch.uint8).contiguous() if zeros else None


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, device=dev, generator=gen)  # noqa: E731
    st = dict(case)
    if case["op"] == "route":
        T, E, K = case["T"], case["E"], case["K"]
        logits = 1.5 * normal(T, E) + 0.5 * normal(E)
        if case["masked"]:
            gone = torch.rand(E, device=dev, generator=gen) < case["masked"]
            gone[0] = False
            logits = logits.masked_fill(gone, -math.inf)
            logits[T // 2:T // 2 + T // 64] = -math.inf          # padding rows: nothing to route
        st["logits"] = logits.to(DTYPES[case["dtype"]])
        spread = 0.05 if case["score"] == "sigmoid" else 0.2 / E
        st["bias"] = spread * normal(E) if case["bias"] else None
        st["grad"] = normal(T, K)
    elif case["op"] == "mix":
        T, E, K = case["T"], case["E"], case["K"]
        popular = -torch.log(torch.rand(T, E, device=dev, generator=gen)) * torch.arange(1, E + 1, device=dev) ** 0.7
        ids = popular.topk(K, dim=1, largest=False).indices.int()
        ids[torch.rand(T, device=dev, generator=gen) < 0.03] = -1            # tokens without adapters
        ids[:, K - 1][torch.rand(T, device=dev, generator=gen) < 0.05] = -1  # tokens with one adapter fewer
        st["ids"], st["weights"] = ids.contiguous(), torch.softmax(normal(T, K), 1)
        st["projections"] = []
        for d_in, d_out in _shapes(case["shapes"]):
            ranks = _ragged(E, case["max_rank"], dev, gen)
            R = int(ranks.sum())
            first = torch.cumsum(ranks, 0) - ranks
            st["projections"].append(dict(
                d_in=d_in, d_out=d_out, ranks=ranks.int(), off_A=first * d_in, off_Bt=first * d_out,
                expert=torch.repeat_interleave(torch.arange(E, device=dev), ranks),
                A=(normal(R, d_in) * d_in ** -0.5).bfloat16(), Bt=(normal(R, d_out) * 0.25).bfloat16(),
                x=normal(T, d_in).bfloat16(), base=normal(T, d_out).bfloat16(),
                grad=normal(T, d_out).bfloat16() if case["train"] else None))
    elif case["op"] == "w4":
        T = case["T"]
        xs, st["projections"] = {}, []
        for i, (d_in, d_out) in enumerate(_shapes(case["shapes"])):
            key = {0: "in", 1: "in", 2: "in", 3: "attn", 4: "mlp", 5: "mlp", 6: "down"}[i]
            if key not in xs:
                x = normal(T, d_in)
                x[:, :: max(d_in // 8, 1)] *= 20.0                # the few large channels of a transformer's activations
                xs[key] = x.bfloat16()
            q, scales, zp = _base_weights(d_in, d_out, case["group"], case["zeros"], dev, gen)
            bias = normal(d_out).bfloat16() if case["bias"] and i < 3 else None
            st["projections"].append(dict(d_in=d_in, d_out=d_out, x=xs[key], q=q, scales=scales, zeros=zp, bias=bias))
    else:
        w = normal(case["d_out"], case["d_in"]) * case["d_in"] ** -0.5
        st["w"] = w.to(DTYPES[case["dtype"]])
    return st


# ---- plain forms ----------------------------------------------------------------------------

def _plain_route(st):
    l, E, K, G = st["logits"].double(), st["E"], st["K"], st["groups"]
    s = torch.softmax(l, 1).nan_to_num(0.0) if st["score"] == "softmax" else torch.sigmoid(l)
    open_ = l > -math.inf
    key = l if st["bias"] is None else s + st["bias"].double()
    key = key.masked_fill(~open_, -math.inf)
    if G > 1:
        c = s if st["bias"] is None else s + st["bias"].double()
        c = c.masked_fill(~open_, -math.inf).view(-1, G, E // G)
        best = c.sort(dim=2, descending=True).values[:, :, :st["group_top"]]
        score = best.masked_fill(best == -math.inf, 0.0).sum(2).masked_fill(best[:, :, 0] == -math.inf, -math.inf)
        order = score.sort(dim=1, descending=True, stable=True).indices[:, :st["top_groups"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, order, True)
        key = key.masked_fill(~keep.repeat_interleave(E // G, 1), -math.inf)
    top = key.sort(dim=1, descending=True, stable=True)
    there = top.values[:, :K] > -math.inf
    ids = top.indices[:, :K]
    sel = s.gather(1, ids).masked_fill(~there, 0.0)
    total = sel.sum(1, keepdim=True).clamp(min=1e-300)
    w = sel / total if st["renorm"] else sel
    out = {"ids": ids.masked_fill(~there, -1).int(), "weights": w.float()}
    if st["train"]:
        g = st["grad"].double().masked_fill(~there, 0.0)
        ds = (g - (g * w).sum(1, keepdim=True)) / total if st["renorm"] else g
        ds = torch.zeros_like(s).scatter_(1, ids, ds.masked_fill(~there, 0.0))
        dl = s * (ds - (s * ds).sum(1, keepdim=True)) if st["score"] == "softmax" else ds * s * (1 - s)
        out["dlogits"] = dl.to(st["logits"].dtype)
    return out


def _plain_mix(st, p):
    E, there = st["E"], st["ids"] >= 0
    ids = st["ids"].clamp(min=0).long()
    w = st["weights"].masked_fill(~there, 0.0)
    per_row = torch.zeros(w.shape[0], E, device=w.device).scatter_add_(1, ids, w)[:, p["expert"]]
    A, Bt, x = p["A"].float(), p["Bt"].float(), p["x"].float()
    t = x @ A.t()
    y = (p["base"].float() + 2.0 * ((t * per_row) @ Bt)).bfloat16()
    if not st["train"]:
        return y
    u = p["grad"].float() @ Bt.t()
    dx = (2.0 * ((u * per_row) @ A)).bfloat16()
    dots = torch.zeros(w.shape[0], E, device=w.device).index_add_(1, p["expert"], t * u)
    return y, dx, (2.0 * dots.gather(1, ids)).masked_fill(~there, 0.0)


def _unpack4(q):
    return torch.stack((q & 15, q >> 4), dim=2).view(q.shape[0], -1)


def _plain_w4(st, p):
    g = st["group"]
    cols = torch.arange(p["d_in"], device=p["q"].device) // g
    z = p["zeros"].float()[:, cols] if p["zeros"] is not None else 8.0
    w = (_unpack4(p["q"]).float() - z) * p["scales"].float()[:, cols]
    y = p["x"].float() @ w.t()
    return (y if p["bias"] is None else y + p["bias"].float()).bfloat16()


def _plain_quant(st):
    w, g = st["w"].double(), st["group"]
    d_out, d_in = w.shape
    ng = _groups_of(d_in, g)
    w = torch.nn.functional.pad(w, (0, ng * g - d_in)).view(d_out, ng, g)
    if st["zeros"]:
        lo, hi = w.amin(2).clamp(max=0), w.amax(2).clamp(min=0)
        scale = ((hi - lo) / 15).float().bfloat16()
    else:
        scale = (w.abs().amax(2) / 7).float().bfloat16()
    s = scale.double()
    inv = torch.where(s > 0, s, 1.0)
    z = (-lo / inv).round().clamp(0, 15) if st["zeros"] else torch.full_like(s, 8.0)
    q = ((w / inv.unsqueeze(2)).round() + z.unsqueeze(2)).clamp(0, 15)
    back = ((q - z.unsqueeze(2)) * s.unsqueeze(2)).view(d_out, ng * g)[:, :d_in]
    out = {"values": back.to(st["w"].dtype).contiguous(), "scales": scale}
    if st["zeros"]:
        out["zeros"] = z.to(torch.uint8)
    return out


# ---- the framework's operators --------------------------------------------------------------

def _own_route(st):
    from post_hoc_rank_b200 import api
    from post_hoc_rank_b200 import loraforge as lf
    r = lf.make_router(st["E"], st["K"], st["score"], n_groups=st["groups"], top_groups=st["top_groups"],
                       group_top=st["group_top"], renorm=st["renorm"])
    ids, w = api.route_experts(st["logits"], r, bias=st["bias"])
    out = {"ids": ids, "weights": w}
    if st["train"]:
        out["dlogits"] = api.route_experts_backward(st["logits"], r, ids, st["grad"])
    return out


def _own_mix(st):
    from post_hoc_rank_b200 import api
    from post_hoc_rank_b200 import loraforge as lf
    ids, w, E = st["ids"], st["weights"], st["E"]
    slices = [lf.make_slice(p["d_out"], 0, p["ranks"], p["off_A"], p["off_Bt"], p["A"], p["Bt"], st["max_rank"])
              for p in st["projections"]]
    ys = [torch.empty_like(p["base"]) for p in st["projections"]]
    api.lora_mixture(ids, w, E, [lf.make_mixture_projection(p["x"], y, sl, base=p["base"])
                                 for p, y, sl in zip(st["projections"], ys, slices)], 2.0)
    if not st["train"]:
        return ys
    dxs = [torch.empty_like(p["x"]) for p in st["projections"]]
    dw = api.lora_mixture_backward(ids, w, E, [lf.make_mixture_grad(p["x"], p["grad"], dx, sl)
                                               for p, dx, sl in zip(st["projections"], dxs, slices)], 2.0)
    return [(y, dx, dw) for y, dx in zip(ys, dxs)]


def _own_w4(st):
    from post_hoc_rank_b200 import api
    from post_hoc_rank_b200 import loraforge as lf
    ys = [torch.empty(p["x"].shape[0], p["d_out"], dtype=torch.bfloat16, device="cuda") for p in st["projections"]]
    api.w4_project([lf.make_w4_projection(p["x"], y, p["q"], p["scales"], st["group"], zeros=p["zeros"], bias=p["bias"])
                    for p, y in zip(st["projections"], ys)])
    return ys


def _own_quant(st):
    from post_hoc_rank_b200 import api
    w4 = api.w4_quantize(st["w"], st["group"], zero_points=st["zeros"])
    out = {"values": api.w4_dequantize(w4, st["w"].dtype), "scales": w4.scales}
    if st["zeros"]:
        out["zeros"] = w4.zeros
    return out


def run(state):
    op = state["op"]
    if op == "route":
        return _own_route(state) if own else _plain_route(state)
    if op == "mix":
        return _own_mix(state) if own else [_plain_mix(state, p) for p in state["projections"]]
    if op == "w4":
        return _own_w4(state) if own else [_plain_w4(state, p) for p in state["projections"]]
    return _own_quant(state) if own else _plain_quant(state)


# ---- what a pass cannot do without ----------------------------------------------------------

def work(case):
    if case["op"] == "route":
        T, E, K = case["T"], case["E"], case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        nbytes = T * E * size + T * K * 8 + (E * 4 if case["bias"] else 0)
        if case["train"]:
            nbytes += T * E * size + T * K * 4      # the gradient, the weights' gradient
        return {"bytes": nbytes, "flops": T * E * (6 if case["train"] else 3)}
    if case["op"] == "mix":
        T, E, K, k = case["T"], case["E"], case["K"], (case["max_rank"] + 1) / 2
        touched = min(E, T * K)
        nbytes, flops = T * K * 8, 0
        for d_in, d_out in _shapes(case["shapes"]):
            nbytes += touched * k * (d_in + d_out) * 2 + T * (d_in + 2 * d_out) * 2
            flops += 2 * T * K * k * (d_in + d_out)
            if case["train"]:
                nbytes += T * (d_in + d_out) * 2 + T * K * 4
                flops += 2 * T * K * k * (d_in + d_out)
        return {"bytes": int(nbytes), "flops": int(flops)}
    if case["op"] == "w4":
        T, nbytes, flops = case["T"], 0, 0
        for d_in, d_out in _shapes(case["shapes"]):
            ng = _groups_of(d_in, case["group"])
            nbytes += d_out * d_in // 2 + d_out * ng * (3 if case["zeros"] else 2) + T * (d_in + d_out) * 2
            flops += 2 * T * d_in * d_out
        return {"bytes": nbytes, "flops": flops}
    n, ng = case["d_in"] * case["d_out"], case["d_out"] * _groups_of(case["d_in"], case["group"])
    size = 4 if case["dtype"] == "f32" else 2
    return {"bytes": 2 * n * size + n // 2 + ng * (3 if case["zeros"] else 2), "flops": 6 * n}


# ---- the definitions in 64 bits -------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "mix": _exact_mix, "w4": _exact_w4, "quant": _exact_quant}[case["op"]](st)


def _exact_route(st):
    l = st["logits"].double()
    T, E, K, G = l.shape[0], st["E"], st["K"], st["groups"]
    rows = torch.arange(T, device=l.device)
    if st["score"] == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True).nan_to_num(neginf=0.0))
        s = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        s = 1 / (1 + torch.exp(-l))
    c = s if st["bias"] is None else s + st["bias"].double()
    shut = l == -math.inf
    if G > 1:
        left = c.masked_fill(shut, -math.inf).view(T, G, -1).clone()
        some = ~torch.isinf(left.amax(2))
        score = torch.zeros(T, G, dtype=torch.float64, device=l.device)
        for _ in range(min(st["group_top"], E // G)):
            m, at = left.max(2)
            score += torch.where(torch.isinf(m), 0.0, m)
            left.scatter_(2, at.unsqueeze(2), -math.inf)
        score = score.masked_fill(~some, -math.inf)
        beats = (score.unsqueeze(1) > score.unsqueeze(2)) | (
            (score.unsqueeze(1) == score.unsqueeze(2)) &
            (torch.arange(G, device=l.device).view(1, 1, G) < torch.arange(G, device=l.device).view(1, G, 1)))
        keep = beats.sum(2) < st["top_groups"]
        shut = shut | ~keep.repeat_interleave(E // G, 1)
    key = (l if st["bias"] is None else c).masked_fill(shut, -math.inf)
    ids, w = [], []
    for _ in range(K):
        best = key.amax(1, keepdim=True)
        at = torch.where(key == best, torch.arange(E, device=l.device), E).amin(1)
        ok = ~torch.isinf(best.squeeze(1))
        ids.append(torch.where(ok, at, -1))
        w.append(torch.where(ok, s[rows, at], 0.0))
        key[rows, at] = -math.inf
    ids, w = torch.stack(ids, 1), torch.stack(w, 1)
    g = torch.where(ids >= 0, st["grad"].double(), 0.0)
    total = w.sum(1, keepdim=True)
    p = torch.where(total > 0, w / total.clamp(min=1e-300), 0.0) if st["renorm"] else w
    out = {"ids": ids.int(), "weights": p}
    if st["train"]:
        d = torch.zeros_like(l)
        for j in range(K):
            on = ids[:, j] >= 0
            at = ids[:, j].clamp(min=0)
            if st["renorm"]:
                v = p[:, j] * (g[:, j] - (p * g).sum(1))
                v = v * (1 - s[rows, at]) if st["score"] == "sigmoid" else v
            else:
                v = p[:, j] * g[:, j]
                v = v * (1 - s[rows, at]) if st["score"] == "sigmoid" else v
            d[rows, at] += torch.where(on, v, 0.0)
        if st["score"] == "softmax" and not st["renorm"]:
            d -= s * (p * g).sum(1, keepdim=True)
        out["dlogits"] = d
    return out


def _exact_mix(st):
    w, outs, dws = st["weights"].double(), [], []
    for p in st["projections"]:
        x, y = p["x"].double(), p["base"].double()
        dx = torch.zeros_like(x)
        dw = torch.zeros_like(w)
        start = 0
        for e, k in enumerate(p["ranks"].tolist()):
            A, B = p["A"][start:start + k].double(), p["Bt"][start:start + k].double()
            start += k
            tok, slot = torch.nonzero(st["ids"] == e, as_tuple=True)
            if not len(tok):
                continue
            t = x[tok] @ A.t()
            y.index_add_(0, tok, 2.0 * w[tok, slot].unsqueeze(1) * (t @ B))
            if st["train"]:
                u = p["grad"][tok].double() @ B.t()
                dx.index_add_(0, tok, 2.0 * w[tok, slot].unsqueeze(1) * (u @ A))
                dw[tok, slot] = 2.0 * (t * u).sum(1)
        outs.append((y, dx) if st["train"] else y)
        dws.append(dw)
    return [(y, dx, sum(dws)) for y, dx in outs] if st["train"] else outs


def _exact_w4(st):
    outs = []
    for p in st["projections"]:
        d_out, d_in, g = p["d_out"], p["d_in"], st["group"]
        w = torch.empty(d_out, d_in, dtype=torch.float64, device=p["q"].device)
        w[:, 0::2] = (p["q"] % 16).double()
        w[:, 1::2] = (p["q"] // 16).double()
        for i in range(_groups_of(d_in, g)):
            part = w[:, i * g:(i + 1) * g]
            part -= 8.0 if p["zeros"] is None else p["zeros"][:, i:i + 1].double()
            part *= p["scales"][:, i:i + 1].double()
        y = torch.nn.functional.linear(p["x"].double(), w)
        outs.append(y if p["bias"] is None else y + p["bias"].double())
    return outs


def _exact_quant(st):
    w, g = st["w"].double(), st["group"]
    back, scales, zeros = torch.empty_like(w), [], []
    for i in range(_groups_of(w.shape[1], g)):
        part = w[:, i * g:(i + 1) * g]
        if st["zeros"]:
            lo, hi = part.amin(1, keepdim=True).clamp(max=0), part.amax(1, keepdim=True).clamp(min=0)
            s = ((hi - lo) / 15).bfloat16().double()
            z = torch.where(s > 0, torch.round(-lo / torch.where(s > 0, s, 1.0)), 0.0).clamp(0, 15)
            zeros.append(z)
        else:
            s = (part.abs().amax(1, keepdim=True) / 7).bfloat16().double()
            z = torch.full_like(s, 8.0)
        code = torch.clamp(torch.round(part / torch.where(s > 0, s, 1.0)) + z, 0, 15)
        back[:, i * g:(i + 1) * g] = (code - z) * s
        scales.append(s)
    out = {"values": back, "scales": torch.cat(scales, 1)}
    if st["zeros"]:
        out["zeros"] = torch.cat(zeros, 1).to(torch.uint8)
    return out
