"""The expert-layer operators as a user calls them: group-limited routing and
its gradient, quantisation to E4M3 with one scale per 128 elements, the products
of block-scaled E4M3 matrices, and the weighted combine with its gradient.

``run`` computes a pass either in its plain form (elementary torch operations in
32 bits, 64 where a rounding or an order is decided) or, with ``own`` true,
through the package's entry points.  Shapes are those of this repository's
workloads: the V3-shaped layer (D=7168, I=2048, 256 experts top-8 in 8 groups),
the fine-grained layer (D=2048, I=1408, 64 experts top-6) and the skewed one
(D=4096, 128 experts top-8)."""
import math

import torch

own = False

BLK = 128            # elements that share a scale
E4M3_MAX = 448.0


def _cdiv(a, b):
    return -(-a // b)


# ------------------------------------------------------------------- cases
def listed():
    return [
        # Routing of one decode step of the V3-shaped layer: latency only.
        dict(name="route_decode_T16_E256", op="route", T=16, E=256, k=8, scores="sigmoid", groups=8, keep=4, top=2,
             renorm=True, scale=2.5, bias=True, dtype="bf16"),
        # ... and of its prefill batch, followed by the grouping of the rows.
        dict(name="route_prefill_T8192_E256", op="route", T=8192, E=256, k=8, scores="sigmoid", groups=8, keep=4, top=2,
             renorm=True, scale=2.5, bias=True, dtype="f32"),
        # Gradient of the skewed layer's plain softmax weights: every logit of a row has one.
        dict(name="route_backward_T16384_E128", op="route_backward", T=16384, E=128, k=8, scores="softmax", groups=1,
             keep=1, top=1, renorm=False, scale=1.0, bias=False, dtype="f32"),
        # Tokens of the fine-grained prefill batch gathered into expert order and quantised.
        dict(name="quantize_gather_24576x2048", op="quantize", kind="gather", T=4096, k=6, K=2048, dtype="bf16"),
        # The gated unit of the V3-shaped experts (one rank of 2), input of the down product.
        dict(name="glu_quantize_32768x2048", op="quantize", kind="glu", R=32768, I=2048),
        # Its gradient over the fine-grained batch.
        dict(name="glu_backward_24576x1408", op="quantize", kind="glu_backward", R=24576, I=1408),
        # Shared expert's gate and up rows for a decode batch: streams the weights.
        dict(name="dense_decode_8x4096x7168", op="matmul", kind="dense", M=8, N=4096, K=7168, out="bf16"),
        # Fine-grained decode step: every expert meets a few rows.
        dict(name="grouped_decode_384_G64", op="matmul", kind="grouped", M=384, G=64, N=2816, K=2048, skew=1.0, out="bf16"),
        # V3-shaped gate/up of one expert-parallel rank of 8 over a prefill batch, ragged groups.
        dict(name="grouped_prefill_8192_G32", op="matmul", kind="grouped", M=8192, G=32, N=4096, K=7168, skew=0.5, out="bf16"),
        # Gradient with respect to the gate/up products' input, fine-grained batch; summed over slots afterwards.
        dict(name="input_gradient_24576_G64", op="matmul", kind="transposed", M=24576, G=64, N=2816, K=2048, skew=0.5, out="f32"),
        # The routed sums of the V3-shaped prefill batch.
        dict(name="combine_8192x8x7168", op="combine", kind="forward", T=8192, k=8, D=7168, dtype="bf16"),
        # Gradient of the fine-grained batch's combine.
        dict(name="combine_backward_4096x6x2048", op="combine", kind="backward", T=4096, k=6, D=2048, dtype="bf16"),
    ]


def _logu(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_backward", "quantize", "quantize", "matmul", "matmul", "matmul", "combine"])
    if op in ("route", "route_backward"):
        groups = rng.choice([1, 1, 2, 4, 8, 5])
        size = rng.randint(2, 512 // groups if groups != 5 else 40)
        E = max(groups * size, 4)
        keep = rng.randint(max(1, groups // 2), groups)
        k = rng.randint(1, min(16, keep * (E // groups)))
        scores = rng.choice(["sigmoid", "softmax"])
        # One renormalised expert weighs `scale` whatever its score: its gradient is zero, with nothing to compare.
        renorm = rng.random() < 0.6 and not (op == "route_backward" and k == 1)
        return dict(op=op, T=_logu(rng, 1, 16384), E=E, k=k, scores=scores, groups=groups, keep=keep,
                    top=rng.choice([1, 2]) if E // groups > 1 else 1, renorm=renorm,
                    scale=round(rng.uniform(0.5, 3.0), 3), bias=rng.random() < 0.5, dtype=rng.choice(["f32", "bf16"]))
    if op == "quantize":
        kind = rng.choice(["gather", "glu", "glu_backward"])
        if kind == "gather":
            return dict(op=op, kind=kind, T=_logu(rng, 1, 4096), k=rng.randint(1, 8), K=16 * _logu(rng, 2, 448),
                        dtype=rng.choice(["bf16", "f32"]))
        return dict(op=op, kind=kind, R=_logu(rng, 1, 24576),
                    I=(16 * _logu(rng, 4, 128) if kind == "glu" else 128 * rng.randint(1, 16)))
    if op == "matmul":
        kind = rng.choice(["dense", "grouped", "transposed"])
        while True:
            G = 1 if kind == "dense" else rng.randint(2, 64)
            c = dict(op=op, kind=kind, M=_logu(rng, 1, 16384), G=G, N=_logu(rng, 64, 4096), K=16 * _logu(rng, 8, 448),
                     skew=round(rng.uniform(0.0, 1.5), 2), out=rng.choice(["bf16", "bf16", "f32"]))
            if kind == "transposed":
                c["N"] = _cdiv(c["N"], 16) * 16
            # No more than the largest listed product, in operations and in weights.
            if c["M"] * c["N"] * c["K"] <= 8192 * 4096 * 7168 and G * c["N"] * c["K"] <= 32 * 4096 * 7168:
                return c
    while True:
        c = dict(op=op, kind=rng.choice(["forward", "backward"]), T=_logu(rng, 1, 8192), k=rng.randint(1, 8),
                 D=8 * _logu(rng, 8, 896), dtype=rng.choice(["bf16", "bf16", "f32"]))
        if c["T"] * c["k"] * c["D"] * (1 if c["kind"] == "forward" else 2) * (2 if c["dtype"] == "f32" else 1) <= 8192 * 8 * 7168:
            return c


# ------------------------------------------------------------------ inputs
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 11)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _grouping(g, T, k, E):
    """A routing of T tokens to k distinct experts of E, in grouped order."""
    idx = torch.rand(T, E, generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    order = torch.argsort(idx.reshape(-1), stable=True)
    row_of_slot = torch.empty(T * k, dtype=torch.int32, device="cuda")
    row_of_slot[order] = torch.arange(T * k, dtype=torch.int32, device="cuda")
    return (order // k).to(torch.int32), row_of_slot.reshape(T, k)


def _codes(v, row_blocks):
    """E4M3 codes (as bytes) and scales of v [..., R, K]: one scale per 128 elements of a row
    (scales [ceil(K/128), R]), or per 128 x 128 where row_blocks."""
    R, K = v.shape[-2:]
    kb, rb = _cdiv(K, BLK), _cdiv(R, BLK)
    v = torch.nn.functional.pad(v, (0, kb * BLK - K, 0, (rb * BLK - R) if row_blocks else 0))
    if row_blocks:
        t = v.reshape(*v.shape[:-2], rb, BLK, kb, BLK)
        s = t.abs().amax(dim=(-3, -1)) / E4M3_MAX
        q = (t / s[..., :, None, :, None]).reshape(v.shape)
    else:
        t = v.reshape(*v.shape[:-1], kb, BLK)
        s = t.abs().amax(dim=-1) / E4M3_MAX
        q = (t / s[..., None]).reshape(v.shape)
    q = q[..., :R, :K].contiguous().to(torch.float8_e4m3fn).view(torch.uint8)
    return q, (s.contiguous() if row_blocks else s.transpose(-1, -2).contiguous())


def _group_sizes(rng, M, G, skew):
    """Rows of each group, ragged: proportional to (rank + 1)^-skew in a seeded order."""
    p = torch.arange(1, G + 1, dtype=torch.float64).pow(-skew)
    p = p[torch.randperm(G, generator=rng)]
    counts = torch.bincount(torch.multinomial(p, M, replacement=True, generator=rng), minlength=G)
    return [int(c) for c in counts]


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    if op in ("route", "route_backward"):
        # Router logits of normalised tokens; the balancing bias of a trained layer is small.
        s = {"c": c, "logits": _randn(g, c["T"], c["E"], dtype=_DT[c["dtype"]]),
             "bias": _randn(g, c["E"]) * 0.05 if c["bias"] else None}
        if op == "route_backward":
            s["idx"], s["w"] = _route_plain(c, s["logits"], s["bias"])
            s["dw"] = _randn(g, c["T"], c["k"])
        return s
    if op == "quantize":
        if c["kind"] == "gather":
            token_of_row, _ = _grouping(g, c["T"], c["k"], max(8, c["k"]))
            # Rows of different sizes, as activations have.
            x = _randn(g, c["T"], c["K"]) * torch.exp(_randn(g, c["T"], 1))
            return {"c": c, "x": x.to(_DT[c["dtype"]]), "token_of_row": token_of_row}
        s = {"c": c, "gu": _randn(g, c["R"], 2 * c["I"], dtype=torch.bfloat16)}
        if c["kind"] == "glu_backward":
            s["dh"] = _randn(g, c["R"], c["I"], dtype=torch.bfloat16)
        return s
    if op == "matmul":
        G, M, N, K = c.get("G", 1), c["M"], c["N"], c["K"]
        con = N if c["kind"] == "transposed" else K
        w, ws = torch.empty(G, N, K, dtype=torch.uint8, device="cuda"), []
        for i in range(G):
            w[i], si = _codes(_randn(g, N, K) * 0.02, True)
            ws.append(si)
        a, sa = _codes(_randn(g, M, con), False)
        s = {"c": c, "a": a, "sa": sa, "w": w, "sw": torch.stack(ws), "offsets": None, "cap": M}
        if c["kind"] != "dense":
            sizes = _group_sizes(torch.Generator().manual_seed(int(seed) + 5), M, G, c["skew"])
            off = [0]
            for n in sizes:
                off.append(off[-1] + n)
            s["offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
            s["cap"] = max(sizes)
        return s
    _, row_of_slot = _grouping(g, c["T"], c["k"], max(8, c["k"]))
    s = {"c": c, "row_of_slot": row_of_slot, "y": _randn(g, c["T"] * c["k"], c["D"], dtype=_DT[c["dtype"]]),
         "w": torch.softmax(_randn(g, c["T"], c["k"]), dim=1)}
    if c["kind"] == "backward":
        s["dout"] = _randn(g, c["T"], c["D"], dtype=torch.bfloat16)
    return s


# ------------------------------------------------------------- plain forms
def _keys(c, logits, bias):
    l = logits.double()
    s = torch.sigmoid(l) if c["scores"] == "sigmoid" else torch.softmax(l, dim=1)
    return s, (s if bias is None else s + bias.double())


def _route_plain(c, logits, bias):
    """Chosen experts and weights; keys in 64 bits, for experts next to each other in order."""
    T, E, G = c["T"], c["E"], c["groups"]
    s, key = _keys(c, logits, bias)
    if G > 1:
        per = key.reshape(T, G, E // G)
        score = per.sort(dim=2, descending=True).values[:, :, :c["top"]].sum(dim=2)
        order = score.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
        kept = torch.zeros(T, G, dtype=torch.bool, device=key.device).scatter_(1, order, True)
        key = torch.where(kept.repeat_interleave(E // G, dim=1), key, -math.inf)
    idx = key.sort(dim=1, descending=True, stable=True).indices[:, :c["k"]]
    w = s.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True)
    return idx.to(torch.int32), (w * c["scale"]).float()


def _group_plain(idx, E):
    T, k = idx.shape
    flat = idx.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=idx.device)
    offsets[1:] = torch.zeros(E, dtype=torch.int64, device=idx.device).scatter_add_(0, flat, torch.ones_like(flat)).cumsum(0)
    row_of_slot = torch.empty(T * k, dtype=torch.int32, device=idx.device)
    row_of_slot[order] = torch.arange(T * k, dtype=torch.int32, device=idx.device)
    return offsets, (order // k).to(torch.int32), row_of_slot.reshape(T, k)


def _route_backward_plain(c, logits, idx, dw):
    l, e = logits.float(), idx.long()
    if c["scores"] == "softmax":
        s = torch.softmax(l, dim=1)
    else:
        s = torch.sigmoid(l)
    sc = s.gather(1, e)
    if c["renorm"]:
        total = sc.sum(dim=1, keepdim=True)
        ds = (dw - (dw * sc).sum(dim=1, keepdim=True) / total) / total
    else:
        ds = dw
    ds = torch.zeros_like(l).scatter(1, e, ds * c["scale"])
    if c["scores"] == "softmax":
        dl = s * (ds - (ds * s).sum(dim=1, keepdim=True))
    else:
        dl = ds * s * (1 - s)
    return dl.to(logits.dtype)


def _quantize_plain(v):
    """v [R, K] fp32 -> E4M3 values and scales [ceil(K/128), R]; the quotient in 64 bits, so that
    a value between two codes is rounded once."""
    R, K = v.shape
    kb = _cdiv(K, BLK)
    t = torch.nn.functional.pad(v, (0, kb * BLK - K)).reshape(R, kb, BLK)
    amax = t.abs().amax(dim=2)
    s = torch.where(amax > 0, (amax.double() / E4M3_MAX).float(), torch.ones_like(amax))
    q = t.double() / s.double()[:, :, None]
    step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
    q = (torch.round(q / step) * step).clamp(-E4M3_MAX, E4M3_MAX)
    return q.reshape(R, kb * BLK)[:, :K].to(torch.float8_e4m3fn), s.t().contiguous()


def _glu_plain(c, gu):
    g, u = gu[:, :c["I"]].float(), gu[:, c["I"]:].float()
    return g * torch.sigmoid(g) * u


def _glu_backward_plain(c, gu, dh):
    g, u, d = gu[:, :c["I"]].float(), gu[:, c["I"]:].float(), dh.float()
    sg = torch.sigmoid(g)
    return torch.cat([d * u * sg * (1 + g * (1 - sg)), d * g * sg], dim=1)


def _wide(codes, scales, row_blocks):
    """The values that codes stand for, in 32 bits."""
    v = codes.view(torch.float8_e4m3fn).float()
    s = scales.repeat_interleave(BLK, dim=-2)[..., :v.shape[-2], :] if row_blocks else scales.t()
    return v * s.repeat_interleave(BLK, dim=-1)[..., :v.shape[-1]]


def _matmul_plain(s):
    c = s["c"]
    a, w = _wide(s["a"], s["sa"], False), _wide(s["w"], s["sw"], True)
    if c["kind"] != "transposed":
        w = w.transpose(1, 2)
    if c["kind"] == "dense":
        return (a @ w[0]).to(_DT[c["out"]])
    # Every group padded to the longest one's rows.
    off, M = s["offsets"].long(), c["M"]
    at = off[:-1, None] + torch.arange(s["cap"], device=a.device)
    inside = at < off[1:, None]
    y = torch.bmm(torch.where(inside[..., None], a[at.clamp(max=M - 1)], 0.0), w)
    row = torch.arange(M, device=a.device)
    group = torch.searchsorted(off[1:], row, right=True)
    return y[group, row - off[group]].to(_DT[c["out"]])


def _combine_plain(s):
    y = s["y"][s["row_of_slot"].long()].float()
    return (y * s["w"][..., None]).sum(dim=1).to(torch.bfloat16)


def _combine_backward_plain(s):
    rows, d = s["row_of_slot"].long(), s["dout"].float()
    dy = torch.empty_like(s["y"])
    dy[rows.reshape(-1)] = (d[:, None, :] * s["w"][..., None]).to(dy.dtype).reshape(-1, d.shape[1])
    return dy, (s["y"][rows].float() * d[:, None, :]).sum(dim=2)


# --------------------------------------------------------------------- run
def _route_args(c):
    return dict(scores=c["scores"], n_groups=c["groups"], topk_groups=c["keep"], group_top=c["top"],
                renormalize=c["renorm"], routed_scale=c["scale"])


def run(state):
    s, c = state, state["c"]
    op = c["op"]
    if own:
        import deterministic_expert_b200 as moe
    if op == "route":
        if own:
            idx, w = moe.route(s["logits"], c["k"], bias=s["bias"], **_route_args(c))
            off, tok, row = moe.group_rows(idx, c["E"])
        else:
            idx, w = _route_plain(c, s["logits"], s["bias"])
            off, tok, row = _group_plain(idx, c["E"])
        return {"idx": idx, "w": w, "offsets": off, "token_of_row": tok, "row_of_slot": row}
    if op == "route_backward":
        if own:
            return {"dlogits": moe.route_backward(s["logits"], s["idx"], s["dw"], **_route_args(c))}
        return {"dlogits": _route_backward_plain(c, s["logits"], s["idx"], s["dw"])}
    if op == "quantize":
        if own:
            if c["kind"] == "gather":
                q, sc = moe.quantize_rows_fp8(s["x"], token_of_row=s["token_of_row"])
            elif c["kind"] == "glu":
                q, sc = moe.glu_quantize_fp8(s["gu"])
            else:
                q, sc = moe.glu_backward_quantize_fp8(s["gu"], s["dh"])
            return {"codes": q.view(torch.float8_e4m3fn), "scales": sc}
        if c["kind"] == "gather":
            q, sc = _quantize_plain(s["x"][s["token_of_row"].long()].float())
        elif c["kind"] == "glu":
            q, sc = _quantize_plain(_glu_plain(c, s["gu"]))
        else:
            q, sc = _quantize_plain(_glu_backward_plain(c, s["gu"], s["dh"]))
        return {"codes": q, "scales": sc}
    if op == "matmul":
        if own:
            return {"out": moe.matmul_fp8(s["a"], s["sa"], s["w"], s["sw"], offsets=s["offsets"],
                                          transposed=c["kind"] == "transposed", out_dtype=_DT[c["out"]])}
        return {"out": _matmul_plain(s)}
    if c["kind"] == "forward":
        if own:
            return {"out": moe.combine_rows(s["y"], s["row_of_slot"], s["w"])}
        return {"out": _combine_plain(s)}
    if own:
        dy, dw = moe.combine_rows_backward(s["dout"], s["y"], s["row_of_slot"], s["w"])
    else:
        dy, dw = _combine_backward_plain(s)
    return {"dy": dy, "dw": dw}


# -------------------------------------------------------------------- work
def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        # Logits in; experts and weights out; the grouping reads the experts once and writes two tables.
        return {"bytes": T * E * size[c["dtype"]] + (4 * E if c["bias"] else 0) + T * k * (8 + 4 + 8) + 4 * (E + 1),
                "flops": 4.0 * T * E}
    if c["op"] == "route_backward":
        T, E, k = c["T"], c["E"], c["k"]
        # Only softmax weights over all experts need the other experts' logits.
        whole = c["scores"] == "softmax" and not c["renorm"]
        read = T * E * size[c["dtype"]] if whole else T * k * size[c["dtype"]]
        return {"bytes": read + T * k * 8 + T * E * size[c["dtype"]], "flops": 4.0 * T * (E if whole else k)}
    if c["op"] == "quantize":
        if c["kind"] == "gather":
            R, K = c["T"] * c["k"], c["K"]
            return {"bytes": c["T"] * K * size[c["dtype"]] + 4 * R + R * K + 4 * R * _cdiv(K, BLK), "flops": 2.0 * R * K}
        R, I = c["R"], c["I"]
        if c["kind"] == "glu":
            return {"bytes": R * 2 * I * 2 + R * I + 4 * R * _cdiv(I, BLK), "flops": 6.0 * R * I}
        return {"bytes": R * 3 * I * 2 + R * 2 * I + 4 * R * _cdiv(2 * I, BLK), "flops": 12.0 * R * I}
    if c["op"] == "matmul":
        G, M, N, K = c.get("G", 1), c["M"], c["N"], c["K"]
        con, outw = (N, K) if c["kind"] == "transposed" else (K, N)
        met = min(G, M)       # groups that can have rows: the others' weights are not needed
        return {"bytes": M * con + 4 * M * _cdiv(con, BLK) + met * (N * K + 4 * _cdiv(N, BLK) * _cdiv(K, BLK))
                + M * outw * size[c["out"]], "flops": 2.0 * M * N * K}
    T, k, D, b = c["T"], c["k"], c["D"], size[c["dtype"]]
    if c["kind"] == "forward":
        return {"bytes": T * k * D * b + T * k * 8 + T * D * 2, "flops": 2.0 * T * k * D}
    return {"bytes": T * k * D * 2 * b + T * D * 2 + T * k * 12, "flops": 3.0 * T * k * D}


# ------------------------------------------------------------------- exact
def _exact_route(c, s):
    l = s["logits"].double()
    e = torch.exp(l - l.max(dim=1, keepdim=True).values)
    sc = 1 / (1 + torch.exp(-l)) if c["scores"] == "sigmoid" else e / e.sum(dim=1, keepdim=True)
    key = sc.clone() if s["bias"] is None else sc + s["bias"].double()
    T, E, G = c["T"], c["E"], c["groups"]
    n = E // G
    if G > 1:
        a = key.reshape(T, G, n)
        score = a.max(dim=2).values
        if c["top"] == 2:
            first = a.argmax(dim=2, keepdim=True)
            score = score + a.scatter(2, first, -math.inf).max(dim=2).values
        better = (score[:, None, :] > score[:, :, None]).sum(dim=2)
        earlier = torch.ones(G, G, device=l.device).tril(-1).bool()
        better = better + ((score[:, None, :] == score[:, :, None]) & earlier).sum(dim=2)
        key = key.masked_fill((better >= c["keep"]).repeat_interleave(n, dim=1), -math.inf)
    idx = torch.empty(T, c["k"], dtype=torch.int64, device=l.device)
    for j in range(c["k"]):
        top = key.max(dim=1, keepdim=True).values
        idx[:, j] = (key == top).int().argmax(dim=1)
        key.scatter_(1, idx[:, j:j + 1], -math.inf)
    w = sc.gather(1, idx) * c["scale"]
    return idx.to(torch.int32), w / sc.gather(1, idx).sum(dim=1, keepdim=True) if c["renorm"] else w


def _exact_quantize(v):
    R, K = v.shape
    codes, scales = [], []
    grid = torch.tensor([m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1],
                        dtype=torch.float64, device=v.device)
    mid = (grid[1:] + grid[:-1]) / 2
    for b in range(0, K, BLK):
        x = v[:, b:b + BLK]
        amax = x.abs().max(dim=1).values
        sc = torch.where(amax > 0, amax.float().double() / E4M3_MAX, torch.ones_like(amax)).float()
        q = (x / sc.double()[:, None]).abs()
        lo, hi = torch.searchsorted(mid, q, right=False), torch.searchsorted(mid, q, right=True)
        i = torch.where(lo == hi, lo, torch.where(lo % 2 == 0, lo, hi))     # a tie: the even code
        codes.append(torch.copysign(grid[i], x))
        scales.append(sc.double())
    return torch.cat(codes, dim=1), torch.stack(scales)


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "route":
        idx, w = _exact_route(c, s)
        return {"idx": idx, "w": w, "offsets": None, "token_of_row": None, "row_of_slot": None}
    if c["op"] == "route_backward":
        with torch.enable_grad():
            l = s["logits"].double().requires_grad_(True)
            p = torch.sigmoid(l) if c["scores"] == "sigmoid" else torch.exp(torch.log_softmax(l, dim=1))
            w = p.gather(1, s["idx"].long())
            if c["renorm"]:
                w = w / w.sum(dim=1, keepdim=True)
            (w * s["dw"].double()).sum().mul(c["scale"]).backward()
        return {"dlogits": l.grad}
    if c["op"] == "quantize":
        if c["kind"] == "gather":
            v = s["x"].double()[s["token_of_row"].long()]
        else:
            with torch.enable_grad():
                gu = s["gu"].double().requires_grad_(True)
                v = torch.nn.functional.silu(gu[:, :c["I"]]) * gu[:, c["I"]:]
                if c["kind"] == "glu_backward":
                    v.backward(s["dh"].double())
                    v = gu.grad
            v = v.detach()
        q, sc = _exact_quantize(v)
        return {"codes": q, "scales": sc}
    if c["op"] == "matmul":
        off = [0, c["M"]] if s["offsets"] is None else s["offsets"].tolist()
        a = s["a"].view(torch.float8_e4m3fn).double()
        sa = s["sa"].double().t()
        outs = []
        for i in range(len(off) - 1):
            w = s["w"][i].view(torch.float8_e4m3fn).double()
            sw = s["sw"][i].double()
            w = w * sw.repeat_interleave(BLK, 0)[:w.shape[0]].repeat_interleave(BLK, 1)[:, :w.shape[1]]
            x = a[off[i]:off[i + 1]] * sa[off[i]:off[i + 1]].repeat_interleave(BLK, 1)[:, :a.shape[1]]
            outs.append(x @ (w if c["kind"] == "transposed" else w.t()))
        return {"out": torch.cat(outs)}
    rows = s["row_of_slot"].long()
    if c["kind"] == "forward":
        out = torch.zeros(c["T"], c["D"], dtype=torch.float64, device="cuda")
        for j in range(c["k"]):
            out += s["w"][:, j:j + 1].double() * s["y"][rows[:, j]].double()
        return {"out": out}
    dy = torch.empty(c["T"] * c["k"], c["D"], dtype=torch.float64, device="cuda")
    dw = torch.empty(c["T"], c["k"], dtype=torch.float64, device="cuda")
    for j in range(c["k"]):
        dy[rows[:, j]] = s["w"][:, j:j + 1].double() * s["dout"].double()
        dw[:, j] = torch.einsum("td,td->t", s["dout"].double(), s["y"][rows[:, j]].double())
    return {"dy": dy, "dw": dw}
