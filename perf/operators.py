"""Cases of the mixture-of-experts and weight-only FP4 operators: what a user's program holds before
each call, the call itself, its plain form in elementary torch operations, and its values in 64 bits.

Operators:
  sort           slots (token, choice) sorted by expert, with the inverse and the experts' offsets
  gather         token rows copied into expert order (dropped slots give zero rows); its gradient
  combine        expert rows summed back per token with the router's weights; its gradient
  linear         y = x . W^T with bf16 / float32 activations and block-scaled FP4 weights
  expert_linear  the same product for rows in expert order, each with its expert's weight

Sizes come from the repository's 8B layer set (hidden 4096, gate+up 28672, down 14336 -> 4096, qkv 6144) and are
otherwise generic.
"""
import math

import torch

own = False

HIDDEN, FFN = 4096, 14336
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decode step of 16 sequences, two experts of eight each: launch latency is everything
        dict(name="sort_decode", op="sort", tokens=16, topk=2, experts=8, drop=0.0),
        # a training micro-batch with many small experts, a few slots dropped by a capacity limit
        dict(name="sort_train", op="sort", tokens=32768, topk=8, experts=128, drop=0.02),
        # dispatch of one 8192-token micro-batch at the 8B layer's width
        dict(name="gather_train", op="gather", tokens=8192, topk=2, experts=8, drop=0.0, hidden=HIDDEN, dtype="bf16"),
        # gradient of a ragged float32 dispatch whose width is not a multiple of the vector length
        dict(name="gather_grad_odd", op="gather_grad", tokens=2047, topk=4, experts=16, drop=0.05, hidden=1001,
             dtype="f32"),
        # a decode batch's return from its experts
        dict(name="combine_decode", op="combine", tokens=33, topk=8, experts=64, drop=0.0, hidden=HIDDEN, dtype="bf16"),
        # backward of the return for one 8192-token micro-batch: gradients of the rows and of the router's weights
        dict(name="combine_grad_train", op="combine_grad", tokens=8192, topk=2, experts=8, drop=0.01, hidden=HIDDEN,
             dtype="bf16"),
        # one new token through the output projection
        dict(name="linear_token", op="linear", rows=1, k=HIDDEN, n=HIDDEN, fmt="e8m0", block=32, layout="1d",
             dtype="bf16"),
        # a few sequences' new tokens through gate+up, weights in 16x16 tiles as trained
        dict(name="linear_batch", op="linear", rows=5, k=HIDDEN, n=28672, fmt="ue5m3", block=16, layout="2d",
             dtype="bf16"),
        # float32 gradient of a short sequence through the transposed view of the down projection
        dict(name="linear_dgrad_f32", op="linear", rows=77, k=HIDDEN, n=FFN, fmt="e4m3", block=16, layout="2dT",
             dtype="f32"),
        # a prompt through qkv
        dict(name="linear_prompt", op="linear", rows=2048, k=HIDDEN, n=6144, fmt="ue5m3", block=16, layout="1d",
             dtype="bf16"),
        # a decode step's few rows through their experts
        dict(name="experts_decode", op="expert_linear", tokens=8, topk=2, experts=8, drop=0.0, k=HIDDEN, n=FFN,
             fmt="ue5m3", block=16, layout="1d", dtype="bf16"),
        # a prompt's rows through eight experts, unevenly routed
        dict(name="experts_prompt", op="expert_linear", tokens=4096, topk=2, experts=8, drop=0.0, k=HIDDEN, n=FFN,
             fmt="e8m0", block=32, layout="1d", dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _log_of(rng, lo, hi, step):
    return step * _log(rng, max(1, lo // step), hi // step)


def draw(rng):
    most_bytes = work(dict(listed()[5]))["bytes"]
    most_flops = work(dict(listed()[-1]))["flops"]
    while True:
        op = rng.choice(["sort", "gather", "gather_grad", "combine", "combine_grad", "linear", "linear", "expert_linear",
                         "expert_linear"])
        c = dict(op=op)
        if op != "linear":
            c.update(topk=rng.choice([1, 2, 3, 4, 6, 8]), drop=rng.choice([0.0, 0.0, 0.03, 0.3]))
            c["experts"] = _log(rng, max(2, c["topk"]), 256)
        if op == "sort":
            c["tokens"] = _log(rng, 1, 32768)
            return c
        c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        if op in ("gather", "gather_grad", "combine", "combine_grad"):
            c["tokens"] = _log(rng, 1, 16384)
            c["hidden"] = rng.choice([_log(rng, 33, 8192), _log_of(rng, 64, 8192, 8)])
            if work(c)["bytes"] <= most_bytes:
                return c
            continue
        c["fmt"] = rng.choice(["ue5m3", "e4m3", "e8m0"])
        c["block"] = 32 if c["fmt"] == "e8m0" else rng.choice([16, 16, 32])
        c["layout"] = rng.choice(["1d", "2d", "2dT"]) if c["block"] == 16 else "1d"
        c["k"] = _log_of(rng, 64, 16384, 64)
        c["n"] = _log_of(rng, 64, 28672, 16) if c["layout"] != "1d" else _log(rng, 33, 28672)
        if op == "linear":
            c["rows"] = _log(rng, 1, 4096)
            if work(c)["flops"] <= most_flops and c["n"] * c["k"] <= 28672 * 4096:
                return c
        else:
            c["experts"] = min(c["experts"], 64)
            c["tokens"] = _log(rng, 1, 4096)
            # the plain form multiplies every row by every expert's weight
            if (work(c)["flops"] * c["experts"] <= 8 * most_flops
                    and c["experts"] * c["n"] * c["k"] <= 8 * FFN * HIDDEN):
                return c


def _scale_bytes(c):
    return c["n"] * c["k"] // (256 if c["layout"] != "1d" else c["block"])


def work(case):
    c = case
    op = c["op"]
    if op != "linear":
        n = c["tokens"] * c["topk"]
    if op == "sort":
        return {"bytes": 4.0 * (3 * n + c["experts"] + 1), "flops": 0.0}
    e = 2 if c["dtype"] == "bf16" else 4
    if op in ("gather", "gather_grad", "combine", "combine_grad"):
        rows = c["tokens"] + n * (2 if op == "combine_grad" else 1)
        extra = {"combine": 4 * n, "combine_grad": 8 * n}.get(op, 0)
        flops = {"gather": 0, "gather_grad": n, "combine": 2 * n, "combine_grad": 3 * n}[op] * c["hidden"]
        return {"bytes": float(rows * c["hidden"] * e + 4 * n + extra), "flops": float(flops)}
    weight = c["n"] * c["k"] // 2 + _scale_bytes(c)
    if op == "linear":
        rows, hit = c["rows"], 1.0
    else:
        rows = n
        hit = c["experts"] * (1.0 - (1.0 - min(1.0, c["topk"] / c["experts"])) ** c["tokens"])
    return {"bytes": float(hit * weight + rows * (c["k"] + c["n"]) * e), "flops": 2.0 * rows * c["n"] * c["k"]}


# ------------------------------------------------------------------ inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _activations(g, rows, width, dtype):
    """Heavy-tailed rows (Student-t, three degrees of freedom) with four outlier channels."""
    x = _randn(g, rows, width)
    x = x * torch.rsqrt((_randn(g, rows, width).square() + _randn(g, rows, width).square()
                         + _randn(g, rows, width).square()) / 3 + 1e-3)
    cols = torch.randint(0, width, (4,), generator=g, device="cuda")
    x[:, cols] *= 20.0
    return x.to(dtype)


def _router(g, tokens, topk, experts, drop):
    """Expert choices of an unevenly loaded router, best first, and their renormalised probabilities."""
    p = torch.softmax(_randn(g, tokens, experts) + 0.5 * _randn(g, 1, experts), dim=1)
    w, ids = torch.topk(p, topk, dim=1)
    if drop > 0:
        ids = torch.where(torch.rand(tokens, topk, generator=g, device="cuda") < drop, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32).contiguous(), (w / w.sum(dim=1, keepdim=True)).contiguous()


def _scale_table(fmt):
    """The scale formats' values by code, ascending (UE5M3 0..0xF7, E4M3 0..0x7E)."""
    bias, codes = (15, 0xF8) if fmt == "ue5m3" else (7, 0x7F)
    return torch.tensor([(c & 7) * 2.0 ** (-2 - bias) if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - bias)
                         for c in range(codes)], dtype=torch.float32, device="cuda")


def _quantize(w, fmt, block, layout):
    """A float32 weight [n, k] as packed codes, scale codes and tensor scale of the given format."""
    n, k = w.shape
    if layout == "1d":
        amax = w.abs().view(n, k // block, block).amax(dim=2)
    else:
        amax = w.abs().view(n // 16, 16, k // 16, 16).amax(dim=3).amax(dim=1)
    if fmt == "e8m0":
        code = (torch.floor(torch.log2(amax.clamp_min(1e-30))) - 2 + 127).clamp(0, 254)
        enc, g = torch.exp2(127 - code), torch.ones(1, device="cuda")
    else:
        table = _scale_table(fmt)
        a = amax.max()
        code = torch.bucketize(amax * (448.0 / a), (table[1:] + table[:-1]) / 2).clamp_min(1)
        enc, g = 6.0 * 448.0 / a / table[code], (a / (6.0 * 448.0)).view(1)
    enc = enc.repeat_interleave(block, dim=1)
    if layout != "1d":
        enc = enc.repeat_interleave(16, dim=0)
    v = w * enc
    values = torch.tensor(E2M1, device="cuda")
    q = torch.bucketize(v.abs(), (values[1:] + values[:-1]) / 2).to(torch.uint8)
    q |= (v < 0).to(torch.uint8) << 3
    if layout == "2dT":
        q = q.t().contiguous()
    return (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous(), code.to(torch.uint8).contiguous(), g


def _weights(g, c, count):
    """`count` quantized weights [n, k], stacked: payload, scale codes, tensor scales."""
    shape = (c["k"], c["n"]) if c["layout"] == "2dT" else (c["n"], c["k"])   # the weight whose transpose is held
    parts = [_quantize(0.02 * _randn(g, *shape), c["fmt"], c["block"], c["layout"]) for _ in range(count)]
    return torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]), torch.cat([p[2] for p in parts])


def _plain_plan(ids, experts):
    flat = ids.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < experts), flat, torch.full_like(flat, experts))
    key, order = torch.sort(key, stable=True)
    at = torch.arange(flat.numel(), device=ids.device)
    at = torch.where(key < experts, at, -1 - at)
    pos = torch.empty_like(order)
    pos[order] = at
    offsets = torch.searchsorted(key, torch.arange(experts + 1, device=ids.device))
    return order.to(torch.int32), pos.to(torch.int32).view(ids.shape), offsets.to(torch.int32)


def prepare(case, seed):
    c = case
    g = _gen(seed)
    s = {"c": c}
    if c["op"] != "linear":
        s["ids"], s["w"] = _router(g, c["tokens"], c["topk"], c["experts"], c["drop"])
        if own:
            import fp4_block_scaled_tensor_amd as fp4
            s["fp4"] = fp4
            if c["op"] != "sort":
                s["plan"] = fp4.expert_sort(s["ids"], c["experts"])
        if c["op"] != "sort":
            s["order"], s["pos"], s["offsets"] = _plain_plan(s["ids"], c["experts"])
    if c["op"] == "sort":
        return s
    dt = DTYPES[c["dtype"]]
    if c["op"] in ("gather", "gather_grad", "combine", "combine_grad"):
        n, h = c["tokens"] * c["topk"], c["hidden"]
        if c["op"] == "gather":
            s["x"] = _activations(g, c["tokens"], h, dt)
        elif c["op"] == "gather_grad":
            s["dxs"] = (1e-3 * _randn(g, n, h)).to(dt)
        else:
            s["ys"] = _activations(g, n, h, dt)
            if c["op"] == "combine_grad":
                s["dy"] = (1e-3 * _randn(g, c["tokens"], h)).to(dt)
        return s
    count = c["experts"] if c["op"] == "expert_linear" else 1
    rows = c["rows"] if c["op"] == "linear" else c["tokens"] * c["topk"]
    s["x"] = _activations(g, rows, c["k"], dt)
    q, sc, gs = _weights(g, c, count)
    if own:
        import fp4_block_scaled_tensor_amd as fp4
        s["fp4"] = fp4
        fmt = {"ue5m3": fp4.UE5M3, "e4m3": fp4.E4M3, "e8m0": fp4.E8M0}[c["fmt"]]
        layout = {"1d": fp4.FP4_SCALES_1D, "2d": fp4.FP4_SCALES_2D, "2dT": fp4.FP4_SCALES_2D_T}[c["layout"]]
        each = [fp4.QTensor(q[e], sc[e], gs[e:e + 1].clone(), fmt, c["block"], layout, c["n"], c["k"])
                for e in range(count)]
        s["weight"] = fp4.stack_experts(each) if c["op"] == "expert_linear" else each[0]
    else:
        s["q"], s["s"], s["g"] = q, sc, gs
    return s


# ------------------------------------------------------------------ the plain forms

def _plain_weight(s, e):
    """Expert e's weight in float32 [n, k]."""
    c = s["c"]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device="cuda")
    q = s["q"][e]
    w = table[torch.stack([q & 15, q >> 4], dim=2).long()].view(c["n"], c["k"])
    code = s["s"][e].long()
    if c["fmt"] == "e8m0":
        sc = torch.exp2((code - 127).float())
    else:
        bias = 15 if c["fmt"] == "ue5m3" else 7
        m, ex = (code & 7).float(), (code >> 3).float()
        sc = torch.where(code < 8, m * 2.0 ** (-2 - bias), (1 + m / 8) * torch.exp2(ex - bias))
    if c["layout"] == "2dT":
        sc = sc.t()
    if c["layout"] != "1d":
        sc = sc.repeat_interleave(16, dim=0)
    return w * sc.repeat_interleave(c["block"], dim=1) * s["g"][e]


def _run_plain(s):
    c = s["c"]
    op = c["op"]
    if op == "sort":
        order, pos, offsets = _plain_plan(s["ids"], c["experts"])
        return {"order": order, "pos": pos, "offsets": offsets}
    if op == "linear":
        return (s["x"].float() @ _plain_weight(s, 0).t()).to(s["x"].dtype)
    at = torch.arange(s["order"].numel(), device="cuda")
    live = (at < s["offsets"][-1])[:, None]
    slot = s["order"].long()
    if op == "expert_linear":
        x = s["x"].float()
        y = torch.zeros(x.shape[0], c["n"], device="cuda")
        for e in range(c["experts"]):
            mine = (at >= s["offsets"][e]) & (at < s["offsets"][e + 1])
            y = torch.where(mine[:, None], x @ _plain_weight(s, e).t(), y)
        return y.to(s["x"].dtype)
    if op == "gather":
        x = s["x"].float()
        return torch.where(live, x[slot // c["topk"]], torch.zeros((), device="cuda")).to(s["x"].dtype)
    kept = (s["pos"] >= 0)[:, :, None]
    pos = torch.where(s["pos"] >= 0, s["pos"], torch.zeros_like(s["pos"])).long()
    if op == "gather_grad":
        rows = torch.where(kept, s["dxs"].float()[pos], torch.zeros((), device="cuda"))
        return rows.sum(dim=1).to(s["dxs"].dtype)
    rows = torch.where(kept, s["ys"].float()[pos], torch.zeros((), device="cuda"))
    if op == "combine":
        return (rows * s["w"][:, :, None]).sum(dim=1).to(s["ys"].dtype)
    dy = s["dy"].float()
    dys = torch.where(live, s["w"].view(-1)[slot][:, None] * dy[slot // c["topk"]], torch.zeros((), device="cuda"))
    return {"dys": dys.to(s["ys"].dtype), "dw": (rows * dy[:, None, :]).sum(dim=2)}


def run(state):
    s = state
    if not own:
        return _run_plain(s)
    fp4, op = s["fp4"], s["c"]["op"]
    if op == "sort":
        p = fp4.expert_sort(s["ids"], s["c"]["experts"])
        return {"order": p.order, "pos": p.pos, "offsets": p.offsets}
    if op == "gather":
        return fp4.expert_gather(s["x"], s["plan"])
    if op == "gather_grad":
        return fp4.expert_gather_grad(s["dxs"], s["plan"])
    if op == "combine":
        return fp4.expert_combine(s["ys"], s["w"], s["plan"])
    if op == "combine_grad":
        dys, dw = fp4.expert_combine_grad(s["dy"], s["ys"], s["w"], s["plan"])
        return {"dys": dys, "dw": dw}
    if op == "linear":
        return fp4.linear(s["x"], s["weight"])
    return fp4.expert_linear(s["x"], s["weight"], s["plan"])


# ------------------------------------------------------------------ the values in 64 bits

def _exact_weight(c, q, code, g):
    """One weight in float64 from the formats' definitions: sign, exponent and mantissa of each code."""
    q = torch.stack([q & 15, q >> 4], dim=-1).reshape(c["n"], c["k"]).to(torch.int64)
    ex, man = (q >> 1) & 3, (q & 1).double()
    v = torch.where(ex == 0, man * 0.5, torch.ldexp(1 + man * 0.5, ex - 1))
    v = torch.where(q >= 8, -v, v)
    code = code.to(torch.int64)
    one = torch.ones((), dtype=torch.float64, device="cuda")
    if c["fmt"] == "e8m0":
        sc = torch.ldexp(one, code - 127)
    else:
        bias = {"ue5m3": 15, "e4m3": 7}[c["fmt"]]
        e, m = code >> 3, (code & 7).double() / 8
        sc = torch.where(e == 0, torch.ldexp(m, torch.full_like(e, 1 - bias)), torch.ldexp(1 + m, e - bias))
    if c["layout"] == "1d":
        return (v.view(c["n"], -1, c["block"]) * sc[:, :, None]).view(c["n"], c["k"]) * g.double()
    grid = sc.t() if c["layout"] == "2dT" else sc
    v = v.view(c["n"] // 16, 16, c["k"] // 16, 16) * grid[:, None, :, None]
    return v.reshape(c["n"], c["k"]) * g.double()


def exact(case, seed):
    global own
    c, held = case, own
    own = False
    try:
        s = prepare(c, seed)
    finally:
        own = held
    op = c["op"]
    if op == "linear":
        return s["x"].double() @ _exact_weight(c, s["q"][0], s["s"][0], s["g"][0]).t()
    ids = s["ids"].reshape(-1).cpu().tolist()
    n, k, experts = len(ids), c["topk"], c["experts"]
    # slots bucket by bucket, the dropped ones last
    buckets = [[] for _ in range(experts + 1)]
    for i, e in enumerate(ids):
        buckets[e if 0 <= e < experts else experts].append(i)
    order = [i for b in buckets for i in b]
    ends = [0]
    for b in buckets[:experts]:
        ends.append(ends[-1] + len(b))
    kept = ends[-1]
    if op == "sort":
        pos = [0] * n
        for p, i in enumerate(order):
            pos[i] = p if p < kept else ~p
        as_int = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")   # noqa: E731
        return {"order": as_int(order), "pos": as_int(pos).view(c["tokens"], k), "offsets": as_int(ends)}
    if op == "expert_linear":
        y = torch.zeros(n, c["n"], dtype=torch.float64, device="cuda")
        for e in range(experts):
            if ends[e + 1] > ends[e]:
                w = _exact_weight(c, s["q"][e], s["s"][e], s["g"][e])
                y[ends[e]:ends[e + 1]] = s["x"][ends[e]:ends[e + 1]].double() @ w.t()
        return y
    live = torch.tensor(order[:kept], dtype=torch.int64, device="cuda")
    token = live // k
    if op == "gather":
        xs = torch.zeros(n, c["hidden"], dtype=torch.float64, device="cuda")
        xs[:kept] = s["x"].double()[token]
        return xs
    if op == "gather_grad":
        dx = torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device="cuda")
        return dx.index_add_(0, token, s["dxs"][:kept].double())
    ys, w = s["ys"][:kept].double(), s["w"].view(-1)[live].double()
    if op == "combine":
        y = torch.zeros(c["tokens"], c["hidden"], dtype=torch.float64, device="cuda")
        return y.index_add_(0, token, ys * w[:, None])
    dy = s["dy"].double()[token]
    dys = torch.zeros(n, c["hidden"], dtype=torch.float64, device="cuda")
    dys[:kept] = w[:, None] * dy
    dw = torch.zeros(n, dtype=torch.float64, device="cuda")
    dw[live] = (ys * dy).sum(dim=1)
    return {"dys": dys, "dw": dw.view(c["tokens"], k)}
