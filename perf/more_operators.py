"""Cases of the routing steps' gradients and of the experts' products with 4-bit weights, and their plain forms.

A pass is one call on the receive layout that the dispatch writes: rank d's
region holds rows [d*cap, (d+1)*cap), grouped by expert and, inside an
expert, ordered by token; pos[g][k] is the row of token g's k-th expert, -1 for
a pair that its rank's region had no room for.  Operations:

* combine_grad   of out[g] = sum_k w[g][k] y[pos[g][k]]: dy[pos[g][k]] = w[g][k] dout[g] and
                 dw[g][k] = <dout[g], y[pos[g][k]]>, 0 for a dropped pair
* dispatch_grad  of packed[pos[g][k]] = x[g]: dx[g] = add[g] + sum_k dpacked[pos[g][k]]
* route_grad     of the top-k weights with respect to the logits and the bias that is added to them
* w4             y[p] = x[p] w[e]^T with w[e][f][k] = r[e][f] s[e][k/group][f] q[e][f][k]: q whole numbers of
                 4 bits, s e4m3, r f32
* w4_swiglu      g|u = x[p] w[e]^T, y = silu(g) * u
"""
import torch

own = False

FILL = 0.5  # what rows without a token hold before the call, and after it


def listed():
    comb = dict(op="combine_grad", skew=0.0)
    disp = dict(op="dispatch_grad", skew=0.0)
    route = dict(op="route_grad", renorm=True, bias="none")
    w4 = dict(y="bf16", skew=0.0, cap=0)
    return [
        # a small batch: 256 tokens, 2 of 16 experts
        dict(comb, name="combine_grad small", N=4, T=64, E=16, R=2, H=1024, y="bf16", cap=0),
        # a training step of 8192 tokens, 8 of 128 experts, regions a quarter larger than the mean
        dict(comb, name="combine_grad train", N=4, T=2048, E=128, R=8, H=4096, y="bf16", cap=20480),
        # odd sizes in f32, skewed so that the first rank is over its capacity and pairs are dropped
        dict(comb, name="combine_grad odd f32 over capacity", N=2, T=511, E=10, R=3, H=1048, y="f32", cap=1200, skew=1.0),
        # a small batch without another gradient to add
        dict(disp, name="dispatch_grad small", N=4, T=64, E=16, R=2, H=1024, x="bf16", add=False, cap=0),
        # a training step of 8192 tokens, 8 of 256 experts, added to the shared expert's and the router's part
        dict(disp, name="dispatch_grad train", N=4, T=2048, E=256, R=8, H=7168, x="bf16", add=True, cap=20480),
        # a prefill-sized batch, softmax over the chosen 8 of 128 experts
        dict(route, name="route_grad softmax renorm", N=4, T=4096, E=128, R=8, score="softmax"),
        # a training step of 65536 tokens, 8 of 256 experts by sigmoid scores, a bias in the selection alone
        dict(route, name="route_grad sigmoid selection bias", N=32, T=2048, E=256, R=8, score="sigmoid", bias="select"),
        # softmax over all of an odd number of experts, a learned bias with its gradient
        dict(route, name="route_grad softmax bias", N=3, T=1367, E=93, R=4, score="softmax", renorm=False, bias="logit"),
        # one matrix and one token: the plain matrix-vector product of a dense layer
        dict(w4, name="w4 dense one token", op="w4", N=1, T=1, E=1, R=1, K=7168, F=4096, group=128),
        # first product of a single token: 8 of a rank's 64 experts, bound by their weights
        dict(w4, name="w4_swiglu one token", op="w4_swiglu", N=1, T=1, E=64, R=8, K=7168, F=2048, group=32),
        # second product of a decode batch: about 128 rows per expert
        dict(w4, name="w4 decode", op="w4", N=8, T=128, E=64, R=8, K=2048, F=7168, group=32, cap=1408),
        # odd sizes, skewed so that some experts get few rows, f32 results for an f32 combine
        dict(w4, name="w4 odd f32", op="w4", N=2, T=37, E=6, R=3, K=1056, F=776, group=32, skew=0.7, y="f32"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["combine_grad", "dispatch_grad", "route_grad", "w4", "w4_swiglu"])
    n = rng.choice([1, 2, 4, 8])
    skew = rng.choice([0.0, 0.0, 0.7, 2.0])
    if op == "route_grad":
        e = n * log(2 if n == 1 else 1, 1024 // n)
        renorm = rng.random() < 0.5
        r = rng.randint(2 if renorm else 1, min(16, e))  # the weight of one expert alone, renormalised, is constant
        t = log(1, 32768 // n)
        while n * t * e > 16 << 20 and t > 1:
            t //= 2
        return dict(op=op, N=n, T=t, E=e, R=r, score=rng.choice(["softmax", "sigmoid"]), renorm=renorm,
                    bias=rng.choice(["none", "select", "logit"]))
    e = n * log(1, (64 if op.startswith("w4") else 256) // n)
    r = rng.randint(1, min(8, e))
    t = log(1, (2048 if op.startswith("w4") else 8192) // n)
    # about 1.5 times a rank's mean share of the rows where there are several ranks; the bound otherwise
    small = rng.random() < 0.5
    if op.startswith("w4"):
        group = rng.choice([32, 64, 128])
        k, f = group * log(1, 7168 // group), 8 * log(4, 512)
        while 2 * n * t * r * k * f * (2 if op == "w4_swiglu" else 1) > 2.4e11 and t > 1:
            t //= 2
        return dict(op=op, N=n, T=t, E=e, R=r, K=k, F=f, group=group, cap=(3 * t * r) // 2 + 1 + e if small else 0,
                    skew=skew, y=rng.choice(["bf16", "f32"]) if op == "w4" else "bf16")
    h = 8 * log(1, 1024)
    kind = rng.choice(["bf16", "bf16", "f32"])
    while n * t * r * h * (2 if kind == "bf16" else 4) > 400 << 20 and t > 1:
        t //= 2
    # the bound on a region's rows is only kept where the buffers stay small
    small = small or n * n * t * max(r, e // n) * h > 1 << 28
    c = dict(op=op, N=n, T=t, E=e, R=r, H=h, cap=(3 * t * r) // 2 + 1 + e if small else 0, skew=skew)
    return dict(c, y=kind) if op == "combine_grad" else dict(c, x=kind, add=rng.random() < 0.5)


def _cap(c):
    return c["cap"] if c["cap"] else c["N"] * c["T"] * max(c["R"], c["E"] // c["N"])


def _width(c):
    """Rows of an expert's weight matrix: gate and up together where there is a gate."""
    return c["F"] * (2 if c["op"] == "w4_swiglu" else 1)


def work(c):
    nt = c["N"] * c["T"]
    pairs = nt * c["R"]
    op = c["op"]
    if op == "route_grad":
        every = c["score"] == "softmax" and not c["renorm"]  # every expert's logit takes part, else the chosen ones'
        bias = c["E"] * 4 if c["bias"] == "logit" else 0
        b = nt * c["E"] * 4 + pairs * 12 + bias  # dlogits and dbias; ids, weights and their gradient
        if every:
            b += nt * c["E"] * 4 + bias
        elif c["score"] == "sigmoid":
            b += pairs * 4 + bias
        return {"bytes": b, "flops": nt * 8 * (c["E"] if every else c["R"])}
    rows = min(pairs, c["N"] * _cap(c))
    if op == "combine_grad":
        el = 2 if c["y"] == "bf16" else 4
        return {"bytes": (nt + 2 * rows) * c["H"] * el + pairs * 12, "flops": 3 * rows * c["H"]}
    if op == "dispatch_grad":
        el = 2 if c["x"] == "bf16" else 4
        return {"bytes": (nt * (2 if c["add"] else 1) + rows) * c["H"] * el + pairs * 4, "flops": rows * c["H"]}
    k, f, w, active = c["K"], c["F"], _width(c), min(c["E"], pairs)
    b = rows * (k * 2 + f * (4 if c["y"] == "f32" else 2)) + active * w * (k // 2 + k // c["group"] + 4)
    return {"bytes": b, "flops": 2 * rows * k * w}


def _choose(c, g):
    """A router's choice: R distinct experts per token, the low ones preferred by `skew`."""
    nt, e = c["N"] * c["T"], c["E"]
    key = torch.rand(nt, e, generator=g, device="cuda").log().neg().log().neg()
    key -= c["skew"] * torch.arange(1, e + 1, device="cuda", dtype=torch.float32).log()
    ids = key.topk(c["R"], dim=1).indices
    offsets = torch.zeros(e + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.bincount(ids.reshape(-1), minlength=e).cumsum(0)
    return ids, offsets


def _positions(c, ids, offsets):
    """Receive row of every pair: grouped by expert in its rank's region, tokens in order."""
    cap, per = _cap(c), c["E"] // c["N"]
    flat = ids.reshape(-1)
    place = torch.empty_like(flat)
    place[flat.argsort(stable=True)] = torch.arange(len(flat), device=flat.device)
    rank = flat // per
    local = place - offsets[rank * per]
    return torch.where(local < cap, rank * cap + local, -1).to(torch.int32).view(ids.shape)


def _pack4(q):
    """Whole numbers in [-8, 7] as words of eight: element 2j at bit 4j, element 2j+1 at bit 16 + 4j."""
    q = q.view(*q.shape[:-1], -1, 8)
    word = torch.zeros(q.shape[:-1], dtype=torch.int32, device=q.device)
    for i in range(8):
        word |= (q[..., i].to(torch.int32) & 15) << (4 * (i // 2) + 16 * (i % 2))
    return word


def _unpack4(word):
    parts = []
    for i in range(8):
        v = (word >> (4 * (i // 2) + 16 * (i % 2))) & 15
        parts.append(v - 16 * (v > 7))
    return torch.stack(parts, dim=-1).flatten(-2)


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    nt, e, r, op = c["N"] * c["T"], c["E"], c["R"], c["op"]

    def randn(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=dev, dtype=dtype)

    if op == "route_grad":
        logits = randn(nt, e, dtype=torch.float32) * 2.0
        bias = None if c["bias"] == "none" else randn(e, dtype=torch.float32) * 0.1
        key = logits
        if c["bias"] == "logit":
            key = logits + bias
        score = torch.softmax(key.double(), 1) if c["score"] == "softmax" else torch.sigmoid(key.double())
        if c["bias"] == "select":
            key = score + bias
        ids = key.topk(r, dim=1).indices
        w = score.gather(1, ids)
        if c["renorm"]:
            w = w / w.sum(1, keepdim=True)
        return dict(case=c, logits=logits, bias=bias, ids=ids.to(torch.int32), w=w.float(),
                    dw=randn(nt, r, dtype=torch.float32), dlogits=torch.empty(nt, e, device=dev),
                    dbias=torch.empty(e, device=dev) if c["bias"] == "logit" else None)
    ids, offsets = _choose(c, g)
    cap = _cap(c)
    rows = c["N"] * cap
    s = dict(case=c, cap=cap)
    if op == "combine_grad":
        t = torch.bfloat16 if c["y"] == "bf16" else torch.float32
        s["pos"] = _positions(c, ids, offsets)
        w = torch.rand(nt, r, generator=g, device=dev) + 0.05
        s["w"] = w / w.sum(1, keepdim=True)
        s["dout"] = randn(nt, c["H"], dtype=t)
        s["y"] = randn(rows, c["H"], dtype=t)
        s["dy"] = torch.full((rows, c["H"]), FILL, dtype=t, device=dev)
        s["dw"] = torch.empty(nt, r, device=dev)
    elif op == "dispatch_grad":
        t = torch.bfloat16 if c["x"] == "bf16" else torch.float32
        s["pos"] = _positions(c, ids, offsets)
        s["dpacked"] = randn(rows, c["H"], dtype=t)
        s["add"] = randn(nt, c["H"], dtype=t) if c["add"] else None
        s["dx"] = torch.empty(nt, c["H"], dtype=t, device=dev)
    else:
        k, f, w, group = c["K"], c["F"], _width(c), c["group"]
        s["offsets"] = offsets.to(torch.int32)
        # the most rows that an expert has, known on the host: the padded plain form needs it
        s["most"] = max(1, min(int((offsets[1:] - offsets[:-1]).max()), cap))
        s["x"] = randn(rows, k)
        # codes of normal weights whose largest magnitude in a group lies near 7
        q = torch.empty(e, w, k, dtype=torch.int8, device=dev)
        for i in range(e):
            q[i] = (randn(w, k) * 2.8).round_().clamp_(-8, 7)
        s["wq"] = _pack4(q)
        del q
        s["ws"] = (448.0 * (0.25 + 0.75 * torch.rand(e, k // group, w, generator=g, device=dev))).to(torch.float8_e4m3fn)
        s["wr"] = (0.5 + torch.rand(e, w, generator=g, device=dev)) * (k ** -0.5 / 800.0)
        t = torch.float32 if c["y"] == "f32" else torch.bfloat16
        s["y"] = torch.full((rows, f), FILL, dtype=t, device=dev)
    return s


def _run_own(s):
    import combine_moe_route_topk_gb300 as moe

    c = s["case"]
    op = c["op"]
    if op == "route_grad":
        dims = moe.make_dims(c["N"], c["T"], c["E"], c["R"], 8)
        fn = moe.MOE_SOFTMAX if c["score"] == "softmax" else moe.MOE_SIGMOID
        if c["bias"] == "select":
            fn |= moe.MOE_BIAS_SELECT_ONLY
        moe.route_grad(dims, s["logits"], s["bias"], fn, c["renorm"], s["ids"], s["w"], s["dw"], s["dlogits"], s["dbias"])
        return [s["dlogits"], s["dbias"]] if s["dbias"] is not None else s["dlogits"]
    if op == "combine_grad":
        dims = moe.make_dims(c["N"], c["T"], c["E"], c["R"], c["H"],
                             y_dtype=moe.MOE_F32 if c["y"] == "f32" else moe.MOE_BF16, cap_rows=s["cap"])
        moe.combine_grad(dims, s["dout"], s["y"], s["pos"], s["w"], s["dy"], s["dw"])
        return [s["dy"], s["dw"]]
    if op == "dispatch_grad":
        dims = moe.make_dims(c["N"], c["T"], c["E"], c["R"], c["H"],
                             x_dtype=moe.MOE_F32 if c["x"] == "f32" else moe.MOE_BF16, cap_rows=s["cap"])
        moe.dispatch_grad(dims, s["dpacked"], s["pos"], s["dx"], s["add"])
        return s["dx"]
    dims = moe.make_dims(c["N"], c["T"], c["E"], c["R"], 8, y_dtype=moe.MOE_F32 if c["y"] == "f32" else moe.MOE_BF16,
                         cap_rows=s["cap"])
    act = moe.MOE_EXPERT_SWIGLU if op == "w4_swiglu" else moe.MOE_EXPERT_LINEAR
    moe.expert_gemm_w4(dims, c["K"], c["F"], act, c["group"], s["x"], s["wq"], s["ws"], s["wr"], s["offsets"], s["y"])
    return s["y"]


def _route_grad(s):
    c = s["case"]
    ids, w, dw = s["ids"].long(), s["w"], s["dw"]
    z = s["logits"] + s["bias"] if c["bias"] == "logit" else s["logits"]
    if c["score"] == "softmax" and not c["renorm"]:
        p = torch.exp(z - z.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
        d = torch.zeros_like(p).scatter_(1, ids, dw)
        d = p * (d - (dw * w).sum(1, keepdim=True))
    else:
        at = w * (dw - (dw * w).sum(1, keepdim=True)) if c["renorm"] else dw * w
        if c["score"] == "sigmoid":
            at = at / (1.0 + torch.exp(z.gather(1, ids)))
        d = torch.zeros_like(z).scatter_(1, ids, at)
    if s["dbias"] is not None:
        return [d, d.double().sum(0).float()]
    return d


def _w4(s):
    c, cap, most, off = s["case"], s["cap"], s["most"], s["offsets"].long()
    n, e, f = c["N"], c["E"], c["F"]
    per = e // n
    dev = off.device
    rank = torch.arange(e, device=dev) // per
    first = off[:-1] - off[rank * per]  # place in the region
    count = torch.minimum(off[1:] - off[:-1], (cap - first).clamp_min(0))
    base = rank * cap + first
    j = torch.arange(most, device=dev)
    inside = j < count.unsqueeze(1)
    rows = torch.where(inside, base.unsqueeze(1) + j, 0)
    x = torch.where(inside.unsqueeze(2), s["x"][rows].float(), 0.0)
    w = _unpack4(s["wq"]).float()
    w = w.view(e, w.shape[1], -1, c["group"]) * s["ws"].float().transpose(1, 2).unsqueeze(3)
    pre = torch.bmm(x, w.view(e, w.shape[1], -1).transpose(1, 2)) * s["wr"].unsqueeze(1)
    if c["op"] == "w4_swiglu":
        pre = pre[..., :f] / (1.0 + torch.exp(-pre[..., :f])) * pre[..., f:]
    p = torch.arange(n * cap, device=dev)
    at = off[p // cap * per] + p % cap  # place in the order of all routed rows
    valid = at < off[(p // cap + 1) * per]
    expert = (torch.searchsorted(off, at, right=True) - 1).clamp(0, e - 1)
    slot = torch.where(valid, p - base[expert], 0).clamp(0, most - 1)
    return torch.where(valid.unsqueeze(1), pre[expert, slot].to(s["y"].dtype), s["y"])


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "route_grad":
        return _route_grad(s)
    if op.startswith("w4"):
        return _w4(s)
    pos = s["pos"].long()
    kept = pos >= 0
    if op == "dispatch_grad":
        d = torch.where(kept.unsqueeze(2), s["dpacked"][pos.clamp_min(0)].float(), 0.0).sum(1)
        return (d if s["add"] is None else d + s["add"].float()).to(s["dx"].dtype)
    dout, w, rows, r = s["dout"].float(), s["w"], len(s["y"]), pos.shape[1]
    dw = (s["y"][pos.clamp_min(0)].float() * dout.unsqueeze(1)).sum(2)
    src = torch.full((rows + 1,), -1, dtype=torch.int64, device=pos.device)
    src.scatter_(0, torch.where(kept, pos, rows).view(-1), torch.arange(pos.numel(), device=pos.device))
    src = src[:rows]
    pair = src.clamp_min(0)
    dy = torch.where((src >= 0).unsqueeze(1), (w.view(-1)[pair].unsqueeze(1) * dout[pair // r]).to(s["dy"].dtype), s["dy"])
    return [dy, torch.where(kept, dw, 0.0)]


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "route_grad":
        # the weights' own gradient, through their definition
        z = s["logits"].double()
        if c["bias"] == "logit":
            z = (s["logits"] + s["bias"]).double()  # the key is rounded to 32 bits
        ids, h = s["ids"].long(), s["dw"].double()
        score = torch.softmax(z, 1) if c["score"] == "softmax" else torch.special.expit(z)
        chosen = score.gather(1, ids)
        if c["renorm"]:  # of v / sum v
            total = chosen.sum(1, keepdim=True)
            h = (h * total - (h * chosen).sum(1, keepdim=True)) / total ** 2
        dscore = torch.zeros_like(z).scatter_(1, ids, h)
        if c["score"] == "softmax":
            d = score * dscore - score * (score * dscore).sum(1, keepdim=True)
        else:
            d = dscore * score * torch.special.expit(-z)
        return [d, d.sum(0)] if s["dbias"] is not None else d
    if op in ("combine_grad", "dispatch_grad"):
        if op == "dispatch_grad":
            dx = torch.zeros(s["dx"].shape, dtype=torch.float64, device="cuda") if s["add"] is None else s["add"].double()
            for k in range(c["R"]):  # one expert's rows at a time
                p = s["pos"][:, k].long()
                has = (p >= 0).nonzero().squeeze(1)
                dx[has] += s["dpacked"][p[has]].double()
            return dx
        dy, dw = s["dy"].double(), torch.zeros(s["dw"].shape, dtype=torch.float64, device="cuda")
        for k in range(c["R"]):
            p = s["pos"][:, k].long()
            has = (p >= 0).nonzero().squeeze(1)
            d = s["dout"][has].double()
            dw[has, k] = (d * s["y"][p[has]].double()).sum(1)
            dy[p[has]] = s["w"][has, k].double().unsqueeze(1) * d
        return [dy, dw]
    off, per, cap, f = s["offsets"].tolist(), c["E"] // c["N"], s["cap"], c["F"]
    y = s["y"].double()
    for e in range(c["E"]):
        start = off[e // per * per]
        lo, hi = min(off[e] - start, cap), min(off[e + 1] - start, cap)
        if lo == hi:
            continue
        rows = slice(e // per * cap + lo, e // per * cap + hi)
        word = s["wq"][e].long() & 0xFFFFFFFF
        w = torch.empty(word.shape[0], c["K"], dtype=torch.float64, device="cuda")
        for i in range(8):
            code = torch.bitwise_right_shift(word, 4 * (i >> 1) + 16 * (i & 1)) & 15
            w[:, i::8] = torch.where(code >= 8, code - 16, code).double()
        w *= s["ws"][e].double().t().repeat_interleave(c["group"], 1)
        w *= s["wr"][e].double().unsqueeze(1)
        pre = s["x"][rows].double() @ w.t()
        y[rows] = pre[:, :f] * torch.special.expit(pre[:, :f]) * pre[:, f:] if op == "w4_swiglu" else pre
    return y
