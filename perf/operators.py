"""Cases of the experts' products between dispatch and combine, and their plain forms.

A pass is one call on the receive layout that the dispatch writes: rank d's
region holds rows [d*cap, (d+1)*cap), grouped by expert; expert_offsets is the
exclusive prefix sum of the experts' row counts.  Operations:

* linear       y[p] = x[p] w[e]^T (bf16 operands, bf16 or f32 results)
* swiglu       g|u = x[p] w[e]^T, y = silu(g) * u (optionally g|u kept for training)
* dgrad        dx[p] = dy[p] w[e]
* wgrad        dw[e] = sum over e's rows of dy[p]^T x[p]
* swiglu_grad  gradient of silu(g) * u
* fp8          y[p] = x[p] w[e]^T of e4m3 codes with f32 scales (1x128 for x, 128x128 for w)
* fp8_swiglu   the same with silu(g) * u requantised to e4m3 + one scale per 128
"""
import torch

own = False

FILL = 0.5  # what rows without a token hold before the call, and after it


def listed():
    base = dict(y="bf16", skew=0.0, save=False)
    return [
        # second product of a small decode batch (256 tokens, 2 of 16 experts), f32 results for an f32 combine
        dict(base, name="linear small decode f32", op="linear", N=4, T=64, E=16, R=2, K=512, F=1024, cap=0, y="f32"),
        # second product of a prefill batch: 131072 routed rows over 128 experts
        dict(base, name="linear prefill", op="linear", N=4, T=4096, E=128, R=8, K=2048, F=4096, cap=40960),
        # first product for a single token: 8 of a rank's 64 experts, bound by their weights
        dict(base, name="swiglu one token", op="swiglu", N=1, T=1, E=64, R=8, K=7168, F=2048, cap=0),
        # first product of a decode batch: about 128 rows per expert
        dict(base, name="swiglu decode", op="swiglu", N=8, T=128, E=64, R=8, K=7168, F=2048, cap=1408),
        # a training step's first product at odd sizes, skewed routing, pre-activations kept
        dict(base, name="swiglu odd train", op="swiglu", N=2, T=37, E=6, R=3, K=1000, F=776, cap=0, skew=0.7, save=True),
        # data gradient of a first product in training
        dict(base, name="dgrad train", op="dgrad", N=4, T=1024, E=32, R=4, K=2048, F=4096, cap=5120),
        # weight gradient of the same step, f32 for the optimiser
        dict(base, name="wgrad train f32", op="wgrad", N=4, T=1024, E=32, R=4, K=2048, F=4096, cap=5120, y="f32"),
        # weight gradient at odd sizes, skewed so that some experts get few rows or none
        dict(base, name="wgrad odd skewed", op="wgrad", N=1, T=777, E=12, R=2, K=520, F=1352, cap=0, skew=3.0),
        # the activation's gradient between the two products' gradients
        dict(base, name="swiglu_grad train", op="swiglu_grad", N=4, T=2048, E=32, R=8, K=8, F=2048, cap=20480),
        # second product of an fp8 decode batch
        dict(base, name="fp8 decode", op="fp8", N=8, T=128, E=64, R=8, K=2048, F=7168, cap=1408),
        # first product of an fp8 prefill batch: about 512 rows per expert
        dict(base, name="fp8_swiglu prefill", op="fp8_swiglu", N=4, T=1024, E=64, R=8, K=7168, F=2048, cap=10240),
        # first product of a few tokens, small experts
        dict(base, name="fp8_swiglu few tokens", op="fp8_swiglu", N=2, T=8, E=16, R=2, K=1024, F=512, cap=0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["linear", "swiglu", "dgrad", "wgrad", "swiglu_grad", "fp8", "fp8_swiglu"])
    n = rng.choice([1, 2, 4, 8])
    e = n * log(1, 64 // n)
    r = rng.randint(1, min(8, e))
    t = log(1, 4096 // n)
    k = 128 * log(1, 48) if op.startswith("fp8") else 8 * log(4, 768)
    f = 128 * log(1, 24) if op == "fp8_swiglu" else 8 * log(4, 384)
    skew = rng.choice([0.0, 0.0, 0.7, 2.0])
    while 2 * n * t * r * k * f * (2 if "swiglu" in op else 1) > 1.0e12 and t > 1:
        t //= 2
    y = rng.choice(["bf16", "f32"]) if op in ("linear", "wgrad", "fp8") else "bf16"
    # about 1.5 times a rank's mean share of the rows where there are several ranks; the bound otherwise
    cap = 0 if rng.random() < 0.5 else (3 * t * r) // 2 + 1 + e
    return dict(op=op, N=n, T=t, E=e, R=r, K=8 if op == "swiglu_grad" else k, F=f, cap=cap, y=y, skew=skew,
                save=op == "swiglu" and rng.random() < 0.5)


def _cap(c):
    return c["cap"] if c["cap"] else c["N"] * c["T"] * max(c["R"], c["E"] // c["N"])


def _width(c):
    """Rows of an expert's weight matrix: gate and up together where there is a gate."""
    return c["F"] * (2 if c["op"] in ("swiglu", "fp8_swiglu") else 1)


def work(c):
    pairs = c["N"] * c["T"] * c["R"]
    rows = min(pairs, c["N"] * _cap(c))
    active = min(c["E"], pairs)
    k, f, w = c["K"], c["F"], _width(c)
    out = 4 if c["y"] == "f32" else 2
    op = c["op"]
    if op == "swiglu_grad":
        return {"bytes": rows * f * 2 * 5, "flops": rows * f * 10}
    flops = 2 * rows * k * w
    if op == "fp8":
        b = rows * (k + k // 32) + active * (w * k + 4 * (-(-w // 128)) * (k // 128)) + rows * f * out
    elif op == "fp8_swiglu":
        b = rows * (k + k // 32) + active * (w * k + w * k // 4096) + rows * (f + f // 32)
    elif op == "wgrad":
        b = rows * (k + f) * 2 + c["E"] * k * f * out
    elif op == "dgrad":
        b = rows * (k + f) * 2 + active * k * f * 2
    else:
        b = rows * k * 2 + active * w * k * 2 + rows * f * out + (rows * w * 2 if c["save"] else 0)
    return {"bytes": b, "flops": flops}


def _quantise(x):
    """Rows of f32 values as e4m3 codes and one f32 scale (amax / 448) per 128."""
    b = x.view(x.shape[0], -1, 128)
    scale = b.abs().amax(dim=2) / 448.0
    inv = torch.where(scale > 0, scale, torch.ones_like(scale))
    q = (b / inv.unsqueeze(2)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return q.view(x.shape), scale


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    n, e, nt, cap = c["N"], c["E"], c["N"] * c["T"], _cap(c)
    rows, k, f, w = n * cap, c["K"], c["F"], _width(c)

    def randn(*shape, scale=1.0, dtype=torch.bfloat16):
        t = torch.randn(*shape, generator=g, device=dev, dtype=torch.float32 if dtype == torch.float32 else torch.bfloat16)
        return t if scale == 1.0 else t.mul_(scale)

    # a router's choice: R distinct experts per token, the low ones preferred by `skew`
    key = torch.rand(nt, e, generator=g, device=dev).log().neg().log().neg()
    key -= c["skew"] * torch.arange(1, e + 1, device=dev, dtype=torch.float32).log()
    ids = key.topk(c["R"], dim=1).indices.reshape(-1)
    counts = torch.bincount(ids, minlength=e)
    offsets = torch.zeros(e + 1, dtype=torch.int32, device=dev)
    offsets[1:] = counts.cumsum(0)
    # the most rows that an expert has, known on the host: the padded plain form needs it
    s = dict(case=c, cap=cap, offsets=offsets, most=max(1, min(int(counts.max()), cap)))
    yt = torch.float32 if c["y"] == "f32" else torch.bfloat16
    op = c["op"]
    if op in ("linear", "swiglu"):
        s["x"] = randn(rows, k)
        s["w"] = randn(e, w, k, scale=k ** -0.5)
        s["y"] = torch.full((rows, f), FILL, dtype=yt, device=dev)
        s["pre"] = torch.full((rows, w), FILL, dtype=torch.bfloat16, device=dev) if c["save"] else None
    elif op == "dgrad":
        s["dy"] = randn(rows, f)
        s["w"] = randn(e, f, k, scale=k ** -0.5)
        s["dx"] = torch.full((rows, k), FILL, dtype=torch.bfloat16, device=dev)
    elif op == "wgrad":
        s["dy"] = randn(rows, f)
        s["x"] = randn(rows, k)
        s["dw"] = torch.full((e, f, k), FILL, dtype=yt, device=dev)
    elif op == "swiglu_grad":
        s["pre"] = randn(rows, 2 * f)
        s["dh"] = randn(rows, f)
        s["dpre"] = torch.full((rows, 2 * f), FILL, dtype=torch.bfloat16, device=dev)
    else:
        q, s["xs"] = _quantise(randn(rows, k, dtype=torch.float32))
        s["xq"] = q.view(torch.uint8)
        s["wq"] = randn(e, w, k, scale=64.0).to(torch.float8_e4m3fn).view(torch.uint8)
        s["ws"] = (0.5 + torch.rand(e, -(-w // 128), k // 128, generator=g, device=dev)) * (k ** -0.5 / 64.0)
        if op == "fp8":
            s["y"] = torch.full((rows, f), FILL, dtype=yt, device=dev)
        else:
            s["y"] = torch.zeros(rows, f, dtype=torch.uint8, device=dev)
            s["ys"] = torch.zeros(rows, f // 128, dtype=torch.float32, device=dev)
    return s


def _run_own(s):
    import combine_moe_route_topk_gb300 as moe

    c = s["case"]
    op, k, f, off = c["op"], c["K"], c["F"], s["offsets"]
    dims = moe.make_dims(c["N"], c["T"], c["E"], c["R"], 8, y_dtype=moe.MOE_F32 if c["y"] == "f32" else moe.MOE_BF16,
                         cap_rows=s["cap"])
    if op == "linear":
        moe.expert_gemm(dims, k, f, moe.MOE_EXPERT_LINEAR, s["x"], s["w"], off, s["y"])
        return s["y"]
    if op == "swiglu":
        moe.expert_gemm(dims, k, f, moe.MOE_EXPERT_SWIGLU, s["x"], s["w"], off, s["y"], s["pre"])
        return [s["y"], s["pre"]] if c["save"] else s["y"]
    if op == "dgrad":
        moe.expert_gemm_dgrad(dims, k, f, s["dy"], s["w"], off, s["dx"])
        return s["dx"]
    if op == "wgrad":
        moe.expert_gemm_wgrad(dims, k, f, s["dy"], s["x"], off, s["dw"])
        return s["dw"]
    if op == "swiglu_grad":
        moe.expert_swiglu_grad(dims, f, s["pre"], s["dh"], off, s["dpre"])
        return s["dpre"]
    if op == "fp8":
        moe.expert_gemm_fp8(dims, k, f, moe.MOE_EXPERT_LINEAR, s["xq"], s["xs"], s["wq"], s["ws"], off, s["y"])
        return s["y"]
    moe.expert_gemm_fp8(dims, k, f, moe.MOE_EXPERT_SWIGLU, s["xq"], s["xs"], s["wq"], s["ws"], off, s["y"], s["ys"])
    return [s["y"].view(torch.float8_e4m3fn), s["ys"]]


class _Groups:
    """Where the experts' rows are, as index tensors: [E][most] padded groups and back."""

    def __init__(self, s):
        c, cap, off = s["case"], s["cap"], s["offsets"].long()
        n, e = c["N"], c["E"]
        dev = off.device
        first = off[:-1] - off[torch.arange(n, device=dev) * (e // n)].repeat_interleave(e // n)  # row in the region
        left = (cap - first).clamp_min(0)
        self.count = torch.minimum(off[1:] - off[:-1], left)  # rows that fit the region
        self.base = torch.arange(n, device=dev).repeat_interleave(e // n) * cap + first
        j = torch.arange(s["most"], device=dev)
        self.inside = j < self.count.unsqueeze(1)  # [E][most]
        self.rows = torch.where(self.inside, self.base.unsqueeze(1) + j, 0)
        p = torch.arange(n * cap, device=dev)
        rank = p // cap
        at = off[rank * (e // n)] + p % cap  # place in the order of all routed rows
        self.valid = at < off[(rank + 1) * (e // n)]
        self.expert = (torch.searchsorted(off, at, right=True) - 1).clamp(0, e - 1)
        self.slot = torch.where(self.valid, p - self.base[self.expert], 0).clamp(0, s["most"] - 1)

    def gather(self, t):
        """Rows of t as f32 [E][most][...], zero where a group has no more rows."""
        return torch.where(self.inside.unsqueeze(2), t[self.rows].float(), 0.0)

    def scatter(self, grouped, like):
        """[E][most][...] back to rows, rows without a token as they were in `like`."""
        return torch.where(self.valid.unsqueeze(1), grouped[self.expert, self.slot].to(like.dtype), like)


def run(s):
    if own:
        return _run_own(s)
    c, gr = s["case"], _Groups(s)
    op, f = c["op"], c["F"]
    if op == "linear":
        return gr.scatter(torch.bmm(gr.gather(s["x"]), s["w"].float().transpose(1, 2)), s["y"])
    if op == "swiglu":
        pre = torch.bmm(gr.gather(s["x"]), s["w"].float().transpose(1, 2))
        h = pre[..., :f] / (1.0 + torch.exp(-pre[..., :f])) * pre[..., f:]
        y = gr.scatter(h, s["y"])
        return [y, gr.scatter(pre, s["pre"])] if c["save"] else y
    if op == "dgrad":
        return gr.scatter(torch.bmm(gr.gather(s["dy"]), s["w"].float()), s["dx"])
    if op == "wgrad":
        return torch.bmm(gr.gather(s["dy"]).transpose(1, 2), gr.gather(s["x"])).to(s["dw"].dtype)
    if op == "swiglu_grad":
        g, u, dh = s["pre"][:, :f].float(), s["pre"][:, f:].float(), s["dh"].float()
        sg = 1.0 / (1.0 + torch.exp(-g))
        d = torch.cat([dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg], dim=1)
        return torch.where(gr.valid.unsqueeze(1), d.to(torch.bfloat16), s["dpre"])
    x = s["xq"].view(torch.float8_e4m3fn).float().view(len(s["xq"]), -1, 128) * s["xs"].unsqueeze(2)
    w = s["wq"].view(torch.float8_e4m3fn).float()
    w *= s["ws"].repeat_interleave(128, dim=2).repeat_interleave(128, dim=1)[:, : w.shape[1]]
    pre = torch.bmm(gr.gather(x.view(len(x), -1)), w.transpose(1, 2))
    if op == "fp8":
        return gr.scatter(pre, s["y"])
    h = pre[..., :f] / (1.0 + torch.exp(-pre[..., :f])) * pre[..., f:]
    q, scale = _quantise(h.reshape(-1, f))
    q = q.float().view(h.shape)
    return [gr.scatter(q, s["y"].view(torch.float8_e4m3fn).float()).to(torch.float8_e4m3fn),
            gr.scatter(scale.view(h.shape[0], h.shape[1], -1), s["ys"])]


def exact(case, seed):
    s = prepare(case, seed)
    c, cap, f = case, s["cap"], case["F"]
    off = s["offsets"].tolist()
    per = c["E"] // c["N"]
    op = c["op"]

    def span(e):
        """Rows of expert e: its place in its rank's region, cut where the region ends."""
        lo = off[e] - off[e // per * per]
        hi = off[e + 1] - off[e // per * per]
        return slice(e // per * cap + min(lo, cap), e // per * cap + min(hi, cap))

    def e4m3(t):
        return t.view(torch.float8_e4m3fn).double()

    if op == "wgrad":
        return torch.stack([s["dy"][span(e)].double().t() @ s["x"][span(e)].double() for e in range(c["E"])])
    if op in ("linear", "swiglu", "fp8"):
        y = s["y"].double()
    if op == "swiglu":
        kept = torch.full((len(y), 2 * f), FILL, dtype=torch.float64, device=y.device) if c["save"] else None
    if op == "dgrad":
        y = s["dx"].double()
    if op == "swiglu_grad":
        y = s["dpre"].double()
    if op == "fp8_swiglu":
        y, scales = e4m3(s["y"]), s["ys"].double()
    for e in range(c["E"]):
        r = span(e)
        if r.start == r.stop:
            continue
        if op == "linear":
            y[r] = s["x"][r].double() @ s["w"][e].double().t()
        elif op == "swiglu":
            pre = s["x"][r].double() @ s["w"][e].double().t()
            y[r] = pre[:, :f] * torch.special.expit(pre[:, :f]) * pre[:, f:]
            if kept is not None:
                kept[r] = pre
        elif op == "dgrad":
            y[r] = s["dy"][r].double() @ s["w"][e].double()
        elif op == "swiglu_grad":
            g, u, dh = s["pre"][r, :f].double(), s["pre"][r, f:].double(), s["dh"][r].double()
            sg = torch.special.expit(g)
            y[r] = torch.cat([dh * u * (sg + g * sg * torch.special.expit(-g)), dh * g * sg], dim=1)
        else:
            xs = s["xs"][r].double()
            x = (e4m3(s["xq"][r]).unflatten(1, (-1, 128)) * xs.unsqueeze(2)).flatten(1)
            w = e4m3(s["wq"][e])
            ws = s["ws"][e].double()
            w = w * ws.repeat_interleave(128, 0)[: w.shape[0]].repeat_interleave(128, 1)
            pre = x @ w.t()
            if op == "fp8":
                y[r] = pre
            else:
                h = (pre[:, :f] * torch.special.expit(pre[:, :f]) * pre[:, f:]).unflatten(1, (-1, 128))
                scales[r] = h.abs().amax(2) / 448.0
                y[r] = (h / scales[r].unsqueeze(2)).flatten(1)
    if op == "swiglu" and c["save"]:
        return [y, kept]
    return [y, scales] if op == "fp8_swiglu" else y
