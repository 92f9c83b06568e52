"""The routing steps' gradients against plain 64-bit formulas and differences.

Errors allowed: an f32 sum of n products, each step rounded (2^-24 of a partial
sum, which never exceeds the sum of magnitudes): (n + 4) 2^-24 sum|a b|; a result
rounded to its type: half a step (expert_ref.check adds it).
"""
import pytest
import torch

import combine_moe_route_topk_gb300 as moe
import expert_ref as ref
from expert_ref import BF16_HALF, F32_HALF, SENTINEL

pytestmark = pytest.mark.gpu
TYPES = {"bf16": (torch.bfloat16, moe.MOE_BF16, BF16_HALF), "f32": (torch.float32, moe.MOE_F32, F32_HALF)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_moe_route_topk_gb300 import _build
    _build.build()
    yield
    assert moe.take_device_error() == moe.MOE_OK


class Routed:
    """Random distinct experts for every token, and their rows by the library's count."""

    def __init__(self, N, T, E, R, H, cap=0, seed=0, skew=0.0, kind="bf16"):
        t, code, self.half = TYPES[kind]
        self.dims = moe.make_dims(N, T, E, R, H, x_dtype=code, y_dtype=code, cap_rows=cap)
        self.t = t
        g = self.g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.NT, self.R, self.H, self.E = N * T, R, H, E
        key = torch.rand(self.NT, E, generator=g, device="cuda") - skew * torch.arange(E, device="cuda") / E
        self.idx = key.topk(R, dim=1).indices.to(torch.int32)
        i = dict(dtype=torch.int32, device="cuda")
        self.pos, self.status = torch.empty(self.NT, R, **i), torch.empty(1, **i)
        moe.dispatch_count(self.dims, self.idx, torch.empty(E, **i), torch.empty(E + 1, **i), torch.empty(N, **i),
                           torch.empty(N + 1, **i), torch.empty(N, N, **i), self.pos, self.status)
        self.rows = N * moe.buffer_sizes(self.dims)["cap_rows"]
        self.has = self.pos >= 0
        self.used = torch.zeros(self.rows, dtype=torch.bool, device="cuda")
        self.used[self.pos[self.has].long()] = True

    def randn(self, *shape, dtype=None):
        return torch.randn(*shape, generator=self.g, device="cuda").to(dtype or self.t)

    def packed(self, width):
        """Rows whose unused ones hold NaN."""
        t = self.randn(self.rows, width)
        t[~self.used] = float("nan")
        return t


# N, T, E, R, H, cap, skew: one token; odd sizes; a row shorter than a block's
# threads, rows that end inside a thread's second vector; more pairs than are
# loaded together; regions that overflow; tokens without any row left
SHAPES = [
    (1, 1, 1, 1, 8, 0, 0.0),
    (1, 3, 5, 2, 16, 0, 0.0),
    (2, 37, 6, 3, 1048, 0, 0.0),
    (4, 64, 16, 2, 1024, 0, 0.0),
    (2, 50, 8, 8, 2056, 0, 0.0),
    (1, 33, 40, 9, 520, 0, 0.0),
    (2, 21, 64, 32, 264, 0, 0.0),
    (2, 100, 10, 3, 136, 60, 2.0),
    (4, 30, 8, 2, 72, 3, 2.0),
    (1, 64, 4, 1, 7168, 5, 0.0),
    (8, 16, 32, 17, 4104, 100, 1.0),
    # many tokens of few bytes: a token is a warp's
    (1, 4099, 7, 2, 1048, 0, 0.0),
    (2, 1101, 10, 5, 264, 900, 2.0),
    (1, 703, 40, 32, 40, 0, 0.0),
    (1, 2050, 3, 1, 2040, 1500, 0.0),
]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", TYPES)
def test_combine_grad(shape, kind):
    N, T, E, R, H, cap, skew = shape
    b = Routed(N, T, E, R, H, cap, 1, skew, kind)
    dout, y, w = b.randn(b.NT, H), b.packed(H), b.randn(b.NT, R, dtype=torch.float32)
    dy, dw = torch.full((b.rows, H), SENTINEL, dtype=b.t, device="cuda"), torch.full((b.NT, R), SENTINEL, device="cuda")
    moe.combine_grad(b.dims, dout, y, b.pos, w, dy, dw)
    src = b.has.nonzero()
    p = b.pos[b.has].long()
    d, yy = dout.double()[src[:, 0]], y.double()[p]
    want = w.double()[b.has].unsqueeze(1) * d
    ref.check(dy[p], want, F32_HALF * want.abs(), b.half, "dy")  # the product is rounded in f32 first
    assert bool((dy[~b.used].float() == SENTINEL).all())
    ref.check(dw[b.has], (d * yy).sum(1), (H + 4) * 2.0 ** -24 * (d * yy).abs().sum(1), F32_HALF, "dtopk_w")
    assert bool((dw[~b.has] == 0).all())


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kind", TYPES)
@pytest.mark.parametrize("add", ["none", "other", "same"])
def test_dispatch_grad(shape, kind, add):
    N, T, E, R, H, cap, skew = shape
    b = Routed(N, T, E, R, H, cap, 2, skew, kind)
    dp = b.packed(H)
    extra = b.randn(b.NT, H)
    dx = extra.clone() if add == "same" else torch.full((b.NT, H), SENTINEL, dtype=b.t, device="cuda")
    moe.dispatch_grad(b.dims, dp, b.pos, dx, {"none": None, "other": extra, "same": dx}[add])
    rows = dp.double()[b.pos.long().clamp_min(0)]
    rows[~b.has] = 0
    want, mag = rows.sum(1), rows.abs().sum(1)
    if add != "none":
        want, mag = want + extra.double(), mag + extra.double().abs()
    ref.check(dx, want, (R + 1) * 2.0 ** -24 * mag, b.half, "dx")


def test_rows_out_of_range_take_no_part():
    b = Routed(1, 4, 4, 2, 64, 0, 3)
    pos = torch.tensor([[-1, -5], [b.rows, 0], [2147483647, -2147483648], [1, 2]], dtype=torch.int32, device="cuda")
    dout, y, w = b.randn(4, 64), b.randn(b.rows, 64), b.randn(4, 2, dtype=torch.float32)
    dy, dw = torch.full_like(y, SENTINEL), torch.full_like(w, SENTINEL)
    moe.combine_grad(b.dims, dout, y, pos, w, dy, dw)
    assert bool((dy[3:] == SENTINEL).all()) and not bool((dy[:3] == SENTINEL).any())
    assert dw[0].tolist() == [0, 0] and float(dw[1, 0]) == 0 and dw[2].tolist() == [0, 0] and float(dw[1, 1]) != 0
    dx = torch.full((4, 64), SENTINEL, dtype=b.t, device="cuda")
    moe.dispatch_grad(b.dims, y, pos, dx)
    assert bool((dx[0] == 0).all()) and bool((dx[2] == 0).all()) and torch.equal(dx[1], y[0])


@pytest.mark.parametrize("kind", TYPES)
def test_rows_beyond_32_bit_offsets(kind):
    """The last rows of regions of more than 2^31 elements, for blocks and for warps a token."""
    for T, R, H in ((4, 2, 4096), (2080, 2, 2056)):
        cap = (1 << 31) // H + 2 * T * R
        b = Routed(1, T, 4, R, H, cap, 5, kind=kind)
        b.pos.copy_(cap - 1 - torch.randperm(T * R, generator=b.g, device="cuda").view(T, R))
        p = b.pos.long()
        y = torch.empty(cap, H, dtype=b.t, device="cuda")
        y[cap - T * R:] = b.randn(T * R, H)
        dout, w = b.randn(T, H), b.randn(T, R, dtype=torch.float32)
        dy, dw = torch.full_like(y, SENTINEL), torch.full((T, R), SENTINEL, device="cuda")
        moe.combine_grad(b.dims, dout, y, b.pos, w, dy, dw)
        want = w.double().unsqueeze(2) * dout.double().unsqueeze(1)
        ref.check(dy[p], want, F32_HALF * want.abs(), b.half, "dy")
        assert all(bool((part == SENTINEL).all()) for part in dy[:cap - T * R].split(1 << 18))
        yy = y[p].double() * dout.double().unsqueeze(1)
        ref.check(dw, yy.sum(2), (H + 4) * 2.0 ** -24 * yy.abs().sum(2), F32_HALF, "dtopk_w")
        del dy
        dx = torch.full((T, H), SENTINEL, dtype=b.t, device="cuda")
        moe.dispatch_grad(b.dims, y, b.pos, dx)
        rows = y[p].double()
        ref.check(dx, rows.sum(1), (R + 1) * 2.0 ** -24 * rows.abs().sum(1), b.half, "dx")


def test_tokens_beyond_32_bit_offsets():
    """More than 2^31 elements of dout, dx and add; all tokens but the last ones have lost their rows."""
    H, last = 2056, 300
    T = (1 << 31) // H + last
    dims = moe.make_dims(1, T, 2, 1, H, cap_rows=last)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    y, w = torch.randn(last, H, generator=g, device="cuda").to(torch.bfloat16), torch.rand(T, 1, generator=g, device="cuda")
    pos = torch.full((T, 1), -1, dtype=torch.int32, device="cuda")
    pos[-last:, 0] = torch.arange(last, dtype=torch.int32, device="cuda").flip(0)
    dout = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    dout[-last:] = torch.randn(last, H, generator=g, device="cuda").to(torch.bfloat16)
    dy, dw = torch.full_like(y, SENTINEL), torch.full((T, 1), SENTINEL, device="cuda")
    moe.combine_grad(dims, dout, y, pos, w, dy, dw)
    d = dout[-last:].double()
    ref.check(dy.flip(0), w[-last:].double() * d, F32_HALF * (w[-last:].double() * d).abs(), BF16_HALF, "dy")
    prod = d * y.flip(0).double()
    ref.check(dw[-last:, 0], prod.sum(1), (H + 4) * 2.0 ** -24 * prod.abs().sum(1), F32_HALF, "dtopk_w")
    assert bool((dw[:-last] == 0).all())
    dx = torch.full_like(dout, SENTINEL)
    moe.dispatch_grad(dims, y, pos, dx, dout)
    ref.check(dx[-last:], d + y.flip(0).double(), 2 * 2.0 ** -24 * (d.abs() + y.flip(0).double().abs()), BF16_HALF, "dx")
    assert all(bool((part == 0).all()) for part in dx[:-last].split(1 << 18))


def test_a_row_that_two_pairs_name_is_added_for_both():
    b = Routed(1, 3, 4, 2, 72, 0, 7)
    dp = b.randn(b.rows, 72)
    pos = torch.tensor([[1, 1], [1, 2], [0, -1]], dtype=torch.int32, device="cuda")
    dx = torch.empty(3, 72, dtype=b.t, device="cuda")
    moe.dispatch_grad(b.dims, dp, pos, dx)
    want = torch.stack([2 * dp[1].double(), dp[1].double() + dp[2].double(), dp[0].double()])
    ref.check(dx, want, 3 * 2.0 ** -24 * want.abs() + 2.0 ** -24 * dp[1:3].double().abs().sum(0), b.half, "dx")


def test_long_rows():
    """Rows of 2^20 elements: sums of a thread's vectors are kept short."""
    H = 1 << 20
    b = Routed(1, 2, 2, 1, H, 0, 4)
    dout, y = b.randn(2, H).abs(), b.randn(b.rows, H).abs()
    w = torch.ones(2, 1, device="cuda")
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    moe.combine_grad(b.dims, dout, y, b.pos, w, dy, dw)
    want = (dout.double() * y.double()[b.pos.long().flatten()]).sum(1, keepdim=True)
    # at most 32 vectors of 8 in a thread's f32 sum, 5 steps over a warp, then 64 bits; the result's rounding
    ref.check(dw, want, (32 * 8 + 5) * 2.0 ** -24 * want, F32_HALF, "dtopk_w")
    assert torch.equal(dy[b.pos.long().flatten()], dout)


# ---- the router -------------------------------------------------------------

def weights(z, idx, score, renorm):
    s = torch.softmax(z, 1) if score == "softmax" else torch.sigmoid(z)
    w = s.gather(1, idx)
    return w / w.sum(1, keepdim=True) if renorm else w


class Router:
    def __init__(self, N, T, E, R, score, renorm, bias, seed=0, scale=2.0):
        self.dims = moe.make_dims(N, T, E, R, 8)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        kw = dict(generator=g, device="cuda")
        self.logits = torch.randn(N * T, E, **kw) * scale
        self.bias = None if bias == "none" else torch.randn(E, **kw) * 0.3
        self.score, self.renorm, self.mode = score, renorm, bias
        self.fn = (moe.MOE_SOFTMAX if score == "softmax" else moe.MOE_SIGMOID) | (
            moe.MOE_BIAS_SELECT_ONLY if bias == "select" else 0)
        self.idx = torch.empty(N * T, R, dtype=torch.int32, device="cuda")
        self.w = torch.empty(N * T, R, device="cuda")
        self.h = torch.randn(N * T, R, **kw)
        self.dl = torch.full((N * T, E), SENTINEL, device="cuda")
        self.db = torch.full((E,), SENTINEL, device="cuda") if bias == "logit" else None

    def route(self):
        moe.route_topk(self.dims, self.logits, self.bias, self.fn, self.renorm, self.idx, self.w)
        return self

    def grad(self):
        moe.route_grad(self.dims, self.logits, self.bias, self.fn, self.renorm, self.idx, self.w, self.h, self.dl, self.db)
        return self

    def z(self):
        return (self.logits + self.bias if self.mode == "logit" else self.logits).double()

    def check(self):
        """Against the formula on the weights that the call was given.

        Allowed: exp within two units (2^-22), every other operation half a unit
        (u = 2^-24).  d is off by ed = (R + 6) u sum|h w|, h - d by that and u |h - d|.
        Chosen entries: w (h - d) / (1 + exp z): 2^-22 + 6 u of the value, and w / (1 + exp z) ed.
        Softmax: p = exp(z - top) / sum: the difference is rounded, u |z - top| of p, for the
        sum at most u times the average of |z - top| under p; exp 2^-22 each; the sum (E / 32 + 6) u;
        three more operations.  Results below the normal range may be off by 2^-126."""
        u, z, h, w = 2.0 ** -24, self.z(), self.h.double(), self.w.double()
        idx, R, E = self.idx.long(), self.idx.shape[1], z.shape[1]
        d, ed = (h * w).sum(1, keepdim=True), (R + 6) * u * (h * w).abs().sum(1, keepdim=True)
        if self.score == "softmax" and not self.renorm:
            p = torch.softmax(z, 1)
            gap = (z.amax(1, keepdim=True) - z)
            mean = (p * gap.clamp(max=1e4)).sum(1, keepdim=True)
            rel = u * gap.clamp(max=1e4) + u * mean + 2 * 2.0 ** -22 + (E / 32 + 6) * u + 4 * u
            he = torch.zeros_like(z).scatter_(1, idx, h)
            want = p * (he - d)
            err = p * ((he - d).abs() * rel + ed + u * (he.abs() + d.abs()))
        else:
            at = w * (h - d) if self.renorm else w * h
            err = w * ed if self.renorm else torch.zeros_like(w)
            if self.score == "sigmoid":
                one = torch.special.expit(-z.gather(1, idx))
                at, err = at * one, err * one
            err = err + at.abs() * (2.0 ** -22 + 6 * u)
            want = torch.zeros_like(z).scatter_(1, idx, at)
            err = torch.zeros_like(z).scatter_(1, idx, err)
        # scores that are all 0 have weights 0 / 0 from the router itself: NaN there, and there alone
        none = torch.isnan(want)
        assert torch.equal(torch.isnan(self.dl), none) and not bool(none[~torch.isnan(w).any(1)].any())
        ref.check(self.dl[~none], want[~none], err[~none] + 2.0 ** -126, F32_HALF, "dlogits")
        if self.db is not None:  # runs of 16 in f32, then 64 bits
            got = self.dl.double()
            assert not bool(none.any())
            ref.check(self.db, got.sum(0), 16 * u * got.abs().sum(0), F32_HALF, "dbias")
        return self


MODES = [(s, r, b) for s in ("softmax", "sigmoid") for r in (False, True) for b in ("none", "logit", "select")]


@pytest.mark.parametrize("N,T,E,R", [(1, 1, 1, 1), (1, 5, 2, 2), (2, 19, 6, 3), (1, 100, 31, 8), (3, 11, 33, 4),
                                     (4, 64, 128, 8), (1, 77, 93, 32), (2, 40, 256, 8), (1, 130, 258, 5),
                                     (8, 33, 384, 8), (1, 9, 513, 16), (2, 300, 1024, 32)])
@pytest.mark.parametrize("score,renorm,bias", MODES)
def test_route_grad(N, T, E, R, score, renorm, bias):
    Router(N, T, E, R, score, renorm, bias, seed=E).route().grad().check()


@pytest.mark.parametrize("score,renorm,bias", MODES)
def test_route_grad_of_extreme_logits(score, renorm, bias):
    """Far apart, masked by -infinity or by the type's lowest value, alone, and all masked but one."""
    r = Router(1, 64, 40, 4, score, renorm, bias, seed=9, scale=40.0)
    low = torch.finfo(torch.float32).min
    r.logits[:16, ::3] = float("-inf")
    r.logits[16:32, 1::3] = low
    r.logits[32, :] = 0.0
    r.logits[33] = -87.0 - torch.arange(40, device="cuda")
    r.logits[34] = 80.0 + torch.arange(40, device="cuda")
    r.logits[35, 4:] = float("-inf")  # as many left as are chosen
    r.logits[36, 5:] = low
    r.route().grad().check()
    masked = (r.logits == float("-inf")) & ~torch.isnan(r.w).any(1, keepdim=True)
    assert bool((r.dl[masked] == 0).all())


def test_route_grad_where_nothing_is_left():
    """Softmax over logits that are all -infinity: zeros whatever the weights are."""
    r = Router(1, 3, 36, 2, "softmax", False, "logit", seed=2)
    r.logits[1] = float("-inf")
    r.route().grad()
    assert bool((r.dl[1] == 0).all()) and bool(torch.isfinite(r.dl).all()) and bool(torch.isfinite(r.db).all())


@pytest.mark.parametrize("E", [3, 36, 93, 1024])
def test_route_grad_of_logits_that_are_not_numbers(E):
    """Softmax over a NaN is NaN, whatever the other logits are: also where nothing but NaN and -infinity is left."""
    r = Router(1, 6, E, 2, "softmax", False, "logit", seed=3)
    r.logits[1] = float("nan")
    r.logits[2] = float("-inf")
    r.logits[2, E - 1] = float("nan")
    r.logits[3, 0] = float("nan")
    r.logits[4] = float("-inf")  # nothing left: zeros
    r.idx.copy_(torch.tensor([[0, E - 1]] * 6, device="cuda"))
    r.w.fill_(0.25)
    r.grad()
    bad = torch.isnan(r.dl)
    assert bool(bad[1:4].all()) and not bool(bad[[0, 4, 5]].any()) and bool((r.dl[4] == 0).all())
    assert bool(torch.isnan(r.db).all())


@pytest.mark.parametrize("score,renorm,bias", MODES)
def test_route_grad_of_repeated_and_invalid_ids(score, renorm, bias):
    """An expert that is named twice gets both parts, ids out of range take no part."""
    r = Router(1, 6, 12, 5, score, renorm, bias, seed=4).route()
    r.idx[0] = torch.tensor([3, 7, 3, 3, 7], device="cuda")
    r.idx[1, 2] = 12
    r.idx[2] = -1
    r.idx[3, 0] = 2 ** 31 - 1
    r.grad()
    for g in range(6):
        keep = [k for k in range(5) if 0 <= int(r.idx[g, k]) < 12]
        z, w, h = r.z()[g].cpu(), r.w[g].double().cpu(), r.h[g].double().cpu()
        d = sum(float(w[k] * h[k]) for k in keep)
        want = -torch.softmax(z, 0) * d if score == "softmax" and not renorm else torch.zeros(12, dtype=torch.float64)
        for k in keep:
            e = int(r.idx[g, k])
            if score == "softmax" and not renorm:
                want[e] += torch.softmax(z, 0)[e] * h[k]
            else:
                v = w[k] * (h[k] - d) if renorm else w[k] * h[k]
                want[e] += v / (1 + torch.exp(z[e])) if score == "sigmoid" else v
        # nothing here is larger than about 10: 20 operations of 2^-24 and the exponentials'
        torch.testing.assert_close(r.dl[g].double().cpu(), want, rtol=0, atol=10 * 30 * 2.0 ** -24)


@pytest.mark.parametrize("score,renorm,bias", MODES)
def test_route_grad_against_differences(score, renorm, bias):
    r = Router(1, 12, 10, 3, score, renorm, bias, seed=6, scale=1.0).route().grad()
    idx, h, z = r.idx.long(), r.h.double(), r.z()
    eps = 2.0 ** -12
    for e in range(10):
        up, down = z.clone(), z.clone()
        up[:, e] += eps
        down[:, e] -= eps
        diff = ((weights(up, idx, score, renorm) - weights(down, idx, score, renorm)) * h).sum(1) / (2 * eps)
        # third derivatives of the weights stay below 6 for each of them: eps^2 / 6 of that; f32 on top
        lim = eps ** 2 * h.abs().sum(1) + 40 * 2.0 ** -24 * (1 + h.abs().sum(1))
        assert bool(((diff - r.dl[:, e].double()).abs() <= lim).all()), e


def test_route_grad_of_arrays_that_are_not_16_byte_aligned():
    for score, renorm in (("softmax", False), ("sigmoid", True)):
        r = Router(1, 20, 64, 4, score, renorm, "logit", seed=8).route()
        r.logits = torch.cat([torch.zeros(1, device="cuda"), r.logits.flatten()])[1:].view(20, 64)
        r.dl = torch.full((20 * 64 + 3,), SENTINEL, device="cuda")[3:].view(20, 64)
        r.grad().check()


@pytest.mark.parametrize("score,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
def test_logits_beyond_32_bit_offsets(score, renorm):
    """More than 2^31 logits: the last tokens' gradient is that of a call with them alone."""
    E, R, last = 1024, 8, 500
    T = (1 << 31) // E + last
    few = Router(1, last, E, R, score, renorm, "logit", seed=11).route().grad().check()
    dims = moe.make_dims(1, T, E, R, 8, cap_rows=8)  # the bound on a region's rows would pass 2^31
    logits, dl = torch.zeros(T, E, device="cuda"), torch.full((T, E), SENTINEL, device="cuda")
    idx, w, h = torch.zeros(T, R, dtype=torch.int32, device="cuda"), torch.zeros(T, R, device="cuda"), torch.zeros(T, R, device="cuda")
    idx[:] = torch.arange(R, device="cuda")
    logits[-last:], idx[-last:], w[-last:], h[-last:] = few.logits, few.idx, few.w, few.h
    db = torch.empty(E, device="cuda")
    moe.route_grad(dims, logits, few.bias, few.fn, renorm, idx, w, h, dl, db)
    assert torch.equal(dl[-last:], few.dl)
    assert all(bool((part == 0).all()) for part in dl[:-last].split(1 << 18))
    # the same numbers in other places of the sum: each of the two within what check allows
    mag = few.dl.double().abs().sum(0)
    assert bool(((db.double() - few.db.double()).abs() <= 2 * (16 * 2.0 ** -24 * mag + F32_HALF * (mag + 1e-30))).all())


def test_long_sums_over_tokens():
    r = Router(1, 200000, 40, 2, "softmax", False, "logit", seed=5).route()
    r.h.abs_()
    r.grad().check()


# ---- together -----------------------------------------------------------------

def test_empty_batch():
    d = moe.make_dims(2, 0, 4, 2, 64)
    e = dict(device="cuda")
    b16, i32 = torch.bfloat16, torch.int32
    none = torch.empty(0, 64, dtype=b16, **e)
    rows = torch.full((2, 64), SENTINEL, dtype=b16, **e)
    ids, w = torch.empty(0, 2, dtype=i32, **e), torch.empty(0, 2, **e)
    moe.combine_grad(d, none, rows, ids, w, torch.empty_like(rows), torch.empty_like(w))
    moe.dispatch_grad(d, rows, ids, none)
    db = torch.full((4,), SENTINEL, **e)
    lg = torch.empty(0, 4, **e)
    moe.route_grad(d, lg, None, moe.MOE_SOFTMAX, True, ids, w, w, lg, db)
    assert db.tolist() == [0, 0, 0, 0]


@pytest.mark.parametrize("score,renorm", [("softmax", True), ("sigmoid", True), ("softmax", False)])
def test_layer_against_automatic_differentiation(score, renorm):
    """A whole layer, forward and back, by the library; its gradients against those of a plain layer in 64
    bits.  Eight arrays on the way are rounded to bf16 (packed rows' product g|u, h, y, out; dy, dh, dpre,
    dpacked), each by at most 2^-8 of its elements: 8 * 2^-8 of a gradient's norm is allowed, twice for the
    parts of products of two rounded factors."""
    N, T, E, R, H, F = 2, 90, 8, 3, 256, 136
    g = torch.Generator(device="cuda")
    g.manual_seed(12)
    kw = dict(generator=g, device="cuda")
    fn = moe.MOE_SOFTMAX if score == "softmax" else moe.MOE_SIGMOID
    d = moe.make_dims(N, T, E, R, H)
    b = moe.Buffers(d, separate_y=True)
    NT, rows = N * T, N * b.sizes["cap_rows"]
    bf = torch.bfloat16
    x = torch.randn(NT, H, **kw).to(bf)
    logits, bias = torch.randn(NT, E, **kw), torch.randn(E, **kw) * 0.2
    w1, w2 = (torch.randn(E, 2 * F, H, **kw) * H ** -0.5).to(bf), (torch.randn(E, H, F, **kw) * F ** -0.5).to(bf)
    dout = torch.randn(NT, H, **kw).to(bf)

    def buf(width, dtype=bf):
        return torch.full((rows, width), float("nan"), dtype=dtype, device="cuda")

    h, pre, dy, dh, dpre, dpacked = buf(F), buf(2 * F), buf(H), buf(F), buf(2 * F), buf(H)
    dw1, dw2 = torch.empty(E, 2 * F, H, device="cuda"), torch.empty(E, H, F, device="cuda")
    dw, dx = torch.empty(NT, R, device="cuda"), torch.empty(NT, H, dtype=bf, device="cuda")
    dl, db = torch.empty(NT, E, device="cuda"), torch.empty(E, device="cuda")

    def step():
        moe.route_topk(d, logits, bias, fn, renorm, b.topk_idx, b.topk_w)
        moe.dispatch_count(d, b.topk_idx, b.expert_counts, b.expert_offsets, b.rank_counts, b.rank_offsets,
                           b.send_counts, b.pos, b.status)
        moe.dispatch_pack(d, x, None, b.pos, b.packed_x, None, b.packed_src)
        off = b.expert_offsets
        moe.expert_gemm(d, H, F, moe.MOE_EXPERT_SWIGLU, b.packed_x, w1, off, h, pre)
        moe.expert_gemm(d, F, H, moe.MOE_EXPERT_LINEAR, h, w2, off, b.y)
        moe.combine(d, b.y, b.pos, b.topk_w, b.out)
        moe.combine_grad(d, dout, b.y, b.pos, b.topk_w, dy, dw)
        moe.expert_gemm_dgrad(d, F, H, dy, w2, off, dh)
        moe.expert_gemm_wgrad(d, F, H, dy, h, off, dw2)
        moe.expert_swiglu_grad(d, F, pre, dh, off, dpre)
        moe.expert_gemm_dgrad(d, H, 2 * F, dpre, w1, off, dpacked)
        moe.expert_gemm_wgrad(d, H, 2 * F, dpre, b.packed_x, off, dw1)
        moe.dispatch_grad(d, dpacked, b.pos, dx)
        moe.route_grad(d, logits, bias, fn, renorm, b.topk_idx, b.topk_w, dw, dl, db)

    step()
    eager = [t.clone() for t in (dx, dl, db, dw1, dw2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    with torch.cuda.graph(graph):
        step()
    for t in (dx, dl, db, dw1, dw2):
        t.fill_(float("nan"))
    graph.replay()
    for a, c in zip(eager, (dx, dl, db, dw1, dw2)):
        assert torch.equal(a, c)

    leaves = [t.double().requires_grad_() for t in (x, logits, bias, w1, w2)]
    xd, ld, bd, a1, a2 = leaves
    wts = weights(ld + bd, b.topk_idx.long(), score, renorm)
    out = torch.zeros(NT, H, dtype=torch.float64, device="cuda")
    for k in range(R):
        for e in range(E):
            tok = (b.topk_idx[:, k] == e).nonzero().flatten()
            gu = xd[tok] @ a1[e].t()
            hh = torch.nn.functional.silu(gu[:, :F]) * gu[:, F:]
            out = out.index_add(0, tok, wts[tok, k:k + 1] * (hh @ a2[e].t()))
    out.backward(dout.double())
    for got, want, name in [(eager[0], xd.grad, "dx"), (eager[1], ld.grad, "dlogits"), (eager[2], bd.grad, "dbias"),
                            (eager[3], a1.grad, "dw1"), (eager[4], a2.grad, "dw2")]:
        rel = float((got.double() - want).norm() / want.norm())
        assert rel <= 16 * 2.0 ** -8, (name, rel)


def test_other_streams_and_calls_at_the_same_time():
    """Two batches on two streams, in turns, give the bits of one after the other."""
    batches = [Routed(2, 300, 16, 4, 2048, 0, s) for s in (1, 2)]
    args = []
    for b in batches:
        args.append((b.randn(b.NT, b.H), b.packed(b.H), torch.rand(b.NT, b.R, generator=b.g, device="cuda")))

    def run(b, a, stream=None):
        dy, dw, dx = torch.full_like(a[1], SENTINEL), torch.empty_like(a[2]), torch.empty_like(a[0])
        torch.cuda.synchronize()
        for _ in range(20):
            moe.combine_grad(b.dims, a[0], a[1], b.pos, a[2], dy, dw, stream=stream)
            moe.dispatch_grad(b.dims, a[1], b.pos, dx, a[0], stream=stream)
        return dy, dw, dx

    alone = [run(b, a) for b, a in zip(batches, args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in batches]
    both = [run(b, a, s) for b, a, s in zip(batches, args, streams)]
    torch.cuda.synchronize()
    for x, y in zip(alone, both):
        for s, t in zip(x, y):
            assert torch.equal(s, t)


def test_binding_refuses_other_shapes_and_types():
    b = Routed(1, 8, 4, 2, 64, 0, 1)
    dout, y, w = b.randn(8, 64), b.randn(b.rows, 64), torch.rand(8, 2, device="cuda")
    dy, dw = torch.empty_like(y), torch.empty_like(w)
    with pytest.raises(ValueError, match="dout must be"):
        moe.combine_grad(b.dims, dout.float(), y, b.pos, w, dy, dw)
    with pytest.raises(ValueError, match="contiguous"):
        moe.combine_grad(b.dims, dout, y.t(), b.pos, w, dy, dw)
    with pytest.raises(ValueError, match="needs"):
        moe.combine_grad(b.dims, dout, y[:-1], b.pos, w, dy, dw)
    with pytest.raises(ValueError, match="dtopk_w is required"):
        moe.combine_grad(b.dims, dout, y, b.pos, w, dy, None)
    with pytest.raises(moe.MoeError, match="overlaps"):
        moe.combine_grad(b.dims, dout, y, b.pos, w, y, dw)
    with pytest.raises(moe.MoeError, match="overlaps"):
        moe.dispatch_grad(b.dims, y, b.pos, y[:8])
