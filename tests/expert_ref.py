"""The experts' products in 64 bits, and how far the kernels may be from them.

Errors allowed, derived for each kernel from its arithmetic:

* a sum of n products held in f32: every addition, in whatever order and
  even truncated, is off by at most one unit in the last place (2^-23) of a
  partial sum, and no partial sum exceeds the sum of magnitudes:
  err <= (n + 4) 2^-23 sum|a b|.  The four cover scale products and, in the
  fp8 product, the multiply-add that joins two blocks.
* a result rounded to bf16: half a step, 2^-8 of its value (f32: 2^-24).
* h = g / (1 + exp(-g)) u from g + eg, u + eu: |silu'| <= 1.1 and |silu(g)| <=
  |g|, so err <= 1.1 eg (|u| + eu) + |g| eu, plus the f32 operations: exp is within
  2 units, an addition and a product within one half each, the division
  within 2 units, which 16 2^-24 |h| covers; a divisor above 2^126 (g below
  -87.3) may give 0, where |h| <= 87.4 2^-126 |u| < 2e-36 |u|.
* requantised h: half a step of e4m3, 2^-4 of the value (2^-10 scales where
  the code is subnormal), on top of h's own error; the step is taken at the
  kernel's scale, itself off by the error of the largest |h| over 448.
"""
from __future__ import annotations

import torch

import combine_moe_route_topk_gb300 as moe

BF16_HALF, F32_HALF, E4M3_HALF = 2.0 ** -8, 2.0 ** -24, 2.0 ** -4
SENTINEL = -77.0


class Batch:
    """Routed rows without a router: `counts[e]` rows for expert e in the
    regions of N ranks of `cap` rows.  pairs = N T R is at least their sum."""

    def __init__(self, N, counts, cap, seed=0, device="cuda"):
        self.N, self.E, self.cap = N, len(counts), cap
        self.L = self.E // N
        self.rows = N * cap
        off = [0]
        for c in counts:
            off.append(off[-1] + c)
        self.off = off
        self.offsets = torch.tensor(off, dtype=torch.int32, device=device)
        self.g = torch.Generator(device=device)
        self.g.manual_seed(seed)
        self.device = device
        self.T = -(-max(1, off[-1]) // N)
        self.valid = torch.zeros(self.rows, dtype=torch.bool, device=device)
        for e in range(self.E):
            self.valid[self.span(e)] = True

    def span(self, e):
        base = self.off[e // self.L * self.L]
        lo, hi = (min(self.off[i] - base, self.cap) for i in (e, e + 1))
        return slice(e // self.L * self.cap + lo, e // self.L * self.cap + hi)

    def dims(self, y_dtype=moe.MOE_BF16):
        return moe.make_dims(self.N, self.T, self.E, 1, 8, y_dtype=y_dtype, cap_rows=self.cap)

    def randn(self, *shape, scale=1.0):
        return (torch.randn(*shape, generator=self.g, device=self.device) * scale).to(torch.bfloat16)

    def row_values(self, width, scale=1.0):
        """bf16 rows; rows without a token hold NaN, infinities and the type's lowest value."""
        t = self.randn(self.rows, width, scale=scale)
        bad = torch.tensor([float("nan"), float("inf"), float("-inf"), torch.finfo(torch.bfloat16).min],
                           device=self.device, dtype=torch.bfloat16)
        out = (~self.valid).nonzero().flatten()
        t[out] = bad[torch.arange(len(out), device=self.device) % 4].unsqueeze(1)
        return t

    def out(self, width, dtype):
        return torch.full((self.rows, width), SENTINEL, dtype=dtype, device=self.device)


def product(b: Batch, x, w):
    """(y, sum of magnitudes), both f64: rows of x times w[e]^T, w [E][F][K]."""
    y = torch.zeros(b.rows, w.shape[1], dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(y)
    for e in range(b.E):
        r = b.span(e)
        if r.stop > r.start:
            a, m = x[r].double(), w[e].double().t()
            y[r], mag[r] = a @ m, a.abs() @ m.abs()
    return y, mag


def sum_error(n, mag):
    return (n + 4) * 2.0 ** -23 * mag


def swiglu(g, u, eg, eu):
    """(h, its error) of the f32 computation from sums that are off by eg, eu."""
    h = g * torch.special.expit(g) * u
    return h, 1.1 * eg * (u.abs() + eu) + g.abs() * eu + 16 * F32_HALF * h.abs() + 2e-36 * u.abs()


def check(got, ref, err, half, what):
    """|got - ref| <= err + half step of the computed value's type."""
    got = got.double()
    lim = err + half * (ref.abs() + err) + 1e-38
    bad = ~((got - ref).abs() <= lim)  # NaN fails too
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: got "
                             f"{got[i].item()!r}, want {ref[i].item()!r} +- {lim[i].item():.3g}")


def check_untouched(b: Batch, t, sentinel=SENTINEL):
    assert bool((t[~b.valid].float() == sentinel).all()), "rows without a token were written"


def quantise(x):
    """bf16/f32 rows as e4m3 codes (uint8) and one f32 scale (amax / 448) per 128."""
    f = x.float().view(x.shape[0], -1, 128)
    s = f.abs().amax(2) / 448.0
    q = (f / torch.where(s > 0, s, torch.ones_like(s)).unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return q.view(x.shape).view(torch.uint8), s


def e4m3(t):
    return t.view(torch.float8_e4m3fn).double()


def dequant_rows(q, s):
    return (e4m3(q).unflatten(1, (-1, 128)) * s.double().unsqueeze(2)).flatten(1)


def dequant_matrix(q, s):
    """[E][W][K] codes with one scale per 128 x 128 block."""
    w = e4m3(q)
    full = s.double().repeat_interleave(128, 1)[:, : w.shape[1]].repeat_interleave(128, 2)
    return w * full
