"""Long sums of the experts' products in bf16: what the tensor core cuts off must not grow with the length.

A sum of n products in parts of 2048: within a part every addition is off by at
most one unit in the last place (2^-23) of a partial sum, and the joining
additions, rounded to nearest, by half a unit each:
err <= (2052 2^-23 + ceil(n / 2048) 2^-24) sum|a b|.  For n = 2^20 that is 2.8e-4 of
a sum of positive terms, where one accumulator loses about 4e-3 of it, as much
as the rounding to bf16 (half a step: 2^-8 of the value, at most)."""
import pytest
import torch

import combine_moe_route_topk_gb300 as moe
import expert_ref as ref
from expert_ref import BF16_HALF, Batch

pytestmark = pytest.mark.gpu
LINEAR, SWIGLU = moe.MOE_EXPERT_LINEAR, moe.MOE_EXPERT_SWIGLU
LONG = (1 << 20) + 72  # ends inside a stage
CHUNK = 1 << 17


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_moe_route_topk_gb300 import _build
    _build.build()
    yield
    assert moe.take_device_error() == moe.MOE_OK


def _part_error(n, mag):
    return (2052 * 2.0 ** -23 + -(-n // 2048) * 2.0 ** -24) * mag


def _positive(*shape, scale=1.0, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    t = torch.empty(*shape, dtype=torch.bfloat16, device="cuda")
    return t.uniform_(0.5, 1.5, generator=g).mul_(scale)


def _product(b, x, w):
    """Rows of x times w[e]^T in 64 bits, by chunks of the reduction (all terms positive: also the sum of magnitudes)."""
    y = torch.zeros(b.rows, w.shape[1], dtype=torch.float64, device="cuda")
    for e in range(b.E):
        r = b.span(e)
        for k in range(0, x.shape[1], CHUNK):
            y[r] += x[r, k:k + CHUNK].double() @ w[e, :, k:k + CHUNK].double().t()
    return y


def test_linear():
    b, F = Batch(1, [40, 0, 300], 350), 72
    x, w, y = _positive(b.rows, LONG), _positive(b.E, F, LONG, seed=1), b.out(F, torch.bfloat16)
    moe.expert_gemm(b.dims(), LONG, F, LINEAR, x, w, b.offsets, y)
    want = _product(b, x, w)
    ref.check(y[b.valid], want[b.valid], _part_error(LONG, want[b.valid]), BF16_HALF, "y")
    ref.check_untouched(b, y)


@pytest.mark.parametrize("save", [False, True])
def test_gated(save):
    b, F = Batch(1, [40, 0, 300], 350), 40
    x, w = _positive(b.rows, LONG), _positive(b.E, 2 * F, LONG, scale=8.0 / LONG, seed=1)
    y, pre = b.out(F, torch.bfloat16), b.out(2 * F, torch.bfloat16) if save else None
    moe.expert_gemm(b.dims(), LONG, F, SWIGLU, x, w, b.offsets, y, pre)
    want = _product(b, x, w)[b.valid]
    err = _part_error(LONG, want)
    h, eh = ref.swiglu(want[:, :F], want[:, F:], err[:, :F], err[:, F:])
    ref.check(y[b.valid], h, eh, BF16_HALF, "h")
    ref.check_untouched(b, y)
    if save:
        ref.check(pre[b.valid], want, err, BF16_HALF, "pre")
        ref.check_untouched(b, pre)


def test_dgrad():
    b, K = Batch(1, [40, 0, 300], 350), 72
    dy, w, dx = _positive(b.rows, LONG), _positive(b.E, LONG, K, seed=1), b.out(K, torch.bfloat16)
    moe.expert_gemm_dgrad(b.dims(), K, LONG, dy, w, b.offsets, dx)
    want = torch.zeros(b.rows, K, dtype=torch.float64, device="cuda")
    for e in range(b.E):
        r = b.span(e)
        for k in range(0, LONG, CHUNK):
            want[r] += dy[r, k:k + CHUNK].double() @ w[e, k:k + CHUNK].double()
    ref.check(dx[b.valid], want[b.valid], _part_error(LONG, want[b.valid]), BF16_HALF, "dx")
    ref.check_untouched(b, dx)


def test_wgrad():
    counts, K, F = [30, 0, LONG - 66, 5], 136, 72
    b = Batch(1, counts, sum(counts))
    dy, x = _positive(b.rows, F), _positive(b.rows, K, seed=1)
    dw = torch.full((b.E, F, K), ref.SENTINEL, dtype=torch.bfloat16, device="cuda")
    moe.expert_gemm_wgrad(b.dims(), K, F, dy, x, b.offsets, dw)
    for e in range(b.E):
        r = b.span(e)
        want = torch.zeros(F, K, dtype=torch.float64, device="cuda")
        for p in range(r.start, r.stop, CHUNK):
            q = slice(p, min(p + CHUNK, r.stop))
            want += dy[q].double().t() @ x[q].double()
        ref.check(dw[e], want, _part_error(counts[e], want), BF16_HALF, f"dw[{e}]")


@pytest.mark.parametrize("n", [1 << 14, (1 << 14) + 8, 50000])
@pytest.mark.parametrize("form", ["linear", "gated", "dgrad"])
def test_both_sides_of_the_length(form, n):
    """The longest sum in one accumulator and the shortest in parts, with signs, empty experts, a region that
    overflows and rows without a token that hold NaN."""
    b = Batch(2, [300, 31, 0, 2], 320)
    out = 136
    x = b.row_values(n)
    if form == "dgrad":
        w, y = b.randn(b.E, n, out, scale=n ** -0.5), b.out(out, torch.bfloat16)
        moe.expert_gemm_dgrad(b.dims(), out, n, x, w, b.offsets, y)
        w = w.transpose(1, 2)
    else:
        w = b.randn(b.E, 2 * out if form == "gated" else out, n, scale=n ** -0.5)
        y = b.out(out, torch.bfloat16)
        moe.expert_gemm(b.dims(), n, out, SWIGLU if form == "gated" else LINEAR, x, w, b.offsets, y)
    want, mag = ref.product(b, x, w)
    # one accumulator: the bound of any order of additions
    err = (_part_error(n, mag) if n > 1 << 14 else ref.sum_error(n, mag))[b.valid]
    want = want[b.valid]
    if form == "gated":
        want, err = ref.swiglu(want[:, :out], want[:, out:], err[:, :out], err[:, out:])
    ref.check(y[b.valid], want, err, BF16_HALF, "y")
    ref.check_untouched(b, y)


@pytest.mark.parametrize("K,F", [(8, 8), (200, 264), (1000, 520)])
def test_wgrad_of_a_batch_that_could_be_long(K, F):
    """Few rows of an expert in a batch that could give it many: the form for long sums, its tile edges."""
    counts = [0, 5, 129, 16, 0, 513, 0]
    b = Batch(1, counts, 1000)
    d = moe.make_dims(1, 70000, b.E, 1, 8, cap_rows=70000)
    rows = 70000
    dy, x = (torch.full((rows, n), float("nan"), dtype=torch.bfloat16, device="cuda") for n in (F, K))
    dy[:sum(counts)], x[:sum(counts)] = b.randn(sum(counts), F), b.randn(sum(counts), K)
    dw = torch.full((b.E, F, K), ref.SENTINEL, dtype=torch.bfloat16, device="cuda")
    moe.expert_gemm_wgrad(d, K, F, dy, x, b.offsets, dw)
    for e in range(b.E):
        r = b.span(e)
        p, q = dy[r].double(), x[r].double()
        ref.check(dw[e], p.t() @ q, ref.sum_error(r.stop - r.start, p.abs().t() @ q.abs()), BF16_HALF, f"dw[{e}]")


def test_the_most_rows():
    """An expert of almost 2^31 rows: its rows and the number of its tiles added up pass 32 bits."""
    rows, first, K, F = (1 << 31) - 1 - 65536, 1000003, 8, 8
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 120 << 30:
        pytest.skip("rows and results take 70 GB")
    d = moe.make_dims(1, rows, 2, 1, 8, cap_rows=rows)
    off = torch.tensor([0, first, rows], dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    x, y = (torch.empty(rows, n, dtype=torch.bfloat16, device="cuda") for n in (K, F))
    step = 1 << 25
    for i in range(0, rows, step):
        x[i:i + step].normal_(generator=g)
        y[i:i + step].fill_(ref.SENTINEL)
    w = torch.randn(2, F, K, generator=g, device="cuda").to(torch.bfloat16)
    moe.expert_gemm(d, K, F, LINEAR, x, w, off, y)
    for i in range(0, rows, step):
        for e, lo, hi in ((0, i, min(i + step, first)), (1, max(i, first), min(i + step, rows))):
            if lo < hi:
                a, m = x[lo:hi].double(), w[e].double().t()
                ref.check(y[lo:hi], a @ m, ref.sum_error(K, a.abs() @ m.abs()), BF16_HALF, f"rows {lo} to {hi}")
