"""The experts' products against plain 64-bit products (tolerances: expert_ref)."""
import pytest
import torch

import combine_moe_route_topk_gb300 as moe
import expert_ref as ref
from expert_ref import BF16_HALF, E4M3_HALF, F32_HALF, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_moe_route_topk_gb300 import _build
    _build.build()
    yield
    assert moe.take_device_error() == moe.MOE_OK


# N, rows per expert, cap.  One row; tile edges on either side of 16, 32, 64,
# 128 and 256 rows; empty experts first, last and in between; a region that
# overflows (inside an expert, and before one); every expert empty.
ROWS = [
    (1, [1], 1),
    (1, [5, 0, 16, 17], 40),
    (2, [0, 33, 64, 65, 0, 1], 200),
    (2, [127, 128, 129, 0], 257),
    (1, [255, 256, 257], 800),
    (2, [300, 31, 15, 2], 320),     # rank 0 loses 11 rows of its second expert
    (2, [50, 9, 3, 0], 40),         # rank 0's second expert lies past the region
    (1, [700], 700),
    (3, [0, 0, 0], 8),
    (4, [3, 0, 0, 2, 0, 0, 7, 1], 12),
    (1, [600, 1, 0, 200], 900),     # many rows on average, and experts with few
]
SIZES = [(8, 8), (64, 128), (72, 136), (200, 264), (512, 96), (1000, 520)]


def _ids(v):
    return str(v).replace(" ", "")


@pytest.mark.parametrize("K,F", SIZES, ids=_ids)
@pytest.mark.parametrize("N,counts,cap", ROWS, ids=_ids)
@pytest.mark.parametrize("f32", [False, True])
def test_linear(N, counts, cap, K, F, f32):
    b = Batch(N, counts, cap)
    x, w = b.row_values(K), b.randn(b.E, F, K, scale=K ** -0.5)
    y = b.out(F, torch.float32 if f32 else torch.bfloat16)
    moe.expert_gemm(b.dims(moe.MOE_F32 if f32 else moe.MOE_BF16), K, F, moe.MOE_EXPERT_LINEAR, x, w, b.offsets, y)
    want, mag = ref.product(b, x, w)
    ref.check(y[b.valid], want[b.valid], ref.sum_error(K, mag)[b.valid], F32_HALF if f32 else BF16_HALF, "y")
    ref.check_untouched(b, y)


@pytest.mark.parametrize("K,F", SIZES, ids=_ids)
@pytest.mark.parametrize("N,counts,cap", ROWS, ids=_ids)
@pytest.mark.parametrize("save", [False, True])
def test_gated(N, counts, cap, K, F, save):
    b = Batch(N, counts, cap)
    x, w = b.row_values(K), b.randn(b.E, 2 * F, K, scale=2 * K ** -0.5)
    y, pre = b.out(F, torch.bfloat16), b.out(2 * F, torch.bfloat16) if save else None
    moe.expert_gemm(b.dims(), K, F, moe.MOE_EXPERT_SWIGLU, x, w, b.offsets, y, pre)
    want, mag = ref.product(b, x, w)
    err = ref.sum_error(K, mag)
    h, eh = ref.swiglu(want[:, :F], want[:, F:], err[:, :F], err[:, F:])
    ref.check(y[b.valid], h[b.valid], eh[b.valid], BF16_HALF, "h")
    ref.check_untouched(b, y)
    if save:
        ref.check(pre[b.valid], want[b.valid], err[b.valid], BF16_HALF, "pre")
        ref.check_untouched(b, pre)


@pytest.mark.parametrize("K,F", SIZES, ids=_ids)
@pytest.mark.parametrize("N,counts,cap", ROWS, ids=_ids)
def test_dgrad(N, counts, cap, K, F):
    b = Batch(N, counts, cap)
    dy, w = b.row_values(F), b.randn(b.E, F, K, scale=K ** -0.5)
    dx = b.out(K, torch.bfloat16)
    moe.expert_gemm_dgrad(b.dims(), K, F, dy, w, b.offsets, dx)
    want, mag = ref.product(b, dy, w.transpose(1, 2))
    ref.check(dx[b.valid], want[b.valid], ref.sum_error(F, mag)[b.valid], BF16_HALF, "dx")
    ref.check_untouched(b, dx)


def _matrix_tiles(b, shift):
    """Least number of tiles of matrix rows with which token tiles of 2^shift rows are the longest that are needed
    (9: tiles of 256 rows take more than four rounds and are sorted by size)."""
    def tiles(k):
        return sum(-(-(b.span(e).stop - b.span(e).start) // 2 ** k) for e in range(b.E))
    pairs = torch.cuda.get_device_properties(0).multi_processor_count // 2
    return 1 if shift == 6 else (4 if shift == 9 else 1) * pairs // tiles(shift - 1) + 1


@pytest.mark.parametrize("form", ["linear", "f32", "gated", "dgrad"])
@pytest.mark.parametrize("shift", [6, 7, 8, 9])
@pytest.mark.parametrize("N,counts,cap", [r for r in ROWS if max(r[1]) > 64], ids=_ids)
def test_token_tiles(N, counts, cap, shift, form):
    """Small batches are cut into tiles of 64 or 128 tokens so that all pairs of blocks get one: each size, by the
    number of columns."""
    b = Batch(N, counts, cap)
    step = 128 if form == "gated" else 256
    F, K = _matrix_tiles(b, shift) * step - 40, 72
    x = b.row_values(K)
    if form == "dgrad":
        w = b.randn(b.E, K, F, scale=K ** -0.5)
        y = b.out(F, torch.bfloat16)
        moe.expert_gemm_dgrad(b.dims(), F, K, x, w, b.offsets, y)
        want, mag = ref.product(b, x, w.transpose(1, 2))
        err = ref.sum_error(K, mag)
    else:
        w = b.randn(b.E, 2 * F if form == "gated" else F, K, scale=K ** -0.5)
        y = b.out(F, torch.float32 if form == "f32" else torch.bfloat16)
        moe.expert_gemm(b.dims(moe.MOE_F32 if form == "f32" else moe.MOE_BF16), K, F,
                        moe.MOE_EXPERT_SWIGLU if form == "gated" else moe.MOE_EXPERT_LINEAR, x, w, b.offsets, y)
        want, mag = ref.product(b, x, w)
        err = ref.sum_error(K, mag)
        if form == "gated":
            want, err = ref.swiglu(want[:, :F], want[:, F:], err[:, :F], err[:, F:])
    ref.check(y[b.valid], want[b.valid], err[b.valid], F32_HALF if form == "f32" else BF16_HALF, "y")
    ref.check_untouched(b, y)


@pytest.mark.parametrize("form", ["linear", "dgrad"])
@pytest.mark.parametrize("N,E,most,F", [(1, 33, 520, 2056), (2, 70, 300, 1288), (4, 1024, 40, 264)])
def test_many_experts(N, E, most, F, form):
    """Experts of mixed sizes, some of them empty, in more tiles than four rounds: sorted by the size of their tiles."""
    g = torch.Generator().manual_seed(E)
    counts = (torch.rand(E, generator=g) * 1.2 * most - 0.2 * most).clamp(min=0).int().tolist()
    b = Batch(N, counts, max(sum(counts[r * E // N:(r + 1) * E // N]) for r in range(N)))
    K = 72
    x = b.row_values(K)
    y = b.out(F, torch.bfloat16)
    if form == "linear":
        w = b.randn(E, F, K, scale=K ** -0.5)
        moe.expert_gemm(b.dims(), K, F, moe.MOE_EXPERT_LINEAR, x, w, b.offsets, y)
    else:
        w = b.randn(E, K, F, scale=K ** -0.5)
        moe.expert_gemm_dgrad(b.dims(), F, K, x, w, b.offsets, y)
        w = w.transpose(1, 2)
    want, mag = ref.product(b, x, w)
    ref.check(y[b.valid], want[b.valid], ref.sum_error(K, mag)[b.valid], BF16_HALF, "y")
    ref.check_untouched(b, y)


@pytest.mark.parametrize("K,F", SIZES, ids=_ids)
@pytest.mark.parametrize("N,counts,cap", ROWS, ids=_ids)
@pytest.mark.parametrize("f32", [False, True])
def test_wgrad(N, counts, cap, K, F, f32):
    b = Batch(N, counts, cap)
    dy, x = b.row_values(F), b.row_values(K)
    dw = torch.full((b.E, F, K), ref.SENTINEL, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    moe.expert_gemm_wgrad(b.dims(), K, F, dy, x, b.offsets, dw)
    for e in range(b.E):
        r = b.span(e)
        d, v = dy[r].double(), x[r].double()
        ref.check(dw[e], d.t() @ v, ref.sum_error(r.stop - r.start, d.abs().t() @ v.abs()),
                  F32_HALF if f32 else BF16_HALF, f"dw[{e}]")


@pytest.mark.parametrize("N,counts,cap", [r for r in ROWS if sum(r[1]) > 0], ids=_ids)
@pytest.mark.parametrize("f32", [False, True])
def test_wgrad_wide(N, counts, cap, f32):
    """So many columns that tiles of 128 do not run at once, for one expert either, and tiles of 256 are taken."""
    test_wgrad(N, counts, cap, 2056, 2568, f32)


@pytest.mark.parametrize("F", [8, 136, 264, 2048, 2056])
@pytest.mark.parametrize("N,counts,cap", ROWS, ids=_ids)
def test_swiglu_grad(N, counts, cap, F):
    b = Batch(N, counts, cap)
    pre, dh = b.row_values(2 * F, scale=3.0), b.row_values(F)
    if b.valid.any():  # extremes: exp overflows, and the sigmoid is 1
        first = int(b.valid.nonzero()[0])
        pre[first, :4] = torch.tensor([-300.0, 300.0, -88.5, 88.5])
    dpre = b.out(2 * F, torch.bfloat16)
    moe.expert_swiglu_grad(b.dims(), F, pre, dh, b.offsets, dpre)
    g, u, d = pre[b.valid, :F].double(), pre[b.valid, F:].double(), dh[b.valid].double()
    s, t = torch.special.expit(g), torch.special.expit(-g)
    # s and 1 - s each carry a few f32 units; 1 - s is absolute, times g
    du_err = 16 * F32_HALF * (d * g * s).abs() + 1e-36 * (d * g).abs()
    dg_err = 16 * F32_HALF * (d * u * s).abs() * (1 + g.abs()) + 1e-36 * (d * u).abs() * (1 + g.abs())
    ref.check(dpre[b.valid, :F], d * u * s * (1 + g * t), dg_err, BF16_HALF, "dg")
    ref.check(dpre[b.valid, F:], d * g * s, du_err, BF16_HALF, "du")
    ref.check_untouched(b, dpre)


@pytest.mark.parametrize("N,E,cap", [(2, 2, 1), (31, 31, 9), (33, 66, 5), (70, 70, 12), (256, 512, 7), (1024, 1024, 4)])
def test_swiglu_grad_ranks(N, E, cap):
    """Many ranks, some without rows and some whose region overflows."""
    g = torch.Generator().manual_seed(N)
    counts = (torch.rand(E, generator=g) * 16 - 4).clamp(min=0).int().tolist()
    b = Batch(N, counts, cap, seed=N)
    F = 136
    pre, dh = b.row_values(2 * F, scale=3.0), b.row_values(F)
    dpre = b.out(2 * F, torch.bfloat16)
    moe.expert_swiglu_grad(b.dims(), F, pre, dh, b.offsets, dpre)
    g, u, d = pre[b.valid, :F].double(), pre[b.valid, F:].double(), dh[b.valid].double()
    s, t = torch.special.expit(g), torch.special.expit(-g)
    ref.check(dpre[b.valid, :F], d * u * s * (1 + g * t), 16 * F32_HALF * (d * u * s).abs() * (1 + g.abs()), BF16_HALF, "dg")
    ref.check(dpre[b.valid, F:], d * g * s, 16 * F32_HALF * (d * g * s).abs(), BF16_HALF, "du")
    ref.check_untouched(b, dpre)


def _fp8_operands(b, K, W):
    x = b.row_values(K)
    x[~b.valid] = 0
    xq, xs = ref.quantise(x)
    xq[~b.valid] = 0x7f  # NaN codes and NaN scales where no token is
    xs[~b.valid] = float("nan")
    wq = (torch.randn(b.E, W, K, generator=b.g, device="cuda") * 64).to(torch.float8_e4m3fn).view(torch.uint8)
    ws = (0.5 + torch.rand(b.E, -(-W // 128), K // 128, generator=b.g, device="cuda")) * (K ** -0.5 / 32)
    return xq, xs, wq, ws


@pytest.mark.parametrize("K,F", [(128, 8), (256, 128), (384, 136), (1152, 264), (640, 520)], ids=_ids)
@pytest.mark.parametrize("N,counts,cap", ROWS, ids=_ids)
@pytest.mark.parametrize("f32", [False, True])
def test_fp8_linear(N, counts, cap, K, F, f32):
    b = Batch(N, counts, cap)
    xq, xs, wq, ws = _fp8_operands(b, K, F)
    y = b.out(F, torch.float32 if f32 else torch.bfloat16)
    moe.expert_gemm_fp8(b.dims(moe.MOE_F32 if f32 else moe.MOE_BF16), K, F, moe.MOE_EXPERT_LINEAR, xq, xs, wq, ws,
                        b.offsets, y)
    want, mag = ref.product(b, ref.dequant_rows(xq, xs), ref.dequant_matrix(wq, ws))
    ref.check(y[b.valid], want[b.valid], ref.sum_error(K, mag)[b.valid], F32_HALF if f32 else BF16_HALF, "y")
    ref.check_untouched(b, y)


@pytest.mark.parametrize("last", [8, 136], ids=["one_block_last", "two_blocks_last"])
@pytest.mark.parametrize("N,counts,cap", [r for r in ROWS if sum(r[1]) > 0], ids=_ids)
@pytest.mark.parametrize("f32", [False, True])
def test_fp8_wide(N, counts, cap, last, f32):
    """So many columns that the tiles of 128 do not run at once and tiles of 256 are taken."""
    b = Batch(N, counts, cap)
    tiles = sum(-(-(b.span(e).stop - b.span(e).start) // 128) for e in range(b.E))
    K, F = 256, torch.cuda.get_device_properties(0).multi_processor_count // tiles // 2 * 256 + 256 + last
    xq, xs, wq, ws = _fp8_operands(b, K, F)
    y = b.out(F, torch.float32 if f32 else torch.bfloat16)
    moe.expert_gemm_fp8(b.dims(moe.MOE_F32 if f32 else moe.MOE_BF16), K, F, moe.MOE_EXPERT_LINEAR, xq, xs, wq, ws,
                        b.offsets, y)
    want, mag = ref.product(b, ref.dequant_rows(xq, xs), ref.dequant_matrix(wq, ws))
    ref.check(y[b.valid], want[b.valid], ref.sum_error(K, mag)[b.valid], F32_HALF if f32 else BF16_HALF, "y")
    ref.check_untouched(b, y)


@pytest.mark.parametrize("K,F", [(128, 128), (384, 256), (1152, 384), (640, 640)], ids=_ids)
@pytest.mark.parametrize("N,counts,cap", ROWS, ids=_ids)
def test_fp8_gated(N, counts, cap, K, F):
    b = Batch(N, counts, cap)
    xq, xs, wq, ws = _fp8_operands(b, K, 2 * F)
    y = torch.full((b.rows, F), 0xA5, dtype=torch.uint8, device="cuda")
    ys = b.out(F // 128, torch.float32)
    moe.expert_gemm_fp8(b.dims(), K, F, moe.MOE_EXPERT_SWIGLU, xq, xs, wq, ws, b.offsets, y, ys)
    want, mag = ref.product(b, ref.dequant_rows(xq, xs), ref.dequant_matrix(wq, ws))
    err = ref.sum_error(K, mag)
    h, eh = ref.swiglu(want[:, :F], want[:, F:], err[:, :F], err[:, F:])
    h, eh = h[b.valid].unflatten(1, (-1, 128)), eh[b.valid].unflatten(1, (-1, 128))
    scale = h.abs().amax(2) / 448
    ref.check(ys[b.valid], scale, eh.amax(2) / 448, 2 * F32_HALF, "scales")
    got_s = ys[b.valid].double().unsqueeze(2)
    got = ref.e4m3(y[b.valid]).unflatten(1, (-1, 128)) * got_s
    ref.check(got, h, eh + got_s * 2.0 ** -10 + 4 * F32_HALF * h.abs(), E4M3_HALF, "codes")
    ref.check_untouched(b, ys)
    assert bool((y[~b.valid] == 0xA5).all())


def test_fp8_gated_many_tiles():
    """Several tiles for each block, in a row: the tokens' largest values of one tile and the next stay apart.  The
    tokens' scales lie 2^-12 to 2^12 apart from tile to tile, so a value of another tile would show."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    K, F, rows = 128, 256, 128 * sms * 2 + 77
    b = Batch(1, [rows], rows)
    xq, xs, wq, ws = _fp8_operands(b, K, 2 * F)
    xs *= torch.exp2(((torch.arange(rows, device="cuda") // 61) % 25 - 12).float()).unsqueeze(1)
    y = torch.full((rows, F), 0xA5, dtype=torch.uint8, device="cuda")
    ys = b.out(F // 128, torch.float32)
    moe.expert_gemm_fp8(b.dims(), K, F, moe.MOE_EXPERT_SWIGLU, xq, xs, wq, ws, b.offsets, y, ys)
    want, mag = ref.product(b, ref.dequant_rows(xq, xs), ref.dequant_matrix(wq, ws))
    err = ref.sum_error(K, mag)
    h, eh = ref.swiglu(want[:, :F], want[:, F:], err[:, :F], err[:, F:])
    h, eh = h.unflatten(1, (-1, 128)), eh.unflatten(1, (-1, 128))
    # the scale's own division: half a unit, and 2^-150 where it is below the normal range
    ref.check(ys, h.abs().amax(2) / 448, eh.amax(2) / 448 + 2.0 ** -149, 2 * F32_HALF, "scales")
    got_s = ys.double().unsqueeze(2)
    ref.check(ref.e4m3(y).unflatten(1, (-1, 128)) * got_s, h, eh + got_s * 2.0 ** -10 + 4 * F32_HALF * h.abs(), E4M3_HALF,
              "codes")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("K,F", [(264, 520), (1024, 1024)], ids=_ids)
@pytest.mark.parametrize("kind", ["whole", "empty", "mixed"])
def test_wgrad_ragged_expert_behind_many_others(kind, K, F, f32):
    """A ragged expert behind some hundred whole (multiples of 16) or empty ones: roles that pass those by wait long."""
    E = 500
    g = torch.Generator().manual_seed(3)
    pick = torch.randint(0, 4, (E,), generator=g).tolist()
    counts = [{"whole": 64, "empty": 0, "mixed": [0, 16, 0, 80][p]}[kind] for p in pick] + [7, 0, 33]
    b = Batch(1, counts, sum(counts))
    dy, x = b.row_values(F), b.row_values(K)
    dw = torch.full((b.E, F, K), ref.SENTINEL, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda")
    moe.expert_gemm_wgrad(b.dims(), K, F, dy, x, b.offsets, dw)
    for e in list(range(0, E, 41)) + [E, E + 1, E + 2]:
        r = b.span(e)
        d, v = dy[r].double(), x[r].double()
        ref.check(dw[e], d.t() @ v, ref.sum_error(r.stop - r.start, d.abs().t() @ v.abs()),
                  F32_HALF if f32 else BF16_HALF, f"dw[{e}]")
    empty = torch.tensor([c == 0 for c in counts], device="cuda")
    assert int(dw[empty].count_nonzero()) == 0
    assert moe.take_device_error() == moe.MOE_OK


def test_swiglu_grad_at_the_ends_of_the_range():
    """g or u the lowest or highest value of the type, or so low that the sigmoid is 0: gradients are finite, and as the
    formula gives them in f32 range, though dh g and dh u are not."""
    low = torch.finfo(torch.bfloat16).min
    g = [low, low, low / 2, -200.0, -200.0, -89.0, -120.0, 200.0, 5.0]
    u = [1.0, -low, 3.0, -low, low, -low, 1e30, 2.0, 1e30]
    d = [4.0, 2.0, -3e38, 3e38, 4.0, -2.0, 3e38, 1e30, 1e7]
    F = 16
    b = Batch(1, [1], 1)
    pre, dh = torch.zeros(1, 2 * F, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, F, dtype=torch.bfloat16, device="cuda")
    for t, at in ((pre[0, :F], g), (pre[0, F:], u), (dh[0], d)):
        t[:len(at)] = torch.tensor(at, dtype=torch.bfloat16)
    dpre = b.out(2 * F, torch.bfloat16)
    moe.expert_swiglu_grad(b.dims(), F, pre, dh, b.offsets, dpre)
    g, u, d = pre[:, :F].double(), pre[:, F:].double(), dh.double()
    s, t = torch.special.expit(g), torch.special.expit(-g)
    # f32 operations as in test_swiglu_grad; a sigmoid below 2^-126 has no more than 2^-149 as its step
    small = 2.0 ** -149
    dg_err = 16 * F32_HALF * (d * u * s).abs() * (1 + g.abs()) + small * (d * u).abs() * (1 + g.abs())
    du_err = 16 * F32_HALF * (d * g * s).abs() + small * (d * g).abs()
    # where exp(-g) passes the range of f32 (g below -88.73) s is 0, and so is the gradient
    zero = g < -88.73
    for got, want, err in ((dpre[:, :F], d * u * s * (1 + g * t), dg_err), (dpre[:, F:], d * g * s, du_err)):
        assert bool(torch.isfinite(got.float()).all())
        assert int(got[zero].count_nonzero()) == 0
        ref.check(got[~zero], want[~zero], err[~zero], BF16_HALF, "gradient")
