"""The experts' product with 4-bit weights against plain 64-bit products (tolerances: expert_ref; a row's scale
multiplies the sum, one more rounding of 2^-24)."""
import threading

import pytest
import torch

import combine_moe_route_topk_gb300 as moe
import expert_ref as ref
from expert_ref import BF16_HALF, F32_HALF, SENTINEL, Batch

pytestmark = pytest.mark.gpu
LINEAR, SWIGLU = moe.MOE_EXPERT_LINEAR, moe.MOE_EXPERT_SWIGLU


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_moe_route_topk_gb300 import _build
    _build.build()
    yield
    assert moe.take_device_error() == moe.MOE_OK


class Weights:
    """Random codes (all sixteen), e4m3 scales from the smallest to the largest, and their values in 64 bits."""

    def __init__(self, b, W, K, group):
        kw = dict(generator=b.g, device="cuda")
        q = torch.randint(-8, 8, (b.E, W, K), dtype=torch.int8, **kw)
        self.wq = moe.pack_w4(q)
        s = (2.0 ** (torch.rand(b.E, K // group, W, **kw) * 6 - 3)).to(torch.float8_e4m3fn)
        s.view(torch.uint8)[..., ::7] = 0x7e  # 448
        s.view(torch.uint8)[:, 0, ::5] = 1    # 2^-9, subnormal
        s.view(torch.uint8)[:, -1, ::6] = 0
        s.view(torch.uint8)[:, 0, 1::11] |= 0x80  # negative ones are scales too
        self.gs = s.view(torch.uint8)
        self.rs = (0.5 + torch.rand(b.E, W, **kw)) * K ** -0.5 / 8
        full = s.double().transpose(1, 2).repeat_interleave(group, 2)
        self.w = q.double() * full * self.rs.double().unsqueeze(2)


def call(b, K, F, act, group, x, w, y, f32=False, **kw):
    moe.expert_gemm_w4(b.dims(moe.MOE_F32 if f32 else moe.MOE_BF16), K, F, act, group, x, w.wq, w.gs, w.rs, b.offsets, y, **kw)


# N, rows per expert, cap: as for the bf16 products, tile edges at 16, 32, 64, 128 rows
ROWS = [
    (1, [1], 1),
    (1, [5, 0, 16, 17], 40),
    (2, [0, 33, 64, 65, 0, 1], 200),
    (2, [127, 128, 129, 0], 257),
    (1, [255, 256, 257], 800),
    (2, [300, 31, 15, 2], 320),
    (2, [50, 9, 3, 0], 40),
    (3, [0, 0, 0], 8),
    (4, [3, 0, 0, 2, 0, 0, 7, 1], 12),
    (1, [48, 112, 49, 113], 400),
]
# at most four rows an expert on average: one tile of eight tokens, edges of it, several tiles, no rows at all
FEW = [
    (1, [8, 0, 1, 7], 40),
    (1, [9, 0, 0, 0, 3], 12),
    (2, [20, 0, 0, 0, 0, 0, 4, 0], 17),   # three tiles, the last cut by the region's end
    (4, [2, 0, 0, 0, 3, 1, 8, 0], 9),
    (1, [0, 0, 0, 17, 0, 0, 0], 64),
    (1, [4], 4),
]
SIZES = [(32, 8, 32), (64, 72, 64), (96, 136, 32), (256, 128, 128), (288, 264, 32), (512, 96, 64), (1152, 200, 128),
         (1056, 64, 32), (2304, 520, 32)]


@pytest.mark.parametrize("K,F,group", SIZES, ids=str)
@pytest.mark.parametrize("N,counts,cap", ROWS + FEW, ids=str)
@pytest.mark.parametrize("form", ["bf16", "f32", "gated"])
def test_product(N, counts, cap, K, F, group, form):
    b = Batch(N, counts, cap)
    x, w = b.row_values(K), Weights(b, 2 * F if form == "gated" else F, K, group)
    y = b.out(F, torch.float32 if form == "f32" else torch.bfloat16)
    call(b, K, F, SWIGLU if form == "gated" else LINEAR, group, x, w, y, form == "f32")
    want, mag = ref.product(b, x, w.w)
    v = b.valid
    err = (ref.sum_error(K, mag) + F32_HALF * want.abs())[v]
    if form == "gated":
        want, err = ref.swiglu(want[v, :F], want[v, F:], err[:, :F], err[:, F:])
        ref.check(y[v], want, err, BF16_HALF, "y")
    else:
        ref.check(y[v], want[v], err, F32_HALF if form == "f32" else BF16_HALF, "y")
    ref.check_untouched(b, y)


@pytest.mark.parametrize("counts", [[(7 * e * e) % 200 if e % 3 == 0 else 0 for e in range(240)],
                                    [e % 11 if e % 3 == 0 else 0 for e in range(240)]], ids=["many", "few"])
def test_many_experts(counts):
    """More tiles than blocks, tiles of every size, most experts without rows."""
    b = Batch(4, counts, 4000)
    K, F = 320, 392
    x, w = b.row_values(K), Weights(b, F, K, 32)
    y = b.out(F, torch.bfloat16)
    call(b, K, F, LINEAR, 32, x, w, y)
    want, mag = ref.product(b, x, w.w)
    v = b.valid
    ref.check(y[v], want[v], (ref.sum_error(K, mag) + F32_HALF * want.abs())[v], BF16_HALF, "y")
    ref.check_untouched(b, y)


@pytest.mark.parametrize("counts,K", [([70, 3], 17408), ([3, 1], 10240), ([3, 1], 17408)], ids=str)
@pytest.mark.parametrize("form", ["bf16", "f32", "gated"])
def test_long_sums_are_taken_in_parts(form, counts, K):
    """Sums of f32 results in parts of 512, those of bf16 ones beyond 16384 likewise.  Within a part an addition is off by
    at most a unit (2^-23) of what the part holds, and the parts are added rounding to nearest."""
    b = Batch(1, counts, 80)
    F = 136
    x, w = b.row_values(K), Weights(b, 2 * F if form == "gated" else F, K, 128)
    y = b.out(F, torch.float32 if form == "f32" else torch.bfloat16)
    call(b, K, F, SWIGLU if form == "gated" else LINEAR, 128, x, w, y, form == "f32")
    want, mag = ref.product(b, x, w.w)
    v = b.valid
    part = 512 if form == "f32" or K > 16384 else K
    err = ((part + 4) * 2.0 ** -23 * mag + K / part * F32_HALF * mag + F32_HALF * want.abs())[v]
    if form == "gated":
        want, err = ref.swiglu(want[v, :F], want[v, F:], err[:, :F], err[:, F:])
        ref.check(y[v], want, err, BF16_HALF, "y")
    else:
        ref.check(y[v], want[v], err, F32_HALF if form == "f32" else BF16_HALF, "y")


@pytest.mark.parametrize("rows", [3, 40])
def test_exact_sums(rows):
    """Whole numbers whose sums fit 24 bits come out exactly: no weight and no product is rounded."""
    b = Batch(1, [rows], rows)
    K, F = 512, 128
    kw = dict(generator=b.g, device="cuda")
    x = torch.randint(-16, 17, (rows, K), **kw).to(torch.bfloat16)
    w = Weights(b, F, K, 32)
    q = torch.randint(-8, 8, (1, F, K), dtype=torch.int8, **kw)
    s = torch.randint(1, 16, (1, K // 32, F), **kw).float()
    w.wq, w.gs, w.rs = moe.pack_w4(q), s.to(torch.float8_e4m3fn), torch.ones(1, F, device="cuda")
    y = b.out(F, torch.float32)
    call(b, K, F, LINEAR, 32, x, w, y, True)
    full = q.double() * s.double().transpose(1, 2).repeat_interleave(32, 2)
    assert torch.equal(y.double(), x.double() @ full[0].t())


@pytest.mark.parametrize("T", [1, 2, 7, 16, 100])
def test_dense_layer(T):
    """N = E = R = 1: a matrix-vector product for one token."""
    K, F, group = 2048, 1032, 128
    d = moe.make_dims(1, T, 1, 1, 8, cap_rows=T)
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    m = torch.randn(1, F, K, generator=g, device="cuda") * K ** -0.5
    wq, gs, rs = moe.quantize_w4(m, group)
    x = torch.randn(T, K, generator=g, device="cuda").to(torch.bfloat16)
    y = torch.empty(T, F, dtype=torch.bfloat16, device="cuda")
    off = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    moe.expert_gemm_w4(d, K, F, LINEAR, group, x, wq, gs, rs, off, y)
    q = torch.empty(F, K, device="cuda", dtype=torch.float64)
    for i in range(8):
        c = (wq[0] >> (4 * (i // 2) + 16 * (i % 2))) & 15
        q[:, i::8] = torch.where(c > 7, c - 16, c).double()
    w = q * gs[0].view(torch.float8_e4m3fn).double().t().repeat_interleave(group, 1) * rs[0].double().unsqueeze(1)
    want, mag = x.double() @ w.t(), x.double().abs() @ w.abs().t()
    ref.check(y, want, ref.sum_error(K, mag) + F32_HALF * want.abs(), BF16_HALF, "y")


def test_layer_between_dispatch_and_combine():
    """Router to combine with 4-bit weights: each call against the formula on what it was given."""
    N, T, E, R, H, F, cap = 4, 24, 16, 4, 256, 136, 90
    d = moe.make_dims(N, T, E, R, H, cap_rows=cap)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    kw = dict(generator=g, device="cuda")
    logits, x = torch.randn(N * T, E, **kw), torch.randn(N * T, H, **kw).to(torch.bfloat16)
    b = moe.Buffers(d, separate_y=True)
    moe.route_topk(d, logits, None, moe.MOE_SOFTMAX, True, b.topk_idx, b.topk_w)
    moe.dispatch_count(d, b.topk_idx, b.expert_counts, b.expert_offsets, b.rank_counts, b.rank_offsets, b.send_counts,
                       b.pos, b.status)
    moe.dispatch_pack(d, x, None, b.pos, b.packed_x, None, b.packed_src)
    rb = Batch(N, b.expert_counts.tolist(), cap)
    w1, w2 = Weights(rb, 2 * F, H, 32), Weights(rb, H, F - F % 32, 32)
    h = rb.out(F, torch.bfloat16)
    moe.expert_gemm_w4(d, H, F, SWIGLU, 32, b.packed_x, w1.wq, w1.gs, w1.rs, b.expert_offsets, h)
    v = rb.valid
    want, mag = ref.product(rb, b.packed_x, w1.w)
    err = (ref.sum_error(H, mag) + F32_HALF * want.abs())[v]
    want, err = ref.swiglu(want[v, :F], want[v, F:], err[:, :F], err[:, F:])
    ref.check(h[v], want, err, BF16_HALF, "h")
    h2 = h[:, : F - F % 32].contiguous()
    moe.expert_gemm_w4(d, F - F % 32, H, LINEAR, 32, h2, w2.wq, w2.gs, w2.rs, b.expert_offsets, b.y)
    want, mag = ref.product(rb, h2, w2.w)
    ref.check(b.y[v], want[v], (ref.sum_error(F, mag) + F32_HALF * want.abs())[v], BF16_HALF, "y")
    moe.combine(d, b.y, b.pos, b.topk_w, b.out)
    rows = b.y.double()[b.pos.long().clamp_min(0)]
    rows[b.pos < 0] = 0
    t = b.topk_w.double().unsqueeze(2)
    ref.check(b.out, (rows * t).sum(1), ref.sum_error(R, (rows.abs() * t).sum(1)), BF16_HALF, "out")


@pytest.mark.parametrize("counts", [[20, 0, 5], [8, 0, 2]])
def test_what_stands_in_other_rows_and_weights_has_no_influence(counts):
    """NaN in rows without a token and in the scales of experts without rows; NaN of one expert's rows stays there."""
    b = Batch(1, counts, 64)
    K, F = 96, 72
    x, w = b.row_values(K), Weights(b, F, K, 32)
    x[b.span(0)][7] = float("nan")
    w.gs[1], w.rs[1] = 0x7f, float("nan")
    y = b.out(F, torch.bfloat16)
    call(b, K, F, LINEAR, 32, x, w, y)
    bad = torch.isnan(y).any(1)
    assert bad.nonzero().flatten().tolist() == [7]
    ref.check_untouched(b, y)


@pytest.mark.parametrize("counts", [[3, 3, 2], [30, 30, 20]])
def test_offsets_of_no_batch_stand_for_no_rows(counts):
    for off in ([0, 5, 3, 8], [0, 4, 8, 1 << 30], [8, 0, 0, 0], [0, -5, 1, 2]):
        b = Batch(1, counts, 90)
        x, w = b.randn(b.rows, 64), Weights(b, 40, 64, 32)
        b.offsets = torch.tensor(off, dtype=torch.int32, device="cuda")
        y = b.out(40, torch.bfloat16)
        call(b, 64, 40, LINEAR, 32, x, w, y)
        assert bool((y == SENTINEL).all()), off


@pytest.mark.parametrize("counts", [[30, 0, 129, 7, 1, 64], [3, 0, 12, 7, 1, 0]])
def test_same_bits_in_graphs_on_streams_and_from_threads(counts):
    b = Batch(2, counts, 200)
    K, F = 544, 264
    x, w1 = b.row_values(K), Weights(b, 2 * F, K, 32)
    want = b.out(F, torch.bfloat16)
    call(b, K, F, SWIGLU, 32, x, w1, want)
    outs = [b.out(F, torch.bfloat16) for _ in range(4)]
    graphs = []
    for y in outs[:2]:  # two graphs, replayed at the same time
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            for _ in range(5):
                call(b, K, F, SWIGLU, 32, x, w1, y)
        graphs.append((gr, s))
    for gr, s in graphs:
        with torch.cuda.stream(s):
            gr.replay()

    def work(y):
        s = torch.cuda.Stream()
        for _ in range(20):
            call(b, K, F, SWIGLU, 32, x, w1, y, stream=s)
        s.synchronize()

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(y,)) for y in outs[2:]]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for y in outs:
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("old,new,T", [([30, 0, 9, 7], [1, 40, 0, 0], 60), ([3, 0, 2, 1], [0, 8, 0, 0], 8)])
def test_captured_call_follows_new_routing(old, new, T):
    b, c = Batch(2, old, 60), Batch(2, new, 60, seed=1)
    b.T = c.T = T
    K, F = 128, 136
    x, w = b.randn(b.rows, K), Weights(b, F, K, 64)
    y = b.out(F, torch.float32)
    gr = torch.cuda.CUDAGraph()
    call(b, K, F, LINEAR, 64, x, w, y, True)
    torch.cuda.synchronize()
    with torch.cuda.graph(gr):
        call(b, K, F, LINEAR, 64, x, w, y, True)
    b.offsets.copy_(c.offsets)
    y.fill_(SENTINEL)
    gr.replay()
    want, mag = ref.product(c, x, w.w)
    v = c.valid
    ref.check(y[v], want[v], (ref.sum_error(K, mag) + F32_HALF * want.abs())[v], F32_HALF, "y")
    ref.check_untouched(c, y)


def test_matrices_beyond_32_bit_offsets():
    """Scales, codes and rows past 2^32 bytes: 300 experts of 8192 x 4096, the last ones alone have rows."""
    E, K, F = 300, 4096, 8192
    counts = [0] * (E - 2) + [3, 2]
    b = Batch(1, counts, 8)
    w = Weights.__new__(Weights)
    w.wq = torch.zeros(E, F, K // 8, dtype=torch.int32, device="cuda")
    w.gs = torch.full((E, K // 32, F), 0x38, dtype=torch.uint8, device="cuda")  # 1
    w.rs = torch.ones(E, F, device="cuda")
    few = Batch(1, [3, 2], 8)
    some = Weights(few, F, K, 32)
    w.wq[-2:], w.gs[-2:], w.rs[-2:] = some.wq, some.gs, some.rs
    x, y = few.row_values(K), few.out(F, torch.bfloat16)
    call(b, K, F, LINEAR, 32, x, w, y)
    want, mag = ref.product(few, x, some.w)
    v = few.valid
    ref.check(y[v], want[v], (ref.sum_error(K, mag) + F32_HALF * want.abs())[v], BF16_HALF, "y")


def test_binding_refuses_other_types():
    b = Batch(1, [4], 4)
    x, w, y = b.randn(4, 64), Weights(b, 16, 64, 32), b.out(16, torch.bfloat16)
    with pytest.raises(ValueError, match="x must be"):
        call(b, 64, 16, LINEAR, 32, x.float(), w, y)
    with pytest.raises(ValueError, match="y must be"):
        call(b, 64, 16, LINEAR, 32, x, w, y, True)
    with pytest.raises(ValueError, match="wq holds"):
        call(b, 128, 16, LINEAR, 32, b.randn(4, 128), w, y)
    with pytest.raises(moe.MoeError, match="group must be"):
        call(b, 64, 16, LINEAR, 8, x, w, y)
    w.wq = w.wq.to(torch.int64)
    with pytest.raises(ValueError, match="wq must be"):
        call(b, 64, 16, LINEAR, 32, x, w, y)


@pytest.mark.parametrize("N,most,E,K,F,group", [(8, 145, 64, 2048, 3584, 32), (1, 40, 32, 4096, 2048, 32), (1, 3, 64, 7168, 1024, 32),
                                                (1, 8, 24, 4096, 2048, 128)])
@pytest.mark.parametrize("form", ["bf16", "f32", "gated"])
def test_long_runs_of_tiles(N, most, E, K, F, group, form):
    """Many tiles in a row for every block, at the pace of a real call: slots of shared memory are filled again as soon as
    their readers have them in registers, not a moment before."""
    g = torch.Generator()
    g.manual_seed(most)
    counts = [max(1, most - int(torch.randint(0, max(1, most // 4), (1,), generator=g))) for _ in range(E)]
    b = Batch(N, counts, sum(counts) // N + 200)
    x, w = b.row_values(K), Weights(b, 2 * F if form == "gated" else F, K, group)
    t = torch.float32 if form == "f32" else torch.bfloat16
    act = SWIGLU if form == "gated" else LINEAR
    y = b.out(F, t)
    call(b, K, F, act, group, x, w, y, form == "f32")
    want, mag = ref.product(b, x, w.w)
    v = b.valid
    err = (ref.sum_error(K, mag) + F32_HALF * want.abs())[v]
    if form == "gated":
        want, err = ref.swiglu(want[v, :F], want[v, F:], err[:, :F], err[:, F:])
        ref.check(y[v], want, err, BF16_HALF, "y")
    else:
        ref.check(y[v], want[v], err, F32_HALF if form == "f32" else BF16_HALF, "y")
    again = b.out(F, t)
    for _ in range(10):
        call(b, K, F, act, group, x, w, again, form == "f32")
        assert torch.equal(again, y)


@pytest.mark.parametrize("T", [33, 64, 65, 128, 200])
@pytest.mark.parametrize("K,F", [(512, 264), (1056, 512), (7168, 1032), (2304, 4096)])
@pytest.mark.parametrize("form", ["bf16", "f32", "gated"])
def test_dense_layer_of_some_tokens(T, K, F, form):
    """Few tiles: two or four blocks share a reduction and join their sums."""
    b = Batch(1, [T], T)
    x, w = b.row_values(K), Weights(b, 2 * F if form == "gated" else F, K, 32)
    y = b.out(F, torch.float32 if form == "f32" else torch.bfloat16)
    act = SWIGLU if form == "gated" else LINEAR
    call(b, K, F, act, 32, x, w, y, form == "f32")
    want, mag = ref.product(b, x, w.w)
    err = ref.sum_error(K, mag) + F32_HALF * want.abs()
    if form == "gated":
        want, err = ref.swiglu(want[:, :F], want[:, F:], err[:, :F], err[:, F:])
    ref.check(y, want, err, F32_HALF if form == "f32" else BF16_HALF, "y")
    again = torch.empty_like(y)
    for _ in range(5):
        call(b, K, F, act, 32, x, w, again, form == "f32")
        assert torch.equal(again, y)


@pytest.mark.parametrize("share", [1, 2, 3, 5, 6, 7, 11])
@pytest.mark.parametrize("K,group", [(96, 32), (384, 128), (1056, 32), (2080, 32), (4160, 64)])
@pytest.mark.parametrize("form", ["bf16", "f32", "gated"])
def test_blocks_of_any_number_of_granules(share, K, group, form):
    """Two experts of one and eight rows; `share` granules of 32 matrix rows a block, and an expert's last a part of one."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    b = Batch(1, [1, 8], 12)
    F = (sms * share // 2 * (16 if form == "gated" else 32)) - 8
    x, w = b.row_values(K), Weights(b, 2 * F if form == "gated" else F, K, group)
    y = b.out(F, torch.float32 if form == "f32" else torch.bfloat16)
    act = SWIGLU if form == "gated" else LINEAR
    call(b, K, F, act, group, x, w, y, form == "f32")
    want, mag = ref.product(b, x, w.w)
    v = b.valid
    err = ref.sum_error(K, mag) + F32_HALF * want.abs()
    if form == "gated":
        want, err = ref.swiglu(want[:, :F], want[:, F:], err[:, :F], err[:, F:])
    ref.check(y[v], want[v], err[v], F32_HALF if form == "f32" else BF16_HALF, "y")
    ref.check_untouched(b, y)


@pytest.mark.parametrize("counts,K,F", [([3, 1], 544, 136), ([40, 70], 544, 136), ([200, 90], 256, 4104)])
@pytest.mark.parametrize("form", ["bf16", "gated"])
def test_arrays_at_their_least_alignment(counts, K, F, form):
    """x, wq and y 16 bytes, group_scales 8 and row_scales 4 past a boundary."""
    b = Batch(1, counts, 300)
    x, w = b.row_values(K), Weights(b, 2 * F if form == "gated" else F, K, 32)

    def moved(t, off):
        buf = torch.empty(t.numel() * t.element_size() + 64, dtype=torch.uint8, device="cuda")
        view = buf[off:off + t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        return view.copy_(t)

    act = SWIGLU if form == "gated" else LINEAR
    y = b.out(F, torch.bfloat16)
    call(b, K, F, act, 32, x, w, y)
    w.wq, w.gs, w.rs = moved(w.wq, 16), moved(w.gs, 8), moved(w.rs, 4)
    again = moved(b.out(F, torch.bfloat16), 16)
    call(b, K, F, act, 32, moved(x, 16), w, again)
    assert torch.equal(again, y)


@pytest.mark.parametrize("counts", [[3, 1], [40, 70], [200, 900]])
def test_first_call_of_a_thread_is_captured(counts):
    """What a call sets up once a thread may be set up during a capture, by a thread that has not used CUDA before."""
    b = Batch(1, counts, 1200)
    K, F = 544, 4104
    x, w = b.row_values(K), Weights(b, F, K, 32)
    want, y = b.out(F, torch.bfloat16), b.out(F, torch.bfloat16)
    call(b, K, F, LINEAR, 32, x, w, want)
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    failed = []

    def work():
        try:
            with torch.cuda.graph(graph, stream=stream):
                call(b, K, F, LINEAR, 32, x, w, y)
        except BaseException as e:  # reported by the test's own thread
            failed.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    assert not failed, failed
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want)
