"""The experts' products as they are used: a whole layer between dispatch and
combine, a training step, a dense layer, graphs, streams and far rows
(tolerances: expert_ref)."""
import pytest
import torch

import combine_moe_route_topk_gb300 as moe
import expert_ref as ref
from expert_ref import BF16_HALF, E4M3_HALF, F32_HALF, Batch

pytestmark = pytest.mark.gpu
LINEAR, SWIGLU = moe.MOE_EXPERT_LINEAR, moe.MOE_EXPERT_SWIGLU


@pytest.fixture(scope="module", autouse=True)
def _built():
    from combine_moe_route_topk_gb300 import _build
    _build.build()
    yield
    assert moe.take_device_error() == moe.MOE_OK


class Layer:
    """Routed tokens of one layer: route, count and pack by the library."""

    def __init__(self, N, T, E, R, H, cap, seed, fp8):
        self.dims = moe.make_dims(N, T, E, R, H, cap_rows=cap)
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.g = g
        self.logits = torch.randn(N * T, E, generator=g, device="cuda")
        self.x = torch.randn(N * T, H, generator=g, device="cuda").to(torch.bfloat16)
        b = self.b = moe.Buffers(self.dims)
        if fp8:
            self.xq = torch.empty(N * cap, H, dtype=torch.uint8, device="cuda")
            self.xs = torch.empty(N * cap, H // 128, device="cuda")
            ws = torch.zeros(b.sizes["fused_workspace_bytes"], dtype=torch.uint8, device="cuda")
            moe.dispatch_fused_quant(self.dims, self.logits, None, moe.MOE_SOFTMAX, True, self.x, b.topk_idx, b.topk_w,
                                     b.expert_counts, b.expert_offsets, b.rank_counts, b.rank_offsets, b.send_counts,
                                     b.pos, b.status, self.xq, self.xs, b.packed_src, ws)
        else:
            moe.route_topk(self.dims, self.logits, None, moe.MOE_SOFTMAX, True, b.topk_idx, b.topk_w)
            moe.dispatch_count(self.dims, b.topk_idx, b.expert_counts, b.expert_offsets, b.rank_counts,
                               b.rank_offsets, b.send_counts, b.pos, b.status)
            moe.dispatch_pack(self.dims, self.x, None, b.pos, b.packed_x, None, b.packed_src)

    def batch(self):
        """The rows as a Batch, for the references (reads the counts back)."""
        return Batch(self.dims.N, self.b.expert_counts.tolist(), self.b.sizes["cap_rows"])

    def check_combine(self, y, out):
        pos, w = self.b.pos.long(), self.b.topk_w.double()
        rows = y.double()[pos.clamp_min(0)]
        rows[pos < 0] = 0
        want, mag = (rows * w.unsqueeze(2)).sum(1), (rows.abs() * w.unsqueeze(2)).sum(1)
        ref.check(out, want, ref.sum_error(w.shape[1], mag), BF16_HALF, "out")


# one token, a decode batch with a region that overflows, a larger batch
@pytest.mark.parametrize("N,T,E,R,H,F,cap", [(1, 1, 8, 3, 128, 128, 3), (4, 16, 16, 4, 256, 384, 70),
                                             (2, 400, 8, 4, 512, 256, 1700)])
def test_fp8_layer(N, T, E, R, H, F, cap):
    lay = Layer(N, T, E, R, H, cap, 3, fp8=True)
    d, b, off = lay.dims, lay.b, lay.b.expert_offsets
    g = dict(generator=lay.g, device="cuda")
    w1 = (torch.randn(E, 2 * F, H, **g) * 64).to(torch.float8_e4m3fn).view(torch.uint8)
    w2 = (torch.randn(E, H, F, **g) * 64).to(torch.float8_e4m3fn).view(torch.uint8)
    s1 = (0.5 + torch.rand(E, 2 * F // 128, H // 128, **g)) * (H ** -0.5 / 32)
    s2 = (0.5 + torch.rand(E, H // 128, F // 128, **g)) * (F ** -0.5 / 64)
    hq = torch.zeros(N * cap, F, dtype=torch.uint8, device="cuda")
    hs = torch.zeros(N * cap, F // 128, device="cuda")
    b.y = torch.zeros(N * cap, H, dtype=torch.bfloat16, device="cuda")
    moe.expert_gemm_fp8(d, H, F, SWIGLU, lay.xq, lay.xs, w1, s1, off, hq, hs)
    moe.expert_gemm_fp8(d, F, H, LINEAR, hq, hs, w2, s2, off, b.y)
    moe.combine(d, b.y, b.pos, b.topk_w, b.out)
    rb = lay.batch()
    v = rb.valid
    pre, mag = ref.product(rb, ref.dequant_rows(lay.xq, lay.xs), ref.dequant_matrix(w1, s1))
    err = ref.sum_error(H, mag)
    h, eh = ref.swiglu(pre[v, :F], pre[v, F:], err[v, :F], err[v, F:])
    got_s = hs[v].double().repeat_interleave(128, 1)
    ref.check(ref.e4m3(hq[v]) * got_s, h, eh + got_s * 2.0 ** -10 + 4 * F32_HALF * h.abs(), E4M3_HALF, "h")
    y, mag = ref.product(rb, ref.dequant_rows(hq, hs), ref.dequant_matrix(w2, s2))
    ref.check(b.y[v], y[v], ref.sum_error(F, mag)[v], BF16_HALF, "y")
    lay.check_combine(b.y, b.out)


@pytest.mark.parametrize("N,T,E,R,H,F,cap", [(1, 1, 8, 3, 128, 72, 3), (4, 16, 16, 4, 264, 136, 70),
                                             (2, 400, 8, 4, 512, 256, 1700)])
def test_bf16_training_step(N, T, E, R, H, F, cap):
    """Forward with the pre-activations kept, then every gradient: each call
    against the formula on what it was given."""
    lay = Layer(N, T, E, R, H, cap, 5, fp8=False)
    d, b, off, x = lay.dims, lay.b, lay.b.expert_offsets, lay.b.packed_x
    rb = lay.batch()
    v = rb.valid
    w1, w2 = rb.randn(E, 2 * F, H, scale=2 * H ** -0.5), rb.randn(E, H, F, scale=F ** -0.5)
    pre, h, y = rb.out(2 * F, torch.bfloat16), rb.out(F, torch.bfloat16), rb.out(H, torch.bfloat16)
    moe.expert_gemm(d, H, F, SWIGLU, x, w1, off, h, pre)
    moe.expert_gemm(d, F, H, LINEAR, h, w2, off, y)
    moe.combine(d, y, b.pos, b.topk_w, b.out)
    lay.check_combine(y, b.out)
    dy = rb.row_values(H)
    dh, dpre, dx = rb.out(F, torch.bfloat16), rb.out(2 * F, torch.bfloat16), rb.out(H, torch.bfloat16)
    dw1 = torch.empty(E, 2 * F, H, device="cuda")
    dw2 = torch.empty(E, H, F, device="cuda")
    moe.expert_gemm_dgrad(d, F, H, dy, w2, off, dh)
    moe.expert_gemm_wgrad(d, F, H, dy, h, off, dw2)
    moe.expert_swiglu_grad(d, F, pre, dh, off, dpre)
    moe.expert_gemm_dgrad(d, H, 2 * F, dpre, w1, off, dx)
    moe.expert_gemm_wgrad(d, H, 2 * F, dpre, x, off, dw1)
    want, mag = ref.product(rb, x, w1)
    ref.check(pre[v], want[v], ref.sum_error(H, mag)[v], BF16_HALF, "pre")
    want, mag = ref.product(rb, h, w2)
    ref.check(y[v], want[v], ref.sum_error(F, mag)[v], BF16_HALF, "y")
    want, mag = ref.product(rb, dy, w2.transpose(1, 2))
    ref.check(dh[v], want[v], ref.sum_error(H, mag)[v], BF16_HALF, "dh")
    want, mag = ref.product(rb, dpre, w1.transpose(1, 2))
    ref.check(dx[v], want[v], ref.sum_error(2 * F, mag)[v], BF16_HALF, "dx")
    for dw, left, right in ((dw2, dy, h), (dw1, dpre, x)):
        for e in range(E):
            r = rb.span(e)
            p, q = left[r].double(), right[r].double()
            ref.check(dw[e], p.t() @ q, ref.sum_error(r.stop - r.start, p.abs().t() @ q.abs()), F32_HALF, f"dw[{e}]")


def test_gradients_against_differences():
    """<gradient, direction> against the difference quotient of the loss
    sum(c * result) in 64 bits.  The product is linear in each operand, so its
    quotient is exact; the gate's is off by its third derivative (below 0.7
    |u| here) times step^2 / 6.  The gradient's own error is its check()
    limit, weighted by the direction."""
    b = Batch(2, [37, 0, 21, 70], 100)
    K, F, step = 72, 40, 2.0 ** -10
    x, w, c = b.row_values(K), b.randn(b.E, F, K, scale=K ** -0.5), b.row_values(F)
    dx, dw = b.out(K, torch.bfloat16), torch.empty(b.E, F, K, device="cuda")
    moe.expert_gemm_dgrad(b.dims(), K, F, c, w, b.offsets, dx)
    moe.expert_gemm_wgrad(b.dims(), K, F, c, x, b.offsets, dw)
    v = b.valid
    for seed in range(3):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        tx = torch.randn(b.rows, K, generator=g, device="cuda", dtype=torch.float64)
        tw = torch.randn(b.E, F, K, generator=g, device="cuda", dtype=torch.float64)

        def loss(xx, ww):
            return (ref.product(b, xx, ww)[0][v] * c[v].double()).sum()

        x64, w64 = x.double(), w.double()
        quotient = (loss(x64 + step * tx, w64) - loss(x64 - step * tx, w64)) / (2 * step)
        got = dx[v].double()
        mag = ref.product(b, c, w.transpose(1, 2))[1][v]
        lim = ((ref.sum_error(F, mag) + BF16_HALF * got.abs() * 1.01) * tx[v].abs()).sum()
        assert abs((got * tx[v]).sum() - quotient) <= lim
        quotient = (loss(x64, w64 + step * tw) - loss(x64, w64 - step * tw)) / (2 * step)
        mags = torch.stack([c[b.span(e)].double().abs().t() @ x[b.span(e)].double().abs() for e in range(b.E)])
        lim = ((ref.sum_error(70, mags) + F32_HALF * dw.double().abs() * 1.01) * tw.abs()).sum()
        assert abs((dw.double() * tw).sum() - quotient) <= lim
    pre, dh, dpre = b.row_values(2 * F), b.row_values(F), b.out(2 * F, torch.bfloat16)
    moe.expert_swiglu_grad(b.dims(), F, pre, dh, b.offsets, dpre)

    def gate(p):
        return (p[:, :F] * torch.special.expit(p[:, :F]) * p[:, F:] * dh[v].double()).sum()

    t = torch.randn(int(v.sum()), 2 * F, device="cuda", dtype=torch.float64)
    p64 = pre[v].double()
    quotient = (gate(p64 + step * t) - gate(p64 - step * t)) / (2 * step)
    got = dpre[v].double()
    u, tg, tu = p64[:, F:], t[:, :F], t[:, F:]
    third = (0.7 * (u.abs() + step * tu.abs()) * tg.abs() ** 3 + 3 * 0.6 * tg ** 2 * tu.abs()) * dh[v].double().abs() / 6
    lim = (BF16_HALF * 1.01 * got.abs() * t.abs()).sum() + step ** 2 * third.sum()
    assert abs((got * t).sum() - quotient) <= lim


def test_dense_layer_is_one_expert():
    rows, K, F = 300, 136, 392
    b = Batch(1, [rows], rows)
    d = moe.make_dims(1, rows, 1, 1, 8, cap_rows=rows)
    x, w, y = b.row_values(K), b.randn(1, F, K, scale=K ** -0.5), b.out(F, torch.bfloat16)
    moe.expert_gemm(d, K, F, LINEAR, x, w, b.offsets, y)
    want, mag = ref.product(b, x, w)
    ref.check(y, want, ref.sum_error(K, mag), BF16_HALF, "y")


def _calls(b, K=256, F=256):
    """Every entry point on one batch: [(call, outputs)]."""
    d = b.dims()
    x, w, dy = b.row_values(K), b.randn(b.E, F, K, scale=K ** -0.5), b.row_values(F)
    w1, pre = b.randn(b.E, 2 * F, K, scale=K ** -0.5), b.row_values(2 * F)
    xz = torch.where(b.valid.unsqueeze(1), x, torch.zeros_like(x))
    xq, xs = ref.quantise(xz)
    wq = (torch.randn(b.E, 2 * F, K, generator=b.g, device="cuda") * 64).to(torch.float8_e4m3fn).view(torch.uint8)
    ws = torch.full((b.E, 2 * F // 128, K // 128), K ** -0.5 / 32, device="cuda")
    y, h, p2, dx, dw, dp = (b.out(F, torch.bfloat16), b.out(F, torch.bfloat16), b.out(2 * F, torch.bfloat16),
                            b.out(K, torch.bfloat16), torch.empty(b.E, F, K, device="cuda"), b.out(2 * F, torch.bfloat16))
    yq, hq, hs = b.out(F, torch.bfloat16), torch.zeros(b.rows, F, dtype=torch.uint8, device="cuda"), b.out(F // 128, torch.float32)
    o = b.offsets
    half = wq[:, :F].contiguous(), ws[:, : F // 128].contiguous()
    return [
        (lambda s=None: moe.expert_gemm(d, K, F, LINEAR, x, w, o, y, stream=s), [y]),
        (lambda s=None: moe.expert_gemm(d, K, F, SWIGLU, x, w1, o, h, p2, stream=s), [h, p2]),
        (lambda s=None: moe.expert_gemm_dgrad(d, K, F, dy, w, o, dx, stream=s), [dx]),
        (lambda s=None: moe.expert_gemm_wgrad(d, K, F, dy, x, o, dw, stream=s), [dw]),
        (lambda s=None: moe.expert_swiglu_grad(d, F, pre, dy, o, dp, stream=s), [dp]),
        (lambda s=None: moe.expert_gemm_fp8(d, K, F, LINEAR, xq, xs, *half, o, yq, stream=s), [yq]),
        (lambda s=None: moe.expert_gemm_fp8(d, K, F, SWIGLU, xq, xs, wq, ws, o, hq, hs, stream=s), [hq, hs]),
    ]


def _bits(outs):
    return [t.clone().view(torch.uint8) for t in outs]


def _same(a, b):
    return all(torch.equal(p, q) for p, q in zip(a, b))


def _clear(outs):
    for t in outs:
        t.view(torch.uint8).fill_(0x5A)


@pytest.fixture()
def batch():
    return Batch(2, [100, 3, 0, 290, 17, 64], 400)


def test_same_call_same_bits_in_graphs_and_on_other_streams(batch):
    for call, outs in _calls(batch):
        _clear(outs)
        call()
        first = _bits(outs)
        _clear(outs)
        call()
        assert _same(_bits(outs), first)
        side = torch.cuda.Stream()
        _clear(outs)
        side.wait_stream(torch.cuda.current_stream())
        call(side)  # passed, not current
        side.synchronize()
        assert _same(_bits(outs), first)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for _ in range(2):
            _clear(outs)
            graph.replay()
            torch.cuda.synchronize()
            assert _same(_bits(outs), first)


def test_captured_call_follows_new_routing(batch):
    """expert_offsets are read on the device: a captured call serves other counts."""
    K, F = 256, 256
    x, w, y = batch.randn(batch.rows, K), batch.randn(batch.E, F, K, scale=K ** -0.5), batch.out(F, torch.bfloat16)
    d, off = batch.dims(), batch.offsets.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.expert_gemm(d, K, F, LINEAR, x, w, off, y)
    for counts in ([100, 3, 0, 290, 17, 64], [0, 0, 0, 0, 0, 0], [1, 390, 5, 30, 0, 0]):
        other = Batch(2, counts, 400)
        off.copy_(other.offsets)
        y.fill_(ref.SENTINEL)
        graph.replay()
        torch.cuda.synchronize()
        want, mag = ref.product(other, x, w)
        ref.check(y[other.valid], want[other.valid], ref.sum_error(K, mag)[other.valid], BF16_HALF, "y")
        ref.check_untouched(other, y)


def test_calls_at_the_same_time(batch):
    """Two of each call, on two streams at once, with inputs and outputs of their own."""
    one, two = _calls(batch), _calls(Batch(3, [65, 0, 200, 9, 300, 1], 320, seed=9))
    want = []
    for call, outs in one + two:
        _clear(outs)
        call()
        want.append(_bits(outs))
        _clear(outs)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for (a, _), (b, _) in zip(one, reversed(two)):
            a(streams[0])
            b(streams[1])
    torch.cuda.synchronize()
    for (_, outs), bits in zip(one + two, want):
        assert _same(_bits(outs), bits)


def test_rows_beyond_32_bit_offsets():
    """Rank 1's rows begin at element 300000 * 8192 > 2^31 of the results."""
    K, F, cap = 64, 8192, 300000
    b = Batch(2, [5, 0, 130, 3], cap)
    x = torch.zeros(b.rows, K, dtype=torch.bfloat16, device="cuda")
    x[b.valid] = b.randn(int(b.valid.sum()), K)
    w, y = b.randn(b.E, F, K, scale=K ** -0.5), torch.zeros(b.rows, F, dtype=torch.bfloat16, device="cuda")
    moe.expert_gemm(b.dims(), K, F, LINEAR, x, w, b.offsets, y)
    dx, dw = torch.zeros(b.rows, K, dtype=torch.bfloat16, device="cuda"), torch.empty(b.E, F, K, device="cuda")
    moe.expert_gemm_dgrad(b.dims(), K, F, y, w, b.offsets, dx)
    moe.expert_gemm_wgrad(b.dims(), K, F, y, x, b.offsets, dw)
    for e in range(b.E):
        r = b.span(e)
        xe, we, ye = x[r].double(), w[e].double(), y[r].double()
        ref.check(ye, xe @ we.t(), ref.sum_error(K, xe.abs() @ we.abs().t()), BF16_HALF, "y")
        ref.check(dx[r], ye @ we, ref.sum_error(F, ye.abs() @ we.abs()), BF16_HALF, "dx")
        ref.check(dw[e], ye.t() @ xe, ref.sum_error(r.stop - r.start, ye.abs().t() @ xe.abs()), F32_HALF, "dw")
    assert int(y[~b.valid].count_nonzero()) == 0


def test_many_experts_and_ranks():
    """1024 experts on 128 ranks, most of them empty."""
    g = torch.Generator().manual_seed(1)
    counts = torch.where(torch.rand(1024, generator=g) < 0.8, 0, torch.randint(1, 40, (1024,), generator=g)).tolist()
    b = Batch(128, counts, 120)
    K, F = 136, 72
    x, w, y = b.row_values(K), b.randn(b.E, F, K, scale=K ** -0.5), b.out(F, torch.bfloat16)
    moe.expert_gemm(b.dims(), K, F, LINEAR, x, w, b.offsets, y)
    want, mag = ref.product(b, x, w)
    ref.check(y[b.valid], want[b.valid], ref.sum_error(K, mag)[b.valid], BF16_HALF, "y")
    ref.check_untouched(b, y)
    pre, dh, dpre = b.row_values(2 * F), b.row_values(F), b.out(2 * F, torch.bfloat16)
    moe.expert_swiglu_grad(b.dims(), F, pre, dh, b.offsets, dpre)
    ref.check_untouched(b, dpre)
    assert bool(torch.isfinite(dpre[b.valid].float()).all())


def test_empty_batch_gives_zero_weight_gradients():
    d = moe.make_dims(2, 0, 4, 2, 8)
    off = torch.zeros(5, dtype=torch.int32, device="cuda")
    none = torch.zeros(2, 8, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((4, 8, 8), 3.0, device="cuda")
    moe.expert_gemm_wgrad(d, 8, 8, none, none, off, dw)
    assert int(dw.count_nonzero()) == 0


def test_scales_of_zero_and_zero_rows():
    """A token of zeros and blocks whose scale is 0 give codes 0 and scale 0, no NaN."""
    b = Batch(1, [20], 20)
    K = F = 256
    x = b.randn(20, K)
    x[3] = 0
    x[5, 128:] = 0
    xq, xs = ref.quantise(x)
    wq = (torch.randn(1, 2 * F, K, generator=b.g, device="cuda") * 64).to(torch.float8_e4m3fn).view(torch.uint8)
    ws = torch.full((1, 2 * F // 128, K // 128), 2.0 ** -10, device="cuda")
    ws[0, 1, :] = 0  # the second block of gate rows: h = silu(0) u = 0
    hq, hs = torch.full((20, F), 0x5A, dtype=torch.uint8, device="cuda"), b.out(F // 128, torch.float32)
    moe.expert_gemm_fp8(b.dims(), K, F, SWIGLU, xq, xs, wq, ws, b.offsets, hq, hs)
    assert int(hs[3].count_nonzero()) == 0 and int((hq[3] & 0x7F).count_nonzero()) == 0
    assert int(hs[:, 1].count_nonzero()) == 0 and int((hq[:, 128:] & 0x7F).count_nonzero()) == 0
    assert bool((hs[:3, 0] > 0).all())


def test_requantised_scales_below_the_normal_range():
    """h near 1e-37: scales of 2^-129 to 2^-134, whose reciprocals overflow f32.
    Beside expert_ref's terms, a denormal scale is rounded by up to 2^-150,
    times a code of at most 448, and h itself by 2^-150."""
    b = Batch(1, [40], 40)
    K = F = 128
    xq, xs = ref.quantise(b.randn(40, K))
    wq = (torch.randn(1, 2 * F, K, generator=b.g, device="cuda") * 64).to(torch.float8_e4m3fn).view(torch.uint8)
    ws = torch.empty(1, 2, 1, device="cuda")
    ws[0, 0], ws[0, 1] = 2.0 ** -10, 2.0 ** -132
    hq, hs = torch.zeros(40, F, dtype=torch.uint8, device="cuda"), b.out(1, torch.float32)
    moe.expert_gemm_fp8(b.dims(), K, F, SWIGLU, xq, xs, wq, ws, b.offsets, hq, hs)
    want, mag = ref.product(b, ref.dequant_rows(xq, xs), ref.dequant_matrix(wq, ws))
    err = ref.sum_error(K, mag) + 2.0 ** -150 * K
    h, eh = ref.swiglu(want[:, :F], want[:, F:], err[:, :F], err[:, F:])
    s = hs.double()
    assert bool((s < 2.0 ** -126).all()) and bool((s > 0).all())
    lim = eh + E4M3_HALF * h.abs() + s * 2.0 ** -10 + 449 * 2.0 ** -150 + 4 * F32_HALF * h.abs()
    assert bool(((ref.e4m3(hq) * s - h).abs() <= lim).all())


def _off(got, want):
    return float((got.double() - want).norm() / want.norm())


def test_f32_results_do_not_lose_with_length():
    """A sum of 16384 is 32 sums of 512 joined in f32 registers.  Each part is as
    far off as a sum of 512 is, and so is their sum; 32 additions rounded to
    nearest add at most 32 2^-24 of it (the partial sums of independent values
    are no larger than the result).  Summed in the tensor core's accumulator
    alone, the result was 1.7e-5 off, eight times what is allowed here."""
    off = {}
    for n in (512, 16384):
        b = Batch(1, [96], 96)
        x, w, y = b.row_values(n), b.randn(1, 64, n), b.out(64, torch.float32)
        moe.expert_gemm(b.dims(moe.MOE_F32), n, 64, LINEAR, x, w, b.offsets, y)
        off["linear", n] = _off(y, x.double() @ w[0].double().t())
        b = Batch(1, [n], n)
        dy, x, dw = b.row_values(64), b.row_values(96), torch.empty(1, 64, 96, device="cuda")
        moe.expert_gemm_wgrad(b.dims(), 96, 64, dy, x, b.offsets, dw)
        off["wgrad", n] = _off(dw[0], dy.double().t() @ x.double())
    for op in ("linear", "wgrad"):
        assert off[op, 16384] <= off[op, 512] + 32 * F32_HALF, off


def test_refusals_on_the_device():
    b = Batch(1, [4], 4)
    x, w, y = b.randn(4, 16), b.randn(1, 8, 16), b.out(8, torch.bfloat16)
    d = b.dims()
    with pytest.raises(ValueError, match="contiguous"):
        moe.expert_gemm(d, 16, 8, LINEAR, x, w.transpose(1, 2), b.offsets, y)
    with pytest.raises(ValueError, match="holds"):
        moe.expert_gemm(d, 16, 8, LINEAR, x[:3], w, b.offsets, y)
    with pytest.raises(ValueError, match="must be torch.bfloat16"):
        moe.expert_gemm(d, 16, 8, LINEAR, x.float(), w, b.offsets, y)
    with pytest.raises(ValueError, match="must be torch.int32"):
        moe.expert_gemm(d, 16, 8, LINEAR, x, w, b.offsets.long(), y)
    with pytest.raises(moe.MoeError, match="16-byte"):
        flat = torch.zeros(4 * 16 + 8, dtype=torch.bfloat16, device="cuda")
        moe.expert_gemm(d, 16, 8, LINEAR, flat[1: 1 + 64].view(4, 16), w, b.offsets, y)
    with pytest.raises(moe.MoeError, match="multiples of 8"):
        moe.expert_gemm(d, 12, 8, LINEAR, x, w, b.offsets, y)


def test_pairs_without_tiles_and_the_kernels_behind_them():
    """One tile, or none, for all pairs of blocks, each launch followed at once by another kernel's blocks with
    barriers of their own at the same places in shared memory: 200 rounds give the same bits as the first."""
    few, none = Batch(1, [3, 0], 4), Batch(2, [0, 0], 4)
    calls = _calls(few, 128, 128) + _calls(none, 128, 128)
    for call, outs in calls:
        _clear(outs)
        call()
    torch.cuda.synchronize()
    want = [_bits(outs) for _, outs in calls]
    for _, outs in calls:
        _clear(outs)
    for i in range(200):
        for call, _ in calls[i % len(calls):] + calls[: i % len(calls)]:
            call()
    for (_, outs), bits in zip(calls, want):
        assert _same(_bits(outs), bits)


@pytest.mark.parametrize("offsets", [[0, 8, 0, 8, 0, 8, 8], [0, 8, 16, 15, 20, 24, 24], [0, 1, 2, 3, 4, 5, 200], [3, 2, 2, 2, 2, 2, 2]])
def test_offsets_of_no_batch_stand_for_no_rows(offsets):
    """Offsets that descend, or span more rows than the batch routes, are no output of the count step; read as they
    are, every expert could seem to have all rows, and the number of tiles pass 32 bits."""
    b = Batch(2, [8, 8, 8, 0, 0, 0], 24)
    for i, (call, outs) in enumerate(_calls(b)):
        if i == 4:  # the activation's gradient takes ranks' regions whole
            continue
        b.offsets.copy_(torch.tensor(offsets, dtype=torch.int32))
        _clear(outs)
        call()
        for t in outs:
            if i == 3:
                assert int(t.count_nonzero()) == 0  # dw: no rows, zeros
            else:
                assert bool((t.view(torch.uint8) == 0x5A).all())


def test_captured_calls_of_two_graphs_at_the_same_time(batch):
    """Two graphs that hold every call, replayed on two streams at once: no call keeps anything another one uses."""
    one, two = _calls(batch), _calls(Batch(3, [65, 0, 200, 9, 300, 1], 320, seed=9))
    want, graphs = [], []
    for calls in (one, two):
        for call, outs in calls:
            _clear(outs)
            call()
            want.append(_bits(outs))
            _clear(outs)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(3):
                for call, _ in calls:
                    call()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        for s, graph in zip(streams, graphs):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, outs), bits in zip(one + two, want):
        assert _same(_bits(outs), bits)


def test_calls_from_two_threads():
    """What the library keeps per thread is set up by the first calls of each, at the same time."""
    import threading
    failed = []

    def work(seed):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                calls = _calls(Batch(2, [100, 3, 0, 290, 17, 64], 400, seed=seed))
                for i in range(20):
                    for call, outs in calls:
                        call()
                        if i == 0:
                            stream.synchronize()
                            outs.append(_bits(outs))
                stream.synchronize()
                for call, (*outs, bits) in calls:
                    assert _same(_bits(outs), bits)
        except BaseException as e:  # reported by the test's own thread
            failed.append(e)

    threads = [threading.Thread(target=work, args=(s,)) for s in (1, 2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
