"""Every kernel of the product with 4-bit weights against plain 64-bit products, and that the sizes reach it (tolerances:
expert_ref; a row's scale multiplies the sum, one more rounding of 2^-24)."""
import subprocess
import threading

import pytest
import torch

import combine_moe_route_topk_gb300 as moe
import expert_ref as ref
from combine_moe_route_topk_gb300 import _build
from expert_ref import BF16_HALF, F32_HALF, SENTINEL, Batch
from test_expert_w4_gpu import LINEAR, SWIGLU, Weights, call
from w4_form import FORMS, expected, form

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    _build.build()
    yield
    assert moe.take_device_error() == moe.MOE_OK


def takes(b, K, F, kind="bf16"):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return form(b.dims(), K, F, kind == "gated", kind == "f32", sms)


def out(b, F, kind):
    return b.out(F, torch.float32 if kind == "f32" else torch.bfloat16)


def run(b, K, F, group, kind, x, w, y, **kw):
    call(b, K, F, SWIGLU if kind == "gated" else LINEAR, group, x, w, y, kind == "f32", **kw)


def weights(b, K, F, group, kind):
    return Weights(b, 2 * F if kind == "gated" else F, K, group)


def compare(b, K, F, kind, x, w, y, err=None):
    """err(sum of magnitudes): of the sums, expert_ref's if not given."""
    want, mag = ref.product(b, x, w.w)
    v = b.valid
    want = want[v]
    err = (err(mag) if err else ref.sum_error(K, mag))[v] + F32_HALF * want.abs()
    if kind == "gated":
        want, err = ref.swiglu(want[:, :F], want[:, F:], err[:, :F], err[:, F:])
    ref.check(y[v], want, err, F32_HALF if kind == "f32" else BF16_HALF, "y")
    ref.check_untouched(b, y)


def form_case(name, kind, seed=0, N=1):
    counts, K, F, group, _ = FORMS[name]
    F = F // 2 if kind == "gated" else F
    b = Batch(N, counts, sum(counts) + 9, seed)
    assert takes(b, K, F, kind) == expected(name, kind == "f32")
    return b, K, F, group


KINDS = ["bf16", "f32", "gated"]


# ---- large tiles: odd and even numbers of units of 128, whole and partial last ones, several tiles of an expert ---------

LARGE_ROWS = [
    (1, [161, 0, 320, 129, 1], 700),
    (1, [160, 159, 321, 16, 480], 1200),
    (2, [300, 31, 415, 0], 320),       # each rank's last expert is cut by its region's end
    (1, [127, 128, 257, 255], 800),
    (4, [640, 0, 0, 33], 700),
]


@pytest.mark.parametrize("K,group", [(32, 32), (96, 32), (128, 128), (192, 64), (256, 128), (288, 32), (384, 128), (544, 32),
                                     (768, 64), (1056, 32), (1152, 128), (2304, 32)])
@pytest.mark.parametrize("N,counts,cap", LARGE_ROWS, ids=str)
@pytest.mark.parametrize("kind", KINDS)
def test_large_tiles(N, counts, cap, K, group, kind):
    F = 1048 if kind == "gated" else 2088  # a part of a tile of matrix rows at the end
    b = Batch(N, counts, cap)
    assert takes(b, K, F, kind) == (128 if kind == "f32" else 160, 1)
    x, w, y = b.row_values(K), weights(b, K, F, group, kind), out(b, F, kind)
    run(b, K, F, group, kind, x, w, y)
    compare(b, K, F, kind, x, w, y)


@pytest.mark.parametrize("K", [16416, 17408])
@pytest.mark.parametrize("kind", ["bf16", "gated"])
def test_large_tiles_of_long_sums(K, kind):
    """bf16 results of sums beyond 16384 terms, in parts of 512: within a part an addition is off by at most a unit (2^-23)
    of what the part holds, and the parts are added rounding to nearest."""
    F = 1672 if kind == "gated" else 3336
    b = Batch(1, [161, 129], 300)
    assert takes(b, K, F, kind) == (128, 1)
    x, w, y = b.row_values(K), weights(b, K, F, 32, kind), out(b, F, kind)
    run(b, K, F, 32, kind, x, w, y)
    compare(b, K, F, kind, x, w, y, lambda mag: (516 * 2.0 ** -23 + (K / 512 + 1) * F32_HALF) * mag)


def test_large_tiles_many_experts():
    """More tiles than blocks, of every size."""
    counts = [(7 * e * e) % 330 for e in range(120)]
    b = Batch(4, counts, 6000)
    K, F = 416, 1032
    assert takes(b, K, F) == (160, 1)
    x, w, y = b.row_values(K), Weights(b, F, K, 32), b.out(F, torch.bfloat16)
    run(b, K, F, 32, "bf16", x, w, y)
    compare(b, K, F, "bf16", x, w, y)


# ---- every form ---------------------------------------------------------------

@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("kind", KINDS)
def test_product(name, kind):
    b, K, F, group = form_case(name, kind)
    x, w, y = b.row_values(K), weights(b, K, F, group, kind), out(b, F, kind)
    run(b, K, F, group, kind, x, w, y)
    compare(b, K, F, kind, x, w, y)
    again = out(b, F, kind)
    for _ in range(5):
        run(b, K, F, group, kind, x, w, again)
        assert torch.equal(again, y)


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_exact_sums(name, kind):
    """Whole numbers whose sums fit 24 bits: no weight, product or sum is rounded, results once."""
    b, K, F, group = form_case(name, kind)
    kw = dict(generator=b.g, device="cuda")
    x = torch.randint(-16, 17, (b.rows, K), **kw).to(torch.bfloat16)
    w = Weights.__new__(Weights)
    q = torch.randint(-8, 8, (b.E, F, K), dtype=torch.int8, **kw)
    s = torch.randint(1, 16, (b.E, K // group, F), **kw).float()
    w.wq, w.gs, w.rs = moe.pack_w4(q), s.to(torch.float8_e4m3fn), torch.ones(b.E, F, device="cuda")
    w.w = q.double() * s.double().transpose(1, 2).repeat_interleave(group, 2)
    y = out(b, F, kind)
    run(b, K, F, group, kind, x, w, y)
    want, mag = ref.product(b, x, w.w)
    assert float(mag.max()) < 2 ** 24
    assert torch.equal(y[b.valid], want[b.valid].to(y.dtype))


@pytest.mark.parametrize("name", FORMS)
def test_what_stands_in_other_rows_and_weights_has_no_influence(name):
    """NaN in rows without a token and in the scales of experts without rows; NaN of one expert's row stays there."""
    b, K, F, group = form_case(name, "bf16")
    x, w = b.row_values(K), Weights(b, F, K, group)
    at = b.span(0).stop - 1
    x[at] = float("nan")
    for e in range(b.E):
        if b.span(e).stop == b.span(e).start:
            w.gs[e], w.rs[e] = 0x7f, float("nan")
    y = b.out(F, torch.bfloat16)
    run(b, K, F, group, "bf16", x, w, y)
    assert torch.isnan(y).any(1).nonzero().flatten().tolist() == [at]
    ref.check_untouched(b, y)


@pytest.mark.parametrize("name", FORMS)
def test_offsets_of_no_batch_stand_for_no_rows(name):
    b, K, F, group = form_case(name, "bf16")
    x, w, good = b.row_values(K), Weights(b, F, K, group), b.offsets.clone()
    for change in ((1, 1 << 30), (b.E, -1), (0, 1 << 29)):
        b.offsets = good.clone()
        b.offsets[change[0]] = change[1]
        y = b.out(F, torch.bfloat16)
        run(b, K, F, group, "bf16", x, w, y)
        assert bool((y == SENTINEL).all()), change


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("kind", KINDS)
def test_captured_call_follows_new_routing(name, kind):
    b, K, F, group = form_case(name, kind)
    c = Batch(1, FORMS[name][0][::-1], b.cap, seed=1)
    c.T = b.T
    x, w, y = c.row_values(K), weights(b, K, F, group, kind), out(b, F, kind)
    run(b, K, F, group, kind, x, w, y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(b, K, F, group, kind, x, w, y)
    b.offsets.copy_(c.offsets)
    y.fill_(SENTINEL)
    graph.replay()
    compare(c, K, F, kind, x, w, y)


@pytest.mark.parametrize("name", FORMS)
def test_same_bits_in_graphs_on_streams_and_from_threads(name):
    kind = "gated"
    b, K, F, group = form_case(name, kind)
    x, w, want = b.row_values(K), weights(b, K, F, group, kind), out(b, F, kind)
    run(b, K, F, group, kind, x, w, want)
    outs, graphs, failed = [out(b, F, kind) for _ in range(4)], [], []
    for y in outs[:2]:  # two graphs, replayed at the same time
        s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=s):
            for _ in range(5):
                run(b, K, F, group, kind, x, w, y)
        graphs.append((graph, s))
    for graph, s in graphs:
        with torch.cuda.stream(s):
            graph.replay()

    def work(y):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                run(b, K, F, group, kind, x, w, y, stream=s)
            s.synchronize()
        except BaseException as e:  # reported by the test's own thread
            failed.append(e)

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work, args=(y,)) for y in outs[2:]]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for y in outs:
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))


# ---- a cluster's second tile ------------------------------------------------------

CLUSTERS = r'''
#include <stdio.h>
#include "expert_w4.cu"
int main() {  // clusters of four blocks of the split kernel that are resident at once
    using namespace moe;
    const auto kern = expert_w4_kernel<64, false, true, true, true>;
    using S = Shape<64, true, true, true>;
    PairLaunch l(S::kThreads, S::kSmem + groups_bytes(1024), nullptr);
    l.attr[1].val.clusterDim.x = 4;
    l.cfg.gridDim = dim3(4);
    PairCache cache;
    if (cache.prepare(reinterpret_cast<const void *>(kern), l.cfg) != cudaSuccess) return 1;
    printf("%d\n", cache.blocks / 2);
}
'''


@pytest.fixture(scope="module")
def clusters(tmp_path_factory):
    d = tmp_path_factory.mktemp("clusters")
    (d / "clusters.cu").write_text(CLUSTERS)
    subprocess.run([_build.nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-o", str(d / "clusters"), str(d / "clusters.cu"), _build.LIB,
                    "-Xlinker", "-rpath=" + _build.PKG], check=True, capture_output=True)
    return int(subprocess.run([str(d / "clusters")], check=True, capture_output=True, text=True).stdout)


@pytest.mark.parametrize("T", [17, 33, 64])
@pytest.mark.parametrize("K", [1024, 1056, 7168])
@pytest.mark.parametrize("kind", KINDS)
def test_clusters_that_join_more_than_once(clusters, T, K, kind):
    """As many tiles as the rule still splits in fours: where fewer clusters are resident (36 on a GPU of 152 SMs), some take
    a second tile, and join in buffers that they have used before."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tiles = sms // 4
    F = tiles * (64 if kind == "gated" else 128) - 24
    b = Batch(1, [T], T)
    assert takes(b, K, F, kind) == (64, 4)
    if clusters >= tiles:
        pytest.skip(f"{clusters} clusters are resident, a split batch has {tiles} tiles at most")
    x, w, y = b.row_values(K), weights(b, K, F, 32, kind), out(b, F, kind)
    run(b, K, F, 32, kind, x, w, y)
    compare(b, K, F, kind, x, w, y)
    again = out(b, F, kind)
    for _ in range(20):
        again.fill_(SENTINEL)
        run(b, K, F, 32, kind, x, w, again)
        assert torch.equal(again, y)


# ---- long arrays -------------------------------------------------------------------

@pytest.mark.parametrize("name,counts,F,want_form", [("few", [3, 1], 1040, (8, 1)), ("split in twos", [40, 31], 1040, (64, 2)),
                                                     ("large tiles", [161, 300], 2064, (160, 1))])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_rows_beyond_32_bit_offsets(name, counts, F, want_form, kind):
    """The second rank's region begins past 2^31 elements of x and y."""
    K, cap = 2304, 1 << 21
    assert cap * F > 1 << 31 and cap * K > 1 << 31
    b = Batch(2, [0, 0] + counts, cap)
    if name == "large tiles" and kind == "f32":
        want_form = (128, 1)
    assert takes(b, K, F, kind) == want_form
    some = Batch(1, counts, sum(counts))
    w = Weights(some, F, K, 32)
    full = Weights.__new__(Weights)
    full.wq, full.gs, full.rs = (torch.cat([torch.zeros_like(t), t]) for t in (w.wq, w.gs, w.rs))
    x = torch.empty(b.rows, K, dtype=torch.bfloat16, device="cuda")
    rows = slice(cap, cap + sum(counts))
    x[rows] = some.row_values(K)
    x[rows.stop:rows.stop + 200] = float("nan")
    y = torch.full((b.rows, F), SENTINEL, dtype=torch.float32 if kind == "f32" else torch.bfloat16, device="cuda")
    run(b, K, F, 32, kind, x, full, y)
    compare(some, K, F, kind, x[rows], w, y[rows])
    for part in (y[:cap], y[rows.stop:]):
        assert all(bool((p == SENTINEL).all()) for p in part.split(1 << 18))
