"""Host-side checks of the experts' products: exports and refusals.  Nothing is launched."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import combine_moe_route_topk_gb300 as moe
from combine_moe_route_topk_gb300 import _build
from conftest import ROOT

OK = ctypes.c_void_p(0x10000)      # aligned, never dereferenced on the host
ODD = ctypes.c_void_p(0x10008)     # not 16-byte aligned
ODD4 = ctypes.c_void_p(0x10002)    # not 4-byte aligned
LINEAR, SWIGLU = moe.MOE_EXPERT_LINEAR, moe.MOE_EXPERT_SWIGLU
INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.lib()


def _dims(**kw):
    return moe.make_dims(**{**dict(N=2, T=8, E=4, R=2, H=8, cap_rows=16), **kw})


def _call(lib, name, d=None, K=128, F=128, act=LINEAR, a=OK, s=OK, b=OK, t=OK, off=OK, out=OK, extra=None, dtype=0):
    d = ctypes.byref(d if d is not None else _dims())
    if name == "gemm":
        return lib.moe_expert_gemm(d, K, F, act, a, b, off, out, extra, None)
    if name == "dgrad":
        return lib.moe_expert_gemm_dgrad(d, K, F, a, b, off, out, None)
    if name == "wgrad":
        return lib.moe_expert_gemm_wgrad(d, K, F, a, b, off, out, dtype, None)
    if name == "swiglu_grad":
        return lib.moe_expert_swiglu_grad(d, F, a, b, off, out, None)
    return lib.moe_expert_gemm_fp8(d, K, F, act, a, s, b, t, off, out, extra, None)


EVERY = ["gemm", "dgrad", "wgrad", "swiglu_grad", "fp8"]


def test_library_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "moe_expert.h")).read()
    names = set(re.findall(r"\b(moe_expert_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert len(names) == 5
    for name in names:
        assert hasattr(lib, name), name


@pytest.mark.parametrize("name", EVERY)
@pytest.mark.parametrize("kw,code,msg", [
    (dict(F=0), INVALID, "multiples of 8"),
    (dict(F=132), INVALID, "multiples of 8"),
    (dict(F=-8), INVALID, "multiples of 8"),
    (dict(F=(1 << 24) + 8), UNSUPPORTED, "2^24"),
    (dict(off=None), INVALID, "expert_offsets"),
    (dict(off=ODD4), INVALID, "expert_offsets"),
    (dict(a=None), INVALID, "NULL"),
    (dict(b=None), INVALID, "NULL"),
    (dict(out=None), INVALID, "NULL"),
    (dict(a=ODD), INVALID, "16-byte"),
    (dict(b=ODD), INVALID, "16-byte"),
    (dict(out=ODD), INVALID, "16-byte"),
    (dict(d=_dims(E=5)), INVALID, "multiple of N"),
    (dict(d=_dims(R=5)), INVALID, "exceeds E"),
    (dict(d=_dims(N=64, T=100000, E=384, R=8, cap_rows=0)), UNSUPPORTED, "2^31"),
])
def test_bad_arguments_are_refused_before_anything_is_enqueued(lib, name, kw, code, msg):
    assert _call(lib, name, **kw) == code
    assert msg in lib.moe_last_error().decode()


@pytest.mark.parametrize("name", ["gemm", "dgrad", "wgrad", "fp8"])
@pytest.mark.parametrize("K", [0, 4, 132, -128])
def test_bad_reduction_length_is_refused(lib, name, K):
    assert _call(lib, name, K=K) == INVALID


def test_fp8_wants_whole_scale_blocks(lib):
    assert _call(lib, "fp8", K=136) == INVALID and "128" in lib.moe_last_error().decode()
    assert _call(lib, "fp8", act=SWIGLU, F=136, extra=OK) == INVALID and "128" in lib.moe_last_error().decode()


@pytest.mark.parametrize("name", ["gemm", "fp8"])
@pytest.mark.parametrize("act", [-1, 2, 16])
def test_unknown_act_is_refused(lib, name, act):
    assert _call(lib, name, act=act) == INVALID and "act" in lib.moe_last_error().decode()


def test_outputs_of_the_gated_form_are_refused_in_the_linear_one(lib):
    assert _call(lib, "gemm", extra=OK) == INVALID and "pre" in lib.moe_last_error().decode()
    assert _call(lib, "fp8", extra=OK) == INVALID and "y_scales" in lib.moe_last_error().decode()
    assert _call(lib, "fp8", act=SWIGLU, extra=None) == INVALID and "NULL" in lib.moe_last_error().decode()
    assert _call(lib, "gemm", act=SWIGLU, extra=ODD) == INVALID


def test_scales_are_required_and_aligned(lib):
    for kw in (dict(s=None), dict(t=None), dict(s=ODD4), dict(t=ODD4), dict(act=SWIGLU, extra=ODD4)):
        assert _call(lib, "fp8", **kw) == INVALID


@pytest.mark.parametrize("name", EVERY)
def test_results_over_another_array_are_refused(lib, name):
    far = [ctypes.c_void_p(0x10000000 * i) for i in range(1, 7)]
    a, b, s, t, out, extra = far
    kw = dict(a=a, b=b, s=s, t=t, out=out)
    for other in ("a", "b") + (("s", "t") if name == "fp8" else ()):
        # the result begins in the last 16 bytes of another array, and the other way round
        if name == "wgrad":
            size = {"a": 32 * 128 * 2, "b": 32 * 128 * 2}[other]
        else:
            size = {"a": 32 * 128 * (1 if name == "fp8" else 4 if name == "swiglu_grad" else 2),
                    "b": (4 * 128 * 128 * (1 if name == "fp8" else 2)) if name != "swiglu_grad" else 32 * 128 * 2,
                    "s": 32 * 4, "t": 4 * 4}[other]
        at = kw[other].value
        for place in (at, at + size - 16, at - 16):
            assert _call(lib, name, **{**kw, "out": ctypes.c_void_p(place)}) == INVALID, (other, place)
            assert "overlaps" in lib.moe_last_error().decode()
    if name in ("gemm", "fp8"):
        for extra in (out, a, b):
            assert _call(lib, name, act=SWIGLU, **kw, extra=extra) == INVALID
            assert "overlaps" in lib.moe_last_error().decode()


@pytest.mark.parametrize("dtype", [-1, 2, 7])
def test_wgrad_refuses_other_result_types(lib, dtype):
    assert _call(lib, "wgrad", dtype=dtype) == INVALID and "dw_dtype" in lib.moe_last_error().decode()


def test_sizes_beyond_a_tensor_map_or_the_tile_count_are_refused(lib):
    assert _call(lib, "gemm", K=1 << 20, F=1 << 20) == UNSUPPORTED and "2^40" in lib.moe_last_error().decode()
    big = _dims(N=1, T=1 << 26, E=64, R=16, cap_rows=1 << 30)
    assert _call(lib, "gemm", d=big, K=64, F=1 << 20) == UNSUPPORTED and "tiles" in lib.moe_last_error().decode()


@pytest.mark.parametrize("name", ["gemm", "dgrad", "swiglu_grad", "fp8"])
def test_an_empty_batch_is_accepted_without_buffers(lib, name):
    assert _call(lib, name, d=_dims(T=0), a=None, b=None, out=None) == moe.MOE_OK


def test_binding_refuses_cpu_tensors_and_other_types():
    d = _dims()
    bf, u8, f32, i32 = (dict(dtype=t) for t in (torch.bfloat16, torch.uint8, torch.float32, torch.int32))
    x, w, y, off = torch.zeros(32, 8, **bf), torch.zeros(4, 8, 8, **bf), torch.zeros(32, 8, **bf), torch.zeros(5, **i32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.expert_gemm(d, 8, 8, LINEAR, x, w, off, y)
    with pytest.raises(ValueError, match="required"):
        moe.expert_gemm(d, 8, 8, LINEAR, None, w, off, y)
    with pytest.raises(ValueError, match="dw must be"):
        moe.expert_gemm_wgrad(d, 8, 8, y, x, off, torch.zeros(4, 8, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.expert_gemm_fp8(d, 128, 8, LINEAR, torch.zeros(32, 128, **u8), torch.zeros(32, 1, **f32),
                            torch.zeros(4, 8, 128, **u8), torch.zeros(4, 1, 1, **f32), off, y)


def _enclosing(text, at):
    """The heads of the blocks around a place of a source without comments."""
    heads, begin = [], 0
    for i, c in enumerate(text[:at]):
        if c in "{};":
            if c == "{":
                heads.append(text[begin:i].strip())
            elif c == "}":
                heads.pop()
            begin = i + 1
    return heads + [text[begin:at].strip()]


@pytest.mark.parametrize("name", ["expert_gemm.cu", "expert_wgrad.cu"])
@pytest.mark.parametrize("needle", ["drain_ring(empty", "mb_drain(done"])
def test_both_blocks_of_a_pair_wait_for_the_leaders_commits(name, needle):
    """The leader's commits arrive in both blocks' shared memory: each block waits for its own last arrivals
    before the closing barrier, which orders threads, not arrivals under way."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, name)).read())

    def of_the_leader(at):
        return any("rank" in h.split(")")[0] for h in _enclosing(text, at) if h.startswith(("if", "else", "}")))

    places = [m.start() for m in re.finditer(re.escape(needle), text)]
    assert places and max(places) < text.rindex("cluster_sync()")
    assert not all(of_the_leader(p) for p in places)
    if "done" in needle:  # and the issuing warp, however late it comes to it, before the block frees TMEM
        assert any(of_the_leader(p) for p in places)


@pytest.mark.parametrize("name", ["expert_gemm.cu", "expert_wgrad.cu", "expert_fp8.cu", "tc_ops.cuh"])
def test_warps_meet_at_bounded_waits_only(name):
    """A named barrier of some warps would wait for ever for one that has given up.  Whole blocks and clusters meet
    before the roles part and after they are all done."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, name)).read())
    assert not re.search(r"\bbar\.|\bbarrier\.(?!cluster)|__syncthreads_|cooperative_groups", text)


@pytest.mark.parametrize("name", EVERY)
def test_results_over_the_offsets_are_refused(lib, name):
    """Blocks read expert_offsets when they start, others may be storing by then."""
    a, b, s, t, out, extra, off = (ctypes.c_void_p(0x10000000 * i) for i in range(1, 8))
    kw = dict(a=a, b=b, s=s, t=t, off=off)
    for at in (off.value - 16, off.value, off.value + 16):  # 5 offsets: 20 bytes
        assert _call(lib, name, out=ctypes.c_void_p(at), **kw) == INVALID, hex(at)
        assert "overlaps" in lib.moe_last_error().decode()
        if name in ("gemm", "fp8"):
            assert _call(lib, name, act=SWIGLU, out=out, extra=ctypes.c_void_p(at), **kw) == INVALID, hex(at)
            assert "overlaps" in lib.moe_last_error().decode()
    if name == "wgrad":
        assert _call(lib, name, d=_dims(T=0), a=None, b=None, out=off, off=off) == INVALID
        assert "overlaps" in lib.moe_last_error().decode()


LIMITS = r'''
#include <stdio.h>
#include <stdlib.h>
#include "tc_ops.cuh"
int main() {  // "w": a wait is over; a number: the steps of the next tile, and the limit then is printed
    moe::WaitLimit limit;
    char word[32];
    printf("%lld %lld\n", moe::kPolls, moe::kStepPolls);
    while (scanf("%31s", word) == 1) {
        if (word[0] == 'w') { limit.waited(); continue; }
        limit.tile(atoi(word));
        printf("%lld\n", limit.polls());
    }
}
'''


def test_limits_of_waits_cover_the_tiles_since_the_last_one(tmp_path):
    """What a role may have to wait for: the stages of all tiles since its last wait (the zeroing warp waits at ragged
    tiles only), and the zeros of every empty tile so far (loads and mma pass them by, storing warps do not)."""
    src = tmp_path / "limits.cu"
    src.write_text(LIMITS)
    subprocess.run([_build.nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-o", str(tmp_path / "limits"), str(src)], check=True,
                   capture_output=True)

    def run(words):
        out = subprocess.run([str(tmp_path / "limits")], input=" ".join(map(str, words)), capture_output=True, text=True,
                             check=True).stdout.split()
        base, step, *limits = map(int, out)
        return [(v - base) / step for v in limits]  # in stages

    assert run([4, 4, 1]) == [4, 8, 9]                        # whole tiles, then a ragged one
    assert run([4, "w", 1, "w", 2]) == [4, 1, 2]              # nothing left over after a wait
    assert run([0] * 1000 + [2, "w", 3])[-2:] == [1002, 1003]  # a thousand matrices of zeros first
    assert run([1 << 24] * 300)[-1] == 300 << 24              # no overflow


def test_every_wait_across_tiles_has_a_limit_of_its_tiles():
    text = re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, "expert_wgrad.cu")).read())
    waits = re.findall(r"mb_wait_warp(?:_pair)?\(([^;]*)\)\s*(?:;|&&|\))", text)
    assert len(waits) == 7
    assert all("limit.polls()" in w for w in waits), waits


def test_waits_for_the_other_blocks_writes_acquire_for_the_cluster():
    """Zeros that block 1 wrote in its shared memory are read by the leader's mma: released for the cluster, they
    have to be acquired for it too (a wait's default is the block)."""
    wgrad, ops = (re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, n)).read()) for n in ("expert_wgrad.cu", "tc_ops.cuh"))
    waits = re.findall(r"(\w+)\(end_peer \+", wgrad)
    waits.remove("at_leader")  # the arrival
    assert [w for w in waits if w != "mb_init"] == ["mb_wait_warp_pair"]
    assert "mbarrier.arrive.release.cluster" in ops and "mbarrier.try_wait.parity.acquire.cluster" in ops


TILES = r'''
#include <stdio.h>
#include "tc_ops.cuh"
int main() {
    int count, most;
    while (scanf("%d %d", &count, &most) == 2) {
        const int tiles = (count + most - 1) / most, rows = moe::tile_rows(count, tiles);
        printf("%d %d\n", tiles, rows);
    }
}
'''


def test_tiles_of_the_longest_groups(tmp_path):
    """A group has up to 2^31 - 65537 rows (what the library accepts); its rows and its tiles added up pass 32 bits."""
    src = tmp_path / "tiles.cu"
    src.write_text(TILES)
    subprocess.run([_build.nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-o", str(tmp_path / "tiles"), str(src)], check=True,
                   capture_output=True)
    top = (1 << 31) - 1 - 65536
    counts = [1, 2, 63, 64, 65, 255, 256, 257, 511, 513, 10 ** 6, top // 2, top - 1000003, top - 1, top]
    cases = [(n, most) for n in counts for most in (64, 128, 256)]
    out = subprocess.run([str(tmp_path / "tiles")], input=" ".join(f"{n} {m}" for n, m in cases), capture_output=True,
                         text=True, check=True).stdout.split()
    for (n, most), tiles, rows in zip(cases, map(int, out[::2]), map(int, out[1::2])):
        assert tiles == -(-n // most) and rows == -(-n // tiles), (n, most)
        assert 0 < rows <= most and rows * (tiles - 1) < n <= rows * tiles
    # every place that cuts a group into tiles uses it
    for name in ("expert_gemm.cu", "expert_fp8.cu"):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, name)).read())
        assert "tile_rows(" in text and not re.search(r"\+ nt - 1", text)


@pytest.mark.parametrize("name", EVERY)
def test_rows_at_the_end_of_32_bits_are_refused(lib, name):
    """The last load of a region may begin a tile behind its last row."""
    top = (1 << 31) - 1 - 65536
    assert _call(lib, name, d=_dims(N=1, T=8, E=4, R=2, cap_rows=top + 1)) == UNSUPPORTED
    assert "N*cap" in lib.moe_last_error().decode()
    assert _call(lib, name, d=_dims(N=1, T=8, E=4, R=2, cap_rows=top), a=None) == INVALID  # gets as far as the pointers
