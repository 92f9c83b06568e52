"""Host-side checks of the experts' product with 4-bit weights: exports, refusals, the weights' form.  Nothing is launched."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import combine_moe_route_topk_gb300 as moe
from combine_moe_route_topk_gb300 import _build
from conftest import ROOT

INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED
LINEAR, SWIGLU = moe.MOE_EXPERT_LINEAR, moe.MOE_EXPERT_SWIGLU
NAMES = ["x", "wq", "group_scales", "row_scales", "expert_offsets", "y"]


def at(i, off=0):  # apart from each other, never dereferenced on the host
    return ctypes.c_void_p(0x10000000 * (i + 1) + off)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.lib()


def _dims(**kw):
    return moe.make_dims(**{**dict(N=2, T=8, E=4, R=2, H=8, cap_rows=16), **kw})


def _call(lib, d=None, K=128, F=128, act=LINEAR, group=32, **kw):
    p = [kw.get(n, at(i)) for i, n in enumerate(NAMES)]
    return lib.moe_expert_gemm_w4(ctypes.byref(d if d is not None else _dims()), K, F, act, group, *p, None)


def test_library_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "moe_expert_w4.h")).read()
    names = set(re.findall(r"\b(moe_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == {"moe_expert_gemm_w4"} and hasattr(lib, "moe_expert_gemm_w4")


@pytest.mark.parametrize("act", [LINEAR, SWIGLU])
def test_bad_arguments_are_refused(lib, act):
    for kw, code, msg in [
            (dict(F=0), INVALID, "multiples of 8"), (dict(F=132), INVALID, "multiples of 8"),
            (dict(K=0), INVALID, "multiples of 8"), (dict(K=48), INVALID, "multiple of group"),
            (dict(K=192, group=128), INVALID, "multiple of group"), (dict(group=0), INVALID, "group must be"),
            (dict(group=-32), INVALID, "group must be"), (dict(group=16), INVALID, "group must be"),
            (dict(group=256, K=256), INVALID, "group must be"), (dict(F=(1 << 24) + 8), UNSUPPORTED, "2^24"),
            (dict(K=(1 << 24) + 32), UNSUPPORTED, "2^24"), (dict(d=_dims(E=5)), INVALID, "multiple of N"),
            (dict(d=_dims(N=1, cap_rows=(1 << 31) - 65536)), UNSUPPORTED, "65536")]:
        assert _call(lib, act=act, **kw) == code, kw
        assert msg in lib.moe_last_error().decode(), kw
    assert _call(lib, act=2) == INVALID and "act" in lib.moe_last_error().decode()


def test_missing_misaligned_and_overlapping_arrays_are_refused(lib):
    for i, n in enumerate(NAMES):
        assert _call(lib, **{n: None}) == INVALID, n
        off = 8 if n in ("x", "wq", "y") else 4 if n == "group_scales" else 2
        assert _call(lib, **{n: at(i, off)}) == INVALID, n
        assert "aligned" in lib.moe_last_error().decode()
        if n != "y":
            for o in (0, 16):
                for act in (LINEAR, SWIGLU):
                    assert _call(lib, act=act, y=at(i, o)) == INVALID, n
                    assert "overlaps" in lib.moe_last_error().decode()


def test_an_empty_batch_is_accepted_without_buffers(lib):
    for act in (LINEAR, SWIGLU):
        assert _call(lib, d=_dims(T=0), act=act, x=None, wq=None, group_scales=None, row_scales=None, y=None) == moe.MOE_OK


def test_binding_refuses_cpu_tensors_and_other_types():
    d = moe.make_dims(1, 1, 1, 1, 8)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        moe.expert_gemm_w4(d, 32, 8, LINEAR, 32, torch.zeros(1, 32, dtype=torch.bfloat16), None, None, None, None, None)


def unpack(words):
    """The header's layout, word by word."""
    out = []
    for word in words.flatten().tolist():
        for i in range(8):
            v = (word >> (4 * (i // 2) + 16 * (i % 2))) & 15
            out.append(v - 16 if v > 7 else v)
    return torch.tensor(out).view(*words.shape[:-1], -1)


def test_words_hold_their_elements():
    g = torch.Generator()
    g.manual_seed(1)
    q = torch.randint(-8, 8, (3, 5, 64), generator=g, dtype=torch.int8)
    words = moe.pack_w4(q)
    assert words.dtype == torch.int32 and words.shape == (3, 5, 8)
    assert torch.equal(unpack(words), q.long())
    one = torch.zeros(8, dtype=torch.int32)
    one[5] = -1  # element 2j + 1, j = 2: bit 16 + 8
    assert int(moe.pack_w4(one)) & 0xFFFFFFFF == 0xF << 24
    for bad in (q.float(), q[..., :12], q.to(torch.int32) + 8):
        with pytest.raises(ValueError):
            moe.pack_w4(bad)


@pytest.mark.parametrize("group", [32, 64, 128])
def test_quantised_weights_are_near(group):
    g = torch.Generator()
    g.manual_seed(2)
    w = torch.randn(2, 24, 256, generator=g) * torch.rand(2, 24, 1, generator=g)
    w[0, 3] = 0  # a row of zeros, a group of zeros, one that is tiny beside the others
    w[1, 5, :group] = 0
    w[1, 6, :group] *= 1e-9
    wq, gs, rs = moe.quantize_w4(w.to(torch.bfloat16), group)
    assert wq.shape == (2, 24, 32) and gs.shape == (2, 256 // group, 24) and rs.shape == (2, 24)
    step = gs.view(torch.float8_e4m3fn).double().transpose(1, 2) * rs.double().unsqueeze(2)  # [E][W][groups]
    got = unpack(wq).double().view(2, 24, -1, group) * step.unsqueeze(3)
    w = w.to(torch.bfloat16).double().view(2, 24, -1, group)
    amax = w.abs().amax(3, keepdim=True)
    assert torch.isfinite(got).all() and bool((got[0, 3] == 0).all()) and bool((got[1, 5, 0] == 0).all())
    # half a step, or what the clamp at -8 and 7 takes off: a scale rounded down by 2^-4 leaves 7 / (1 - 2^-4) = 7.47,
    # cut to 7; a scale below the smallest one is zero or up to twice too large
    lim = torch.maximum(0.5 * step, amax.squeeze(3) / 14.9) * (1 + 1e-5)
    lim[1, 6, 0] = amax[1, 6, 0, 0]
    assert bool(((got - w).abs() <= lim.unsqueeze(3)).all())
    for bad in (w[0, 0], torch.zeros(1, 8, 48)):
        with pytest.raises(ValueError):
            moe.quantize_w4(bad, group)


@pytest.mark.parametrize("name", ["expert_w4.cu", "expert_w4_few.cu", "w4_ops.cuh"])
def test_warps_meet_at_bounded_waits_only(name):
    """A named barrier of some warps would wait for ever for one that has given up.  Whole blocks and clusters meet
    before the roles part and after they are all done."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, name)).read())
    assert not re.search(r"\bbar\.|\bbarrier\.(?!cluster)|__syncthreads_|cooperative_groups", text)
    assert text.count("__syncthreads()") <= 2
    for wait in re.findall(r"while \([^\n]*mb_try[^\n]*", text):
        assert "left > 0" in wait


@pytest.mark.parametrize("name", ["expert_w4.cu", "expert_w4_few.cu"])
def test_slots_are_given_back_by_a_lane_that_depends_on_the_words(name):
    """An arrival right behind the loads from a slot may pass them: where a warp has read, the arriving lane is chosen by
    a vote on what it read."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, name)).read())
    assert len(re.findall(r"if \(lane == reader_lane\([^;]*\)\) mb_arrive\(c?empty", text)) == 1
    assert len(re.findall(r"mb_arrive\(c?empty", text)) == 2  # the other one is of warps that read nothing


def test_a_warps_reads_are_ordered_before_its_one_arrival():
    """One lane arrives for 32 that have read.  A vote orders no memory, __syncwarp does."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(_build.CSRC, "w4_ops.cuh")).read())
    body = re.search(r"int reader_lane\(uint32_t loaded\) \{(.*?)\n\}", text, re.S).group(1)
    assert "__syncwarp()" in body and "__all_sync" in body


BOUNDS = """
#include <stdio.h>
#include "expert_w4.cu"
namespace moe {
template <int kTok, bool kParts, bool kF32, bool kSplit>
void show() {
    using S = Shape<kTok, kParts, kF32, kSplit>;
    printf("%d %d %d %d %d %d\\n", kTok, kParts, kF32, kSplit, S::kSmem + groups_bytes(1024), most_shared_w4(S::kBars));
}
void show_all() {
    show<160, false, false, false>(), show<128, true, false, false>(), show<128, true, true, false>();
    show<64, false, false, false>(), show<64, true, false, false>(), show<64, true, true, false>();
    show<64, false, false, true>(), show<64, true, false, true>(), show<64, true, true, true>();
}
}
int main() { moe::show_all(); }
"""


def test_a_blocks_shared_memory_fits_beside_its_static_words(lib, tmp_path):
    """227 KB hold the largest dynamic part that a kernel asks for and the static words that the compiler finds."""
    (tmp_path / "bounds.cu").write_text(BOUNDS)
    r = subprocess.run([_build.nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-Xptxas", "-v", "-o", str(tmp_path / "bounds"),
                        str(tmp_path / "bounds.cu"), _build.LIB, "-Xlinker", "-rpath=" + os.path.dirname(_build.LIB)],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    static = {}
    for kernel, info in re.findall(r"Compiling entry function '(\w*expert_w4_kernel\w*)'.*?Used ([^\n]*)", r.stdout + r.stderr, re.S):
        tok, _, parts, f32, split = re.search(r"Li(\d+)ELb(\d)ELb(\d)ELb(\d)ELb(\d)E", kernel).groups()
        key = (tok, parts, f32, split)
        static[key] = max(static.get(key, 0), int(re.search(r"(\d+) bytes smem", info).group(1)))
    shown = subprocess.run([str(tmp_path / "bounds")], capture_output=True, text=True, check=True).stdout.splitlines()
    assert len(shown) == len(static) == 9
    for line in shown:
        *key, dynamic, most = line.split()
        assert int(dynamic) <= int(most), key
        assert int(most) + static[tuple(key)] <= 227 * 1024, key
