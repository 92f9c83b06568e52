"""Host-side checks of the routing steps' gradients: exports and refusals.  Nothing is launched."""
import ctypes
import os
import re

import pytest
import torch

import combine_moe_route_topk_gb300 as moe
from combine_moe_route_topk_gb300 import _build
from conftest import ROOT

INVALID = moe.MOE_ERR_INVALID_ARG


def at(i, off=0):  # apart from each other, never dereferenced on the host
    return ctypes.c_void_p(0x10000000 * (i + 1) + off)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.lib()


def _dims(**kw):
    return moe.make_dims(**{**dict(N=2, T=8, E=4, R=2, H=64, cap_rows=16), **kw})


# arguments in order; None where NULL is allowed
ARRAYS = {"combine": ["dout", "y", "pos", "topk_w", "dy", "dtopk_w"],
          "dispatch": ["dpacked", "pos", "add", "dx"],
          "route": ["logits", "bias", "topk_idx", "topk_w", "dtopk_w", "dlogits", "dbias"]}
OPTIONAL = {"add", "bias", "dbias"}
RESULTS = {"combine": ["dy", "dtopk_w"], "dispatch": ["dx"], "route": ["dlogits", "dbias"]}
ROWS = {"dout", "y", "dy", "dpacked", "add", "dx"}  # read by 16 bytes


def _call(lib, name, d=None, fn=0, **kw):
    d = ctypes.byref(d if d is not None else _dims())
    p = {n: kw.get(n, at(i)) for i, n in enumerate(ARRAYS[name])}
    assert set(kw) <= set(p)
    if name == "combine":
        return lib.moe_combine_grad(d, *p.values(), None)
    if name == "dispatch":
        return lib.moe_dispatch_grad(d, *p.values(), None)
    v = list(p.values())
    return lib.moe_route_grad(d, v[0], v[1], fn, 1, *v[2:], None)


def test_library_exports_every_declared_symbol(lib):
    text = open(os.path.join(ROOT, "include", "moe_grad.h")).read()
    names = set(re.findall(r"\b(moe_[a-z_]+)\s*\(", re.sub(r"/\*.*?\*/", "", text, flags=re.S)))
    assert names == {"moe_combine_grad", "moe_dispatch_grad", "moe_route_grad"}
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("name", ARRAYS)
def test_missing_and_misaligned_arrays_are_refused(lib, name):
    for i, n in enumerate(ARRAYS[name]):
        if n not in OPTIONAL:
            assert _call(lib, name, **{n: None}) == INVALID, n
            assert "NULL" in lib.moe_last_error().decode()
        assert _call(lib, name, **{n: at(i, 8 if n in ROWS else 2)}) == INVALID, n
        assert "aligned" in lib.moe_last_error().decode()


@pytest.mark.parametrize("name", ARRAYS)
def test_results_over_another_array_are_refused(lib, name):
    for out in RESULTS[name]:
        for i, n in enumerate(ARRAYS[name]):
            if n == out:
                continue
            if (n, out) != ("add", "dx"):
                assert _call(lib, name, **{out: at(i)}) == INVALID, (out, n)
                assert "overlaps" in lib.moe_last_error().decode()
            assert _call(lib, name, **{out: at(i, 16 if out in ROWS else 4)}) == INVALID, (out, n)  # in part
            assert "overlaps" in lib.moe_last_error().decode()


def test_other_arguments(lib):
    assert _call(lib, "route", fn=7) == INVALID
    assert "score_fn" in lib.moe_last_error().decode()
    assert _call(lib, "route", fn=moe.MOE_BIAS_SELECT_ONLY) == INVALID
    assert "dbias must be NULL" in lib.moe_last_error().decode()
    assert _call(lib, "dispatch", d=_dims(H=128, x_dtype=moe.MOE_FP8E4M3_BLK128)) == INVALID
    assert "x_dtype" in lib.moe_last_error().decode()
    for name in ARRAYS:
        assert _call(lib, name, d=_dims(H=60)) == INVALID
        assert _call(lib, name, d=_dims(E=5)) == INVALID


@pytest.mark.parametrize("name", ["combine", "dispatch"])
def test_an_empty_batch_is_accepted_without_buffers(lib, name):
    assert _call(lib, name, d=_dims(T=0), **{n: None for n in ARRAYS[name]}) == moe.MOE_OK
    assert _call(lib, "route", d=_dims(T=0), **{n: None for n in ARRAYS["route"]}) == moe.MOE_OK


def test_binding_refuses_cpu_tensors():
    d = moe.make_dims(1, 4, 4, 2, 64)
    x, w = torch.zeros(16, 64, dtype=torch.bfloat16), torch.zeros(4, 2)
    i = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.combine_grad(d, x[:4], x, i, w, x, w)
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.dispatch_grad(d, x, i, x[:4])
    with pytest.raises(ValueError, match="CUDA tensor"):
        moe.route_grad(d, torch.zeros(4, 4), None, 0, True, i, w, w, torch.zeros(4, 4))
