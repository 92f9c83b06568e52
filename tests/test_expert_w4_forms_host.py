"""The rule that chooses a kernel of the product with 4-bit weights: which form takes which batch.  Nothing is launched."""
import pytest

import combine_moe_route_topk_gb300 as moe
from expert_ref import Batch
from w4_form import FORMS, expected, form

SMS = 152


def dense(T, K, F, gated=False, f32=False, sms=SMS):
    return form(moe.make_dims(1, T, 1, 1, 8, cap_rows=T), K, F, gated, f32, sms)


@pytest.mark.parametrize("name", FORMS)
@pytest.mark.parametrize("kind", ["bf16", "f32", "gated"])
def test_each_form_is_reached(name, kind):
    counts, K, F, group, _ = FORMS[name]
    b = Batch(1, counts, sum(counts) + 9, device="cpu")
    assert K % group == 0
    assert form(b.dims(), K, F // 2 if kind == "gated" else F, kind == "gated", kind == "f32", SMS) == expected(name, kind == "f32")


def test_forms_of_a_dense_layer():
    """One matrix of 4096 x 7168 and more and more tokens."""
    got = [dense(T, 7168, 4096) for T in (1, 8, 32, 128, 256, 300, 4096)]
    assert got == [(8, 1), (8, 1), (64, 4), (64, 2), (64, 1), (160, 1), (160, 1)]
    assert dense(4096, 7168, 4096, f32=True) == (128, 1) and dense(4096, 16384 + 32, 4096) == (128, 1)
    assert dense(4096, 7168, 4096, gated=True) == (160, 1)


def test_limits_of_the_kernel_for_few_rows():
    assert dense(1, 1 << 15, 64) == (8, 1) and dense(1, (1 << 15) + 32, 64)[0] == 64
    # eight tokens' lines leave too little room for codes
    assert dense(8, 1 << 13, 64)[0] == 64 and dense(1, 1 << 13, 64) == (8, 1)


@pytest.mark.parametrize("sms", [1, 2, 16, 148, 152, 160, 304])
def test_a_split_never_has_more_blocks_than_sms(sms):
    for T in (1, 9, 64, 65, 200, 1000, 5000):
        for K in (32, 256, 288, 1024, 1056, 7168, 40960):
            for F in (8, 264, 4096, 16384):
                for gated in (False, True):
                    tokens, split = dense(T, K, F, gated, sms=sms)
                    assert split == 1 or tokens == 64
                    assert -(-K // 256) >= split  # every block has a stage of codes
                    if split > 1:
                        assert -(-T // 64) * -(-F // (64 if gated else 128)) * split <= sms
