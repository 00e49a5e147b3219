"""Attention with other scores where a factor, a cap or a score is at the end of its range."""
import math

import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv
from test_gpu_decode_ops import BF16, DEV, FP8
from test_gpu_decode_ops_4bit import FP4, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(params=[0, 1], ids=["tiles", "any shape"])
def variant(request):
    nv.set_variant(request.param)
    yield request.param
    nv.set_variant(0)


@pytest.mark.parametrize("cache", [FP8, FP4])
@pytest.mark.parametrize("cap", [0.0, 50.0, 1000.0])
def test_a_head_scale_of_nan_makes_its_head_nan(variant, cache, cap):
    # the score's factor is NaN, whatever the cap makes of finite ones; the other head's rows do not change by a bit
    q, kc, vc, table, ln, ks, vs = _inputs([70, 3], 2, 4, 2, 64, cache, 16, 31)
    lse = [torch.empty((4, 4), device=DEV) for _ in range(2)]
    kw = dict(softcap=cap, v_scale=vs)
    clean = nv.paged_attention(q, kc, vc, table, ln, k_scale=ks, lse=lse[0], **kw)
    spoiled = ks.clone()
    spoiled[1] = math.nan
    got = nv.paged_attention(q, kc, vc, table, ln, k_scale=spoiled, lse=lse[1], **kw)
    assert bool(torch.isnan(got[:, 2:].float()).all()) and bool(torch.isnan(lse[1][:, 2:]).all())
    assert torch.equal(got[:, :2], clean[:, :2]) and torch.equal(lse[1][:, :2], lse[0][:, :2])
    assert nv.device_status() == 0


@pytest.mark.parametrize("cap", [1e-46, -1e-46, 5e-324, 1e300, -1e300, 2.0 ** -40 * (1 - 2.0 ** -24), 2.0 ** 40 * (1 + 2.0 ** -23)])
def test_caps_that_no_float_in_the_range_holds_are_refused(cap):
    q, kc, vc, table, ln, _, _ = _inputs([5, 6], 2, 4, 2, 64, BF16, 16, 8)
    with pytest.raises(nv.NVFP4Error) as e:
        nv.paged_attention(q, kc, vc, table, ln, softcap=cap)
    assert e.value.status == 2
    # (integers and zeros of either sign are numbers like others)
    want = nv.paged_attention(q, kc, vc, table, ln, softcap=0.0)
    assert torch.equal(nv.paged_attention(q, kc, vc, table, ln, softcap=-0.0), want)
    assert torch.equal(nv.paged_attention(q, kc, vc, table, ln, softcap=0), want)
