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


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
@pytest.mark.parametrize("cap", [8.0, 50.0, 100.0, 256.0, 1000.0])
def test_a_capped_score_has_the_bits_that_are_stated(variant, cache, cap):
    # one key a sequence, of one value: lse is the score itself. x = s / cap takes 6 roundings of 2^-24 (the factor, its
    # quotient by the cap, the product), tanh's series below 0.3 four, cap and lse's unit 5: 16 of the score, 24 with
    # room for their meeting. Beyond 0.3 tanh is within 2^-22 of 1; with up to 64 over 4 bits that is so of any score.
    x = torch.exp2(torch.linspace(-14, 3, 70, device=DEV))
    q = torch.zeros((140, 1, 64), device=DEV, dtype=BF16)
    q[:, 0, 0] = (torch.cat([x, -x]) * cap / 1.5).to(BF16)
    n = len(q)
    kc, vc = nv.kv_cache(n, 1, 16, 64, cache)
    k = torch.zeros((n, 1, 64), device=DEV)
    k[:, :, 0] = 1.5  # exact in every type
    table = torch.arange(n, dtype=torch.int32, device=DEV)[:, None]
    none = torch.empty(0, device=DEV)
    nv.rope_append(None, k, k, torch.zeros(n, dtype=torch.int32, device=DEV), none, kc, vc, table)
    lse = torch.empty((n, 1), device=DEV)
    nv.paged_attention(q, kc, vc, table, torch.ones(n, dtype=torch.int32, device=DEV), 1.0, softcap=cap, lse=lse)
    assert nv.device_status() == 0
    s = q[:, 0, :1].double() * 1.5
    z = cap * torch.tanh(s / cap)
    near = s.abs() >= 0.29 * cap
    if cache is FP4 and cap <= 64 and variant == 0:
        near[:] = True
    err = (lse.double() - z).abs() - near * cap * 2.0 ** -22
    if cache is not BF16 and variant == 0:
        # f16 weights, and what l and the reference m refer to, carry 2^7: m - 7 in base 2, where |m| is below 1, has steps
        # of 2^-21 and is off by 2^-22 of a power of two, 0.7 of it in lse; with larger |m| by 2^-24 of |m| + 7
        err -= 0.7 * torch.clamp((z.abs() * 1.4427 + 7) * 2.0 ** -24, min=2.0 ** -22)
    assert bool((err <= 24 * 2.0 ** -24 * z.abs()).all()), float((err / z.abs()).max() * 2 ** 24)
