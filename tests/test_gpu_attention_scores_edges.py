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


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
@pytest.mark.parametrize("cap", [2.0 ** -40, 8.0, 50.0, 100.0, 1000.0, 2.0 ** 40])
@pytest.mark.parametrize("scale", [1e30, -1e30, 1e-30, -1e-30])
def test_scores_beyond_the_cap_and_of_nothing(variant, cache, cap, scale):
    # every third key is zero, the others are +-1.5 along the signs of the first head's query; the second head's is its
    # opposite. So raw scores are 0 or +-1.5 sum|q| scale: their magnitude is beyond 2^40 or below 2^-80.
    n, D, g = 41, 64, torch.Generator(device=DEV)
    g.manual_seed(17)
    q = torch.randn((1, 1, D), generator=g, device=DEV).to(BF16)
    kind = torch.arange(n, device=DEV) % 3 - 1
    k = (1.5 * kind[:, None].float() * torch.sign(q[0].float()))[:, None]
    v = torch.randn((n, 1, D), generator=g, device=DEV).to(BF16).float()
    kc, vc = nv.kv_cache(3, 1, 16, D, cache)
    table, at = torch.arange(3, dtype=torch.int32, device=DEV)[None], torch.arange(n, dtype=torch.int32, device=DEV)
    nv.rope_append(None, k, v, at, torch.empty(0, device=DEV), kc, vc, table)
    k_held, v_held = (t[:, 0].double() for t in nv.cache_read(at, kc, vc, table))
    assert torch.equal(k_held, k[:, 0].double())
    lse = torch.empty((1, 2), device=DEV)
    got = nv.paged_attention(torch.cat([q, -q], dim=1), kc, vc, table, torch.tensor([n], dtype=torch.int32, device=DEV), scale,
                             softcap=cap, lse=lse)
    assert nv.device_status() == 0
    s = torch.cat([q, -q], dim=1)[0].double() @ k_held.T * scale
    z = cap * torch.tanh(s / cap)
    # beyond the cap z is +-cap, as tanh is 1 there to 2^-22 (a short form's error, too, is 2^-22 of the cap); below it z
    # is nothing. lse has roundings of its size and of the 2^7 that weights are raised by, 8 steps of 2^-24 of them.
    far = float(z.abs().max()) if abs(scale) > 1 else 0.0
    want = torch.logsumexp(z, dim=1)
    off = 2.0 ** -21 * min(far, cap) + (2.0 ** -21 * cap if cache is FP4 and cap <= 64 else 0.0)
    assert bool(((lse[0].double() - want).abs() <= off + 8 * 2.0 ** -24 * (want.abs() * 1.4427 + 8)).all()), (lse, want)
    # weights: scores off by `off`, 11 bits; then the output's rounding
    p = torch.softmax(z, dim=1)
    tol = (p @ v_held.abs()) * (2 * off + 2.0 ** -11 + 2.0 ** -18) + (p @ v_held).abs() * 2.0 ** -8 + 2.0 ** -30
    assert bool(((got[0].double() - p @ v_held).abs() <= tol).all())


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
@pytest.mark.parametrize("cap,biased", [(50.0, False), (100.0, True), (1000.0, False)])
@pytest.mark.parametrize("scale", [3e38, -3e38])
def test_a_score_of_zero_by_a_factor_beyond_fp32(variant, cache, cap, biased, scale):
    # in base-2 units the largest scales are beyond fp32's range; scores of zero stay zero, others reach the cap
    n, D = 20, 64
    q = torch.ones((1, 1, D), device=DEV, dtype=BF16)
    k = torch.zeros((n, 1, D), device=DEV)
    k[7] = math.copysign(1.5, -scale)  # a score of -cap, of weight exp(-cap)
    v = torch.arange(n, device=DEV)[:, None, None].expand(-1, 1, D) % 4 * 0.5 + 1.5  # exact in every type
    kc, vc = nv.kv_cache(2, 1, 16, D, cache)
    table, at = torch.arange(2, dtype=torch.int32, device=DEV)[None], torch.arange(n, dtype=torch.int32, device=DEV)
    nv.rope_append(None, k, v.contiguous(), at, torch.empty(0, device=DEV), kc, vc, table)
    lse = torch.empty((1, 1), device=DEV)
    got = nv.paged_attention(q, kc, vc, table, torch.tensor([n], dtype=torch.int32, device=DEV), scale, softcap=cap,
                             slopes=torch.full((1,), 0.25, device=DEV) if biased else None, lse=lse)
    z = torch.zeros(n, dtype=torch.float64, device=DEV)
    z[7] = -cap
    if biased:
        z -= 0.25 * torch.arange(n - 1, -1, -1, device=DEV)
    assert abs(float(lse) - float(torch.logsumexp(z, 0))) <= 2.0 ** -18  # 8 steps of 2^-24 of a lse below 4 and of 7
    want = (torch.softmax(z, 0)[:, None] * v[:, 0].double()).sum(0)
    assert bool(((got[0, 0].double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -17)).all())


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("scale", [3e38, -3e38])
def test_plain_scores_of_zero_by_a_factor_beyond_fp32(variant, cache, biased, scale):
    # as above without a cap: the other key's score is beyond fp32 and its weight nothing
    n, D = 20, 64
    q = torch.ones((1, 1, D), device=DEV, dtype=BF16)
    k = torch.zeros((n, 1, D), device=DEV)
    k[7] = math.copysign(1.5, -scale)
    v = (torch.arange(n, device=DEV)[:, None, None].expand(-1, 1, D) % 4 * 0.5 + 1.5).contiguous()
    kc, vc = nv.kv_cache(2, 1, 16, D, cache)
    table, at = torch.arange(2, dtype=torch.int32, device=DEV)[None], torch.arange(n, dtype=torch.int32, device=DEV)
    nv.rope_append(None, k, v, at, torch.empty(0, device=DEV), kc, vc, table)
    lse = torch.empty((1, 1), device=DEV)
    got = nv.paged_attention(q, kc, vc, table, torch.tensor([n], dtype=torch.int32, device=DEV), scale,
                             slopes=torch.full((1,), 0.25, device=DEV) if biased else None, lse=lse)
    z = torch.zeros(n, dtype=torch.float64, device=DEV)
    z[7] = -math.inf
    if biased:
        z -= 0.25 * torch.arange(n - 1, -1, -1, device=DEV)
    assert abs(float(lse) - float(torch.logsumexp(z, 0))) <= 2.0 ** -18
    want = (torch.softmax(z, 0)[:, None] * v[:, 0].double()).sum(0)
    assert bool(((got[0, 0].double() - want).abs() <= want * (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -17)).all())
