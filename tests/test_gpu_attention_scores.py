"""Attention with capped scores and with a bias that falls with distance, over caches of every type.

References, tolerances and inputs are those of test_gpu_decode_ops_4bit.
"""
import math

import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv
from test_gpu_decode_ops import BF16, DEV, FP8, U16
from test_gpu_decode_ops_4bit import FP4, _check, _inputs

pytestmark = pytest.mark.gpu
FORMS = [(30.0, False), (0.0, True), (5.0, True)]


def _slopes(hq, signed=False):
    s = torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEV) / hq)
    if signed:
        s[1::2] *= -0.01
    return s


def _scored(lengths, rows, hq, hk, D, page, cap, biased, cache, signed=False, **kw):
    _check(lengths, rows, hq, hk, D, page, cache=cache, cap=cap, slopes=_slopes(hq, signed) if biased else None, q_gain=4.0, **kw)


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
@pytest.mark.parametrize("cap,biased", FORMS)
@pytest.mark.parametrize("D", [64, 128, 256, 80])
@pytest.mark.parametrize("rows,hq,hk", [(1, 8, 2), (4, 6, 1), (8, 16, 2), (8, 32, 1)])
def test_scores(cache, cap, biased, D, rows, hq, hk):
    _scored([37, 0, 1, 300, 16, 2], rows, hq, hk, D, 16, cap, biased, cache, seed=D + rows)


@pytest.mark.parametrize("cache", [BF16, FP8])
def test_scores_on_the_kernel_for_any_shape(cache):
    for cap, biased in FORMS:
        _scored([40, 7], 2, 4, 2, 33, 5, cap, biased, cache)
        _scored([40, 7], 2, 4, 2, 320, 16, cap, biased, cache)


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
@pytest.mark.parametrize("window", [1, 16, 100])
def test_scores_with_windows(cache, window):
    for cap, biased in FORMS:
        _scored([0, 1, 33, 400], 4, 6, 2, 128, 16, cap, biased, cache, window=window, seed=window)


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
def test_slopes_of_either_sign(cache):
    _scored([700, 33], 3, 8, 2, 128, 16, 0.0, True, cache, signed=True)


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
@pytest.mark.parametrize("cap", [2.0 ** -40, 0.01, 1.0, 1000.0, 2.0 ** 40])
def test_caps_from_the_smallest_to_the_largest(cache, cap):
    _scored([90, 3], 2, 4, 2, 64, 16, cap, False, cache)


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
@pytest.mark.parametrize("scale", [0.0, -0.3])
def test_scores_with_other_scales(cache, scale):
    for cap, biased in FORMS:
        _scored([90, 3], 2, 4, 2, 64, 16, cap, biased, cache, scale=scale)


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
def test_scores_over_a_long_context_and_many_items(cache):
    _scored([131071, 40000], 1, 8, 2, 128, 64, 30.0, True, cache)
    for seqs in (32, 33):
        _scored([(1000 + 397 * i) % 2100 for i in range(seqs)], 4, 32, 8, 128, 16, 30.0, True, cache)


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
def test_neither_form_is_plain_attention(cache):
    q, kc, vc, table, ln, ks, vs = _inputs([300, 5], 2, 8, 2, 128, cache, 16, 4)
    want = nv.paged_attention(q, kc, vc, table, ln, k_scale=ks, v_scale=vs)
    assert torch.equal(nv.paged_attention(q, kc, vc, table, ln, k_scale=ks, v_scale=vs, softcap=0.0, slopes=None), want)
    # slopes of zero change nothing but roundings of the exponent
    got = nv.paged_attention(q, kc, vc, table, ln, k_scale=ks, v_scale=vs, slopes=torch.zeros(8, device=DEV))
    assert torch.allclose(got.float(), want.float(), rtol=2 * U16, atol=2.0 ** -10)


@pytest.mark.parametrize("window", [0, 24])
@pytest.mark.parametrize("cap,biased", FORMS)
def test_what_a_row_does_not_see_does_not_reach_it(cap, biased, window):
    rows, n, page, D, hk = 4, 61, 16, 128, 2
    q, kc, vc, table, ln, _, _ = _inputs([n], rows, 8, hk, D, BF16, page, 21)
    kw = dict(window=window, softcap=cap, slopes=_slopes(8) if biased else None)
    clean = nv.paged_attention(q, kc, vc, table, ln, **kw)
    for value in (math.nan, math.inf, 3e38):
        for c in (kc, vc):
            c[int(table[0, (n - 1) // page]), :, (n - 1) % page] = value
        got = nv.paged_attention(q, kc, vc, table, ln, **kw)
        assert torch.equal(got[:rows - 1], clean[:rows - 1]), value
    assert nv.device_status() == 0


def test_infinite_scores_reach_the_cap():
    # a key of -inf scores -cap and not -inf: it keeps a weight, and a row of nothing else is their mean
    n, D = 40, 64
    q, kc, vc, table, ln, _, _ = _inputs([n], 1, 2, 1, D, BF16, 16, 5)
    q.fill_(1.0)
    for i in range(3):
        kc[int(table[0, i])] = -math.inf
    lse = torch.empty((1, 2), device=DEV)
    got = nv.paged_attention(q, kc, vc, table, ln, softcap=2.0, lse=lse)
    vals = vc[table[0].long()].double()[:, 0].reshape(-1, D)[:n]
    assert torch.allclose(got[0].double(), vals.mean(0).expand(2, -1), rtol=2 * U16, atol=2.0 ** -9)
    assert torch.allclose(lse.double(), torch.full_like(lse, -2 + math.log(n)).double(), atol=1e-5)
    # with a bias alone they still weigh nothing
    got = nv.paged_attention(q, kc, vc, table, ln, slopes=_slopes(2), lse=lse)
    assert not got.float().any() and bool((lse == -math.inf).all())


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
@pytest.mark.parametrize("scale,cap", [(1e30, 2.0 ** -40), (1e30, 50.0), (1e-30, 2.0 ** 40)])
def test_extreme_scales_and_caps(cache, scale, cap):
    # scores far beyond the cap are +-cap, those of zero stay zero: every other key is zero
    q, kc, vc, table, ln, ks, vs = _inputs([32], 1, 2, 1, 64, cache, 16, 9)
    kc.view(torch.uint8).zero_()
    lse = torch.empty((1, 2), device=DEV)
    got = nv.paged_attention(q, kc, vc, table, ln, scale, softcap=cap, k_scale=ks, v_scale=vs, lse=lse)
    assert torch.allclose(lse, torch.full_like(lse, math.log(32)), atol=1e-5) and torch.isfinite(got.float()).all()


def test_refusals():
    q, kc, vc, table, ln, _, _ = _inputs([5, 6], 2, 4, 2, 64, BF16, 16, 8)
    one = torch.ones(4, device=DEV)
    for bad in (dict(slopes=one[:3]), dict(slopes=one.to(BF16)), dict(slopes=one.cpu()), dict(slopes=one[None]), dict(slopes=1.0),
                dict(slopes=torch.ones(8, device=DEV)[::2]), dict(softcap=None), dict(softcap="1")):
        with pytest.raises((TypeError, ValueError)):
            nv.paged_attention(q, kc, vc, table, ln, **bad)
    for cap in (-1.0, math.nan, math.inf, 2.0 ** -41, 2.0 ** 41):
        with pytest.raises(nv.NVFP4Error) as e:
            nv.paged_attention(q, kc, vc, table, ln, softcap=cap)
        assert e.value.status == 2


def test_scores_on_another_stream_and_captured():
    q, kc, vc, table, ln, ks, vs = _inputs([500, 30], 2, 8, 2, 128, FP4, 16, 7)
    kw = dict(k_scale=ks, v_scale=vs, softcap=9.0, slopes=_slopes(8))
    want = nv.paged_attention(q, kc, vc, table, ln, **kw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = nv.paged_attention(q, kc, vc, table, ln, stream=side, **kw)
    side.synchronize()
    assert torch.equal(got, want)
    ws, graph = nv.attention_workspace(2, 2, 8, 2, 128), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = nv.paged_attention(q, kc, vc, table, ln, workspace=ws, **kw)
    for _ in range(3):
        kept.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept, want)
    assert nv.device_status() == 0
