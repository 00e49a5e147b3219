"""Appends to 8-bit and 4-bit caches by head scales from the ends of fp32's range: the codes are those of the fp32 quotient, in
both kernels."""
import math

import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv
from test_gpu_decode_ops import BF16, DEV, F32, FP8, _gen, _randn
from test_gpu_decode_ops_4bit import FP4, _bytes_at, _records_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("variant", [0, 1])
@pytest.mark.parametrize("xt", [F32, BF16])
@pytest.mark.parametrize("D", [128, 24 * 2])
@pytest.mark.parametrize("cache", [FP8, FP4])
def test_codes_by_extreme_scales(cache, D, xt, variant):
    scales = torch.tensor([math.inf, 3e38, 2.0 ** 100, 1.0, 2.0 ** -100, 2.0 ** -126, 2.0 ** -140, 2.0 ** -149], device=DEV)
    T, hk = 16, len(scales)
    x = _randn((T, hk, D), _gen(5)) * torch.exp2(torch.arange(-120, 120, 15, device=DEV).float())[:, None, None]
    x[0, :, 3], x[1], x[2, :, 7] = math.inf, 0.0, -math.inf
    x = x.to(xt)
    kc, vc = nv.kv_cache(1, hk, 16, D, cache)
    table, pos = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    nv.set_variant(variant)
    try:
        nv.rope_append(None, x, x, pos, torch.empty(0, device=DEV), kc, vc, table, k_scale=scales, v_scale=scales)
    finally:
        nv.set_variant(0)
    assert nv.device_status() == 0
    for c in (kc, vc):
        if cache is FP8:
            want = (x.float() / scales[:, None]).clamp(-448, 448).to(FP8)
            got = c[0].transpose(0, 1).contiguous()
            nan = torch.isnan(want.float())
            assert torch.equal(torch.isnan(got.float()), nan)
            # as values: the correction of a quotient of -0 is +0 - 0, which is +0, so its code may have either sign
            assert torch.equal(got.float()[~nan], want.float()[~nan])
            continue
        codes, blocks = _records_of(x, scales)
        nan = (x.float() / scales[:, None]).unflatten(2, (-1, 16)).isnan().any(dim=3)
        for t in range(T):
            gc, gb = _bytes_at(c, 0, t)
            assert bool((gb[nan[t]] & 0x7f == 0x7f).all())
            fine = ~nan[t]
            assert torch.equal(gb[fine], blocks[t][fine]), t
            same = fine.repeat_interleave(16, dim=1)
            assert torch.equal(gc[same], codes[t][same]), t
