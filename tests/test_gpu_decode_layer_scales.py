"""The range of a 4-bit cache, and what a head scale makes of it, through the decoder layer's own cache."""
import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv
from nvfp4_weight_only_gemv_gb300.decode_layer import DecodeLayer

pytestmark = pytest.mark.gpu


def _through(layer, rows, scale, dtype=torch.uint8):
    cache = layer.make_cache(1, len(rows), 16, dtype, scale=scale)
    at = torch.arange(len(rows), dtype=torch.int32, device="cuda")
    layer.fill_cache(cache, rows, rows, at, torch.zeros_like(at))
    k, v = nv.cache_read(at, *cache[:3], k_scale=cache[3], v_scale=cache[4])
    assert nv.device_status() == 0 and torch.equal(k, v)
    return k.double()


@pytest.mark.parametrize("size", [2.0 ** -14, 1.0, 2.0 ** 14])
def test_rows_of_any_magnitude_with_a_scale(size):
    layer = DecodeLayer(hidden=256, q_heads=4, kv_heads=2, head_dim=64, ffn=256)
    gen = torch.Generator().manual_seed(3)
    rows = (size * torch.randn(20, 2, 64, generator=gen)).cuda()
    got = _through(layer, rows, size)
    # a code is off by 1 / 6 of its block's largest value at most, and its scale by 2^-4 of itself; bf16 rounds once more
    top = rows.double().view(20, 2, 4, 16).abs().amax(dim=3, keepdim=True).expand(-1, -1, -1, 16).reshape(20, 2, 64)
    assert float(((got - rows.double()).abs() / top).max()) < (1 / 6 + 2.0 ** -4) * (1 + 2.0 ** -4) + 2.0 ** -8


def test_the_range_without_a_scale_is_the_one_that_is_stated():
    layer = DecodeLayer(hidden=256, q_heads=4, kv_heads=2, head_dim=64, ffn=256)
    sizes = torch.tensor([6 * 2.0 ** -10, 6 * 2.0 ** -10 * (1 + 2.0 ** -20), 0.09375, 2688.0, 4000.0], device="cuda")
    got = _through(layer, sizes[:, None, None].expand(-1, 2, 64).contiguous(), None)
    # zeros; the smallest scale, 2^-9, by 3 (of 3 + 3 * 2^-20); 2^-6 by 6; 448 by 6, exact; 448 by 6, saturated
    want = torch.tensor([0.0, 3 * 2.0 ** -9, 0.09375, 2688.0, 2688.0], device="cuda").double()
    assert torch.equal(got, want[:, None, None].expand_as(got))


def test_eight_bits_take_a_scale_too():
    layer = DecodeLayer(hidden=256, q_heads=4, kv_heads=2, head_dim=64, ffn=256)
    rows = torch.full((4, 2, 64), 3 * 2.0 ** -12, device="cuda")
    assert torch.equal(_through(layer, rows, 2.0 ** -12, torch.float8_e4m3fn), rows.double())
    assert layer.make_cache(1, 4, 16, torch.float8_e4m3fn)[3].tolist() == pytest.approx([0.05, 0.05])
    assert layer.make_cache(1, 4, 16, torch.uint8)[3] is None
