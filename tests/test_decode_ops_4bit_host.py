"""Host side of the 4-bit cache and of attention's other scores, without a GPU: the C entry points' checks and the
Python checks on CPU tensors."""
import math

import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv
from nvfp4_weight_only_gemv_gb300 import decode_ops
from test_decode_ops_host import ATTEND, P, _append, _attend

READ = dict(zip("k_cache v_cache k_scale v_scale positions seq_ids page_table k_out v_out kps vps ts cache_type tokens seqs "
                "kv_heads head_dim pages max_pages page_size".split(),
                [P, P, 0, 0, P, 0, P, P, P, 2048, 2048, 4, 1, 2, 1, 2, 64, 4, 4, 16]))


def _read(**kw):
    return nv.library().nvfp4_cache_read(decode_ops._READ(*{**READ, **kw}.values()), None)


def _scored(softcap=0.0, slopes=0, **kw):
    return nv.library().nvfp4_paged_attention_scored(decode_ops._ATTEND(*{**ATTEND, **kw}.values()),
                                                     decode_ops._SCORES(slopes, softcap), None)


@pytest.mark.parametrize("kw,status", [
    (dict(k_cache=0), 1), (dict(v_cache=0), 1), (dict(positions=0), 1), (dict(page_table=0), 1), (dict(k_out=0), 1), (dict(v_out=0), 1),
    (dict(tokens=-1), 2), (dict(page_size=0), 2), (dict(seqs=0), 2), (dict(tokens=3, seqs=2), 2), (dict(head_dim=-1), 2), (dict(pages=-1), 2),
    (dict(kv_heads=-1), 2), (dict(max_pages=-1), 2), (dict(cache_type=3, head_dim=72), 2), (dict(cache_type=3, page_size=24), 2),
    (dict(cache_type=0), 4), (dict(cache_type=4), 4), (dict(k_scale=P), 4), (dict(v_scale=P), 4),
    (dict(head_dim=1032), 5), (dict(max_pages=1 << 21), 5), (dict(kv_heads=40000), 5),
    (dict(tokens=0), 0), (dict(head_dim=0), 0), (dict(kv_heads=0), 0), (dict(tokens=0, cache_type=3, k_scale=P), 0)])
def test_cache_read_arguments(kw, status):
    assert _read(**kw) == status


def test_four_bit_caches_have_whole_records():
    empty = dict(tokens=0), dict(seqs=0)  # calls without work, which are not launched
    for kw, status in ((dict(), 0), (dict(k_scale=P, v_scale=P), 0), (dict(head_dim=72), 2), (dict(page_size=8), 2), (dict(page_size=40), 2)):
        assert _append(cache_type=3, **empty[0], **kw) == status
        assert _attend(cache_type=3, **empty[1], **kw) == status
    assert _append(cache_type=4, **empty[0]) == 4 and _attend(cache_type=4, **empty[1]) == 4


@pytest.mark.parametrize("cap,status", [(0.0, 0), (50.0, 0), (2.0 ** -40, 0), (2.0 ** 40, 0), (-1.0, 2), (math.nan, 2), (math.inf, 2),
                                        (2.0 ** -41, 2), (2.0 ** 41, 2), (-0.0, 0)])
def test_caps(cap, status):
    assert _scored(cap, seqs=0) == status and _scored(cap, P, seqs=0) == status


def test_scored_attention_checks_what_attention_checks():
    for kw, status in ((dict(q=0), 1), (dict(rows=9), 2), (dict(workspace=P + 16), 3), (dict(cache_type=0), 4), (dict(head_dim=520), 5)):
        assert _scored(1.0, P, **kw) == status
    lib = nv.library()
    assert lib.nvfp4_cache_read(None, None) == 1 and lib.nvfp4_paged_attention_scored(None, None, None) == 1
    empty = decode_ops._ATTEND(*{**ATTEND, "seqs": 0}.values())
    assert lib.nvfp4_paged_attention_scored(empty, None, None) == 0


def test_kv_cache_of_four_bits():
    k, v = nv.kv_cache(3, 2, 32, 128, torch.uint8, device="cpu")
    assert k.shape == v.shape == (3, 2, 32, 72) and k.dtype == torch.uint8
    assert k.stride(0) == 2 * 2 * 32 * 72 and v.data_ptr() - k.data_ptr() == 2 * 32 * 72
    for page, dim in ((8, 128), (16, 72), (40, 64)):
        with pytest.raises(ValueError):
            nv.kv_cache(3, 2, page, dim, torch.uint8, device="cpu")
    with pytest.raises(TypeError):
        nv.kv_cache(3, 2, 16, 64, torch.int8, device="cpu")


def test_cpu_tensors_are_refused():
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(2, 2, 16, 36, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        nv.cache_read(i, c, c, i.view(1, 2))
    with pytest.raises(TypeError):
        nv.cache_read([0, 1], c, c, i.view(1, 2))
