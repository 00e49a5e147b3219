"""Host side of the decode step's operators, without a GPU: the C entry points' checks on structs
with pointers that are never read, the Python checks on CPU tensors, and the frequency rule."""
import math

import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv
from nvfp4_weight_only_gemv_gb300 import decode_ops

P = 4096  # never dereferenced: every call below fails its checks or has nothing to do

NORM = dict(zip("x residual weight residual_out y scales ldx ldr ldro ldy x_type residual_type w_type y_type rows cols "
                "group eps".split(), [P, 0, P, 0, P, 0, 64, 0, 0, 64, 1, 1, 0, 1, 2, 64, 0, 1e-6]))
APPEND = dict(zip("q k v positions seq_ids inv_freq q_norm k_norm q_out k_cache v_cache k_scale v_scale page_table qt qh "
                  "kt kh vt vh kps vps ts x_type norm_type cache_type tokens seqs q_heads kv_heads head_dim rotary_half "
                  "interleaved pages max_pages page_size mscale eps".split(),
                  [P, P, P, P, 0, P, 0, 0, P, P, P, 0, 0, P, 512, 64, 128, 64, 128, 64, 2048, 2048, 4, 1, 0, 1, 2, 1, 8, 2,
                   64, 32, 0, 4, 4, 16, 1.0, 1e-6]))
ATTEND = dict(zip("q k_cache v_cache k_scale v_scale page_table lengths out lse workspace qt qh kps vps ts ws_bytes "
                  "cache_type seqs rows q_heads kv_heads head_dim pages max_pages page_size window scale".split(),
                  [P, P, P, 0, 0, P, P, P, 0, P, 512, 64, 2048, 2048, 4, 1 << 40, 1, 2, 1, 8, 2, 64, 4, 4, 16, 0, 0.125]))


def _norm(**kw):
    return nv.library().nvfp4_rms_norm(decode_ops._NORM(*{**NORM, **kw}.values()), None)


def _append(**kw):
    return nv.library().nvfp4_rope_append(decode_ops._APPEND(*{**APPEND, **kw}.values()), None)


def _attend(**kw):
    return nv.library().nvfp4_paged_attention(decode_ops._ATTEND(*{**ATTEND, **kw}.values()), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), 1), (dict(weight=0), 1), (dict(y=0), 1), (dict(residual=P), 1), (dict(y_type=2), 1),
    (dict(rows=-1), 2), (dict(cols=-8), 2), (dict(eps=-1.0), 2), (dict(eps=math.nan), 2), (dict(group=16), 2),
    (dict(y_type=2, scales=P, group=8), 2), (dict(y_type=2, scales=P, group=512), 2), (dict(y_type=2, scales=P, group=48), 2),
    (dict(ldy=63), 2), (dict(ldx=-1), 2), (dict(residual=P, residual_out=P, ldro=1), 2),
    (dict(x_type=2), 4), (dict(w_type=3), 4), (dict(y_type=5), 4), (dict(residual=P, residual_out=P, residual_type=2), 4),
    (dict(cols=32769, ldx=40000, ldy=40000), 5), (dict(rows=0), 0), (dict(cols=0), 0)])
def test_rms_norm_arguments(kw, status):
    assert _norm(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(k=0), 1), (dict(v=0), 1), (dict(positions=0), 1), (dict(inv_freq=0), 1), (dict(q_out=0), 1), (dict(k_cache=0), 1),
    (dict(v_cache=0), 1), (dict(page_table=0), 1),
    (dict(tokens=-1), 2), (dict(rotary_half=33), 2), (dict(page_size=0), 2), (dict(seqs=0), 2), (dict(tokens=3, seqs=2), 2),
    (dict(eps=math.nan), 2), (dict(head_dim=-1), 2), (dict(pages=-1), 2),
    (dict(x_type=2), 4), (dict(cache_type=0), 4), (dict(q_norm=P, norm_type=2), 4),
    (dict(head_dim=1032), 5), (dict(max_pages=1 << 21), 5), (dict(q_heads=70000), 5),
    (dict(tokens=0), 0), (dict(head_dim=0, rotary_half=0), 0), (dict(q=0, kv_heads=0), 0)])
def test_rope_append_arguments(kw, status):
    assert _append(**kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), 1), (dict(k_cache=0), 1), (dict(v_cache=0), 1), (dict(page_table=0), 1), (dict(lengths=0), 1),
    (dict(out=0), 1), (dict(workspace=0), 1),
    (dict(rows=9), 2), (dict(q_heads=7), 2), (dict(seqs=-1), 2), (dict(kv_heads=0), 2), (dict(page_size=0), 2),
    (dict(window=-1), 2), (dict(ws_bytes=0), 2), (dict(workspace=P + 16), 3),
    (dict(cache_type=0), 4), (dict(head_dim=520), 5), (dict(max_pages=1 << 21), 5),
    (dict(seqs=0), 0), (dict(rows=0), 0), (dict(q_heads=0, kv_heads=0), 0), (dict(head_dim=0), 0)])
def test_paged_attention_arguments(kw, status):
    assert _attend(**kw) == status


def test_null_structs():
    lib = nv.library()
    for f in (lib.nvfp4_rms_norm, lib.nvfp4_rope_append, lib.nvfp4_paged_attention):
        assert f(None, None) == 1


def test_cpu_tensors_are_refused():
    x, w = torch.zeros(2, 64), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        nv.rms_norm(x, w)
    c = torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        nv.rope_append(None, x.view(2, 1, 64), x.view(2, 1, 64), i, w, c, c, i.view(1, 2))
    with pytest.raises(ValueError, match="CUDA"):
        nv.paged_attention(c[0], c, c, i.view(1, 2), i)


def test_rope_frequencies():
    f, m = nv.rope_frequencies(128, 1e6, device="cpu")
    assert m == 1.0 and f.shape == (64,) and float(f[0]) == 1.0
    assert torch.allclose(f.double(), torch.tensor([1e6 ** (-i / 64) for i in range(64)], dtype=torch.float64), rtol=1e-7)
    lin, m = nv.rope_frequencies(128, 1e6, factor=4.0, device="cpu")
    assert m == 1.0 and torch.allclose(lin * 4, f)
    mix, m = nv.rope_frequencies(128, 1e4, factor=4.0, original_length=4096, device="cpu")
    f, _ = nv.rope_frequencies(128, 1e4, device="cpu")
    assert m == pytest.approx(0.1 * math.log(4.0) + 1)
    ratio = (f / mix).double()
    turns = 4096 * f.double() / (2 * math.pi)
    assert torch.allclose(ratio[turns > 33], torch.ones(()).double()) and torch.allclose(ratio[turns < 0.9], torch.full((), 4.0).double())
    assert bool((ratio[1:] >= ratio[:-1] - 1e-6).all())
    for bad in (0, 7, -2):
        with pytest.raises(ValueError):
            nv.rope_frequencies(bad)


def test_workspace_bytes_refuse_what_the_call_refuses():
    assert nv.attention_workspace_bytes(64, 8, 64, 8, 128) > 0
    for bad in ((1, 9, 8, 8, 128), (1, 1, 7, 2, 128), (-1, 1, 8, 8, 128), (1, 1, 8, 8, 520)):
        with pytest.raises(ValueError):
            nv.attention_workspace_bytes(*bad)
