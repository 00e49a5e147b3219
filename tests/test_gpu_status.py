"""The device status word: every operator's bits, in one read, and a call whose first use is inside a capture."""
import subprocess
import sys

import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv
from conftest import ROOT

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.bfloat16, torch.float8_e4m3fn, torch.uint8]


def _place(dtype, page_id):
    kc, vc = nv.kv_cache(2, 1, 16, 64, dtype)
    table = torch.tensor([[page_id]], dtype=torch.int32, device=DEV)
    return kc, vc, table, torch.zeros(1, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("variant", [0, 1])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("call", ["append", "read", "attention", "scores"])
def test_a_bad_page_is_reported_once(call, dtype, variant):
    rows = torch.ones((1, 1, 64), dtype=torch.bfloat16, device=DEV)
    one = torch.ones(1, dtype=torch.int32, device=DEV)

    def run(page_id):
        kc, vc, table, zero = _place(dtype, page_id)
        if call == "append":
            nv.rope_append(None, rows, rows, zero, torch.empty(0, device=DEV), kc, vc, table)
        elif call == "read":
            nv.cache_read(zero, kc, vc, table)
        else:
            nv.paged_attention(rows, kc, vc, table, one, softcap=5.0 if call == "scores" else 0.0)

    assert nv.device_status() == 0
    nv.set_variant(variant)
    try:
        run(0)
        assert nv.device_status() == 0
        run(2)
        assert nv.device_status() == nv.DEV_BAD_PAGE and nv.device_status() == 0
    finally:
        nv.set_variant(0)


def test_bits_of_several_operators_meet():
    kc, vc, table, zero = _place(torch.uint8, 9)
    nv.cache_read(zero, kc, vc, table)
    g = torch.Generator().manual_seed(1)
    w = torch.randint(256, (2, 64, 128), generator=g, dtype=torch.uint8).to(DEV)
    s = torch.full((2, 64, 16), 0x38, dtype=torch.uint8, device=DEV)
    nv.moe_gemv(w, s, torch.ones(2, device=DEV), torch.tensor([5], dtype=torch.int32, device=DEV),
                torch.ones((1, 256), dtype=torch.bfloat16, device=DEV), False, 1)
    assert nv.device_status() == nv.DEV_BAD_PAGE | nv.DEV_BAD_EXPERT and nv.device_status() == 0


FIRST_IN_A_CAPTURE = """
import torch, nvfp4_weight_only_gemv_gb300 as nv
kc, vc = nv.kv_cache(2, 1, 16, 64, getattr(torch, {dtype!r}))
table = torch.zeros((1, 1), dtype=torch.int32, device="cuda")
zero, one = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
rows, freq = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda"), torch.empty(0, device="cuda")
ws = nv.attention_workspace(1, 1, 1, 1, 64)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    nv.rope_append(None, rows, rows, zero, freq, kc, vc, table)
    k, v = nv.cache_read(zero, kc, vc, table)
    y = nv.paged_attention(rows, kc, vc, table, one, workspace=ws)
    z = nv.paged_attention(rows, kc, vc, table, one, softcap=3.0, workspace=ws)
for bad in (0, 8, 0):
    table.fill_(bad)
    graph.replay()
    torch.cuda.synchronize()
    assert nv.device_status() == (nv.DEV_BAD_PAGE if bad else 0)
    assert all(bool((t == 0 if bad else t > 0.9).all()) for t in (k, v, y, z)), (bad, k, v, y, z)
"""


@pytest.mark.parametrize("dtype", ["bfloat16", "uint8"])
def test_a_process_whose_first_calls_are_captured(dtype):
    out = subprocess.run([sys.executable, "-c", FIRST_IN_A_CAPTURE.format(dtype=dtype)], cwd=ROOT, capture_output=True,
                         text=True, timeout=250)
    assert out.returncode == 0, out.stderr[-2000:]
