"""Products called on another stream than the current one: what they allocate belongs to that stream."""
import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv
from nvfp4_weight_only_gemv_gb300 import synth
from test_gpu_decode_ops_edges import _owner

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _calls():
    p = synth.dense_problem(256, 512, 2, 0, DEV)
    f = synth.ffn_problem(1024, 512, 1, 4, DEV)
    m = synth.moe_problem(8, 128, 512, 2, 4, False, seed=2, device=DEV)
    plane, table = (t.to(DEV) for t in synth.sdict_form(synth.sdict_problem(256, 512, 2, 3)["s"]))
    d = synth.sdict_problem(256, 512, 2, 3, DEV)
    md = synth.moe_problem(4, 128, 512, 2, 2, False, seed=3, device=DEV, fill="all", max_codes=16)
    idx, tab = (t.to(DEV) for t in synth.sdict_form(md["s"].cpu()))
    gate = [f[k] for k in ("wg", "sg", "gg", "wu", "su", "gu", "x")]
    ffn = [f[k] for k in ("wg", "sg", "gg", "wu", "su", "gu", "wd", "sd", "gd", "x")]
    return {"gemv": lambda **k: nv.gemv(p["w"], p["s"], p["g"], p["x"], **k),
            "gemv_gate_up": lambda **k: nv.gemv_gate_up(*gate, **k),
            "gemv_gate_up_swiglu": lambda **k: nv.gemv_gate_up_swiglu(*gate, 1.5, **k),
            "ffn_swiglu": lambda **k: nv.ffn_swiglu(*ffn, 2.0, **k),
            "ffn_swiglu_static": lambda **k: nv.ffn_swiglu_static(*ffn, **k),
            "moe_gemv": lambda **k: nv.moe_gemv(m["w"], m["s"], m["gs"], m["ids"], m["x"], False, 4, **k),
            "gemv_sdict": lambda **k: nv.gemv_sdict(d["w"], plane, table, d["g"], d["x"], **k),
            "moe_gemv_sdict": lambda **k: nv.moe_gemv_sdict(md["w"], idx, tab, md["gs"], md["ids"], md["x"], False, 2, **k)}


@pytest.mark.parametrize("name", ["gemv", "gemv_gate_up", "gemv_gate_up_swiglu", "ffn_swiglu", "ffn_swiglu_static", "moe_gemv",
                                  "gemv_sdict", "moe_gemv_sdict"])
@pytest.mark.parametrize("handle", [False, True])
def test_a_product_on_another_stream_does_not_use_the_current_one(name, handle):
    # the current stream is busy and its pool's free blocks are full of ones
    call = _calls()[name]
    want = {t: call(out_dtype=t) for t in (torch.float32, torch.bfloat16)}
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    blocks = [torch.full((n,), 0xff, dtype=torch.uint8, device=DEV) for n in (512, 1024, 3072, 4096, 8192) for _ in range(4)]
    torch.cuda.synchronize()
    del blocks
    torch.cuda._sleep(200_000_000)  # 0.1 s of the current stream
    got = {t: call(out_dtype=t, stream=side.cuda_stream if handle else side) for t in want}
    side.synchronize()
    assert not torch.cuda.current_stream().query(), "waited for the current stream"
    for t in want:
        assert got[t].dtype == t and _owner(got[t]) == side.cuda_stream
        assert torch.equal(got[t], want[t])
    kept = torch.empty_like(want[torch.float32])
    assert call(out=kept, stream=side) is kept
    side.synchronize()
    assert torch.equal(kept, want[torch.float32])
    assert nv.device_status() == 0
