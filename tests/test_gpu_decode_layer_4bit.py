"""A decoder layer's step over a 4-bit cache with capped and biased scores, through the package's calls, against the
same step in 64 bits on the keys and values that the cache gives back."""
import json
import subprocess
import sys

import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv
from conftest import ROOT
from nvfp4_weight_only_gemv_gb300 import synth
from nvfp4_weight_only_gemv_gb300.decode_layer import DecodeLayer
from test_gpu_decode_layer import _norm, _product

import oracle

pytestmark = pytest.mark.gpu


def _step_ref(layer, x, residual, positions, rows_of, inv_freq):
    """rows_of(b): the keys and values of sequence b [tokens, kv heads, D] as the cache holds them after the append."""
    m, d, g = x.shape[0], layer.head_dim, layer.q_heads // layer.kv_heads
    w_in, w_post, w_q, _ = layer.norms
    h = x.double() + (residual.double() if residual is not None else 0)
    res = h.to(torch.bfloat16)
    q = _norm(_product(layer.wq, _norm(h, w_in).to(torch.bfloat16)).view(m, -1, d), w_q)
    angle = positions.double()[:, None, None] * inv_freq.double().cpu()
    c, s = torch.cos(angle), torch.sin(angle)
    a, b2 = q[..., :d // 2], q[..., d // 2:]
    q = torch.cat([a * c - b2 * s, b2 * c + a * s], dim=-1).to(torch.bfloat16).double()
    out, slopes = torch.zeros(m, layer.q_heads, d, dtype=torch.float64), layer.slopes.double().cpu()
    seqs = len(set(rows_of))
    rows = m // seqs
    for b in range(seqs):
        kk, vv = rows_of[b]
        for r in range(rows):
            n = len(kk) - rows + r + 1
            for hq in range(layer.q_heads):
                z = layer.softcap * torch.tanh(kk[:n, hq // g] @ q[b * rows + r, hq] * d ** -0.5 / layer.softcap)
                z = z - slopes[hq] * torch.arange(n - 1, -1, -1)
                out[b * rows + r, hq] = torch.softmax(z, 0) @ vv[:n, hq // g]
    o = _product(layer.wo, out.to(torch.bfloat16).view(m, -1))
    h = o + res.double()
    y = _norm(h, w_post).to(torch.bfloat16)
    f = [t.cpu().numpy() if isinstance(t, torch.Tensor) else t for w in (layer.gate, layer.up, layer.down) for t in w]
    return torch.from_numpy(oracle.ffn_swiglu(*f, synth.bf16_bits(y), float("inf"))[0]), h.to(torch.bfloat16).double()


@pytest.mark.parametrize("seqs,rows", [(1, 1), (2, 3)])
def test_two_layers_of_a_decode_step(seqs, rows):
    past, page = 40, 16
    slopes = torch.exp2(-torch.arange(1, 9, device="cuda").float())
    layers = [DecodeLayer(hidden=256, q_heads=8, kv_heads=2, head_dim=64, ffn=512, seed=i, softcap=4.0, slopes=slopes)
              for i in range(2)]
    inv_freq, _ = nv.rope_frequencies(64, 1e6)
    gen = torch.Generator().manual_seed(5)
    x0 = torch.randn(seqs * rows, 256, generator=gen).to(torch.bfloat16)
    positions = (past + torch.arange(rows, dtype=torch.int32)).repeat(seqs)
    lengths = torch.full((seqs,), past + rows, dtype=torch.int32, device="cuda")
    ws, fws = nv.attention_workspace(seqs, rows, 8, 2, 64), nv.ffn_workspace(seqs * rows, 512)
    x, res, xr, rr = x0.cuda(), None, x0.double(), None
    at = torch.arange(past, dtype=torch.int32, device="cuda").repeat(seqs)
    sid = torch.arange(seqs, dtype=torch.int32, device="cuda").repeat_interleave(past)
    every = torch.arange(past + rows, dtype=torch.int32, device="cuda")
    for layer in layers:
        cache = layer.make_cache(seqs, past + rows, page, torch.uint8)
        old = [torch.randn(seqs * past, 2, 64, generator=gen).to(torch.bfloat16).cuda() for _ in "kv"]
        layer.fill_cache(cache, *old, at, sid)
        x, res = layer.step(x, res, positions.cuda(), lengths, inv_freq, cache, ws, fws)
        held = {b: tuple(t.double().cpu() for t in nv.cache_read(every, *cache[:3], torch.full_like(every, b))) for b in range(seqs)}
        # the new rows differ from 64 bits by their quantisation alone, which test_gpu_decode_ops_4bit bounds
        xr, rr = _step_ref(layer, xr, rr, positions, held, inv_freq)
    assert nv.device_status() == 0
    # what differs is which way values near a rounding to bf16 go, 2^-8 each at five places a layer
    for got, ref in ((x, xr), (res, rr)):
        err = (got.double().cpu() - ref).norm() / ref.norm()
        assert float(err) < 5 * 2 * 2.0 ** -8, float(err)


def test_the_command_runs():
    out = subprocess.run([sys.executable, "-m", "nvfp4_weight_only_gemv_gb300.decode_layer", "--layers", "2", "--steps", "3",
                          "--context", "300", "--seqs", "2", "--rows", "2", "--cache", "fp4", "--softcap", "30", "--alibi"],
                         cwd=ROOT, capture_output=True, text=True, timeout=250)
    assert out.returncode == 0, out.stderr[-2000:]
    line = json.loads(out.stdout.strip().splitlines()[-1])
    assert line["us_per_layer"] > 0 and line["cache"] == "fp4" and line["softcap"] == 30.0 and line["alibi"] is True
