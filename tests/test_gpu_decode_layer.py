"""A decoder layer's step through the package's calls, against the same step in 64 bits."""
import json
import subprocess
import sys

import numpy as np
import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv
import oracle
from conftest import ROOT
from nvfp4_weight_only_gemv_gb300 import synth
from nvfp4_weight_only_gemv_gb300.decode_layer import DecodeLayer

pytestmark = pytest.mark.gpu


def _bf16(x):
    return torch.from_numpy(np.asarray(x)).to(torch.bfloat16)


def _product(weight, x):
    w, s, g = weight
    y, _ = oracle.gemv(w.cpu().numpy(), s.cpu().numpy(), g, synth.bf16_bits(x))
    return torch.from_numpy(y)


def _norm(h, w):
    return h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * w.double().cpu()


def _step_ref(layer, x, residual, positions, keys, vals, inv_freq):
    """keys, vals: per sequence [tokens, kv heads, D] of earlier tokens; roundings to bf16 where the
    calls have them."""
    m, d, g = x.shape[0], layer.head_dim, layer.q_heads // layer.kv_heads
    w_in, w_post, w_q, w_k = layer.norms
    h = x.double() + (residual.double() if residual is not None else 0)
    res = h.to(torch.bfloat16)
    y = _norm(h, w_in).to(torch.bfloat16)
    q, k, v = (_product(w, y).view(m, -1, d) for w in (layer.wq, layer.wk, layer.wv))
    angle = positions.double()[:, None, None] * inv_freq.double().cpu()
    c, s = torch.cos(angle), torch.sin(angle)

    def turn(u):
        a, b = u[..., :d // 2], u[..., d // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], dim=-1).to(torch.bfloat16).double()

    q, k, v = turn(_norm(q, w_q)), turn(_norm(k, w_k)), v.to(torch.bfloat16).double()
    rows, out = m // len(keys), torch.zeros(m, layer.q_heads, d, dtype=torch.float64)
    for b in range(len(keys)):
        own = slice(b * rows, (b + 1) * rows)
        kk, vv = torch.cat([keys[b].double(), k[own]]), torch.cat([vals[b].double(), v[own]])
        for r in range(rows):
            n = len(kk) - rows + r + 1
            for hq in range(layer.q_heads):
                z = kk[:n, hq // g] @ q[b * rows + r, hq] * d ** -0.5
                out[b * rows + r, hq] = torch.softmax(z, 0) @ vv[:n, hq // g]
    o = _product(layer.wo, out.to(torch.bfloat16).view(m, -1))
    h = o + res.double()
    y = _norm(h, w_post).to(torch.bfloat16)
    f = [t.cpu().numpy() if isinstance(t, torch.Tensor) else t for w in (layer.gate, layer.up, layer.down) for t in w]
    return torch.from_numpy(oracle.ffn_swiglu(*f, synth.bf16_bits(y), float("inf"))[0]), h.to(torch.bfloat16).double()


@pytest.mark.parametrize("seqs,rows", [(1, 1), (2, 3), (8, 1)])
def test_two_layers_of_a_decode_step(seqs, rows):
    past, page = 40, 16
    layers = [DecodeLayer(hidden=256, q_heads=8, kv_heads=2, head_dim=64, ffn=512, seed=i) for i in range(2)]
    inv_freq, _ = nv.rope_frequencies(64, 1e6)
    gen = torch.Generator().manual_seed(5)
    x0 = torch.randn(seqs * rows, 256, generator=gen).to(torch.bfloat16)
    positions = (past + torch.arange(rows, dtype=torch.int32)).repeat(seqs)
    lengths = torch.full((seqs,), past + rows, dtype=torch.int32, device="cuda")
    ws, fws = nv.attention_workspace(seqs, rows, 8, 2, 64), nv.ffn_workspace(seqs * rows, 512)
    x, res, xr, rr = x0.cuda(), None, x0.double(), None
    for layer in layers:
        cache = layer.make_cache(seqs, past + rows, page)
        old = [torch.randn(2, seqs, past, 2, 64, generator=gen).to(torch.bfloat16)][0]
        for c, t in zip(cache[:2], old):
            for b in range(seqs):
                for j in range(past):
                    c[int(cache[2][b, j // page]), :, j % page] = t[b, j].cuda()
        x, res = layer.step(x, res, positions.cuda(), lengths, inv_freq, cache, ws, fws)
        xr, rr = _step_ref(layer, xr, rr, positions, list(old[0]), list(old[1]), inv_freq)
    assert nv.device_status() == 0
    # every call is within its own bound of the reference; what differs is which way values near a
    # rounding to bf16 go, 2^-8 each at five places a layer
    for got, ref in ((x, xr), (res, rr)):
        err = (got.double().cpu() - ref).norm() / ref.norm()
        assert float(err) < 5 * 2 * 2.0 ** -8, float(err)


def test_the_command_runs():
    out = subprocess.run([sys.executable, "-m", "nvfp4_weight_only_gemv_gb300.decode_layer", "--layers", "2", "--steps", "3",
                          "--context", "300", "--seqs", "2", "--rows", "2", "--cache", "fp8"],
                         cwd=ROOT, capture_output=True, text=True, timeout=250)
    assert out.returncode == 0, out.stderr[-2000:]
    line = json.loads(out.stdout.strip().splitlines()[-1])
    assert line["us_per_layer"] > 0 and line["cache"] == "fp8"
