"""One decoder layer's step from this package's calls, and a command that times it.

    python -m nvfp4_weight_only_gemv_gb300.decode_layer [--seqs 1] [--rows 1] [--context 8191]
                                                        [--cache bf16|fp8] [--layers 8] [--steps 50]

For the newest ``rows`` tokens of each of ``seqs`` sequences (seqs * rows <= 8 rows in all):

    y, res = rms_norm(x + res)                         x: the previous layer's product, fp32
    q, k, v = Wq y, Wk y, Wv y                         gemv
    q = rope_append(q, k, v)                           per-head norm, rotary positions, cache append
    a = paged_attention(q)                             over the cache, the new tokens included
    y, res = rms_norm(Wo a + res)                      gemv, norm with the residual's addition
    x = ffn_swiglu(y)                                  gate/up, SwiGLU, down

The sizes are those of the dense model in "llama.cpp eval-callback — ggml op level": 32 query and 8
kv heads of 128 values with per-head norms, hidden size 4096, FFN 12288. Weights are random.
"""
from __future__ import annotations

import argparse
import json

import torch

import nvfp4_weight_only_gemv_gb300 as nv
from nvfp4_weight_only_gemv_gb300 import synth


class DecodeLayer:
    """Random NVFP4 weights of one layer and the cache of its sequences."""

    def __init__(self, hidden=4096, q_heads=32, kv_heads=8, head_dim=128, ffn=12288, seed=0, device="cuda"):
        self.hidden, self.q_heads, self.kv_heads, self.head_dim, self.ffn = hidden, q_heads, kv_heads, head_dim, ffn

        def weight(n, k, s):
            p = synth.dense_problem(n, k, 1, seed * 100 + s, device=device)
            return p["w"], p["s"], p["g"]

        q, kv = q_heads * head_dim, kv_heads * head_dim
        self.wq, self.wk, self.wv = weight(q, hidden, 1), weight(kv, hidden, 2), weight(kv, hidden, 3)
        self.wo = weight(hidden, q, 4)
        self.gate, self.up, self.down = weight(ffn, hidden, 5), weight(ffn, hidden, 6), weight(hidden, ffn, 7)
        gen = torch.Generator().manual_seed(seed)
        self.norms = [(1 + 0.1 * torch.randn(n, generator=gen)).to(torch.bfloat16).to(device)
                      for n in (hidden, hidden, head_dim, head_dim)]  # input, post-attention, q, k

    def make_cache(self, seqs, tokens, page_size=64, dtype=torch.bfloat16, device="cuda"):
        """A cache of `tokens` places per sequence: (k, v, page table, k scales, v scales)."""
        per_seq = -(-tokens // page_size)
        k, v = nv.kv_cache(seqs * per_seq, self.kv_heads, page_size, self.head_dim, dtype, device)
        table = torch.arange(seqs * per_seq, dtype=torch.int32, device=device).view(seqs, per_seq)
        scale = torch.full((self.kv_heads,), 0.05, device=device) if dtype == torch.float8_e4m3fn else None
        return k, v, table, scale, scale

    def step(self, x, residual, positions, lengths, inv_freq, cache, workspace, ffn_workspace, mscale=1.0):
        """x [rows, hidden] float32 or bfloat16 and the residual stream (bfloat16; None in front of the
        first layer) -> the same pair behind this layer. positions int32 [rows], lengths int32 [seqs]
        with the new tokens counted. Rows of a sequence stand together."""
        m, d = x.shape[0], self.head_dim
        k_cache, v_cache, table, k_scale, v_scale = cache
        w_in, w_post, w_q, w_k = self.norms
        if residual is None:
            residual = x.to(torch.bfloat16)
            y = nv.rms_norm(x, w_in).y
        else:
            y, residual, _ = nv.rms_norm(x, w_in, residual=residual)
        q, k, v = (nv.gemv(*w, y).view(m, -1, d) for w in (self.wq, self.wk, self.wv))
        q = nv.rope_append(q, k, v, positions, inv_freq, k_cache, v_cache, table, mscale=mscale, q_norm=w_q, k_norm=w_k,
                           k_scale=k_scale, v_scale=v_scale)
        a = nv.paged_attention(q, k_cache, v_cache, table, lengths, k_scale=k_scale, v_scale=v_scale, workspace=workspace)
        o = nv.gemv(*self.wo, a.view(m, -1))
        y, residual, _ = nv.rms_norm(o, w_post, residual=residual)
        return nv.ffn_swiglu(*self.gate, *self.up, *self.down, y, workspace=ffn_workspace), residual


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--seqs", type=int, default=1)
    ap.add_argument("--rows", type=int, default=1)
    ap.add_argument("--context", type=int, default=8191)
    ap.add_argument("--cache", choices=("bf16", "fp8"), default="bf16")
    ap.add_argument("--layers", type=int, default=8)
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args(argv)
    if not 1 <= a.seqs * a.rows <= 8 or a.context < a.rows:
        ap.error("seqs * rows must be 1..8 and the context hold the rows")
    dtype = torch.bfloat16 if a.cache == "bf16" else torch.float8_e4m3fn
    layers = [DecodeLayer(seed=i) for i in range(a.layers)]
    caches = [l.make_cache(a.seqs, a.context + 1, dtype=dtype) for l in layers]
    for k, v, *_ in caches:
        for c in (k, v):
            c.copy_(torch.randn(c.shape, device="cuda").to(dtype))
    l0 = layers[0]
    inv_freq, mscale = nv.rope_frequencies(l0.head_dim, 1e6)
    lengths = torch.full((a.seqs,), a.context, dtype=torch.int32, device="cuda")
    positions = (a.context - a.rows + torch.arange(a.rows, dtype=torch.int32)).repeat(a.seqs).cuda()
    ws = nv.attention_workspace(a.seqs, a.rows, l0.q_heads, l0.kv_heads, l0.head_dim)
    fws = nv.ffn_workspace(a.seqs * a.rows, l0.ffn)
    x0 = torch.randn(a.seqs * a.rows, l0.hidden, device="cuda", dtype=torch.bfloat16)

    def step():
        x, res = x0, None
        for layer, cache in zip(layers, caches):
            x, res = layer.step(x, res, positions, lengths, inv_freq, cache, ws, fws, mscale)
        return x, res

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x, res = step()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(3):
        graph.replay()
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    flags = nv.device_status()
    if flags or not torch.isfinite(x).all():
        raise SystemExit(f"device status {flags}, finite {bool(torch.isfinite(x).all())}")
    print(json.dumps({"us_per_layer": begin.elapsed_time(end) * 1e3 / (a.steps * a.layers), "layers": a.layers, "seqs": a.seqs,
                      "rows": a.rows, "context": a.context, "cache": a.cache}))


if __name__ == "__main__":
    main()
