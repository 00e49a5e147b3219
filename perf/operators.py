"""The decode step's operators around the NVFP4 products, in plain torch and through the package.

Three operators that stand between one projection and the next:

* ``norm``: root-mean-square norm of a row, with the residual's addition and the new residual
  stream, stored in bf16 for the next projection or in E4M3 with scales;
* ``append``: per-head norm and rotary positions of q and k, and the append of k and v to a paged
  cache (bf16, or E4M3 with a scale per key/value head);
* ``attend``: attention of the newest 1..8 tokens of each sequence over that cache.

``own`` chooses between the plain forms (elementary torch operations in 32 bits, rounded once at
the end) and the calls a user of the package makes.
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
BF16 = torch.bfloat16
DTYPES = {"f32": torch.float32, "bf16": BF16, "fp8": E4M3, "none": None}
BYTES = {"f32": 4, "bf16": 2, "fp8": 1, "none": 0}
SCALE_FLOOR = 2.0 ** -64


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # The norm after one token's down projection: fp32 product in, bf16 row out.
        dict(name="norm_one_token", op="norm", rows=1, cols=4096, x="f32", residual="bf16", out="bf16", group=0),
        # Drafted tokens into an 8-bit projection, one scale per token; a width that is no power of two.
        dict(name="norm_drafts_fp8", op="norm", rows=5, cols=2816, x="bf16", residual="bf16", out="fp8", group=0),
        # A prompt's rows between two layers.
        dict(name="norm_prompt", op="norm", rows=8192, cols=4096, x="bf16", residual="bf16", out="bf16", group=0),
        # A prompt of odd length with an fp32 residual stream, quantised per 128 columns.
        dict(name="norm_prompt_fp8", op="norm", rows=4099, cols=4096, x="f32", residual="f32", out="fp8", group=128),
        # One decoded token at position 32,767: the three projections' fp32 outputs, per-head norm, half layout.
        dict(name="append_one_token", op="append", tokens=1, seqs=1, past=32767, heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=False, norm=True, x="f32", fused=False, cache="bf16", page=16),
        # Five drafted tokens for each of seven users: interleaved pairs on half of the head, 8-bit cache.
        dict(name="append_drafts_fp8", op="append", tokens=35, seqs=7, past=4001, heads=24, kv_heads=8, dim=128,
             rotary=64, interleaved=True, norm=False, x="bf16", fused=True, cache="fp8", page=32),
        # Three prompts of unequal length at once, from a fused q|k|v projection.
        dict(name="append_prompts", op="append", tokens=8192, seqs=3, past=0, heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=False, norm=True, x="bf16", fused=True, cache="bf16", page=64),
        # The start of one user's answer: latency, an odd length.
        dict(name="attend_one_short", op="attend", seqs=1, length=257, ragged=False, rows=1, heads=32, kv_heads=8,
             dim=128, cache="bf16", page=16, window=0),
        # One user with a long context: the cache's length has to be split over the whole GPU.
        dict(name="attend_one_long", op="attend", seqs=1, length=131071, ragged=False, rows=1, heads=32, kv_heads=8,
             dim=128, cache="bf16", page=64, window=0),
        # Sixteen users between an empty context and 8191 tokens.
        dict(name="attend_ragged", op="attend", seqs=16, length=8191, ragged=True, rows=1, heads=32, kv_heads=8,
             dim=128, cache="bf16", page=32, window=0),
        # Verification of three tokens for each of eight users, narrow heads, a sliding window.
        dict(name="attend_drafts", op="attend", seqs=8, length=20011, ragged=True, rows=3, heads=40, kv_heads=8,
             dim=64, cache="bf16", page=16, window=4096),
        # A full batch on an 8-bit cache, four tokens to verify for each user.
        dict(name="attend_batch_fp8", op="attend", seqs=64, length=8191, ragged=False, rows=4, heads=32, kv_heads=8,
             dim=128, cache="fp8", page=64, window=0),
    ]


def _log_int(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    op = rng.choice(["norm", "append", "attend", "attend"])
    if op == "norm":
        cols = 16 * rng.choice([_log_int(rng, 16, 191), _log_int(rng, 193, 1024)])
        rows = _log_int(rng, 1, max(1, min(8192, 33_000_000 // cols)))
        out = rng.choice(["bf16", "f32", "fp8"])
        group = rng.choice([0, 128]) if out == "fp8" and cols % 128 == 0 else 0
        return dict(op=op, rows=rows, cols=cols, x=rng.choice(["f32", "bf16"]),
                    residual=rng.choice(["none", "bf16", "f32"]), out=out, group=group)
    cache = rng.choice(["bf16", "fp8"])
    dim = rng.choice([64, 80, 96, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.randint(1, 8)
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "append":
        tokens = _log_int(rng, 1, max(1, min(8192, 50_000_000 // ((heads + 2 * kv_heads) * dim))))
        return dict(op=op, tokens=tokens, seqs=rng.randint(1, min(16, tokens)), past=_log_int(rng, 1, 20000),
                    heads=heads, kv_heads=kv_heads, dim=dim, rotary=rng.choice([dim, dim // 2]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.5, x=rng.choice(["f32", "bf16"]),
                    fused=rng.random() < 0.5, cache=cache, page=page)
    rows = rng.randint(1, 8)
    seqs = _log_int(rng, 1, 64)
    most = 800_000_000 // (2 * kv_heads * dim * BYTES[cache] * seqs)
    # the scores of all rows are held at once by the plain form: 2^29 of them at most
    most = min(most, (1 << 29) // (seqs * heads * rows), 131071)
    return dict(op=op, seqs=seqs, length=_log_int(rng, 1, max(1, most)), ragged=rng.random() < 0.5, rows=rows,
                heads=heads, kv_heads=kv_heads, dim=dim, cache=cache, page=page,
                window=rng.choice([0, 0, _log_int(rng, 16, 8192)]))


# ----------------------------------------------------------------------------------- inputs

def _lengths(case):
    """The sequences' lengths, new tokens included: all alike, or spread from 0 to the case's."""
    n, most = case["seqs"], case["length"]
    if not case["ragged"]:
        return [most] * n
    return [most * i // (n - 1) if n > 1 else most for i in range(n)]


def _counts(case):
    """How many of the tokens each sequence appends, and how many it has before."""
    t, n = case["tokens"], case["seqs"]
    if t % n == 0 and case["past"]:
        return [t // n] * n, [case["past"] + 37 * i for i in range(n)]
    counts = [1 + (t - n) * (i + 1) // (n * (n + 1) // 2) for i in range(n)]
    counts[-1] += t - sum(counts)
    return counts, [case["past"] // (i + 1) for i in range(n)]


def _pages(tokens_of, page, gen, dev):
    """A page table whose pages lie in no order in the pool; -1 where a sequence has no page."""
    need = [-(-n // page) for n in tokens_of]
    total = sum(need)
    order = torch.randperm(total + 3, generator=gen, device=dev).to(torch.int32)
    used = torch.arange(max(1, *need), device=dev) < torch.tensor(need, device=dev)[:, None]
    table = torch.full(used.shape, -1, dtype=torch.int32, device=dev)
    table[used] = order[:total]
    return table, total + 3


def _cache(pages, case, gen, dev):
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    x = torch.empty(shape, dtype=BF16, device=dev)
    x.normal_(generator=gen)
    return x if case["cache"] == "bf16" else (x * 8).to(E4M3)


def _kv_scales(case, gen, dev):
    if case["cache"] != "fp8":
        return None, None
    r = torch.rand((2, case["kv_heads"]), generator=gen, device=dev) * 0.1 + 0.08
    return r[0].contiguous(), r[1].contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = dict(case=case)
    if case["op"] == "norm":
        t, h = case["rows"], case["cols"]
        # hidden states have a few channels far larger than the rest
        gain = 1 + 20 * (torch.rand(h, generator=gen, device=dev) < 0.004).float()
        s["x"] = (randn(t, h) * gain).to(DTYPES[case["x"]])
        s["residual"] = None if case["residual"] == "none" else (randn(t, h) * 3 * gain).to(DTYPES[case["residual"]])
        s["weight"] = (1 + 0.2 * randn(h)).to(BF16)
        s["out"] = torch.empty(t, h, dtype=DTYPES[case["out"]], device=dev)
        s["residual_out"] = None if s["residual"] is None else torch.empty_like(s["residual"])
        s["scales"] = None
        if case["out"] == "fp8":
            s["scales"] = torch.empty(t, h // case["group"] if case["group"] else 1, device=dev)
        return s
    if case["op"] == "append":
        counts, past = _counts(case)
        t, hq, hk, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]
        dt = DTYPES[case["x"]]
        if case["fused"]:
            qkv = randn(t, (hq + 2 * hk) * d).to(dt)
            s["q"], s["k"], s["v"] = (x.view(t, -1, d) for x in qkv.split([hq * d, hk * d, hk * d], dim=1))
        else:
            s["q"], s["k"], s["v"] = (randn(t, n, d).to(dt) for n in (hq, hk, hk))
        s["positions"] = torch.cat([torch.arange(p, p + c, dtype=torch.int32) for c, p in zip(counts, past)]).to(dev)
        s["seq_ids"] = torch.repeat_interleave(torch.arange(len(counts), dtype=torch.int32), torch.tensor(counts)).to(dev)
        half = case["rotary"] // 2
        s["inv_freq"] = (1e6 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)).float()
        s["q_norm"], s["k_norm"] = ((1 + 0.2 * randn(d)).to(BF16) for _ in "qk") if case["norm"] else (None, None)
        s["table"], pages = _pages([c + p for c, p in zip(counts, past)], case["page"], gen, dev)
        s["k_cache"], s["v_cache"] = _cache(pages, case, gen, dev), _cache(pages, case, gen, dev)
        s["k_scale"], s["v_scale"] = _kv_scales(case, gen, dev)
        s["out"] = torch.empty(t, hq, d, dtype=BF16, device=dev)
        return s
    lengths = _lengths(case)
    random.Random(seed).shuffle(lengths)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    s["table"], pages = _pages(lengths, case["page"], gen, dev)
    s["k_cache"], s["v_cache"] = _cache(pages, case, gen, dev), _cache(pages, case, gen, dev)
    s["k_scale"], s["v_scale"] = _kv_scales(case, gen, dev)
    t = case["seqs"] * case["rows"]
    s["q"] = (2 * randn(t, case["heads"], case["dim"])).to(BF16)
    s["scale"] = case["dim"] ** -0.5
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(t, case["heads"], device=dev)
    # scratch that a decoding program zeroes once and keeps for all its layers and steps
    s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------------------ plain forms

def _e4m3(x):
    return x.clamp(-448.0, 448.0).to(E4M3)


def _norm_plain(s):
    case, h = s["case"], s["x"].float()
    res = None
    if s["residual"] is not None:
        h = h + s["residual"].float()
        res = h.to(s["residual"].dtype)
    y = h * torch.rsqrt(h.square().mean(dim=-1, keepdim=True) + 1e-6) * s["weight"].float()
    if case["out"] != "fp8":
        return [y.to(DTYPES[case["out"]]), res, None]
    g = y.view(y.shape[0], -1, case["group"] or y.shape[1])
    scales = (g.abs().amax(dim=-1) / 448.0).clamp_min(SCALE_FLOOR)
    return [_e4m3(g / scales[..., None]).view(y.shape), res, scales]


def _rms_heads(x, weight):
    if weight is None:
        return x
    return x * torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + 1e-6) * weight.float()


def _rotate(x, cos, sin, case):
    r = case["rotary"]
    rot, rest = x[..., :r], x[..., r:]
    if case["interleaved"]:
        a, b = rot[..., 0::2], rot[..., 1::2]
        out = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = rot[..., :r // 2], rot[..., r // 2:]
        out = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([out, rest], dim=-1)


def _append_plain(s):
    case = s["case"]
    angle = s["positions"].float()[:, None] * s["inv_freq"]
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    q = _rotate(_rms_heads(s["q"].float(), s["q_norm"]), cos, sin, case)
    k = _rotate(_rms_heads(s["k"].float(), s["k_norm"]), cos, sin, case)
    v = s["v"].float()
    pos = s["positions"].long()
    page, slot = s["table"][s["seq_ids"].long(), pos // case["page"]].long(), pos % case["page"]
    if case["cache"] == "fp8":
        k, v = _e4m3(k / s["k_scale"][:, None]).view(torch.uint8), _e4m3(v / s["v_scale"][:, None]).view(torch.uint8)
        s["k_cache"].view(torch.uint8)[page, :, slot] = k
        s["v_cache"].view(torch.uint8)[page, :, slot] = v
    else:
        s["k_cache"][page, :, slot] = k.to(BF16)
        s["v_cache"][page, :, slot] = v.to(BF16)
    return [q.to(BF16), s["k_cache"], s["v_cache"]]


def _gather(cache, table, scale):
    """[B, kv heads, keys, D] in 32 bits, pages in the sequences' order."""
    at = table.clamp_min(0).long()
    x = cache.view(torch.uint8)[at].view(E4M3) if cache.dtype == E4M3 else cache[at]
    x = x.transpose(1, 2).flatten(2, 3).float()
    return x if scale is None else x * scale[:, None, None]


def _attend_plain(s):
    case = s["case"]
    b, m, hk, d = case["seqs"], case["rows"], case["kv_heads"], case["dim"]
    g = case["heads"] // hk
    k, v = _gather(s["k_cache"], s["table"], s["k_scale"]), _gather(s["v_cache"], s["table"], s["v_scale"])
    q = s["q"].float().view(b, m, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, m * g, d)
    key = torch.arange(k.shape[2], device=k.device)
    last = (s["lengths"][:, None] - m + torch.arange(m, device=k.device))[..., None]
    seen = key <= last
    if case["window"]:
        seen = seen & (key > last - case["window"])
    seen = seen[:, None, :, None, :].expand(b, 1, m, g, -1).reshape(b, 1, m * g, -1)
    score = (q @ k.transpose(2, 3) * s["scale"]).masked_fill(~seen, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(dim=-1, keepdim=True)
    out = torch.where(total > 0, (p @ v) / total, torch.zeros_like(total))
    lse = top + torch.log(total)
    back = (b, hk, m, g)
    out = out.view(*back, d).permute(0, 2, 1, 3, 4).reshape(b * m, hk * g, d)
    return [out.to(BF16), lse.view(back).permute(0, 2, 1, 3).reshape(b * m, hk * g)]


def run(s):
    case = s["case"]
    if not own:
        return {"norm": _norm_plain, "append": _append_plain, "attend": _attend_plain}[case["op"]](s)
    import nvfp4_weight_only_gemv_gb300 as nv
    if case["op"] == "norm":
        return nv.rms_norm(s["x"], s["weight"], 1e-6, residual=s["residual"], residual_out=s["residual_out"],
                           out=s["out"], scales=s["scales"], group=case["group"])
    if case["op"] == "append":
        q = nv.rope_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["k_cache"], s["v_cache"],
                           s["table"], s["seq_ids"], interleaved=case["interleaved"], q_norm=s["q_norm"],
                           k_norm=s["k_norm"], eps=1e-6, k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
        return [q, s["k_cache"], s["v_cache"]]
    out = nv.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["scale"],
                             window=case["window"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                             workspace=s["workspace"], out=s["out"], lse=s["lse"])
    return [out, s["lse"]]


# ------------------------------------------------------------------------- 64 bits, and work

def _exact_norm(s):
    case = s["case"]
    h = s["x"].double()
    if s["residual"] is not None:
        h = h + s["residual"].double()
    mean = (h * h).sum(dim=1) / case["cols"]
    y = h / torch.sqrt(mean + 1e-6)[:, None] * s["weight"].double()
    res = h if s["residual"] is not None else None
    if case["out"] != "fp8":
        return [y, res, None]
    parts = y.reshape(case["rows"], -1, case["group"] or case["cols"])
    scales = parts.abs().max(dim=2).values / 448.0
    return [(parts / scales.unsqueeze(2)).reshape(y.shape), res, scales]


def _exact_heads(x, weight, cos, sin, case):
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(dim=2, keepdim=True) + 1e-6) * weight.double()
    r = case["rotary"]
    i = torch.arange(r // 2, device=x.device)
    a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
    y = x.clone()
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., a] * sin + x[..., b] * cos
    return y


def _exact_append(s):
    case = s["case"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle), torch.sin(angle)
    q = _exact_heads(s["q"], s["q_norm"], cos, sin, case)
    k = _exact_heads(s["k"], s["k_norm"], cos, sin, case)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    p = s["positions"].long()
    at = s["table"][s["seq_ids"].long(), torch.div(p, case["page"], rounding_mode="floor")].long()
    ks, vs = (1.0 if x is None else x.double()[:, None] for x in (s["k_scale"], s["v_scale"]))
    kc[at, :, p % case["page"]] = k / ks
    vc[at, :, p % case["page"]] = s["v"].double() / vs
    return [q, kc, vc]


def _pages_of(cache, pages, head):
    return cache.view(torch.uint8)[pages, head].view(E4M3) if cache.dtype == E4M3 else cache[pages, head]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "append":
        return _exact_append(s)
    m, d, page, g = case["rows"], case["dim"], case["page"], case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=out.device)
    for b, n in enumerate(s["lengths"].tolist()):
        pages = s["table"][b, :-(-n // page)].long()
        for h in range(case["kv_heads"]):
            k, v = (_pages_of(c, pages, h).double().reshape(-1, d)[:n] for c in (s["k_cache"], s["v_cache"]))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for r in range(m):
                hi = n - m + r + 1
                lo = max(0, hi - case["window"]) if case["window"] else 0
                if hi > lo:
                    z = s["q"][b * m + r, h * g:(h + 1) * g].double() @ k[lo:hi].T * s["scale"]
                    lse[b * m + r, h * g:(h + 1) * g] = torch.logsumexp(z, dim=1)
                    out[b * m + r, h * g:(h + 1) * g] = torch.softmax(z, dim=1) @ v[lo:hi]
    return [out, lse]


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * case["cols"]
        per = BYTES[case["x"]] + 2 * BYTES[case["residual"]] + BYTES[case["out"]]
        scales = case["rows"] * (case["cols"] // (case["group"] or case["cols"])) * 4 if case["out"] == "fp8" else 0
        return {"bytes": n * per + 2 * case["cols"] + scales, "flops": 5 * n}
    d, hq, hk = case["dim"], case["heads"], case["kv_heads"]
    if case["op"] == "append":
        t = case["tokens"]
        moved = t * d * (BYTES[case["x"]] * (hq + 2 * hk) + 2 * hq + 2 * hk * BYTES[case["cache"]])
        rotated = t * (hq + hk) * case["rotary"] * 3
        return {"bytes": moved + 8 * t + 2 * case["rotary"], "flops": rotated + (4 * t * (hq + hk) * d if case["norm"] else 0)}
    m, keys, pairs = case["rows"], 0, 0
    for n in _lengths(case):
        w = case["window"] or n
        keys += min(n, w + m - 1)
        pairs += sum(min(max(0, n - m + r + 1), w) for r in range(m))
    rows = case["seqs"] * m * hq
    return {"bytes": keys * hk * d * 2 * BYTES[case["cache"]] + rows * (4 * d + 4), "flops": 4 * d * hq * pairs}
