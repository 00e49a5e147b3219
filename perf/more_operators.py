"""Attention over a paged cache held in 4 bits, and attention with other scores, in plain torch and
through the package.

Three operators of a decode step:

* ``append``: per-head norm and rotary positions of q and k, the append of k and v to a paged NVFP4 cache,
  and the appended rows read back as what the cache stands for;
* ``attend``: attention of the newest 1..8 tokens of each sequence over that cache;
* ``scores``: the same attention, over a cache of any type, with scores that are capped by a tanh, get a
  bias that falls with the distance of a key, or both.

``own`` chooses between the plain forms (elementary torch operations, rounded once at the end) and the
calls a user of the package makes.

The 4-bit cache: 16 keys of a head are a record of 9 D bytes, first their E2M1 codes [16][D / 2] (element
2j in the low nibble of byte j), then a block scale in E4M3 for each 16 elements, [D / 16][16 keys]. An
element stands for code * block scale * the head's scale. A cache is uint8 [pages, kv heads, page, 9 D / 16].
"""
import math
import random

import torch

own = False

E4M3 = torch.float8_e4m3fn
BF16 = torch.bfloat16
DTYPES = {"f32": torch.float32, "bf16": BF16}
#: bytes per value in a cache, in sixteenths
SIXTEENTHS = {"bf16": 32, "fp8": 16, "fp4": 9}
BYTES = {"f32": 4, "bf16": 2}
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # The start of one user's answer: latency, an odd length.
        dict(name="attend_one_short", op="attend", seqs=1, length=257, ragged=False, rows=1, heads=32, kv_heads=8,
             dim=128, cache="fp4", page=16, window=0, cap=0.0, slopes=False),
        # One user with a long context, which is what a cache of 4 bits is for.
        dict(name="attend_one_long", op="attend", seqs=1, length=131071, ragged=False, rows=1, heads=32, kv_heads=8,
             dim=128, cache="fp4", page=64, window=0, cap=0.0, slopes=False),
        # Sixteen users between an empty context and 8191 tokens.
        dict(name="attend_ragged", op="attend", seqs=16, length=8191, ragged=True, rows=1, heads=32, kv_heads=8,
             dim=128, cache="fp4", page=32, window=0, cap=0.0, slopes=False),
        # Verification of three tokens for each of eight users, narrow heads, a sliding window.
        dict(name="attend_drafts", op="attend", seqs=8, length=20011, ragged=True, rows=3, heads=40, kv_heads=8,
             dim=64, cache="fp4", page=16, window=4096, cap=0.0, slopes=False),
        # A full batch, four tokens to verify for each user.
        dict(name="attend_batch", op="attend", seqs=64, length=8191, ragged=False, rows=4, heads=32, kv_heads=8,
             dim=128, cache="fp4", page=64, window=0, cap=0.0, slopes=False),
        # One user of a model that caps its scores, wide heads.
        dict(name="capped_one", op="scores", seqs=1, length=4097, ragged=False, rows=1, heads=16, kv_heads=4,
             dim=256, cache="bf16", page=16, window=0, cap=50.0, slopes=False),
        # Its layers with a sliding window, sixteen users.
        dict(name="capped_windows", op="scores", seqs=16, length=8191, ragged=True, rows=1, heads=32, kv_heads=8,
             dim=128, cache="bf16", page=32, window=4096, cap=50.0, slopes=False),
        # A model whose heads see near keys first, a batch over an 8-bit cache.
        dict(name="distance_batch", op="scores", seqs=32, length=4095, ragged=False, rows=1, heads=32, kv_heads=8,
             dim=128, cache="fp8", page=64, window=0, cap=0.0, slopes=True),
        # Both at once over the 4-bit cache, five drafted tokens for each of seven users, pages of no power of two.
        dict(name="both_drafts", op="scores", seqs=7, length=12001, ragged=True, rows=5, heads=24, kv_heads=8,
             dim=128, cache="fp4", page=48, window=0, cap=30.0, slopes=True),
        # One decoded token at position 32,767: the three projections' fp32 outputs, per-head norm, half layout.
        dict(name="append_one_token", op="append", tokens=1, seqs=1, past=32767, heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=False, norm=True, x="f32", fused=False, page=16),
        # Five drafted tokens for each of seven users: interleaved pairs on half of the head.
        dict(name="append_drafts", op="append", tokens=35, seqs=7, past=4001, heads=24, kv_heads=8, dim=128,
             rotary=64, interleaved=True, norm=False, x="bf16", fused=True, page=32),
        # Three prompts of unequal length at once, from a fused q|k|v projection.
        dict(name="append_prompts", op="append", tokens=8192, seqs=3, past=0, heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=False, norm=True, x="bf16", fused=True, page=64),
    ]


def _log_int(rng, lo, hi):
    return int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "scores", "scores"])
    dim = rng.choice([64, 80, 96, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.randint(1, 8)
    page = rng.choice([16, 32, 48, 64, 128])
    if op == "append":
        tokens = _log_int(rng, 1, max(1, min(8192, 50_000_000 // ((heads + 2 * kv_heads) * dim))))
        return dict(op=op, tokens=tokens, seqs=rng.randint(1, min(16, tokens)), past=_log_int(rng, 1, 20000),
                    heads=heads, kv_heads=kv_heads, dim=dim, rotary=rng.choice([dim, dim // 2]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.5, x=rng.choice(["f32", "bf16"]),
                    fused=rng.random() < 0.5, page=page)
    cache = "fp4" if op == "attend" else rng.choice(["bf16", "fp8", "fp4"])
    cap, slopes = (0.0, False) if op == "attend" else rng.choice([(50.0, False), (0.0, True), (20.0, True)])
    rows = rng.randint(1, 8)
    seqs = _log_int(rng, 1, 64)
    most = 600_000_000 * 16 // (2 * kv_heads * dim * SIXTEENTHS[cache] * seqs)
    # the scores of all rows are held at once by the plain form, several times: 2^28 of them at most
    most = min(most, (1 << 28) // (seqs * heads * rows), 131071)
    return dict(op=op, seqs=seqs, length=_log_int(rng, 1, max(1, most)), ragged=rng.random() < 0.5, rows=rows,
                heads=heads, kv_heads=kv_heads, dim=dim, cache=cache, page=page,
                window=rng.choice([0, 0, _log_int(rng, 16, 8192)]), cap=cap, slopes=slopes)


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


def _records(codes, scales):
    """Codes uint8 [pages, heads, page, D / 2] and block scales E4M3 [pages, heads, page, D / 16] as a cache."""
    p, h, page, half = codes.shape
    codes = codes.reshape(p, h, page // 16, 8 * 2 * half)
    scales = scales.view(torch.uint8).view(p, h, page // 16, 16, half // 8).transpose(3, 4)
    return torch.cat([codes, scales.reshape(p, h, page // 16, 2 * half)], dim=3).view(p, h, page, 9 * half // 8)


def _cache(pages, case, gen, dev):
    shape = (pages, case["kv_heads"], case["page"], case["dim"])
    if case.get("cache", "fp4") == "fp4":
        # what a normal block's values become: the largest at 6, and scales around a sixth of the largest value
        u = torch.empty(*shape[:3], case["dim"] // 2, 2, device=dev).normal_(generator=gen)
        code = ((u.abs() * 2.4).clamp(max=7).to(torch.uint8)) | (u < 0).to(torch.uint8) << 3
        scales = 0.2 + 0.25 * torch.rand((*shape[:3], case["dim"] // 16), generator=gen, device=dev)
        return _records(code[..., 0] | code[..., 1] << 4, scales.to(E4M3))
    x = torch.empty(shape, dtype=BF16, device=dev)
    x.normal_(generator=gen)
    return x if case["cache"] == "bf16" else (x * 8).to(E4M3)


def _kv_scales(case, gen, dev):
    cache = case.get("cache", "fp4")
    if cache == "bf16":
        return None, None
    r = torch.rand((2, case["kv_heads"]), generator=gen, device=dev)
    r = r * 0.1 + 0.08 if cache == "fp8" else 0.7 + 0.6 * r
    return r[0].contiguous(), r[1].contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    s = dict(case=case)
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "append":
        counts, past = _counts(case)
        t, dt = case["tokens"], DTYPES[case["x"]]
        # keys have a few channels far larger than the rest
        gain = 1 + 11 * (torch.rand(d, generator=gen, device=dev) < 0.04).float()
        gain[d // 3] = 12
        q, k, v = randn(t, hq, d), randn(t, hk, d), randn(t, hk, d)
        s["q_norm"] = s["k_norm"] = None
        if case["norm"]:
            s["q_norm"], s["k_norm"] = (1 + 0.2 * randn(d)).to(BF16), ((1 + 0.2 * randn(d)) * gain).to(BF16)
        else:
            k = k * gain
        s["q"], s["k"], s["v"] = q.to(dt), k.to(dt), v.to(dt)
        if case["fused"]:
            qkv = torch.cat([s[n].view(t, -1) for n in "qkv"], dim=1)
            s["q"], s["k"], s["v"] = (x.view(t, -1, d) for x in qkv.split([hq * d, hk * d, hk * d], dim=1))
        s["positions"] = torch.cat([torch.arange(p, p + c, dtype=torch.int32) for c, p in zip(counts, past)]).to(dev)
        s["seq_ids"] = torch.repeat_interleave(torch.arange(len(counts), dtype=torch.int32), torch.tensor(counts)).to(dev)
        half = case["rotary"] // 2
        s["inv_freq"] = (1e6 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)).float()
        s["table"], pages = _pages([c + p for c, p in zip(counts, past)], case["page"], gen, dev)
        s["k_cache"], s["v_cache"] = _cache(pages, case, gen, dev), _cache(pages, case, gen, dev)
        s["k_scale"], s["v_scale"] = _kv_scales(case, gen, dev)
        s["out"] = torch.empty(t, hq, d, dtype=BF16, device=dev)
        s["k_out"], s["v_out"] = (torch.empty(t, hk, d, dtype=BF16, device=dev) for _ in "kv")
        return s
    lengths = _lengths(case)
    random.Random(seed).shuffle(lengths)
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
    s["table"], pages = _pages(lengths, case["page"], gen, dev)
    s["k_cache"], s["v_cache"] = _cache(pages, case, gen, dev), _cache(pages, case, gen, dev)
    s["k_scale"], s["v_scale"] = _kv_scales(case, gen, dev)
    t = case["seqs"] * case["rows"]
    # capped scores reach into the cap's bend
    s["q"] = ((12 if case["cap"] else 2) * randn(t, hq, d)).to(BF16)
    s["scale"] = d ** -0.5
    s["slopes"] = 2.0 ** (-8.0 * torch.arange(1, hq + 1, device=dev) / hq) if case["slopes"] else None
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(t, hq, device=dev)
    # scratch that a decoding program zeroes once and keeps for all its layers and steps
    s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    return s


# ------------------------------------------------------------------------------ plain forms

def _widen(rows, dim):
    """Records uint8 [..., groups of 16 keys, 9 D] -> [..., keys, D] in 32 bits, without the head's scale."""
    byte = rows[..., :8 * dim].int()
    code = torch.stack([byte & 15, byte >> 4], dim=-1).view(*rows.shape[:-1], 16, dim // 16, 16)
    value = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=rows.device)[code]
    scale = rows[..., 8 * dim:].contiguous().view(E4M3).float().view(*rows.shape[:-1], dim // 16, 16).transpose(-1, -2)
    return (value * scale[..., None]).view(*rows.shape[:-2], -1, dim)


def _code(x):
    """E2M1 codes of x, to nearest, ties to the even code, beyond 6 to 6."""
    a = x.abs()
    code = sum((a > b).to(torch.uint8) for b in (0.25, 1.25, 2.5, 5.0)) + sum((a >= b).to(torch.uint8) for b in (0.75, 1.75, 3.5))
    return code | (x < 0).to(torch.uint8) << 3


def _store(cache, page, slot, x, scale):
    """Quantises x [tokens, heads, D] into the tokens' places."""
    d = x.shape[2]
    x = (x / scale[:, None]).unflatten(2, (d // 16, 16))
    block = (x.abs().amax(dim=3) / 6.0).clamp(max=448.0).to(E4M3)
    b = block.float()[..., None]
    code = _code(torch.where(b > 0, x / b, torch.zeros_like(x))).flatten(2)
    rec = cache.view(cache.shape[0], cache.shape[1], -1, 9 * d)
    group, key = slot // 16, slot % 16
    at = torch.arange(d // 2, device=x.device)
    head = torch.arange(x.shape[1], device=x.device)[None, :, None]
    rec[page[:, None, None], head, group[:, None, None], key[:, None, None] * (d // 2) + at] = code[..., 0::2] | code[..., 1::2] << 4
    at = 8 * d + 16 * torch.arange(d // 16, device=x.device)
    rec[page[:, None, None], head, group[:, None, None], at + key[:, None, None]] = block.view(torch.uint8)


def _rows_back(cache, page, slot, dim, scale):
    rec = cache.view(cache.shape[0], cache.shape[1], -1, 9 * dim)[page, :, slot // 16]
    rows = _widen(rec[:, :, None], dim)[torch.arange(len(page), device=page.device), :, slot % 16]
    return (rows * scale[:, None]).to(BF16)


def _rms_heads(x, weight):
    if weight is None:
        return x
    return x / torch.sqrt(x.square().mean(dim=-1, keepdim=True) + 1e-6) * weight.double()


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
    # keys in 64 bits up to their quotients: a code next to a border goes by the last bits
    case, d = s["case"], s["case"]["dim"]
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()
    cos, sin = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    q = _rotate(_rms_heads(s["q"].double(), s["q_norm"]), cos, sin, case)
    k = _rotate(_rms_heads(s["k"].double(), s["k_norm"]), cos, sin, case)
    pos = s["positions"].long()
    page, slot = s["table"][s["seq_ids"].long(), pos // case["page"]].long(), pos % case["page"]
    _store(s["k_cache"], page, slot, k.float(), s["k_scale"])
    _store(s["v_cache"], page, slot, s["v"].float(), s["v_scale"])
    return [q.to(BF16), _rows_back(s["k_cache"], page, slot, d, s["k_scale"]), _rows_back(s["v_cache"], page, slot, d, s["v_scale"])]


def _gather(cache, table, scale, dim):
    """[B, kv heads, keys, D] in 32 bits, pages in the sequences' order."""
    at = table.clamp_min(0).long()
    if cache.dtype == torch.uint8:
        rows = cache[at].transpose(1, 2)
        x = _widen(rows.reshape(*rows.shape[:3], -1, 9 * dim).flatten(2, 3), dim)
    else:
        x = cache.view(torch.uint8)[at].view(E4M3) if cache.dtype == E4M3 else cache[at]
        x = x.transpose(1, 2).flatten(2, 3).float()
    return x if scale is None else x * scale[:, None, None]


def _attend_plain(s):
    case = s["case"]
    b, m, hk, d = case["seqs"], case["rows"], case["kv_heads"], case["dim"]
    g = case["heads"] // hk
    k, v = _gather(s["k_cache"], s["table"], s["k_scale"], d), _gather(s["v_cache"], s["table"], s["v_scale"], d)
    q = s["q"].float().view(b, m, hk, g, d).permute(0, 2, 1, 3, 4).reshape(b, hk, m * g, d)
    key = torch.arange(k.shape[2], device=k.device)
    last = (s["lengths"][:, None] - m + torch.arange(m, device=k.device))[..., None]
    seen = key <= last
    if case["window"]:
        seen = seen & (key > last - case["window"])
    seen = seen[:, None, :, None, :].expand(b, 1, m, g, -1).reshape(b, 1, m * g, -1)
    score = q @ k.transpose(2, 3) * s["scale"]
    if case["cap"]:
        score = case["cap"] * torch.tanh(score / case["cap"])
    if s["slopes"] is not None:
        away = (last - key).float()[:, None, :, None, :]
        score = score - (s["slopes"].view(1, hk, 1, g, 1) * away).reshape(b, hk, m * g, -1)
    score = score.masked_fill(~seen, -math.inf)
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
        return _append_plain(s) if case["op"] == "append" else _attend_plain(s)
    import nvfp4_weight_only_gemv_gb300 as nv
    if case["op"] == "append":
        q = nv.rope_append(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["k_cache"], s["v_cache"],
                           s["table"], s["seq_ids"], interleaved=case["interleaved"], q_norm=s["q_norm"],
                           k_norm=s["k_norm"], eps=1e-6, k_scale=s["k_scale"], v_scale=s["v_scale"], out=s["out"])
        k, v = nv.cache_read(s["positions"], s["k_cache"], s["v_cache"], s["table"], s["seq_ids"], k_scale=s["k_scale"],
                             v_scale=s["v_scale"], k_out=s["k_out"], v_out=s["v_out"])
        return [q, k, v]
    out = nv.paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lengths"], s["scale"],
                             window=case["window"], softcap=case["cap"], slopes=s["slopes"], k_scale=s["k_scale"],
                             v_scale=s["v_scale"], workspace=s["workspace"], out=s["out"], lse=s["lse"])
    return [out, s["lse"]]


# ------------------------------------------------------------------------- 64 bits, and work

def _to_e4m3(x):
    """Non-negative x rounded to E4M3 values in 64 bits, to nearest, ties to even, beyond 448 to 448."""
    step = torch.exp2(torch.floor(torch.log2(x.clamp_min(2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(max=448.0)


def _to_e2m1(x):
    """x rounded to E2M1 values in 64 bits, to nearest, ties to even, beyond 6 to 6."""
    a = x.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.sign(x) * (torch.round(a / step) * step).clamp(max=6.0)


def _exact_rows(x, scale):
    y = (x / scale.double()[:, None]).reshape(*x.shape[:2], -1, 16)
    b = _to_e4m3(y.abs().max(dim=3, keepdim=True).values / 6)
    y = torch.where(b > 0, _to_e2m1(y / b.clamp_min(2.0 ** -9)) * b, 0.0)
    return y.reshape(x.shape) * scale.double()[:, None]


def _exact_heads(x, weight, cos, sin, case):
    x = x.double()
    if weight is not None:
        x = x * torch.rsqrt((x * x).sum(dim=2, keepdim=True) / case["dim"] + 1e-6) * weight.double()
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
    return [q, _exact_rows(k, s["k_scale"]), _exact_rows(s["v"].double(), s["v_scale"])]


def _keys_of(cache, pages, head, n, dim):
    """The first n keys (or values) of a head in 64 bits, out of the pages in order."""
    if cache.dtype != torch.uint8:
        rows = cache.view(torch.uint8)[pages, head].view(E4M3) if cache.dtype == E4M3 else cache[pages, head]
        return rows.double().reshape(-1, dim)[:n]
    rec = cache[pages, head].reshape(-1, 9 * dim)
    code = torch.empty((rec.shape[0], 16, dim), dtype=torch.int64, device=rec.device)
    byte = rec[:, :8 * dim].reshape(-1, 16, dim // 2).long()
    code[..., 0::2], code[..., 1::2] = byte % 16, byte // 16
    e, f = code % 8 // 2, code % 2
    value = torch.where(e > 0, torch.exp2(e.double() - 1) * (1 + f / 2), f / 2) * (1 - 2 * (code // 8)).double()
    scale = rec[:, 8 * dim:].reshape(-1, dim // 16, 16).contiguous().view(E4M3).double().permute(0, 2, 1)
    return (value * scale.repeat_interleave(16, dim=2)).reshape(-1, dim)[:n]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(s)
    m, d, page, g = case["rows"], case["dim"], case["page"], case["heads"] // case["kv_heads"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["lse"].shape, -math.inf, dtype=torch.float64, device=out.device)
    for b, n in enumerate(s["lengths"].tolist()):
        pages = s["table"][b, :-(-n // page)].long()
        for h in range(case["kv_heads"]):
            k, v = (_keys_of(c, pages, h, n, d) for c in (s["k_cache"], s["v_cache"]))
            if s["k_scale"] is not None:
                k, v = k * s["k_scale"][h].double(), v * s["v_scale"][h].double()
            for r in range(m):
                hi = n - m + r + 1
                lo = max(0, hi - case["window"]) if case["window"] else 0
                if hi <= lo:
                    continue
                at = slice(h * g, (h + 1) * g)
                z = s["q"][b * m + r, at].double() @ k[lo:hi].T * s["scale"]
                if case["cap"]:
                    z = torch.tanh(z / case["cap"]) * case["cap"]
                if s["slopes"] is not None:
                    away = torch.arange(hi - lo - 1, -1, -1, device=z.device, dtype=torch.float64)
                    z = z - s["slopes"][at].double()[:, None] * away
                lse[b * m + r, at] = torch.logsumexp(z, dim=1)
                out[b * m + r, at] = torch.softmax(z, dim=1) @ v[lo:hi]
    return [out, lse]


def work(case):
    d, hq, hk = case["dim"], case["heads"], case["kv_heads"]
    if case["op"] == "append":
        t = case["tokens"]
        moved = t * d * (BYTES[case["x"]] * (hq + 2 * hk) + 2 * hq + 2 * hk * 2) + t * hk * 2 * d * 9 // 16
        rotated = t * (hq + hk) * case["rotary"] * 3
        return {"bytes": moved + 8 * t + 2 * case["rotary"], "flops": rotated + (4 * t * (hq + hk) * d if case["norm"] else 0)}
    m, keys, pairs = case["rows"], 0, 0
    for n in _lengths(case):
        w = case["window"] or n
        keys += min(n, w + m - 1)
        pairs += sum(min(max(0, n - m + r + 1), w) for r in range(m))
    rows = case["seqs"] * m * hq
    return {"bytes": keys * hk * d * 2 * SIXTEENTHS[case["cache"]] // 16 + rows * (4 * d + 4), "flops": 4 * d * hq * pairs}
