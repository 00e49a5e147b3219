"""The 4-bit cache: append, rows read back, and attention over it, against plain implementations.

Tolerances come from the arithmetic, before any run, with the units of test_gpu_decode_ops. An E2M1 code is off by
at most half a step of the quotient's binade (0.25 below 2, 0.5 below 4, 1 up to 6), an E4M3 block scale by 2^-4 of
itself, or 2^-10 below 2^-6.
"""
import math

import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv
from test_gpu_decode_ops import BF16, DEV, F32, FP8, U16, U32, U8, _gen, _heads_ref, _randn, _table, _turn_ref, _within

pytestmark = pytest.mark.gpu
FP4 = torch.uint8
CODES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64)


def _split(cache):
    """(code values [pages, heads, page, D], block scales [pages, heads, page, D / 16]) of a 4-bit cache, 64 bits."""
    p, h, page, n = cache.shape
    d = n // 9 * 16
    rec = cache.reshape(p, h, page // 16, 9 * d)
    byte = rec[..., :8 * d].reshape(p, h, page, d // 2).long()
    codes = CODES.to(cache.device)[torch.stack([byte & 15, byte >> 4], dim=-1)].flatten(3)
    scales = rec[..., 8 * d:].reshape(p, h, page // 16, d // 16, 16).transpose(3, 4).reshape(p, h, page, d // 16)
    return codes, scales.contiguous().view(FP8).double()


def _values(cache):
    """What any cache holds, without the heads' scales, in 64 bits."""
    if cache.dtype is not FP4:
        return cache.double()
    codes, scales = _split(cache)
    return codes * scales.repeat_interleave(16, dim=3)


def _fill(cache, gen, used=None, spread=1.0):
    """Random codes and block scales; a NaN scale for keys that `used` [pages, page] leaves out."""
    p, h, page, n = cache.shape
    d = n // 9 * 16
    byte = torch.randint(256, (p, h, page // 16, 8 * d), generator=gen, device=DEV, dtype=torch.uint8)
    s = (spread * (0.1 + 0.4 * torch.rand((p, h, page, d // 16), generator=gen, device=DEV))).to(FP8)
    s = torch.where(torch.rand(s.shape, generator=gen, device=DEV) < 0.1, -s.float(), s.float()).to(FP8)
    if used is not None:
        s = torch.where(used[:, None, :, None], s.float(), math.nan).to(FP8)
    s = s.view(torch.uint8).reshape(p, h, page // 16, 16, d // 16).transpose(3, 4).reshape(p, h, page // 16, d)
    cache.copy_(torch.cat([byte, s], dim=3).reshape(cache.shape))


# ------------------------------------------------------------------------------------ append

def _e2m1(q):
    """Codes of fp32 quotients, to nearest, ties to the even code, beyond 6 to 6 (no NaN)."""
    a = q.abs()
    code = sum((a > b).to(torch.uint8) for b in (0.25, 1.25, 2.5, 5.0)) + sum((a >= b).to(torch.uint8) for b in (0.75, 1.75, 3.5))
    return code | torch.signbit(q).to(torch.uint8) << 3


def _records_of(x, scale):
    """Codes [T, heads, D] and block scale bytes [T, heads, D / 16] that appending fp32 x means."""
    t = (x.float() / scale[:, None]).unflatten(2, (-1, 16))
    b = (t.abs().amax(dim=3) / 6.0).clamp(max=448.0).to(FP8)
    w = b.float()[..., None]
    return _e2m1(torch.where(w > 0, t / w, t.abs() * 0)).flatten(2), b.view(torch.uint8)


def _bytes_at(cache, page, slot):
    """The codes and scale bytes of one key of every head."""
    d = cache.shape[3] // 9 * 16
    rec = cache[page].reshape(cache.shape[1], -1, 9 * d)[:, slot // 16]
    byte = rec[:, :8 * d].reshape(-1, 16, d // 2)[:, slot % 16]
    return torch.stack([byte & 15, byte >> 4], dim=-1).flatten(1), rec[:, 8 * d:].reshape(-1, d // 16, 16)[:, :, slot % 16]


def _check_append(T, hq, hk, D, half, interleaved, xt, fused, page, norm, positions, seqs, seq_ids=None, offset=0, scaled=True):
    g = _gen(T * 7919 + D + half + page)
    if fused:
        w = (hq + 2 * hk) * D
        qkv = _randn((T, w + offset), g, xt)[:, offset:]
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([hq * D, hk * D, hk * D], dim=1))
    else:
        q, k, v = (_randn((T, n, D), g, xt) for n in (hq, hk, hk))
    inv_freq = (1e4 ** (-torch.arange(half, device=DEV).double() / max(half, 1))).float()
    pos = torch.tensor(positions, dtype=torch.int32, device=DEV)
    sid = None if seq_ids is None else torch.tensor(seq_ids, dtype=torch.int32, device=DEV)
    owner = seq_ids if seq_ids is not None else [t // (T // seqs) for t in range(T)]
    need = [max([p // page + 1 for p, o in zip(positions, owner) if o == b and p >= 0], default=0) for b in range(seqs)]
    table, pages = _table(need, g)
    kc, vc = nv.kv_cache(pages, hk, page, D, FP4)
    kc.fill_(0xa5)
    vc.fill_(0xa5)
    qn, kn = ((1 + 0.2 * _randn((D,), g)).to(BF16 if D % 64 else F32) for _ in "qk") if norm else (None, None)
    ks, vs = (0.5 + torch.rand(hk, generator=g, device=DEV) for _ in "kv") if scaled else (None, None)
    got = nv.rope_append(q, k, v, pos, inv_freq, kc, vc, table, sid, interleaved=interleaved, q_norm=qn, k_norm=kn,
                         eps=1e-6, k_scale=ks, v_scale=vs)
    assert nv.device_status() == 0
    one = torch.ones(hk, device=DEV)
    ks, vs = (one if s is None else s for s in (ks, vs))
    live, at = pos >= 0, pos.clamp_min(0)
    uq, uk = _heads_ref(q, qn, 1e-6), _heads_ref(k, kn, 1e-6)
    q_ref, q_size = _turn_ref(uq, at, inv_freq, interleaved, 1.0)
    k_ref, k_size = _turn_ref(uk, at, inv_freq, interleaved, 1.0)
    rel = 24 * U32  # as in the bf16 append's test
    _within(got, q_ref * live[:, None, None], q_size * rel + q_ref.abs() * U16 + 2.0 ** -133, "q")
    v_codes, v_blocks = _records_of(v, vs)
    k_codes, k_blocks = _split(kc)
    touched = torch.zeros((pages, page), dtype=torch.bool, device=DEV)
    for t in range(T):
        if positions[t] < 0:
            continue
        p, s = int(table[owner[t], positions[t] // page]), positions[t] % page
        touched[p, s] = True
        # values: the very bytes
        c, b = _bytes_at(vc, p, s)
        assert torch.equal(b, v_blocks[t]) and torch.equal(c, v_codes[t]), t
        # keys, whose last bits come out of the rotation: each block's scale and, by it, each code
        ref = (k_ref[t] / ks.double()[:, None]).unflatten(1, (-1, 16))
        off = (k_size[t] / ks.double()[:, None]).unflatten(1, (-1, 16)) * (rel + 2 * U32)
        b, top = k_blocks[p, :, s], ref.abs().amax(dim=2) / 6
        _within(b, top, top * U8 + 2.0 ** -10 + off.amax(dim=2), "block scales")
        back, quotient = k_codes[p, :, s].unflatten(1, (-1, 16)) * b[..., None], ref.abs() / b[..., None]
        step = torch.where(quotient <= 2, 0.25, torch.where(quotient <= 4, 0.5, torch.where(quotient <= 6, 1.0, quotient - 6)))
        _within(back, ref, step * b[..., None] + 2 * off, "codes")
    idle = ~touched[:, None, :].expand(-1, hk, -1)
    for c in (kc, vc):
        rec = c.reshape(pages, hk, page // 16, 9 * D)
        byte = rec[..., :8 * D].reshape(pages, hk, page, -1)
        scale = rec[..., 8 * D:].reshape(pages, hk, page // 16, -1, 16).transpose(3, 4).reshape(pages, hk, page, -1)
        assert bool((byte[idle] == 0xa5).all()) and bool((scale[idle] == 0xa5).all()), "wrote elsewhere"


@pytest.mark.parametrize("D,half,interleaved", [(128, 64, False), (128, 64, True), (128, 32, False), (128, 32, True),
                                                (64, 32, False), (96, 48, True), (96, 48, False), (80, 40, False),
                                                (256, 64, False), (128, 0, False), (48, 20, False), (48, 3, True),
                                                (16, 8, False), (512, 256, False), (112, 56, True), (144, 16, False),
                                                (112, 56, False), (80, 24, False), (144, 72, False), (48, 8, False), (80, 40, True),
                                                (80, 20, False), (80, 20, True), (256, 60, False), (16, 4, False), (64, 28, True)])
@pytest.mark.parametrize("xt,fused,norm", [(F32, False, True), (BF16, True, False), (BF16, True, True)])
def test_append(D, half, interleaved, xt, fused, norm):
    _check_append(6, 5, 2, D, half, interleaved, xt, fused, 16, norm, [0, 1, 2, 15, 16, 40], 2, scaled=not norm)


@pytest.mark.parametrize("page", [16, 48, 128])
@pytest.mark.parametrize("T", [1, 13, 97])
def test_append_ragged(page, T):
    lens = [3 * T // 4, 0, T - 3 * T // 4]
    sid = [b for b, n in enumerate(lens) for _ in range(n)]
    pos = [p + 5 * b for b, n in enumerate(lens) for p in range(n)]
    if T > 5:
        pos[2] = -1  # padding
    _check_append(T, 8, 4, 128, 64, False, BF16, True, page, True, pos, 3, sid)


@pytest.mark.parametrize("offset", [1, 4])
def test_append_odd_strides(offset):
    _check_append(4, 3, 1, 64, 32, False, BF16, True, 16, False, [70000, 3, 900, 65535], 2, offset=offset)


@pytest.mark.parametrize("variant", [0, 1])
@pytest.mark.parametrize("xt", [F32, BF16])
def test_appended_bytes_are_the_quotients(variant, xt):
    # values at and beside the middles of two codes, blocks whose scale is a tie, vanishes or is beyond 448, and
    # the types' extremes
    g = _gen(78)
    T, hk, D = 64, 16, 128
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0], device=DEV)
    x = mid[torch.randint(len(mid), (T, hk, D), generator=g, device=DEV)]
    x = x * (1 + torch.randint(-1, 2, x.shape, generator=g, device=DEV) * 2.0 ** -20)
    x = x * torch.where(torch.rand(x.shape, generator=g, device=DEV) < 0.5, -1.0, 1.0)
    x[..., ::16] = 6.0
    e = torch.randint(-12, 11, (T, hk, D // 16), generator=g, device=DEV).float()
    x = x * torch.exp2(e).repeat_interleave(16, dim=2) * (1 + torch.randint(0, 17, e.shape, generator=g, device=DEV) / 16).repeat_interleave(16, dim=2)
    x[0], x[1], x[2, :, ::3], x[3, :, 5], x[4] = 0.0, 1e-30, 3e38, math.inf, 2.0 ** -9 * 6 * 0.5
    x = x.to(xt)
    scale = torch.rand(hk, generator=g, device=DEV) + 0.5
    scale[::2] = 1.0
    scale[3], scale[7], scale[11] = 2.0 ** -126, 2.0 ** -140, 2.0 ** 120
    kc, vc = nv.kv_cache(4, hk, 16, D, FP4)
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    nv.set_variant(variant)
    try:
        nv.rope_append(None, x, -x, pos, torch.empty(0, device=DEV), kc, vc, table, k_scale=scale, v_scale=scale)
    finally:
        nv.set_variant(0)
    for c, ref in ((kc, x), (vc, -x)):
        codes, blocks = _records_of(ref, scale)
        for t in range(T):
            gc, gb = _bytes_at(c, t // 16, t % 16)
            assert torch.equal(gb, blocks[t]), t
            assert torch.equal(gc, codes[t]), t
    assert nv.device_status() == 0


@pytest.mark.parametrize("variant", [0, 1])
def test_a_nan_makes_its_block_nan(variant):
    k = torch.ones((1, 2, 64), device=DEV)
    k[0, 1, 20] = math.nan
    kc, vc = nv.kv_cache(1, 2, 16, 64, FP4)
    zero = torch.zeros(1, dtype=torch.int32, device=DEV)
    nv.set_variant(variant)
    try:
        nv.rope_append(None, k, k, zero, torch.empty(0, device=DEV), kc, vc, zero[None])
    finally:
        nv.set_variant(0)
    for got in nv.cache_read(zero, kc, vc, zero[None]):
        bad = torch.isnan(got[0].float())
        assert bool(bad[1, 16:32].all()) and int(bad.sum()) == 16
        # a block of ones: 1/6 lies nearest to the E4M3 value 0.171875, 1 / 0.171875 = 5.82 nearest to 6
        assert bool((got[0, 0] == 6 * 0.171875).all())


# -------------------------------------------------------------------------------- rows read back

@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
@pytest.mark.parametrize("D,page", [(128, 16), (64, 48), (80, 32), (16, 16), (256, 128), (1024, 16)])
@pytest.mark.parametrize("T", [1, 6, 300])
def test_cache_read(cache, D, page, T):
    g = _gen(D + page + T)
    hk, seqs, pages = 3, 4, 9
    kc, vc = nv.kv_cache(pages, hk, page, D, cache)
    for c in (kc, vc):
        if cache is FP4:
            _fill(c, g, spread=900.0)
        else:
            c.copy_(_randn(c.shape, g).to(cache))
    table = torch.randint(pages, (seqs, 2), generator=g, device=DEV).int()
    pos = torch.randint(-2, 2 * page, (T,), generator=g, device=DEV).int()
    sid = torch.randint(seqs, (T,), generator=g, device=DEV).int()
    ks, vs = (None, None) if cache is BF16 else (0.5 + torch.rand(hk, generator=g, device=DEV) for _ in "kv")
    for variant in (0, 1):
        nv.set_variant(variant)
        try:
            got = nv.cache_read(pos, kc, vc, table, sid, k_scale=ks, v_scale=vs)
        finally:
            nv.set_variant(0)
        assert nv.device_status() == 0
        at = pos.clamp_min(0).long()
        page_of = table[sid.long(), at // page].long()
        for x, c, s in zip(got, (kc, vc), (ks, vs)):
            want = _values(c)[page_of, :, at % page].float()
            if s is not None:
                want = want * s[:, None]
            want = torch.where(pos[:, None, None] < 0, torch.zeros_like(want), want).to(BF16)
            assert torch.equal(x, want)
    # in the sequences' order, into given tensors, on another stream
    if T % seqs == 0:
        side, outs = torch.cuda.Stream(), [torch.full((T, hk, D), math.nan, dtype=BF16, device=DEV) for _ in "kv"]
        torch.cuda.synchronize()
        order = torch.arange(seqs, device=DEV).repeat_interleave(T // seqs).int()
        back = nv.cache_read(pos, kc, vc, table, k_scale=ks, v_scale=vs, k_out=outs[0], v_out=outs[1], stream=side)
        side.synchronize()
        assert back[0] is outs[0] and back[1] is outs[1]
        for a, b in zip(outs, nv.cache_read(pos, kc, vc, table, order, k_scale=ks, v_scale=vs)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
@pytest.mark.parametrize("offset", [1, 8, 16])
def test_cache_read_into_outputs_on_any_boundary(cache, offset):
    g = _gen(offset)
    T, hk, D, page = 5, 2, 64, 16
    kc, vc = nv.kv_cache(3, hk, page, D, cache)
    for c in (kc, vc):
        _fill(c, g) if cache is FP4 else c.copy_(_randn(c.shape, g).to(cache))
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    pos = torch.tensor([40, 3, -1, 17, 0], dtype=torch.int32, device=DEV)
    want = nv.cache_read(pos, kc, vc, table)
    mem = [torch.full((T * hk * D + 64,), math.nan, dtype=BF16, device=DEV) for _ in "kv"]
    outs = [m[offset:offset + T * hk * D].view(T, hk, D) for m in mem]
    nv.cache_read(pos, kc, vc, table, k_out=outs[0], v_out=outs[1])
    for m, o, w in zip(mem, outs, want):
        assert torch.equal(o, w) and bool(torch.isnan(m[:offset]).all()) and bool(torch.isnan(m[offset + T * hk * D:]).all())


@pytest.mark.parametrize("cache", [BF16, FP8])
def test_cache_read_of_odd_heads_and_pages(cache):
    g = _gen(3)
    kc, vc = nv.kv_cache(4, 2, 7, 33, cache)
    for c in (kc, vc):
        c.copy_(_randn(c.shape, g).to(cache))
    table = torch.tensor([[3, 1]], dtype=torch.int32, device=DEV)
    pos = torch.arange(14, dtype=torch.int32, device=DEV)
    for x, c in zip(nv.cache_read(pos, kc, vc, table), (kc, vc)):
        assert torch.equal(x, c[table[0].long()].transpose(1, 2).reshape(14, 2, 33).to(BF16))


@pytest.mark.parametrize("cache", [BF16, FP8, FP4])
def test_cache_read_of_no_place_sets_the_status_and_gives_zeros(cache):
    kc, vc = nv.kv_cache(3, 2, 16, 64, cache)
    for c in (kc, vc):
        c.view(torch.uint8).fill_(0x38)
    table = torch.tensor([[0, 1], [2, 7]], dtype=torch.int32, device=DEV)
    pos = torch.tensor([32, 0, 16, 3, 5], dtype=torch.int32, device=DEV)  # past the table; good; bad page; bad seqs
    sid = torch.tensor([0, 0, 1, 2, -1], dtype=torch.int32, device=DEV)
    k, v = nv.cache_read(pos, kc, vc, table, sid)
    assert nv.device_status() == nv.DEV_BAD_PAGE and nv.device_status() == 0
    for x in (k, v):
        # (0x38 as codes is -0 and 1.5: no bit pattern of zero either)
        assert bool(x[1].view(torch.int16).ne(0).all()) and not x[[0, 2, 3, 4]].view(torch.int16).any()
    empty = nv.kv_cache(0, 2, 16, 64, cache)
    k, v = nv.cache_read(pos[:2], *empty, table[:1, :0])
    assert not k.any() and not v.any() and nv.device_status() == nv.DEV_BAD_PAGE
    assert nv.cache_read(pos[:0], kc, vc, table)[0].shape == (0, 2, 64)


# ----------------------------------------------------------------------------------- attention

def _ref(q, kd, vd, table, lengths, rows, scale, window, ks, vs, p_err, cap=0.0, slopes=None):
    """out, its tolerance, lse and its tolerance in 64 bits, row by row, from values kd, vd [pages, heads, page, D]."""
    T, hq, D = q.shape
    hk, page = kd.shape[1], kd.shape[2]
    g = hq // hk
    out = torch.zeros((T, hq, D), dtype=torch.float64, device=DEV)
    tol = torch.full_like(out, 2.0 ** -133)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=DEV)
    ltol = torch.zeros_like(lse)
    for b, n in enumerate(lengths):
        pages = table[b, :-(-n // page)].long()
        for h in range(hk):
            keys, vals = (c[pages, h].reshape(-1, D)[:n] for c in (kd, vd))
            if ks is not None:
                keys, vals = keys * ks[h].double(), vals * vs[h].double()
            for r in range(rows):
                hi = n - rows + r + 1
                lo = max(0, hi - window) if window else 0
                if hi <= lo:
                    continue
                t, hs, m = b * rows + r, slice(h * g, (h + 1) * g), hi - lo
                qq, kk, vv = q[t, hs].double(), keys[lo:hi], vals[lo:hi]
                z = qq @ kk.T * scale
                # fp32 dot products of D terms and the scaling; q in f16 next to its maximum
                dz = ((D + 8) * U32 * (qq.abs() @ kk.abs().T) * abs(scale) + 4 * U32 * z.abs()
                      + 2.0 ** -24 * qq.abs().amax(dim=1, keepdim=True) * kk.abs().sum(dim=1) * abs(scale))
                if cap:
                    # the quotient by the cap (3 roundings of an argument under a tanh: x / cosh(x)^2 < 0.45), the
                    # tanh itself (2 units of 1), the product back
                    z = cap * torch.tanh(z / cap)
                    dz = dz + cap * 0.45 * 4 * U32 + cap * 4 * U32
                if slopes is not None:
                    bias = slopes[hs].double()[:, None] * torch.arange(lo - hi + 1, 1, device=DEV)
                    z = z + bias
                    dz = dz + 2 * U32 * bias.abs()  # the slope in base-2 units, and the sum below
                dz = dz + 4 * U32 * z.abs()
                # the exponent's own sum is as exact as the largest term in it
                dz = dz + 2 * U32 * z.amax(dim=1, keepdim=True).abs()
                p = torch.softmax(z, dim=1)
                mean = (p * dz).sum(dim=1, keepdim=True)
                lse[t, hs] = torch.logsumexp(z, dim=1)
                ltol[t, hs] = mean.squeeze(1) + (8 + m) * U32 + lse[t, hs].abs() * 4 * U32
                out[t, hs] = p @ vv
                size = p @ vv.abs()
                tol[t, hs] += (p * dz) @ vv.abs() + size * (mean + p_err + (m + 16) * U32) + out[t, hs].abs() * U16
                if p_err > 2.0 ** -12:
                    tol[t, hs] += 2.0 ** -32 * p.amax(dim=1, keepdim=True) * vv.abs().sum(dim=0)
    return out, tol, lse, ltol


P_ERR = {BF16: 2.0 ** -15, FP8: 2.0 ** -11, FP4: 2.0 ** -11}


def _inputs(lengths, rows, hq, hk, D, cache, page, seed, max_pages=0):
    """Random caches; what lies past a sequence's end, and every page of nobody, is NaN."""
    g = _gen(seed)
    need = [-(-n // page) for n in lengths]
    table, pages = _table(need, g)
    if max_pages > table.shape[1]:
        table = torch.nn.functional.pad(table, (0, max_pages - table.shape[1]), value=-1)
    kc, vc = nv.kv_cache(pages, hk, page, D, cache)
    used = torch.zeros((pages, page), dtype=torch.bool, device=DEV)
    for b, n in enumerate(lengths):
        for i in range(need[b]):
            used[int(table[b, i]), :min(page, n - i * page)] = True
    for c in (kc, vc):
        if cache is FP4:
            _fill(c, g, used)
        else:
            x = _randn(c.shape, g) * (16 if cache is FP8 else 1)
            x[~used[:, None, :].expand(-1, hk, -1)] = math.nan
            c.copy_(x.to(cache))
    lo, more = (0.04, 0.05) if cache is FP8 else (0.5, 1.0)
    ks, vs = (None, None) if cache is BF16 else (lo + more * torch.rand(hk, generator=g, device=DEV) for _ in "kv")
    q = (2 * _randn((len(lengths) * rows, hq, D), g)).to(BF16)
    return q, kc, vc, table, torch.tensor(lengths, dtype=torch.int32, device=DEV), ks, vs


def _check(lengths, rows, hq, hk, D, page, window=0, scale=None, seed=0, cache=FP4, cap=0.0, slopes=None, q_gain=1.0, max_pages=0):
    q, kc, vc, table, ln, ks, vs = _inputs(lengths, rows, hq, hk, D, cache, page, seed, max_pages)
    q = (q.float() * q_gain).to(BF16)
    kw = dict(window=window, softcap=cap, slopes=slopes, k_scale=ks, v_scale=vs)
    kw["workspace"] = nv.attention_workspace(len(lengths), rows, hq, hk, D)
    got = [(torch.full_like(q, math.nan), torch.full((q.shape[0], hq), math.nan, device=DEV)) for _ in range(2)]
    for out, lse in got:
        nv.paged_attention(q, kc, vc, table, ln, scale, out=out, lse=lse, **kw)
    assert nv.device_status() == 0
    ref, tol, lref, ltol = _ref(q, _values(kc), _values(vc), table, lengths, rows, D ** -0.5 if scale is None else scale,
                                window, ks, vs, P_ERR[cache], cap, slopes)
    _within(got[0][0], ref, tol, "out")
    _within(got[0][1], lref, ltol, "lse")
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1]), "the same call twice differs"


@pytest.mark.parametrize("D", [64, 128, 256, 80, 96, 16, 48, 192, 512])
@pytest.mark.parametrize("rows,hq,hk", [(1, 8, 8), (1, 32, 8), (3, 10, 2), (5, 8, 1), (8, 16, 2), (2, 7, 7)])
def test_attention(D, rows, hq, hk):
    _check([37, 0, 1, 300, 16, 2], rows, hq, hk, D, 16, seed=D + rows)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 257, 1000, 4099])
def test_attention_lengths(n):
    _check([n], 1, 8, 2, 128, 32, seed=n)
    _check([n, n // 2], 4, 4, 1, 64, 16, seed=n + 1)
    _check([n], 2, 4, 2, 256, 64, seed=n + 2)


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("D", [64, 128, 256, 112])
def test_attention_page_sizes(page, D):
    _check([page, page + 1, 3 * page - 1, 97], 2, 8, 2, D, page, seed=page, max_pages=200)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 1000])
@pytest.mark.parametrize("rows", [1, 4, 8])
def test_attention_windows(window, rows):
    _check([0, 1, 5, 16, 33, 400], rows, 6, 2, 128, 16, window=window, seed=window + rows)


@pytest.mark.parametrize("rows,hq,hk,D", [(1, 32, 1, 128), (8, 32, 2, 128), (8, 16, 1, 128), (8, 20, 1, 64), (1, 71, 1, 64),
                                          (8, 32, 1, 128), (8, 8, 1, 256), (3, 64, 1, 256), (1, 4, 2, 320), (8, 40, 2, 80)])
def test_attention_of_many_rows(rows, hq, hk, D):
    _check([260, 3, 77], rows, hq, hk, D, 16, seed=hq)


def test_attention_of_many_sequences():
    _check([(i * 37) % 150 for i in range(700)], 1, 4, 1, 64, 16, seed=3)


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_attention_scales(scale):
    _check([200, 9], 2, 8, 2, 64, 16, scale=scale, seed=11)


@pytest.mark.parametrize("rows,hq,hk,D", [(1, 8, 8, 128), (4, 32, 8, 128), (8, 32, 8, 128), (8, 16, 8, 64), (1, 8, 8, 64),
                                          (4, 16, 8, 256), (8, 40, 4, 128), (3, 64, 4, 96)])
def test_ctas_that_walk_through_items(rows, hq, hk, D):
    for seqs in (32, 33):
        _check([(1000 + 397 * i) % 2100 for i in range(seqs)], rows, hq, hk, D, 64 if seqs == 32 else 16, seed=rows + D)


@pytest.mark.parametrize("rows,hq,hk,window", [(1, 8, 2, 0), (4, 8, 1, 0), (3, 4, 2, 70000)])
def test_a_long_context(rows, hq, hk, window):
    _check([131071, 40000], rows, hq, hk, 128, 64, window=window, seed=rows)


@pytest.mark.parametrize("window", [0, 24])
def test_what_a_row_does_not_see_does_not_reach_it(window):
    # the newest key (and, with a window, old ones) hold NaN scales: rows that do not see them are as without
    rows, n, page, D, hk = 4, 61, 16, 128, 2
    q, kc, vc, table, ln, ks, vs = _inputs([n], rows, 8, hk, D, FP4, page, 21)
    clean = nv.paged_attention(q, kc, vc, table, ln, window=window, k_scale=ks, v_scale=vs)
    old = [n - 1] + ([3, 36] if window else [])
    for j in old:
        for c in (kc, vc):
            c[int(table[0, j // page])].reshape(hk, 1, 9 * D)[:, 0, 8 * D + j % 16::16] = 0x7f
    got = nv.paged_attention(q, kc, vc, table, ln, window=window, k_scale=ks, v_scale=vs)
    for r in range(rows):
        at = n - rows + r
        if any(j <= at and (not window or j > at - window) for j in old):
            assert torch.isnan(got[r].float()).all(), r
        else:
            assert torch.equal(got[r], clean[r]), r
    assert nv.device_status() == 0


def test_bad_pages_and_lengths():
    q, kc, vc, table, ln, _, _ = _inputs([40, 20], 1, 4, 2, 128, FP4, 16, 6)
    clean = nv.paged_attention(q, kc, vc, table, ln)
    spoiled = table.clone()
    spoiled[0, 1] = 1000
    got = nv.paged_attention(q, kc, vc, spoiled, ln)
    assert nv.device_status() == nv.DEV_BAD_PAGE
    assert torch.equal(got[1], clean[1]) and torch.isfinite(got.float()).all()
    # the bad page's keys are as if they were not there
    keep = torch.tensor([[int(table[0, 0]), int(table[0, 2])]], dtype=torch.int32, device=DEV)
    less = nv.paged_attention(q[:1], kc, vc, keep, ln[:1] - 16)
    assert torch.allclose(got[0].float(), less[0].float(), rtol=2 * U16, atol=2.0 ** -10)
    long = torch.tensor([4000, -3], dtype=torch.int32, device=DEV)
    got = nv.paged_attention(q, kc, vc, table, long)
    assert nv.device_status() == nv.DEV_BAD_PAGE and not got[1].float().any() and nv.device_status() == 0


@pytest.mark.parametrize("pages,max_pages", [(0, 0), (0, 3), (4, 0)])
def test_an_empty_cache_or_table(pages, max_pages):
    D = 64
    kc, vc = nv.kv_cache(pages, 2, 16, D, FP4)
    table = torch.zeros((2, max_pages), dtype=torch.int32, device=DEV)
    q, ln = torch.ones((4, 4, D), dtype=BF16, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    lse = torch.full((4, 4), math.nan, device=DEV)
    out = nv.paged_attention(q, kc, vc, table, ln, lse=lse)
    assert not out.any() and bool((lse == -math.inf).all()) and nv.device_status() == 0
    k, freq = torch.ones((2, 2, D), dtype=BF16, device=DEV), torch.ones(32, device=DEV)
    for at, status in ((-1, 0), (0, nv.DEV_BAD_PAGE)):
        pos = torch.full((2,), at, dtype=torch.int32, device=DEV)
        nv.rope_append(q[:2], k, k, pos, freq, kc, vc, table)
        assert nv.device_status() == status
    assert not kc.any() and not vc.any()


def test_offsets_past_32_bits():
    # pages of 2^20 bytes: the last of 5000 starts past 2^32
    page, D = 16, 64
    pool = torch.zeros(5000, 1 << 20, dtype=FP4, device=DEV)
    row = 9 * D // 16
    kc, vc = (pool.as_strided((5000, 1, page, row), (1 << 20, page * row, row, 1), at) for at in (0, 1 << 19))
    g = _gen(8)
    ids = [4999, 4100, 17]
    for c in (kc, vc):
        some = torch.empty((3, 1, page, row), dtype=FP4, device=DEV)
        _fill(some, g)
        c[ids] = some
    table = torch.tensor([ids], dtype=torch.int32, device=DEV)
    q = _randn((2, 4, D), g, BF16)
    ln = torch.tensor([45], dtype=torch.int32, device=DEV)
    got = nv.paged_attention(q, kc, vc, table, ln)
    kd, vd = (torch.zeros((5000, 1, page, D), dtype=torch.float64, device=DEV) for _ in "kv")
    kd[ids], vd[ids] = _values(kc[ids]), _values(vc[ids])
    ref, tol, _, _ = _ref(q, kd, vd, table, [45], 2, D ** -0.5, 0, None, None, P_ERR[FP4])
    _within(got, ref, tol)
    k = _randn((1, 1, D), g, BF16)
    pos = torch.tensor([3], dtype=torch.int32, device=DEV)
    nv.rope_append(None, k, k, pos, torch.empty(0, device=DEV), kc, vc, table)
    codes, blocks = _records_of(k, torch.ones(1, device=DEV))
    for c in (kc, vc):
        gc, gb = _bytes_at(c, 4999, 3)
        assert torch.equal(gc, codes[0]) and torch.equal(gb, blocks[0])
    assert torch.equal(nv.cache_read(pos, kc, vc, table)[0][0].double(), _values(kc[4999:])[0, :, 3])


@pytest.mark.parametrize("offset,stride", [(0, 0), (1, 0), (0, 1), (8, 8), (16, 16)])
def test_caches_on_any_boundary_and_with_strides_of_their_own(offset, stride):
    # keys and values in separate pools, whose pages begin on other boundaries and lie apart by other strides
    g = _gen(offset + 40 * stride)
    page, D, hk, pages = 32, 128, 2, 6
    row = 9 * D // 16
    size = hk * page * row

    def pool(extra):
        mem = torch.zeros(pages * (size + extra) + 64, dtype=FP4, device=DEV)
        return mem.as_strided((pages, hk, page, row), (size + extra, page * row, row, 1), offset)

    kc, vc = pool(stride), pool(2 * stride)
    T, table = 70, torch.tensor([[4, 1, 5]], dtype=torch.int32, device=DEV)
    k, v = (_randn((T, hk, D), g, BF16) for _ in "kv")
    at = torch.arange(T, dtype=torch.int32, device=DEV)
    nv.rope_append(None, k, v, at, torch.empty(0, device=DEV), kc, vc, table)
    even = nv.kv_cache(pages, hk, page, D, FP4)
    nv.rope_append(None, k, v, at, torch.empty(0, device=DEV), *even, table)
    assert torch.equal(kc, even[0]) and torch.equal(vc, even[1])
    for a, b in zip(nv.cache_read(at, kc, vc, table), nv.cache_read(at, *even, table)):
        assert torch.equal(a, b)
    q, ln = _randn((2, 8, D), g, BF16), torch.tensor([T], dtype=torch.int32, device=DEV)
    got = nv.paged_attention(q, kc, vc, table, ln)
    ref, tol, _, _ = _ref(q, _values(even[0]), _values(even[1]), table, [T], 2, D ** -0.5, 0, None, None, P_ERR[FP4])
    _within(got, ref, tol)
    assert nv.device_status() == 0


# ------------------------------------------------------------------------------- used together

def test_append_read_and_attend_together_in_a_graph():
    # a prompt appended, its rows read back, then decode steps over it: eager, on another stream and captured
    g = _gen(12)
    hq, hk, D, page, T = 8, 2, 128, 16, 50
    kc, vc = nv.kv_cache(5, hk, page, D, FP4)
    table = torch.tensor([[4, 0, 2, 1, 3]], dtype=torch.int32, device=DEV)
    freq, _ = nv.rope_frequencies(D)
    q, k, v = (_randn((T, n, D), g, BF16) for n in (hq, hk, hk))
    nv.rope_append(q, k, v, torch.arange(T, dtype=torch.int32, device=DEV), freq, kc, vc, table)
    ws = nv.attention_workspace(1, 2, hq, hk, D)
    pos, ln = torch.tensor([T, T + 1], dtype=torch.int32, device=DEV), torch.tensor([T + 2], dtype=torch.int32, device=DEV)
    q, k, v = (_randn((2, n, D), g, BF16) for n in (hq, hk, hk))
    every = torch.arange(T + 2, dtype=torch.int32, device=DEV)

    def step():
        turned = nv.rope_append(q, k, v, pos, freq, kc, vc, table)
        rows = nv.cache_read(every, kc, vc, table)
        return turned, *rows, nv.paged_attention(turned, kc, vc, table, ln, softcap=20.0, workspace=ws)

    want = step()
    turned, keys, vals, out = (t.double() for t in want)
    for r in range(2):
        z = torch.einsum("hgd,khd->hgk", turned[r].view(hk, -1, D), keys[:T + 1 + r]) * D ** -0.5
        p = torch.softmax(20 * torch.tanh(z / 20), 2)
        ref = torch.einsum("hgk,khd->hgd", p, vals[:T + 1 + r]).reshape(hq, D)
        size = torch.einsum("hgk,khd->hgd", p, vals[:T + 1 + r].abs()).reshape(hq, D)
        # codes times scales of 1 are bf16 values, so the rows are what attention reads: weights of 11 bits, the output
        _within(out[r], ref, ref.abs() * U16 + size * (2.0 ** -11 + 2.0 ** -16), "out")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for t in kept:
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, kept)) and nv.device_status() == 0


def test_the_workspace_is_shared_with_other_caches_and_left_ready():
    ws = max((nv.attention_workspace(2, 4, 16, 2, D) for D in (64, 128, 256)), key=len)
    calls = []
    for i, (cache, D, lengths) in enumerate([(FP4, 128, [900, 30]), (BF16, 128, [5000, 3]), (FP4, 256, [70, 2000]), (FP8, 64, [9, 900])]):
        q, kc, vc, table, ln, ks, vs = _inputs(lengths, 4, 16, 2, D, cache, 16, i)
        calls.append(lambda w, a=(q, kc, vc, table, ln), ks=ks, vs=vs: nv.paged_attention(*a, k_scale=ks, v_scale=vs, workspace=w))
    want = [c(None) for c in calls]
    for i in (0, 1, 0, 2, 3, 2, 0, 1):
        assert torch.equal(calls[i](ws), want[i]), i
    assert nv.device_status() == 0


def test_wait_budget():
    q, kc, vc, table, ln, ks, vs = _inputs([3000, 30], 1, 8, 2, 128, FP4, 16, 7)
    ws = nv.attention_workspace(2, 1, 8, 2, 128)
    want = nv.paged_attention(q, kc, vc, table, ln, workspace=ws)
    try:
        nv.set_wait_budget_ns(0)
        nv.paged_attention(q, kc, vc, table, ln, workspace=ws)
        nv.device_status()  # copies that had come already are no timeout
    finally:
        nv.set_wait_budget_ns(None)
    assert torch.equal(nv.paged_attention(q, kc, vc, table, ln, workspace=ws), want)
    assert nv.device_status() == 0


def test_refusals():
    q, kc, vc, table, ln, _, _ = _inputs([5, 6], 2, 4, 2, 64, FP4, 16, 8)
    pos, k = torch.tensor([0, 1], dtype=torch.int32, device=DEV), torch.ones((2, 2, 64), dtype=BF16, device=DEV)
    freq = torch.ones(32, device=DEV)
    for bad in (dict(k_cache=kc[..., :35], v_cache=vc[..., :35]), dict(v_cache=vc.to(BF16)), dict(k_cache=kc[:, :, :8], v_cache=vc[:, :, :8]),
                dict(q=q[..., :32]), dict(k_scale=torch.ones(3, device=DEV)), dict(k_cache=kc.cpu(), v_cache=vc.cpu()),
                dict(v_cache=vc.view(FP8))):
        with pytest.raises((TypeError, ValueError)):
            nv.paged_attention(**{**dict(q=q, k_cache=kc, v_cache=vc, page_table=table, lengths=ln), **bad})
        if "q" not in bad:
            with pytest.raises((TypeError, ValueError)):
                nv.rope_append(**{**dict(q=None, k=k, v=k, positions=pos, inv_freq=freq, k_cache=kc, v_cache=vc, page_table=table), **bad})
            with pytest.raises((TypeError, ValueError)):
                nv.cache_read(**{**dict(positions=pos, k_cache=kc, v_cache=vc, page_table=table), **bad})
    for bad in (dict(positions=pos.long()), dict(positions=pos[None]), dict(positions=[0, 1]), dict(page_table=table[0]), dict(seq_ids=pos[:1]),
                dict(page_table=table[:1].expand(3, -1)), dict(k_out=torch.empty((2, 2, 64), device=DEV)),
                dict(v_out=torch.empty((2, 2, 32), dtype=BF16, device=DEV)), dict(k_out=torch.empty((2, 2, 128), dtype=BF16, device=DEV)[..., ::2]),
                dict(k_cache=None), dict(v_scale=freq)):
        with pytest.raises((TypeError, ValueError)):
            nv.cache_read(**{**dict(positions=pos, k_cache=kc, v_cache=vc, page_table=table), **bad})
    b16 = nv.kv_cache(1, 2, 16, 64)
    with pytest.raises(ValueError):
        nv.cache_read(pos, *b16, table, k_scale=torch.ones(2, device=DEV))


# ------------------------------------------------------------------------------ beside the usual

def test_a_long_prompt_on_both_kernels():
    # a warp takes a whole token where tokens are many: the same values, and the same keys but for their last bits
    g = _gen(31)
    T, hq, hk, D, page = 3001, 4, 3, 128, 64
    q, k, v = (_randn((T, n, D), g, BF16) for n in (hq, hk, hk))
    at = torch.randperm(T, generator=g, device=DEV).int()
    freq, _ = nv.rope_frequencies(D)
    table = torch.randperm(48, generator=g, device=DEV).int()[None, :47]
    norm, scale = (1 + 0.2 * _randn((D,), g)).to(BF16), 0.5 + torch.rand(hk, generator=g, device=DEV)
    got = []
    for variant in (0, 1):
        kc, vc = nv.kv_cache(48, hk, page, D, FP4)
        nv.set_variant(variant)
        try:
            out = nv.rope_append(q, k, v, at, freq, kc, vc, table, k_norm=norm, k_scale=scale, v_scale=scale)
        finally:
            nv.set_variant(0)
        got.append((out, *nv.cache_read(at, kc, vc, table, k_scale=scale, v_scale=scale)))
    assert nv.device_status() == 0
    (qa, ka, va), (qb, kb, vb) = got
    assert torch.equal(va, vb)
    # queries: each kernel's fp32 value, up to 24 roundings of magnitudes below 8 off, rounded to bf16
    _within(qa, qb.double(), qb.double().abs() * 2 * U16 + 2 * 24 * U32 * 8, "q")
    # a key beside a border takes the other code of two, or its block the other scale: one in 10^5, not more
    assert float((ka != kb).float().mean()) < 1e-4
    back = vb.double() / scale.double()[:, None]
    top = (v.double() / scale.double()[:, None]).view(T, hk, 8, 16).abs().amax(dim=3, keepdim=True)
    off = (back - v.double() / scale.double()[:, None]).view(T, hk, 8, 16).abs()
    # half a step of the largest binade, 1 / 6 of the largest value, of a scale 2^-4 off, and the row's bf16
    assert bool((off <= top * ((1 / 6) * (1 + U8) + U8 + U16)).all())


def test_the_same_token_twice_leaves_one_of_its_places_whole():
    # all bytes of the place are one of the tokens': codes of either, the scale of either
    g = _gen(5)
    k = _randn((2, 1, 16), g, BF16)
    kc, vc = nv.kv_cache(1, 1, 16, 16, FP4)
    zero = torch.zeros(2, dtype=torch.int32, device=DEV)
    nv.rope_append(None, k, k, zero, torch.empty(0, device=DEV), kc, vc, zero[:1][None], zero)
    codes, blocks = _records_of(k, torch.ones(1, device=DEV))
    for c in (kc, vc):
        gc, gb = _bytes_at(c, 0, 0)
        assert bool(((gc == codes[0]) | (gc == codes[1])).all()) and bool(((gb == blocks[0]) | (gb == blocks[1])).all())
        assert not c.reshape(-1)[8:128].any() and nv.device_status() == 0


def test_two_graphs_share_a_workspace():
    calls = []
    for i, (lengths, rows, cap) in enumerate([([3000, 30], 1, 0.0), ([700, 1, 0, 90], 4, 20.0)]):
        q, kc, vc, table, ln, ks, vs = _inputs(lengths, rows, 8, 2, 128, FP4, 16, i)
        calls.append((q, kc, vc, table, ln, dict(k_scale=ks, v_scale=vs, softcap=cap)))
    ws = max((nv.attention_workspace(len(c[4]), len(c[0]) // len(c[4]), 8, 2, 128) for c in calls), key=len)
    want = [nv.paged_attention(*c[:5], **c[5]) for c in calls]
    graphs, kept = [], []
    for c in calls:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kept.append(nv.paged_attention(*c[:5], workspace=ws, **c[5]))
        graphs.append(graph)
    for i in (0, 1, 1, 0, 0, 1):
        kept[i].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(kept[i], want[i]), i
    assert nv.device_status() == 0


def test_two_calls_at_once_with_workspaces_of_their_own():
    q, kc, vc, table, ln, ks, vs = _inputs([9000, 2000], 2, 8, 2, 128, FP4, 16, 3)
    want = nv.paged_attention(q, kc, vc, table, ln, k_scale=ks, v_scale=vs)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = [nv.paged_attention(q, kc, vc, table, ln, k_scale=ks, v_scale=vs, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got) and nv.device_status() == 0


def test_rows_read_on_another_stream_are_its_own():
    from test_gpu_decode_ops_edges import _owner
    _, kc, vc, table, _, ks, vs = _inputs([40], 1, 2, 2, 64, FP4, 16, 3)
    at = torch.arange(40, dtype=torch.int32, device=DEV)
    want = nv.cache_read(at, kc, vc, table, k_scale=ks, v_scale=vs)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = nv.cache_read(at, kc, vc, table, k_scale=ks, v_scale=vs, stream=side)
    mixed = nv.cache_read(at, kc, vc, table, k_scale=ks, v_scale=vs, stream=side.cuda_stream, k_out=torch.empty_like(want[0]))
    side.synchronize()
    for g, w in zip((*got, *mixed), (*want, *want)):
        assert torch.equal(g, w)
    assert _owner(got[0]) == _owner(got[1]) == _owner(mixed[1]) == side.cuda_stream


def test_nothing_to_do():
    kc, vc = nv.kv_cache(2, 2, 16, 64, FP4)
    none = torch.zeros((0, 3), dtype=torch.int32, device=DEV)
    q, i = torch.empty((0, 4, 64), dtype=BF16, device=DEV), torch.empty(0, dtype=torch.int32, device=DEV)
    assert nv.paged_attention(q, kc, vc, none, i, softcap=3.0).shape == (0, 4, 64)
    assert nv.rope_append(None, q[:, :2], q[:, :2], i, torch.empty(0, device=DEV), kc, vc, none) is None
    k, v = nv.cache_read(i, kc, vc, none)
    assert k.shape == v.shape == (0, 2, 64) and nv.device_status() == 0
    with pytest.raises(ValueError):
        nv.cache_read(torch.zeros(1, dtype=torch.int32, device=DEV), kc, vc, none)
