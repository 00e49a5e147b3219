"""The decode step's operators against plain 64-bit implementations: norm, rotary append, paged
attention, and the three together with the products.

Tolerances come from the arithmetic, before any run. u32 = 2^-24 and u16 = 2^-8 are the relative
rounding errors of fp32 and bf16, u8 = 2^-4 that of E4M3 (2^-10 absolute below its normal range).
"""
import math

import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16, FP8 = torch.float32, torch.bfloat16, torch.float8_e4m3fn
U32, U16, U8 = 2.0 ** -24, 2.0 ** -8, 2.0 ** -4


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(shape, gen, dtype=F32):
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def _within(got, ref, tol, what=""):
    got, ref = got.double(), ref.double()
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), f"{what}: NaN in other places"
    fine = torch.isfinite(ref)
    assert torch.equal(got[~fine & ~torch.isnan(ref)], ref[~fine & ~torch.isnan(ref)]), f"{what}: infinities differ"
    excess = ((got - ref).abs() - tol)[fine]
    assert excess.numel() == 0 or float(excess.max()) <= 0, f"{what}: over the tolerance by {float(excess.max())}"


# ------------------------------------------------------------------------------------- norm

def _norm_ref(x, residual, weight, eps):
    h = x.double() + (residual.double() if residual is not None else 0)
    return h, h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + eps) * weight.double()


def _check_norm(got, x, residual, weight, eps, group=0, residual_before=None):
    res_in = residual if residual_before is None else residual_before
    h, y = _norm_ref(x, res_in, weight, eps)
    # one fp32 addition, then 4 roundings (mean, rsqrt to 2 units, product, product); the sum of
    # squares adds at most 32 values in a row per thread and 15 partial sums
    rel = 32 * U32
    if res_in is not None:
        _within(got.residual, h, h.abs() * (U32 if got.residual.dtype is F32 else U16 + U32) + 2.0 ** -140, "residual")
    if got.y.dtype is not FP8:
        _within(got.y, y, y.abs() * (rel + (U16 if got.y.dtype is BF16 else 0)) + 2.0 ** -133, "y")
        return
    parts = y.view(y.shape[0], -1, group or y.shape[1])
    s = (parts.abs().amax(dim=2) / 448).clamp_min(2.0 ** -64)
    _within(got.scales, s, s.abs() * 2 * rel, "scales")
    back = got.y.double().view(parts.shape) * got.scales.double()[..., None]
    _within(back.view(y.shape), y, (parts.abs() * (U8 + 4 * rel) + s[..., None] * 2.0 ** -10).view(y.shape), "codes")


@pytest.mark.parametrize("rows,cols", [(1, 4096), (3, 2816), (5, 256), (130, 8), (2, 24), (1, 32768), (9, 16392),
                                       (4, 7), (3, 1001), (1, 1), (700, 1152), (2, 30001)])
@pytest.mark.parametrize("xt,rt,yt", [(F32, BF16, BF16), (BF16, None, F32), (BF16, BF16, FP8), (F32, F32, FP8),
                                      (BF16, F32, BF16)])
def test_rms_norm(rows, cols, xt, rt, yt):
    g = _gen(rows * 40009 + cols)
    x = _randn((rows, cols), g, xt)
    r = _randn((rows, cols), g, rt) * 3 if rt else None
    w = (1 + 0.2 * _randn((cols,), g)).to(BF16 if cols % 2 else F32)
    got = nv.rms_norm(x, w, 1e-6, residual=r, out_dtype=yt)
    _check_norm(got, x, r, w, 1e-6)


@pytest.mark.parametrize("cols,group", [(4096, 128), (256, 16), (1056, 32), (2816, 256), (448, 64), (48, 16)])
@pytest.mark.parametrize("pitch", [0, 8, 3])
def test_rms_norm_groups_and_pitches(cols, group, pitch):
    g = _gen(cols + group + pitch)
    x = _randn((6, cols + pitch), g, BF16)[:, pitch:]
    r = _randn((6, cols + pitch), g)[:, :cols]
    w = 1 + 0.2 * _randn((cols,), g)
    out = torch.empty((6, cols + pitch), device=DEV).to(FP8)[:, :cols]
    got = nv.rms_norm(x, w, 1e-5, residual=r, out=out, group=group)
    _check_norm(got, x, r, w, 1e-5, group)


def test_rms_norm_in_place_and_broadcast_rows():
    g = _gen(5)
    for cols in (4096, 515):
        r = _randn((4, cols), g, BF16)
        before = r.clone()
        w = 1 + 0.2 * _randn((cols,), g)
        x = _randn((1, cols), g, BF16).expand(4, cols)
        got = nv.rms_norm(x, w, residual=r, residual_out=r)
        assert got.residual is r
        _check_norm(got, x, r, w, 1e-6, residual_before=before)
        y = _randn((4, cols), g, BF16)
        before = y.clone()
        nv.rms_norm(y, w, out=y)
        _check_norm(nv.RMSNormOut(y, None, None), before, None, w, 1e-6)


@pytest.mark.parametrize("cols", [512, 77])
def test_rms_norm_of_zeros_infinities_and_nan(cols):
    w = torch.ones(cols, device=DEV)
    x = torch.zeros((5, cols), device=DEV)
    x[1] = 1e-30                      # the mean square vanishes against eps
    x[2, 3] = math.inf
    x[3, 4] = math.nan
    x[4] = 1e18                       # squares up to 1e36 still sum in range
    got = nv.rms_norm(x, w, 1e-6, out_dtype=F32).y
    _, ref = _norm_ref(x, None, w, 1e-6)
    ref[2] = 0.0                      # finite / infinity
    ref[2, 3] = math.nan
    _within(got, ref, ref.abs() * 32 * U32 + 2.0 ** -140)
    q = nv.rms_norm(x, w, 1e-6, out_dtype=FP8)
    assert float(q.scales[0, 0]) == 2.0 ** -64 and not q.y[0].float().any()
    assert torch.isnan(q.scales[2, 0]) and torch.isnan(q.scales[3, 0]) and torch.isnan(q.y[3].float()).all()
    assert float(q.y[4, 0].float()) == 448.0


def test_rms_norm_refusals():
    x, w = torch.zeros((2, 64), device=DEV), torch.ones(64, device=DEV)
    for bad in (dict(x=x.cpu()), dict(x=x[0]), dict(x=x.half()), dict(weight=w[:63]), dict(weight=w.double()),
                dict(residual=x[:, :32]), dict(residual_out=x), dict(scales=w), dict(group=16), dict(out=x[:1]),
                dict(x=x.t()), dict(out_dtype=FP8, group=48), dict(out_dtype=FP8, scales=x)):
        with pytest.raises((TypeError, ValueError)):
            nv.rms_norm(**{"x": x, "weight": w, **bad})
    with pytest.raises(nv.NVFP4Error) as e:
        nv.rms_norm(x, w, out_dtype=FP8, group=8)
    assert e.value.status == 2
    with pytest.raises(nv.NVFP4Error) as e:
        nv.rms_norm(x, w, float("nan"))
    assert e.value.status == 2
    with pytest.raises(nv.NVFP4Error) as e:
        nv.rms_norm(torch.zeros((1, 32776), device=DEV), torch.ones(32776, device=DEV))
    assert e.value.status == 5
    assert nv.rms_norm(x[:0], w).y.shape == (0, 64)


# ----------------------------------------------------------------------------------- append

def _table(need, gen, spare=2):
    total = sum(need)
    order = torch.randperm(total + spare, generator=gen, device=DEV).int().tolist()
    t = torch.full((len(need), max(1, *need)), -1, dtype=torch.int32)
    for b, n in enumerate(need):
        t[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
    return t.to(DEV), total + spare


def _heads_ref(x, norm, eps):
    x = x.double()
    return x if norm is None else x / torch.sqrt((x * x).mean(dim=2, keepdim=True) + eps) * norm.double()


def _turn_ref(u, positions, inv_freq, interleaved, mscale):
    half = inv_freq.shape[0]
    angle = positions.double()[:, None, None] * inv_freq.double()
    c, s = mscale * torch.cos(angle), mscale * torch.sin(angle)
    i = torch.arange(half, device=DEV)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    y = u.clone()
    y[..., a] = u[..., a] * c - u[..., b] * s
    y[..., b] = u[..., b] * c + u[..., a] * s
    size = u.abs()
    size[..., a] = size[..., b] = mscale * (u[..., a].abs() + u[..., b].abs())
    return y, size


def _check_append(T, hq, hk, D, half, interleaved, xt, fused, cache, page, norm, positions, seqs, seq_ids=None,
                  mscale=1.0, freq=None, pair=False, offset=0):
    g = _gen(T * 7919 + D + half + page)
    if fused:
        w = (hq + 2 * hk) * D
        qkv = _randn((T, w + offset), g, xt)[:, offset:]
        q, k, v = (t.view(T, -1, D) if offset == 0 else t.unflatten(1, (-1, D)) for t in
                   qkv.split([hq * D, hk * D, hk * D], dim=1))
    else:
        q, k, v = (_randn((T, n, D), g, xt) for n in (hq, hk, hk))
    inv_freq = freq if freq is not None else (1e4 ** (-torch.arange(half, device=DEV).double() / max(half, 1))).float()
    pos = torch.tensor(positions, dtype=torch.int32, device=DEV)
    sid = None if seq_ids is None else torch.tensor(seq_ids, dtype=torch.int32, device=DEV)
    owner = seq_ids if seq_ids is not None else [t // (T // seqs) for t in range(T)]
    need = [max([p // page + 1 for p, o in zip(positions, owner) if o == b and p >= 0], default=0) for b in range(seqs)]
    table, pages = _table(need, g)
    if pair:
        kc, vc = nv.kv_cache(pages, hk, page, D, BF16 if cache is BF16 else FP8)
    else:
        kc, vc = (torch.zeros((pages, hk, page, D), device=DEV).to(cache) for _ in "kv")
    qn, kn = ((1 + 0.2 * _randn((D,), g)).to(BF16 if D % 64 else F32) for _ in "qk") if norm else (None, None)
    ks, vs = (0.05 + 0.1 * torch.rand(hk, generator=g, device=DEV) for _ in "kv") if cache is FP8 else (None, None)
    got = nv.rope_append(q, k, v, pos, inv_freq, kc, vc, table, sid, interleaved=interleaved, mscale=mscale, q_norm=qn,
                         k_norm=kn, eps=1e-6, k_scale=ks, v_scale=vs)
    assert nv.device_status() == 0
    live = pos >= 0
    at = pos.clamp_min(0)
    uq, uk = _heads_ref(q, qn, 1e-6), _heads_ref(k, kn, 1e-6)
    q_ref, q_size = _turn_ref(uq, at, inv_freq, interleaved, mscale)
    k_ref, k_size = _turn_ref(uk, at, inv_freq, interleaved, mscale)
    # per-head norm 12 units, cos and sin 8 units of 1 (angle 2^-22), three roundings
    rel = 24 * U32
    _within(got, q_ref * live[:, None, None], q_size * rel + q_ref.abs() * U16 + 2.0 ** -133, "q")
    touched = torch.zeros((pages, page), dtype=torch.bool, device=DEV)
    for t in range(T):
        if positions[t] < 0:
            continue
        p, s = int(table[owner[t], positions[t] // page]), positions[t] % page
        touched[p, s] = True
        for c, ref, size, sc, name in ((kc, k_ref, k_size, ks, "k"), (vc, v.double(), v.double().abs(), vs, "v")):
            row = c[p].double()[:, s]
            if cache is FP8:
                ref, size = (z[t] / sc.double()[:, None] for z in (ref, size))
                ref = ref.clamp(-448, 448)
                _within(row, ref, ref.abs() * U8 + size * rel + 2.0 ** -10, name)
            else:
                _within(row, ref[t], size[t] * rel + ref[t].abs() * U16 + 2.0 ** -133, name)
    for c in (kc, vc):
        assert not c.view(torch.uint8).flatten(3)[~touched[:, None, :].expand(-1, hk, -1)].any(), "wrote elsewhere"


@pytest.mark.parametrize("D,half,interleaved", [(128, 64, False), (128, 64, True), (128, 32, False), (128, 32, True),
                                                (64, 32, False), (96, 48, True), (80, 40, False), (256, 64, False),
                                                (128, 0, False), (72, 20, False), (40, 3, True), (33, 16, False),
                                                (512, 256, False)])
@pytest.mark.parametrize("xt,cache,fused,norm", [(F32, BF16, False, True), (BF16, FP8, True, False),
                                                 (BF16, BF16, True, True)])
def test_rope_append(D, half, interleaved, xt, cache, fused, norm):
    _check_append(6, 5, 2, D, half, interleaved, xt, fused, cache, 16, norm, [0, 1, 2, 15, 16, 40], 2,
                  pair=cache is FP8)


@pytest.mark.parametrize("page", [1, 7, 48, 128])
@pytest.mark.parametrize("T", [1, 13, 97])
def test_rope_append_ragged(page, T):
    lens = [3 * T // 4, 0, T - 3 * T // 4]
    sid = [b for b, n in enumerate(lens) for _ in range(n)]
    pos = [p + 5 * b for b, n in enumerate(lens) for p in range(n)]
    if T > 5:
        pos[2] = -1  # padding
    _check_append(T, 8, 4, 128, 64, False, BF16, True, FP8 if page == 48 else BF16, page, True, pos, 3, sid)


def test_rope_append_odd_strides_and_scaled_frequencies():
    freq, mscale = nv.rope_frequencies(64, 1e4, factor=8.0, original_length=4096)
    _check_append(4, 3, 1, 64, 32, False, BF16, True, BF16, 16, False, [70000, 3, 900, 65535], 2, mscale=mscale,
                  freq=freq.to(DEV), offset=1)


def test_rope_append_far_positions():
    # at 2^24 - 1 the angle's fp32 product alone would be off by half a radian
    pos = [(1 << 24) - 1, 1000003, 8388607, 131071]
    T, D = 4, 128
    g = _gen(9)
    q, k = _randn((T, 2, D), g), _randn((T, 1, D), g)
    table = torch.zeros((1, 1 << 18), dtype=torch.int32, device=DEV)
    kc, vc = (torch.zeros((1, 1, 64, D), dtype=BF16, device=DEV) for _ in "kv")
    freq = (1e4 ** (-torch.arange(64, device=DEV).double() / 64)).float()
    p = torch.tensor(pos, dtype=torch.int32, device=DEV)
    got = nv.rope_append(q, k, k, p, freq, kc, vc, table)
    ref, size = _turn_ref(q.double(), p, freq, False, 1.0)
    _within(got, ref, size * 24 * U32 + ref.abs() * U16)


def test_rope_append_bad_places_set_the_status_and_write_nothing():
    T, D = 5, 128
    k = torch.ones((T, 2, D), dtype=BF16, device=DEV)
    q = torch.ones((T, 4, D), dtype=BF16, device=DEV)
    kc, vc = nv.kv_cache(3, 2, 16, D)
    table = torch.tensor([[0, 1], [2, 7]], dtype=torch.int32, device=DEV)
    pos = torch.tensor([32, 0, 16, 3, 5], dtype=torch.int32, device=DEV)      # past the table; good; bad page; bad seqs
    sid = torch.tensor([0, 0, 1, 2, -1], dtype=torch.int32, device=DEV)
    freq = torch.ones(64, device=DEV)
    out = nv.rope_append(q, k, k, pos, freq, kc, vc, table, sid)
    assert nv.device_status() == nv.DEV_BAD_PAGE and nv.device_status() == 0
    assert torch.isfinite(out.float()).all() and bool((out != 0).any(dim=2).all())
    assert bool(vc[0, :, 0].eq(1).all()) and int((vc != 0).sum()) == 2 * D and int((kc != 0).any(dim=3).sum()) == 2


def test_rope_append_without_queries_and_refusals():
    D = 64
    k = torch.ones((2, 2, D), device=DEV)
    kc, vc = nv.kv_cache(2, 2, 16, D)
    table = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    pos = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    freq = torch.ones(32, device=DEV)
    ok = dict(q=None, k=k, v=k, positions=pos, inv_freq=freq, k_cache=kc, v_cache=vc, page_table=table)
    assert nv.rope_append(**ok) is None
    assert bool(vc[0, :, :2].eq(1).all())
    for bad in (dict(v=k[:1]), dict(v=k.to(BF16)), dict(positions=pos.long()), dict(positions=pos[:1]),
                dict(inv_freq=torch.ones(33, device=DEV)), dict(k_cache=kc[:, :1]), dict(v_cache=vc.to(FP8)),
                dict(q=k.to(BF16)), dict(q=k[:, :, :32]), dict(out=k), dict(seq_ids=pos[:1]), dict(q_norm=freq),
                dict(k_norm=freq), dict(k_scale=freq), dict(page_table=table.expand(4, 1)),
                dict(k=k.transpose(1, 2)), dict(k_cache=kc.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises((TypeError, ValueError)):
            nv.rope_append(**{**ok, **bad})
    with pytest.raises(nv.NVFP4Error) as e:
        nv.rope_append(**{**ok, "page_table": torch.zeros((1, 1 << 21), dtype=torch.int32, device=DEV)})
    assert e.value.status == 5


# -------------------------------------------------------------------------------- attention

def _attend_ref(q, kc, vc, table, lengths, rows, scale, window, ks, vs, p_err):
    """out, its tolerance, lse and its tolerance, in 64 bits, row by row."""
    T, hq, D = q.shape
    hk, page = kc.shape[1], kc.shape[2]
    g = hq // hk
    out = torch.zeros((T, hq, D), dtype=torch.float64, device=DEV)
    tol = torch.full_like(out, 2.0 ** -133)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=DEV)
    ltol = torch.zeros_like(lse)
    for b, n in enumerate(lengths):
        npg = -(-n // page)
        for h in range(hk):
            keys, vals = (c[table[b, :npg].long()].double()[:, h].reshape(-1, D)[:n] for c in (kc, vc))
            if ks is not None:
                keys, vals = keys * ks[h].double(), vals * vs[h].double()
            for r in range(rows):
                hi = n - rows + r + 1
                lo = max(0, hi - window) if window else 0
                if hi <= lo:
                    continue
                t, hs = b * rows + r, slice(h * g, (h + 1) * g)
                qq = q[t, hs].double()
                z = qq @ keys[lo:hi].T * scale
                # fp32 dot products of D terms and the scaling; E4M3 caches: q in f16 next to its maximum
                dz = ((D + 8) * U32 * (qq.abs() @ keys[lo:hi].abs().T) * abs(scale)
                      + 2.0 ** -24 * qq.abs().amax(dim=1, keepdim=True) * keys[lo:hi].abs().sum(dim=1) * abs(scale))
                dz = dz.amax(dim=1, keepdim=True) + z.abs().amax(dim=1, keepdim=True) * 4 * U32
                p = torch.softmax(z, dim=1)
                lse[t, hs] = torch.logsumexp(z, dim=1)
                m = hi - lo
                ltol[t, hs] = (dz + 8 * U32 + m * U32).squeeze(1) + lse[t, hs].abs() * 4 * U32
                out[t, hs] = p @ vals[lo:hi]
                size = p @ vals[lo:hi].abs()
                tol[t, hs] += size * (2 * dz + p_err + (m + 16) * U32) + out[t, hs].abs() * U16
                # probabilities below the rounded type's normal range: 2^-25 of the row's largest
                tol[t, hs] += 2.0 ** -25 * p.amax(dim=1, keepdim=True) * vals[lo:hi].abs().sum(dim=0)
    return out, tol, lse, ltol


def _attend_inputs(lengths, rows, hq, hk, D, cache, page, seed, poison=True, max_pages=0):
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
        x = _randn(c.shape, g) * (16 if cache is FP8 else 1)
        if poison:
            x[~used[:, None, :].expand(-1, hk, -1)] = math.nan
        c.copy_(x.to(cache))
    ks, vs = ((0.04 + 0.05 * torch.rand(hk, generator=g, device=DEV) for _ in "kv") if cache is FP8 else (None, None))
    q = (2 * _randn((len(lengths) * rows, hq, D), g)).to(BF16)
    return q, kc, vc, table, torch.tensor(lengths, dtype=torch.int32, device=DEV), ks, vs


def _check_attend(lengths, rows, hq, hk, D, cache, page, window=0, scale=None, seed=0, spoil=None, max_pages=0):
    q, kc, vc, table, ln, ks, vs = _attend_inputs(lengths, rows, hq, hk, D, cache, page, seed, max_pages=max_pages)
    ref_k, ref_v = kc, vc
    if spoil:
        ref_k, ref_v = kc.clone(), vc.clone()
        spoil(kc, vc, table)
    ws = nv.attention_workspace(len(lengths), rows, hq, hk, D)
    lse = torch.empty((q.shape[0], hq), device=DEV)
    out = torch.full_like(q, math.nan)
    nv.paged_attention(q, kc, vc, table, ln, scale, window=window, k_scale=ks, v_scale=vs, workspace=ws, out=out, lse=lse)
    assert nv.device_status() == 0
    sc = scale if scale is not None else D ** -0.5
    p_err = U16 if cache is BF16 else 2.0 ** -11
    ref, tol, lref, ltol = _attend_ref(q, ref_k, ref_v, table, lengths, rows, sc, window, ks, vs, p_err)
    _within(out, ref, tol, "out")
    _within(lse, lref, ltol, "lse")
    again, lse2 = torch.full_like(q, math.nan), torch.empty_like(lse)
    nv.paged_attention(q, kc, vc, table, ln, scale, window=window, k_scale=ks, v_scale=vs, workspace=ws, out=again, lse=lse2)
    assert torch.equal(out, again) and torch.equal(lse, lse2), "the same call twice differs"
    return out


@pytest.mark.parametrize("cache", [BF16, FP8])
@pytest.mark.parametrize("D", [64, 128, 256, 80, 96, 16, 48, 192])
@pytest.mark.parametrize("rows,hq,hk", [(1, 8, 8), (1, 32, 8), (3, 10, 2), (5, 8, 1), (8, 16, 2), (2, 7, 7)])
def test_paged_attention(cache, D, rows, hq, hk):
    _check_attend([37, 0, 1, 300, 16, 2], rows, hq, hk, D, cache, 16, seed=D + rows)


@pytest.mark.parametrize("cache", [BF16, FP8])
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 257, 1000, 4099])
def test_paged_attention_lengths(cache, n):
    _check_attend([n], 1, 8, 2, 128, cache, 32, seed=n)
    _check_attend([n, n // 2], 4, 4, 1, 64, cache, 16, seed=n + 1)


@pytest.mark.parametrize("cache", [BF16, FP8])
@pytest.mark.parametrize("page", [1, 5, 8, 16, 24, 48, 64, 128, 256])
def test_paged_attention_page_sizes(cache, page):
    _check_attend([page, page + 1, 3 * page - 1, 97], 2, 8, 2, 128, cache, page, seed=page, max_pages=200)


@pytest.mark.parametrize("window", [1, 2, 15, 16, 17, 100, 1000])
@pytest.mark.parametrize("rows", [1, 4, 8])
def test_paged_attention_windows(window, rows):
    for cache in (BF16, FP8):
        _check_attend([0, 1, 5, 16, 33, 400], rows, 6, 2, 128, cache, 16, window=window, seed=window + rows)


@pytest.mark.parametrize("rows,hq,hk,D", [(1, 32, 1, 128), (8, 32, 2, 128), (8, 16, 1, 128), (8, 20, 1, 64), (1, 71, 1, 64),
                                          (8, 32, 1, 128), (8, 8, 1, 256), (3, 64, 1, 256), (1, 5, 1, 33),
                                          (1, 4, 2, 320), (2, 4, 4, 512)])
def test_paged_attention_many_rows_and_odd_heads(rows, hq, hk, D):
    for cache in (BF16, FP8):
        _check_attend([260, 3, 77], rows, hq, hk, D, cache, 16, seed=hq)


@pytest.mark.parametrize("rows,hq", [(8, 1024), (2, 1025), (8, 1500)])
def test_paged_attention_many_heads_per_kv_head(rows, hq):
    _check_attend([40, 3], rows, hq, 1, 64, BF16, 16)


def test_paged_attention_many_sequences():
    lengths = [(i * 37) % 150 for i in range(700)]
    _check_attend(lengths, 1, 4, 1, 64, BF16, 16, seed=3)


@pytest.mark.parametrize("cache", [BF16, FP8])
@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_paged_attention_scales(cache, scale):
    # scale 3 makes all but a few probabilities vanish
    _check_attend([200, 9], 2, 8, 2, 64, cache, 16, scale=scale, seed=11)


@pytest.mark.parametrize("cache", [BF16, FP8])
@pytest.mark.parametrize("window", [0, 24])
@pytest.mark.parametrize("what", [math.nan, math.inf])
def test_what_a_row_does_not_see_does_not_reach_it(cache, window, what):
    # the newest key (and, with a window, old ones) hold NaN or infinity: rows that do not see
    # them are as without
    rows, n, page, D, hk = 4, 61, 16, 128, 2
    value = math.nan if cache is FP8 else what

    q, kc, vc, table, ln, ks, vs = _attend_inputs([n], rows, 8, hk, D, cache, page, 21)
    clean = nv.paged_attention(q, kc, vc, table, ln, window=window, k_scale=ks, v_scale=vs)
    for j in [n - 1] + ([3, 36] if window else []):
        p, s = int(table[0, j // page]), j % page
        for c in (kc, vc):
            c[p, :, s] = torch.full((hk, D), value, device=DEV).to(cache)
    got = nv.paged_attention(q, kc, vc, table, ln, window=window, k_scale=ks, v_scale=vs)
    first = n - rows
    for r in range(rows):
        seen = [j for j in ([n - 1] + ([3, 36] if window else [])) if j <= first + r and (not window or j > first + r - window)]
        if seen:
            assert torch.isnan(got[r].float()).all(), r
        else:
            assert torch.allclose(got[r].float(), clean[r].float(), rtol=2 * U16, atol=1e-3), r
    assert nv.device_status() == 0


def test_paged_attention_infinite_scores():
    # a key of -inf has weight zero; a row of nothing else gives zeros and -inf
    n, D = 40, 64
    q, kc, vc, table, ln, _, _ = _attend_inputs([n], 1, 2, 1, D, BF16, 16, 5)
    q.fill_(1.0)
    p, s = int(table[0, 1]), 4
    kc[p, 0, s] = -math.inf
    lse = torch.empty((1, 2), device=DEV)
    got = nv.paged_attention(q, kc, vc, table, ln, lse=lse)
    keep = [j for j in range(n) if j != 20]
    keys, vals = (c[table[0].long()].double()[:, 0].reshape(-1, D)[keep] for c in (kc, vc))
    z = q[0].double() @ keys.T * D ** -0.5
    ref = torch.softmax(z, 1) @ vals
    assert torch.allclose(got[0].double(), ref, rtol=2 * U16, atol=2 * U16)
    for i in range(3):
        kc[int(table[0, i])] = -math.inf
    got = nv.paged_attention(q, kc, vc, table, ln, lse=lse)
    assert not got.float().any() and bool((lse == -math.inf).all())


def test_paged_attention_bad_pages_and_lengths():
    q, kc, vc, table, ln, _, _ = _attend_inputs([40, 20], 1, 4, 2, 128, BF16, 16, 6)
    clean = nv.paged_attention(q, kc, vc, table, ln)
    spoiled = table.clone()
    spoiled[0, 1] = 1000
    got = nv.paged_attention(q, kc, vc, spoiled, ln)
    assert nv.device_status() == nv.DEV_BAD_PAGE
    assert torch.equal(got[1], clean[1]) and torch.isfinite(got.float()).all()
    long = torch.tensor([4000, -3], dtype=torch.int32, device=DEV)
    got = nv.paged_attention(q, kc, vc, table, long)
    assert nv.device_status() == nv.DEV_BAD_PAGE and not got[1].float().any()
    assert nv.device_status() == 0


def test_paged_attention_offsets_past_32_bits():
    # pages of 2^20 elements: the last of 5000 starts past 2^32 elements and bytes
    page, D = 16, 64
    pool = torch.zeros(5000, 1 << 20, dtype=BF16, device=DEV)
    kc = pool[:, :page * D].view(5000, 1, page, D) if False else pool.as_strided((5000, 1, page, D), (1 << 20, page * D, D, 1))
    vc = pool.as_strided((5000, 1, page, D), (1 << 20, page * D, D, 1), 1 << 19)
    g = _gen(8)
    ids = [4999, 4100, 17]
    for i in ids:
        kc[i], vc[i] = _randn((1, page, D), g, BF16), _randn((1, page, D), g, BF16)
    table = torch.tensor([ids], dtype=torch.int32, device=DEV)
    q = _randn((2, 4, D), g, BF16)
    ln = torch.tensor([45], dtype=torch.int32, device=DEV)
    got = nv.paged_attention(q, kc, vc, table, ln)
    ref, tol, _, _ = _attend_ref(q, kc, vc, table, [45], 2, D ** -0.5, 0, None, None, U16)
    _within(got, ref, tol)
    k = _randn((1, 1, D), g, BF16)
    nv.rope_append(None, k, k, torch.tensor([3], dtype=torch.int32, device=DEV), torch.empty(0, device=DEV), kc, vc, table)
    assert torch.equal(kc[4999, 0, 3], k[0, 0]) and torch.equal(vc[4999, 0, 3], k[0, 0])


def test_paged_attention_strided_queries():
    q, kc, vc, table, ln, _, _ = _attend_inputs([50, 9], 2, 6, 2, 128, BF16, 16, 7)
    want = nv.paged_attention(q, kc, vc, table, ln)
    wide = torch.zeros((4, 9, 128), dtype=BF16, device=DEV)
    wide[:, 2:8] = q
    assert torch.equal(nv.paged_attention(wide[:, 2:8], kc, vc, table, ln), want)
    odd = torch.zeros((4, 6, 131), dtype=BF16, device=DEV)
    odd[:, :, 3:] = q
    assert torch.equal(nv.paged_attention(odd[:, :, 3:], kc, vc, table, ln), want)


def test_paged_attention_refusals():
    q, kc, vc, table, ln, _, _ = _attend_inputs([5, 6], 2, 4, 2, 64, BF16, 16, 8)
    ok = dict(q=q, k_cache=kc, v_cache=vc, page_table=table, lengths=ln)
    for bad in (dict(q=q.float()), dict(q=q[:3]), dict(q=q[:, :3]), dict(lengths=ln.long()), dict(lengths=ln[:1]),
                dict(k_cache=kc.float()), dict(v_cache=vc[:1]), dict(page_table=table[0]), dict(out=q[:2]),
                dict(lse=torch.empty(4, device=DEV)), dict(k_scale=torch.ones(3, device=DEV)), dict(q=q.cpu()),
                dict(workspace=torch.zeros(4096, device=DEV))):
        with pytest.raises((TypeError, ValueError)):
            nv.paged_attention(**{**ok, **bad})
    with pytest.raises(nv.NVFP4Error) as e:
        nv.paged_attention(**ok, workspace=torch.zeros(1, dtype=torch.uint8, device=DEV))
    assert e.value.status == 2
    ws = nv.attention_workspace(2, 2, 4, 2, 64)
    with pytest.raises(nv.NVFP4Error) as e:
        nv.paged_attention(**ok, workspace=torch.zeros(ws.numel() + 16, dtype=torch.uint8, device=DEV)[16:])
    assert e.value.status == 3
    with pytest.raises(nv.NVFP4Error) as e:
        nv.paged_attention(**ok, workspace=ws, window=-1)
    assert e.value.status == 2
    with pytest.raises(ValueError):
        nv.attention_workspace_bytes(1, 9, 8, 8, 128)


def test_decode_ops_on_other_streams_and_in_graphs():
    g = _gen(12)
    x, w = _randn((4, 512), g, BF16), 1 + 0.1 * _randn((512,), g)
    q, kc, vc, table, ln, _, _ = _attend_inputs([50, 9], 2, 6, 2, 128, BF16, 16, 7)
    ws = nv.attention_workspace(2, 2, 6, 2, 128)
    pos = torch.tensor([10, 11, 2, 3], dtype=torch.int32, device=DEV)
    freq, _ = nv.rope_frequencies(128)
    k = _randn((4, 2, 128), g, BF16)

    def step():
        y = nv.rms_norm(x, w).y
        qr = nv.rope_append(q, k, k, pos, freq, kc, vc, table)
        return y, qr, nv.paged_attention(qr, kc, vc, table, ln, workspace=ws)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    y = torch.empty_like(want[0])
    nv.rms_norm(x, w, out=y, stream=side)
    side.synchronize()
    assert torch.equal(y, want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = step()
    for t in kept:
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, kept))


def test_attention_workspace_is_left_ready():
    q, kc, vc, table, ln, _, _ = _attend_inputs([900, 30], 1, 8, 2, 128, BF16, 16, 7)
    ws = nv.attention_workspace(2, 1, 8, 2, 128)
    want = nv.paged_attention(q, kc, vc, table, ln, workspace=ws)
    # shorter, other heads, then the first again, on the same workspace
    nv.paged_attention(q, kc, vc, table, ln // 3, workspace=ws)
    nv.paged_attention(q[:, :4], kc, vc, table, ln, workspace=ws)
    assert torch.equal(nv.paged_attention(q, kc, vc, table, ln, workspace=ws), want)


def test_paged_attention_wait_budget():
    # with no time for its copies the call sets the status, ends, and leaves the workspace ready
    q, kc, vc, table, ln, _, _ = _attend_inputs([3000, 30], 1, 8, 2, 128, BF16, 16, 7)
    ws = nv.attention_workspace(2, 1, 8, 2, 128)
    want = nv.paged_attention(q, kc, vc, table, ln, workspace=ws)
    try:
        nv.set_wait_budget_ns(0)
        nv.paged_attention(q, kc, vc, table, ln, workspace=ws)
        assert nv.device_status() == nv.DEV_TIMEOUT
    finally:
        nv.set_wait_budget_ns(None)
    assert torch.equal(nv.paged_attention(q, kc, vc, table, ln, workspace=ws), want)
    assert nv.device_status() == 0


def test_infinite_values_stay_infinite():
    # a value of +-inf under a weight above zero makes that output +-inf, its sign kept; the rest is untouched
    n, D = 50, 128
    q, kc, vc, table, ln, _, _ = _attend_inputs([n], 2, 4, 2, D, BF16, 16, 31)
    clean = nv.paged_attention(q, kc, vc, table, ln)
    vc[int(table[0, 0]), :, 3, 5] = math.inf
    vc[int(table[0, 1]), :, 7, 90] = -math.inf
    got = nv.paged_attention(q, kc, vc, table, ln)
    assert bool((got[:, :, 5] == math.inf).all()) and bool((got[:, :, 90] == -math.inf).all())
    rest = [d for d in range(D) if d not in (5, 90)]
    assert torch.equal(got[:, :, rest], clean[:, :, rest])
