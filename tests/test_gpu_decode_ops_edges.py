"""Where the decode step's operators can go wrong beyond single calls of ordinary sizes and values.

Tolerances come from the arithmetic, before any run, with the units of test_gpu_decode_ops.
"""
import math

import pytest
import torch

import nvfp4_weight_only_gemv_gb300 as nv
from test_gpu_decode_ops import BF16, DEV, FP8, U16, U32, _attend_inputs, _check_attend, _gen, _randn, _within

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- one workspace, several shapes

def _shape(lengths, rows, hq, hk, D, cache, seed):
    q, kc, vc, table, ln, ks, vs = _attend_inputs(lengths, rows, hq, hk, D, cache, 16, seed)

    def call(ws):
        out, lse = torch.full_like(q, math.nan), torch.full((q.shape[0], hq), math.nan, device=DEV)
        nv.paged_attention(q, kc, vc, table, ln, k_scale=ks, v_scale=vs, workspace=ws, out=out, lse=lse)
        return out, lse

    return call, nv.attention_workspace_bytes(len(lengths), rows, hq, hk, D)


@pytest.mark.parametrize("a,b", [
    # as many parts as there are CTAs: 3, 2 and 1 of them an SM
    (([20000], 4, 32, 8, 128, BF16), ([20000], 1, 32, 8, 128, BF16)),
    (([9000], 8, 16, 2, 64, BF16), ([9000], 1, 4, 1, 256, FP8)),
    # few items, then many: a batch that grows and shrinks
    (([3000], 1, 32, 8, 128, FP8), ([200 + i for i in range(128)], 1, 32, 8, 128, FP8)),
    (([700] * 3, 2, 64, 1, 64, BF16), ([150] * 40, 8, 16, 2, 128, BF16)),
])
def test_attention_workspace_serves_every_shape(a, b):
    calls = [_shape(*a, seed=3), _shape(*b, seed=4)]
    want = [call(torch.zeros(n, dtype=torch.uint8, device=DEV)) for call, n in calls]
    ws = torch.zeros(max(n for _, n in calls), dtype=torch.uint8, device=DEV)
    for i in (0, 1, 0, 0, 1, 1, 0):
        got = calls[i][0](ws)
        for g, w in zip(got, want[i]):
            assert torch.equal(g, w), f"shape {i}: {int(torch.isnan(g).sum())} values were never written"
    assert nv.device_status() == 0


# --------------------------------------------------------------------------- windows without an end

@pytest.mark.parametrize("cache", [BF16, FP8])
@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("rows", [4, 8])
def test_the_widest_window_is_no_window(rows, page, cache):
    # sequences shorter than the rows too: their first row stands at a position below zero
    q, kc, vc, table, ln, ks, vs = _attend_inputs([0, 1, 300, rows - 1], rows, 8, 2, 128, cache, page, 9)
    want = nv.paged_attention(q, kc, vc, table, ln, k_scale=ks, v_scale=vs)
    for window in (2 ** 31 - 1, 2 ** 31 - rows, 1 << 24, 300):
        got = nv.paged_attention(q, kc, vc, table, ln, window=window, k_scale=ks, v_scale=vs)
        assert torch.equal(got, want), window
    assert nv.device_status() == 0


# ------------------------------------------------------------- what a row does not see, finite

@pytest.mark.parametrize("window", [0, 24])
@pytest.mark.parametrize("rows,D", [(4, 128), (8, 64), (2, 256)])
@pytest.mark.parametrize("value", [3e38, -3e38])
def test_huge_values_behind_the_mask_do_not_reach_a_row(rows, D, window, value):
    # the newest key (and, with a window, old ones) hold the largest values: rows that do not see them
    # are, bit for bit, as without
    n, page, hk = 61, 16, 2
    q, kc, vc, table, ln, _, _ = _attend_inputs([n], rows, 8, hk, D, BF16, page, 21)
    clean = nv.paged_attention(q, kc, vc, table, ln, window=window)
    old = [n - 1] + ([n - rows - 23, n - 26] if window else [])
    for j in old:
        vc[int(table[0, j // page]), :, j % page] = value
    got = nv.paged_attention(q, kc, vc, table, ln, window=window)
    for r in range(rows):
        at = n - rows + r
        if not any(j <= at and (not window or j > at - window) for j in old):
            assert torch.equal(got[r], clean[r]), (r, float((got[r].float() - clean[r].float()).abs().max()))
    assert nv.device_status() == 0


def test_huge_values_under_a_vanished_weight():
    # a key 200 nats below the others weighs e^-200 = 0 in fp32, and 3e38 times that is nothing
    n, D = 40, 64
    q, kc, vc, table, ln, _, _ = _attend_inputs([n], 1, 2, 1, D, BF16, 16, 5)
    q.fill_(1.0)
    p, s = int(table[0, 1]), 4
    kc[p, 0, s] = -25.0  # -25 * 64 / 8 = -200
    vc[p, 0, s] = 3e38
    got = nv.paged_attention(q, kc, vc, table, ln)
    vc[p, 0, s] = 0.0
    assert torch.equal(got, nv.paged_attention(q, kc, vc, table, ln))


# --------------------------------------------------------------------- weights far below the largest

@pytest.mark.parametrize("cache", [BF16, FP8])
@pytest.mark.parametrize("rows,group,D", [(1, 4, 128), (4, 1, 64), (8, 4, 128), (2, 1, 256)])
def test_a_long_tail_behind_one_heavy_key(cache, rows, group, D):
    # one key outweighs each other by 2^26 and holds zeros: the output is the tail's alone. So many items that a
    # warp takes a good part of one. A weight is off by 2^-15 of itself (two bf16 numbers) or 2^-11
    # (f16), and, f16, by half a step of 2^-24 where the largest is at least 2^7: 2^-32 of the largest.
    n, page, hk, seqs = 4000, 16, 64, 8
    g = _gen(n + D + rows)
    kc, vc = nv.kv_cache(n // page, hk, page, D, cache)
    kc.copy_((_randn(kc.shape, g) * 0.02).to(cache))
    vc.copy_((0.5 + torch.rand(vc.shape, generator=g, device=DEV)).to(cache))
    kc[0, :, 5] = torch.full((D,), 18.0 / D ** 0.5, device=DEV).to(cache)  # 26 log 2 = 18.02
    vc[0, :, 5] = torch.zeros(D, device=DEV).to(cache)
    q = torch.ones((seqs * rows, hk * group, D), dtype=BF16, device=DEV)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV).expand(seqs, -1)
    ln = torch.full((seqs,), n, dtype=torch.int32, device=DEV)
    lse = torch.empty((seqs * rows, hk * group), device=DEV)
    got = nv.paged_attention(q, kc, vc, table, ln, lse=lse)
    assert nv.device_status() == 0
    got, lse = got.view(seqs, rows, hk, group, D), lse.view(seqs, rows, hk, group)
    keys, vals = (c.double().transpose(0, 1).reshape(hk, n, D) for c in (kc, vc))
    for r in range(rows):
        hi = n - rows + r + 1
        z = keys[:, :hi].sum(dim=2) * D ** -0.5  # every query is ones
        p = torch.softmax(z, 1)
        ref = torch.einsum("hk,hkd->hd", p, vals[:, :hi])  # no value is below zero: also the sum of magnitudes
        # fp32 dot products, and at most hi / 16 terms of a sum in a row
        dz = float((D + 8) * U32 * keys[:, :hi].abs().sum(dim=2).max() * D ** -0.5) + float(z.abs().max()) * 4 * U32
        tol = ref * (U16 + 2 * dz + (2.0 ** -15 if cache is BF16 else 2.0 ** -11) + (hi / 16 + 16) * U32)
        if cache is FP8:
            tol = tol + 2.0 ** -32 * vals[:, :hi].sum(dim=1)
        _within(got[:, r], ref[None, :, None].expand(seqs, -1, group, -1), tol[None, :, None], "out")
        want = torch.logsumexp(z, dim=1)[None, :, None].expand(seqs, -1, group)
        _within(lse[:, r], want, dz + (hi / 16 + 16) * U32 + want.abs() * 4 * U32, "lse")


# ------------------------------------------------------------------- CTAs that take several items

@pytest.mark.parametrize("cache", [BF16, FP8])
@pytest.mark.parametrize("rows,hq,hk,D", [(1, 8, 8, 128), (4, 32, 8, 128), (8, 32, 8, 128), (8, 16, 8, 64), (1, 8, 8, 64),
                                          (4, 16, 8, 256), (8, 40, 4, 128), (3, 64, 4, 96)])
def test_ctas_that_walk_through_items(cache, rows, hq, hk, D):
    # more (sequence, kv head) items than whole ones fit the CTAs, of unequal lengths: runs begin and end
    # inside items, and a CTA's rings, query rows and joins follow one another; up to 32 sequences
    # and beyond take their schedule on different ways
    for seqs in (32, 33):
        _check_attend([(1000 + 397 * i) % 2100 for i in range(seqs)], rows, hq, hk, D, cache, 32 if seqs == 32 else 16, seed=rows + D)


@pytest.mark.parametrize("cache", [BF16, FP8])
@pytest.mark.parametrize("rows", [1, 8])
def test_ctas_that_walk_through_windows(cache, rows):
    _check_attend([(500 + 1237 * i) % 5000 for i in range(30)], rows, 32, 8, 128, cache, 16, window=1500, seed=rows)


# ---------------------------------------------------------------------------------- 8-bit appends

@pytest.mark.parametrize("variant", [0, 1])
def test_appended_codes_are_the_quotients(variant):
    # values at and beside the middle of two codes, where a quotient off by a unit takes the other one; scales
    # down to the smallest
    g = _gen(77)
    T, hk, D = 64, 16, 128
    scale = torch.rand(hk, generator=g, device=DEV) * 0.9 + 0.05
    scale[3], scale[7] = 2.0 ** -126, 2.0 ** -140
    mid = torch.tensor([(8 + m + 0.5) / 8 * 2.0 ** e for m in range(8) for e in range(-6, 8)], device=DEV)
    x = mid[torch.randint(len(mid), (T, hk, D), generator=g, device=DEV)] * scale[:, None]
    kc, vc = nv.kv_cache(4, hk, 16, D, FP8)
    table = torch.arange(4, dtype=torch.int32, device=DEV)[None]
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    nv.set_variant(variant)
    try:
        nv.rope_append(None, x, -x, pos, torch.empty(0, device=DEV), kc, vc, table, k_scale=scale, v_scale=scale)
    finally:
        nv.set_variant(0)
    want = (x / scale[:, None]).clamp(-448, 448)
    for c, ref in ((kc, want), (vc, -want)):
        rows = c.transpose(1, 2).reshape(T, hk, D)
        assert torch.equal(rows.view(torch.uint8), ref.to(FP8).view(torch.uint8)), int((rows.float() != ref.to(FP8).float()).sum())
    assert nv.device_status() == 0


# ------------------------------------------------------------------------------------ other streams

def _owner(t):
    """The stream whose memory pool a tensor's block belongs to."""
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


@pytest.mark.parametrize("handle", [False, True])
def test_a_call_on_another_stream_does_not_use_the_current_one(handle):
    # the current stream is busy and its pool's free blocks are full of ones: a workspace zeroed there would be
    # ready after the kernel on the side stream had counted in it
    q, kc, vc, table, ln, _, _ = _attend_inputs([3000, 30], 1, 8, 2, 128, BF16, 16, 7)
    x, r, w = q.view(2, -1), q.view(2, -1).clone(), torch.ones(1024, device=DEV)
    pos, freq = ln - 1, torch.empty(0, device=DEV)
    k = q[:, :2].contiguous()
    want = nv.paged_attention(q, kc, vc, table, ln)
    normed = nv.rms_norm(x, w, residual=r, out_dtype=FP8)
    nv.rope_append(q, k, k, pos, freq, kc.clone(), vc.clone(), table)  # a kernel's first launch may wait for the device
    side = torch.cuda.Stream()
    on = side.cuda_stream if handle else side
    torch.cuda.synchronize()
    n = nv.attention_workspace_bytes(2, 1, 8, 2, 128)
    blocks = [torch.full((n,), 0xff, dtype=torch.uint8, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    del blocks
    torch.cuda._sleep(200_000_000)  # 0.1 s of the current stream
    got = nv.paged_attention(q, kc, vc, table, ln, stream=on)
    norm2 = nv.rms_norm(x, w, residual=r, out_dtype=FP8, stream=on)
    turned = nv.rope_append(q, k, k, pos, freq, kc, vc, table, stream=on)
    side.synchronize()
    assert not torch.cuda.current_stream().query(), "waited for the current stream"
    for t in (got, *norm2, turned):
        assert _owner(t) == side.cuda_stream
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.equal(turned, q)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(norm2, normed))
    assert nv.device_status() == 0


def test_a_call_on_another_stream_keeps_what_it_is_given():
    q, kc, vc, table, ln, _, _ = _attend_inputs([300, 30], 1, 8, 2, 128, BF16, 16, 7)
    want = nv.paged_attention(q, kc, vc, table, ln)
    side, ws = torch.cuda.Stream(), nv.attention_workspace(2, 1, 8, 2, 128)
    torch.cuda.synchronize()
    for kw in (dict(), dict(workspace=ws), dict(out=torch.empty_like(q)), dict(workspace=ws, out=torch.empty_like(q))):
        got = nv.paged_attention(q, kc, vc, table, ln, stream=side, **kw)
        side.synchronize()
        assert torch.equal(got, want) and (got is kw["out"] if "out" in kw else _owner(got) == side.cuda_stream)
    got = nv.paged_attention(q, kc, vc, table, ln, stream=0)  # the default stream's handle
    torch.cuda.synchronize()
    assert torch.equal(got, want) and _owner(got) == 0


# ---------------------------------------------------------------------------------------- refusals

def test_rope_append_refuses_what_has_no_truth_value():
    k = torch.ones((2, 2, 64), device=DEV)
    kc, vc = nv.kv_cache(2, 2, 16, 64)
    table = torch.zeros((1, 1), dtype=torch.int32, device=DEV)
    pos, freq = torch.tensor([0, 1], dtype=torch.int32, device=DEV), torch.ones(32, device=DEV)
    with pytest.raises(RuntimeError, match="ambiguous"):
        nv.rope_append(None, k, k, pos, freq, kc, vc, table, interleaved=torch.tensor([True, False]))
    torch.cuda.synchronize()
    assert not kc.any() and not vc.any()


def test_scales_next_to_a_bf16_cache_are_refused():
    q, kc, vc, table, ln, _, _ = _attend_inputs([5, 6], 1, 4, 2, 64, BF16, 16, 8)
    one = torch.ones(2, device=DEV)
    for kw in (dict(k_scale=one), dict(v_scale=one)):
        with pytest.raises(ValueError, match="float8"):
            nv.paged_attention(q, kc, vc, table, ln, **kw)
        with pytest.raises(ValueError, match="float8"):
            nv.rope_append(q, q[:, :2], q[:, :2], ln - 1, torch.ones(32, device=DEV), kc, vc, table, **kw)


# ------------------------------------------------------------------------------ nothing cached yet

@pytest.mark.parametrize("pages,max_pages", [(0, 0), (0, 3), (4, 0)])
@pytest.mark.parametrize("cache", [BF16, FP8])
def test_an_empty_cache_or_table(pages, max_pages, cache):
    D, ws = 64, nv.attention_workspace(2, 2, 4, 2, 64)
    kc, vc = nv.kv_cache(pages, 2, 16, D, cache)
    table = torch.zeros((2, max_pages), dtype=torch.int32, device=DEV)
    q, ln = torch.ones((4, 4, D), dtype=BF16, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV)
    lse = torch.full((4, 4), math.nan, device=DEV)
    out = nv.paged_attention(q, kc, vc, table, ln, workspace=ws, lse=lse)
    assert not out.any() and bool((lse == -math.inf).all()) and nv.device_status() == 0
    # padding is appended nowhere, a token without a place is reported
    k, freq = torch.ones((2, 2, D), dtype=BF16, device=DEV), torch.ones(32, device=DEV)
    for at, status in ((-1, 0), (0, nv.DEV_BAD_PAGE)):
        pos = torch.full((2,), at, dtype=torch.int32, device=DEV)
        nv.rope_append(q[:2], k, k, pos, freq, kc, vc, table)
        assert nv.device_status() == status
    assert not kc.float().any() and not vc.float().any()


# ---------------------------------------------------------------------- precision of the weights

@pytest.mark.parametrize("cache", [BF16, FP8])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_weights_carry_their_bits(D, cache):
    # two keys of nearly the same score with values 1 and -1: the output, (1 - e) / (1 + e) for a weight e of the
    # second, is a small difference that shows e's own rounding, 2^-16 (two bf16 numbers) or 2^-12 (f16) at most
    H = 64
    kc, vc = nv.kv_cache(1, 1, 16, D, cache)
    kc[0, 0, :2, 0] = torch.tensor([1.0, 0.875], device=DEV).to(cache)
    vc[0, 0, 0], vc[0, 0, 1] = (torch.full((D,), v, device=DEV).to(cache) for v in (1.0, -1.0))
    q = torch.zeros((1, H, D), dtype=BF16, device=DEV)
    q[0, :, 0] = torch.linspace(0.05, 0.4, H, device=DEV).to(BF16)
    table, ln = torch.zeros((1, 1), dtype=torch.int32, device=DEV), torch.full((1,), 2, dtype=torch.int32, device=DEV)
    got = nv.paged_attention(q, kc, vc, table, ln, 1.0)[0].double()
    e = torch.exp(-0.125 * q[0, :, 0].double())[:, None]
    ref = (1 - e) / (1 + e)
    # an error x of e moves the output by 2 x / (1 + e)^2 < 0.6 x; scores and exp2 are good to 2^-21
    bits = 16 if cache is BF16 else 12
    tol = ref * U16 / 2 + 0.6 * (2.0 ** -bits + 2.0 ** -21)
    _within(got, ref.expand(-1, D), tol)
    # what one bf16 number a weight would give is outside
    rough = e.to(BF16).double()
    off = ((1 - rough) / (1 + rough) - ref).abs()
    assert bool((off > tol).any())


@pytest.mark.parametrize("cache", [BF16, FP8])
@pytest.mark.parametrize("rows,hq,hk,window", [(1, 8, 2, 0), (4, 8, 1, 0), (3, 4, 2, 70000)])
def test_a_long_context(cache, rows, hq, hk, window):
    _check_attend([131071, 40000], rows, hq, hk, 128, cache, 64, window=window, seed=rows)


# ------------------------------------------------------------------------------------ 8-bit norms

@pytest.mark.parametrize("pitch", [0, 3])
@pytest.mark.parametrize("rows,cols,group", [(4096, 4096, 128), (4096, 4096, 0), (3, 4096, 16), (60, 30016, 0)])
def test_normed_codes_are_the_quotients(rows, cols, group, pitch):
    # the same rows in fp32, divided by the scales that came with the codes; both kernels
    g = _gen(rows + cols + group)
    x = _randn((rows, cols + pitch), g)[:, pitch:]
    w = 1 + 0.2 * _randn((cols,), g)
    got = nv.rms_norm(x, w, out_dtype=FP8, group=group)
    y = nv.rms_norm(x, w, out_dtype=torch.float32).y.view(rows, -1, group or cols)
    top = y.abs().amax(dim=2).double() / 448
    _within(got.scales, top, top * 2 * U32, "scales")  # 1 / 448 is rounded, and the product
    want = (y / got.scales[..., None]).to(FP8).view(rows, cols)
    assert torch.equal(got.y.view(torch.uint8), want.view(torch.uint8)), int((got.y.float() != want.float()).sum())


def test_normed_codes_beside_infinities():
    # a weight that overflows one value: the row's scale is infinite, what is finite over it is zero
    x, w = torch.ones((2, 64), device=DEV), torch.ones(64, device=DEV)
    x[1] = 2.0 ** 40
    w[5] = 3e38
    x[:, 5] = 2 * x[:, 5]
    for cols in (64, 63):
        got = nv.rms_norm(x[:, :cols].contiguous(), w[:cols].contiguous(), 0.0, out_dtype=FP8)
        y = nv.rms_norm(x[:, :cols].contiguous(), w[:cols].contiguous(), 0.0, out_dtype=torch.float32).y
        want = (y / got.scales).to(FP8).float()
        assert bool(torch.isinf(got.scales).all()) and bool(torch.isinf(y[:, 5]).all())
        assert torch.equal(torch.isnan(got.y.float()), torch.isnan(want)) and torch.equal(got.y.float().nan_to_num(), want.nan_to_num())
