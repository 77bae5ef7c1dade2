"""Serving operators on a B200 against plain binary64 forms: rotary positions,
the append to a paged cache, attention over it and the join of two partial
results, each within the bounds derived in serving_util; then the whole run of
them beside the codec."""
import math

import numpy as np
import pytest
import torch

import oracle
from kv_quantization_tile_b200 import hq
from serving_util import (U32, assert_within, attend, make_cache, randn, rotate, rotate_tolerance, starts, theta_of)

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
YARN = {"kind": "yarn", "factor": 16.0, "slow": 1.0, "fast": 32.0, "original": 4096}
BANDS = {"kind": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "original": 8192}


def i32(*v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def new_status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ----------------------------------------------------------------- rotation
@pytest.mark.parametrize("d,r", [(64, 64), (128, 128), (128, 32), (256, 256), (256, 16), (80, 48), (16, 16)])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("din,dout", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("tokens,heads,scaling", [(1, 1, None), (37, 5, YARN)])
def test_rope(d, r, layout, din, dout, tokens, heads, scaling):
    x = randn(tokens, heads, d, seed=d + r, dtype=din)
    pos = torch.randint(-1000, 200000, (tokens,), generator=torch.Generator().manual_seed(3))
    y = torch.full((tokens, heads, d), float("nan"), dtype=dout, device=DEV)
    hq.hq_rope(x.to(DEV), pos.to(DEV), hq.rope_table(r, 500000.0, scaling, layout), y)
    theta, amp = theta_of(r, 500000.0, scaling)
    ref = rotate(x, pos, theta, amp, layout)
    assert_within(y, ref, rotate_tolerance(x, ref, theta, amp, layout, pos, dout))


def test_rope_many_tokens_and_heads_take_the_wide_blocks():
    x = randn(2377, 3, 64, seed=5)
    pos = torch.arange(2377)
    y = torch.empty_like(x, device=DEV)
    hq.hq_rope(x.to(DEV), pos.to(DEV), hq.rope_table(64), y)
    theta, amp = theta_of(64, 10000.0)
    ref = rotate(x, pos, theta, amp, "half")
    assert_within(y, ref, rotate_tolerance(x, ref, theta, amp, "half", pos, BF))


def test_rope_far_positions_keep_their_angle():
    """At positions around 2^31 a binary32 angle would be off by radians; the
    reference takes the angle from exact integers, 50 digits."""
    import mpmath
    mpmath.mp.dps = 50
    pos = torch.tensor([2 ** 31 - 1, -(2 ** 31), 2 ** 30 + 7, 123456789])
    x = randn(4, 2, 64, seed=1, dtype=F32)
    y = torch.empty_like(x, device=DEV)
    theta, amp = theta_of(64, 10000.0)
    hq.hq_rope(x.to(DEV), pos.to(DEV), hq.rope_table(64), y)
    ref = x.double().clone()
    for t, p in enumerate(pos.tolist()):
        for i, th in enumerate(theta):
            a = mpmath.mpf(p) * mpmath.mpf(float(th))
            c, s = float(mpmath.cos(a)), float(mpmath.sin(a))
            x1, x2 = x[t, :, i].double(), x[t, :, i + 32].double()
            ref[t, :, i], ref[t, :, i + 32] = x1 * c - x2 * s, x2 * c + x1 * s
    # theta / 2 pi is rounded to 2^-64 turns and a few 2^-64 of itself: 2^31
    # positions turn that into 2^-30 turns, 6e-9 radians
    mag = x.double().abs()
    tol = torch.cat([mag[..., :32] + mag[..., 32:]] * 2, -1) * (10 * U32 + 2e-8) + U32 * ref.abs()
    assert_within(y, ref, tol)


@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rope_strides_and_in_place(layout):
    qkv = randn(33, 12 * 64, seed=9).to(DEV)
    x = qkv[:, 64:64 * 6].view(33, 5, 64)  # some heads of a fused projection
    pos = torch.arange(33, device=DEV) * 31
    table = hq.rope_table(64, layout=layout)
    before = qkv.clone()
    dense = torch.empty(33, 5, 64, dtype=BF, device=DEV)
    hq.hq_rope(x, pos, table, dense)
    by_head = torch.zeros(5, 33, 64, dtype=BF, device=DEV)  # [heads, tokens, d]
    hq.hq_rope(x, pos, table, by_head.transpose(0, 1))
    assert torch.equal(by_head.transpose(0, 1), dense)
    one = x[:, :1].expand(33, 4, 64)  # one head read four times
    four = torch.empty(33, 4, 64, dtype=BF, device=DEV)
    hq.hq_rope(one, pos, table, four)
    assert all(torch.equal(four[:, h], dense[:, 0]) for h in range(4))
    assert torch.equal(qkv, before)
    hq.hq_rope(x, pos, table, x)
    assert torch.equal(x, dense)
    x.copy_(before[:, 64:64 * 6].view(33, 5, 64))
    assert torch.equal(qkv, before)  # nothing beside the heads was written


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling", [None, YARN])
def test_rope_inverse_is_the_gradient(layout, scaling):
    """Against autograd of the formula in binary64, and against differences of
    the forward kernel (linear: (f(x + h e) - f(x)) / h has no truncation error,
    only the outputs' roundings, 2 * 12 U32 amp (|x1| + |x2| + h) / h)."""
    x, dy = randn(7, 3, 64, seed=2, dtype=F32), randn(7, 3, 64, seed=3, dtype=F32)
    pos = torch.tensor([0, 1, 5, 100, 4095, 70000, 1000000])
    theta, amp = theta_of(64, 10000.0, scaling)
    table = hq.rope_table(64, scaling=scaling, layout=layout)
    dx = torch.empty_like(x, device=DEV)
    hq.hq_rope(dy.to(DEV), pos.to(DEV), table, dx, inverse=True)
    xr = x.double().requires_grad_()
    a = pos.double()[:, None, None] * torch.as_tensor(theta)
    c, s = amp * torch.cos(a), amp * torch.sin(a)
    i1, i2 = (slice(0, 32), slice(32, 64)) if layout == "half" else (slice(0, 64, 2), slice(1, 64, 2))
    y = torch.zeros(7, 3, 64, dtype=torch.float64)
    y[..., i1] = xr[..., i1] * c - xr[..., i2] * s
    y[..., i2] = xr[..., i2] * c + xr[..., i1] * s
    y.backward(dy.double())
    assert_within(dx, xr.grad, rotate_tolerance(dy, xr.grad, theta, amp, layout, pos, F32))
    h = 8.0
    for i in (0, 1, 31, 32, 63):
        xp = x.clone()
        xp[..., i] += h
        y0, y1 = torch.empty_like(x, device=DEV), torch.empty_like(x, device=DEV)
        hq.hq_rope(x.to(DEV), pos.to(DEV), table, y0)
        hq.hq_rope(xp.to(DEV), pos.to(DEV), table, y1)
        diff = ((y1.double() - y0.double()).cpu() * dy.double()).sum(-1) / h
        bound = 24 * U32 * amp * ((x.abs().max() * 2 + h) / h).double() * dy.double().abs().sum(-1) * 2
        assert ((diff - dx[..., i].double().cpu()).abs() <= bound).all()


# ----------------------------------------------------------------- append
@pytest.mark.parametrize("d,page,kvh,qh", [(128, 16, 2, 8), (64, 64, 3, 0), (256, 128, 1, 5)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("slot_major", [False, True])
@pytest.mark.parametrize("rotated", [False, True])
def test_append(d, page, kvh, qh, dtype, slot_major, rotated):
    tokens, pages = 29, 5
    qkv = randn(tokens, (qh + 2 * kvh) * d, seed=d, dtype=dtype).to(DEV)
    q = qkv[:, :qh * d].view(tokens, qh, d)
    k = qkv[:, qh * d:(qh + kvh) * d].view(tokens, kvh, d)
    v = qkv[:, (qh + kvh) * d:].view(tokens, kvh, d)
    shape = (pages, page, kvh, d) if slot_major else (pages, kvh, page, d)
    kp, vp = randn(*shape, seed=50).to(DEV), randn(*shape, seed=51).to(DEV)
    if slot_major:
        kp, vp = kp.permute(0, 2, 1, 3), vp.permute(0, 2, 1, 3)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(4))[:tokens]
    slots[3] = -1  # padding tokens
    slots[7] = -5
    slots[11] = pages * page  # past the pool: skipped and reported
    slots[12] = 2 ** 60
    pos = torch.arange(tokens) * 977
    q_out = torch.full((tokens, qh, d), 7.0, dtype=BF, device=DEV)
    r, theta, amp, layout = d, *theta_of(d, 500000.0, BANDS), "interleaved"
    table = hq.rope_table(r, 500000.0, BANDS, layout) if rotated else None
    k0, v0 = kp.cpu().clone(), vp.cpu().clone()
    st = new_status()
    hq.hq_kv_append(k, v, slots.to(DEV), hq.Pages(kp, vp), positions=pos.to(DEV) if rotated else None, rope=table,
                    q=q if qh else None, q_out=q_out if qh else None, status=st)
    assert int(st) == hq.HQ_ST_INDEX
    turn = (lambda x: rotate(x, pos, theta, amp, layout)) if rotated else lambda x: x.double().cpu()
    tol = (lambda x, ref: rotate_tolerance(x, ref, theta, amp, layout, pos, BF)) if rotated \
        else (lambda x, ref: 2.0 ** -8 * ref.abs())
    kr, vr, qr = turn(k), v.double().cpu(), turn(q)
    tk, tq = tol(k, kr), tol(q, qr) if qh else None
    want_k, want_v = k0.double(), v0.double()
    tol_k, tol_v = torch.zeros_like(want_k), torch.zeros_like(want_v)
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            want_k[s // page, :, s % page], tol_k[s // page, :, s % page] = kr[t], tk[t]
            want_v[s // page, :, s % page], tol_v[s // page, :, s % page] = vr[t], 2.0 ** -8 * vr[t].abs()
        elif qh:
            assert (q_out[t] == 7.0).all()  # a skipped token's query is left as it was
    assert_within(kp, want_k, tol_k)
    assert_within(vp, want_v, tol_v)
    if qh:
        kept = (slots >= 0) & (slots < pages * page)
        assert_within(q_out[kept.to(DEV)], qr[kept], tq[kept])


def test_append_without_tokens_and_status():
    pool = hq.alloc_pages(2, 16, 2, 64)
    x = torch.empty(0, 2, 64, dtype=BF, device=DEV)
    hq.hq_kv_append(x, x, torch.empty(0, dtype=torch.int64, device=DEV), pool)
    x = torch.ones(1, 2, 64, dtype=BF, device=DEV)
    hq.hq_kv_append(x, x, torch.tensor([99], device=DEV), pool)  # out of the pool, nobody asked
    torch.cuda.synchronize()


# ----------------------------------------------------------------- attention
def run_attention(q_lens, kv_lens, kvh, group, d, page, causal=True, window=0, scale=None, seed=0, behind=2,
                  slot_major=False, k_scale=1.0, max_q=None, max_kv=None, out_dtype=BF, stale=float("nan")):
    kp, vp, table, K, V = make_cache(kv_lens, kvh, d, page, seed, slot_major=slot_major, k_scale=k_scale, stale=stale)
    heads, n = kvh * group, sum(q_lens)
    q = randn(n + behind, heads, d, seed=seed + 77)
    scale = d ** -0.5 if scale is None else scale
    max_q = max(q_lens) if max_q is None else max_q
    max_kv = max(kv_lens) if max_kv is None else max_kv
    out = torch.full((n + behind, heads, d), 3.0, dtype=out_dtype, device=DEV)
    lse = torch.full((n + behind, heads), 5.0, device=DEV)
    ws = hq.alloc_paged_attention_workspace(len(q_lens), n + behind, max_q, max_kv, kvh, group, d)
    ws.fill_(255)
    st = new_status()
    hq.hq_paged_attention(q.to(DEV), starts(q_lens).to(DEV), torch.tensor(kv_lens, dtype=torch.int32, device=DEV),
                          hq.Pages(kp.to(DEV), vp.to(DEV)), table.to(DEV), scale, out, ws, max_q=max_q, max_kv=max_kv,
                          causal=causal, window=window, lse=lse, status=st)
    assert int(st) == 0
    ref, ref_lse, tol_b, tol_f, tol_l = attend(q[:n], K, V, q_lens, scale, causal, window)
    assert_within(out[:n], ref, tol_b if out_dtype == BF else tol_f, "out")
    assert_within(lse[:n], ref_lse, tol_l, "lse")
    assert (out[n:] == 3.0).all() and (lse[n:] == 5.0).all()  # rows behind the last sequence


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 3, 4, 8])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_attention_single_tokens(d, group, page):
    run_attention([1, 1, 1, 1, 1], [1, 17, 63, 300, 1029], 2, group, d, page, seed=d + group)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens", [([3, 7, 1], [3, 200, 65]), ([5, 20], [130, 20]), ([40, 2, 17], [40, 700, 90])])
@pytest.mark.parametrize("group", [1, 4])
def test_attention_drafts(d, q_lens, kv_lens, group):
    run_attention(q_lens, kv_lens, 2, group, d, 32, seed=d + group)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens", [([130], [130]), ([257, 1, 33], [513, 77, 900]), ([64, 300, 5], [64, 301, 700])])
@pytest.mark.parametrize("group,page", [(1, 16), (4, 64), (3, 128), (8, 256)])
def test_attention_chunks(d, q_lens, kv_lens, group, page):
    run_attention(q_lens, kv_lens, 2, group, d, page, seed=d + group)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [400, 30]), ([9, 2], [300, 10]), ([200, 150], [600, 150])])
@pytest.mark.parametrize("window", [1, 5, 64, 129, 100000])
def test_attention_window(d, q_lens, kv_lens, window):
    run_attention(q_lens, kv_lens, 1, 4, d, 16, window=window, seed=window)


@pytest.mark.parametrize("q_lens,max_kv,window", [([1, 1], 16384, 16382), ([1, 1], 16384, (1 << 63) - 1),
                                                  ([150, 2], 4096, (1 << 63) - 1), ([150, 2], 4096, 1 << 31)])
def test_attention_windows_about_the_bounds(q_lens, max_kv, window):
    run_attention(q_lens, [400, 77], 8, 4, 128, 64, window=window, max_kv=max_kv)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 4], [90, 33]), ([100, 70], [300, 20])])
@pytest.mark.parametrize("window", [0, 40])
def test_attention_without_causal_mask(q_lens, kv_lens, window):
    run_attention(q_lens, kv_lens, 2, 2, 128, 16, causal=False, window=window)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens", [([0, 1, 0, 2], [5, 0, 0, 1]), ([4, 1], [2, 0]), ([150, 0, 140], [3, 9, 0])])
def test_attention_rows_that_see_nothing(d, q_lens, kv_lens):
    """No cached token, more new tokens than cached ones, empty sequences."""
    run_attention(q_lens, kv_lens, 2, 2, d, 16, max_kv=16)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2], [300, 70]), ([140], [300])])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-6, 3.0])
def test_attention_scales(q_lens, kv_lens, scale):
    run_attention(q_lens, kv_lens, 2, 2, 128, 32, scale=scale)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens", [[1, 6], [160, 90]])
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_attention_peaked_scores_move_the_maximum(d, q_lens, out_dtype):
    """Scores of +-hundreds: the running maximum jumps many times."""
    run_attention(q_lens, [700, 410], 1, 4, d, 16, k_scale=16.0, out_dtype=out_dtype)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens", [[1], [70]])
def test_attention_keys_that_grow_along_the_sequence(d, q_lens):
    """Each later key scores higher, so every tile raises the maximum."""
    kv, page = 900, 16
    kp, vp, table, K, V = make_cache([kv], 1, d, page, 3)
    ramp = torch.arange(kv).view(-1, 1, 1) * 0.02
    K[0] = (torch.ones(kv, 1, d) * ramp).to(BF)
    for i in range(-(-kv // page)):
        m = min(page, kv - i * page)
        kp[int(table[0, i]), :, :m] = K[0][i * page:i * page + m].transpose(0, 1)
    q = torch.ones(sum(q_lens), 2, d, dtype=BF)
    out, lse = torch.empty_like(q, device=DEV), torch.empty(sum(q_lens), 2, device=DEV)
    ws = hq.alloc_paged_attention_workspace(1, q.shape[0], q.shape[0], kv, 1, 2, d)
    hq.hq_paged_attention(q.to(DEV), starts(q_lens).to(DEV), i32(kv), hq.Pages(kp.to(DEV), vp.to(DEV)), table.to(DEV),
                          0.5, out, ws, max_q=q.shape[0], max_kv=kv, lse=lse)
    ref, ref_lse, tol, _, tol_l = attend(q, K, V, q_lens, 0.5)
    assert_within(out, ref, tol)
    assert_within(lse, ref_lse, tol_l)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 3], [500, 129]), ([150], [333])])
@pytest.mark.parametrize("stale", [float("inf"), -float("inf"), torch.finfo(BF).min])
def test_attention_ignores_what_stale_slots_hold(q_lens, kv_lens, stale):
    run_attention(q_lens, kv_lens, 2, 2, 128, 64, stale=stale)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2], [300, 70]), ([140, 20], [300, 64])])
def test_attention_slot_major_pages(q_lens, kv_lens):
    run_attention(q_lens, kv_lens, 3, 2, 128, 16, slot_major=True)


def test_attention_long_sequence_over_many_blocks():
    run_attention([1], [20011], 1, 4, 128, 16, seed=5)
    run_attention([9], [9001], 1, 2, 64, 64, seed=6)
    run_attention([1, 1, 1], [5000, 3, 12345], 2, 8, 256, 128, seed=7)
    run_attention([129], [5003], 1, 4, 128, 32, seed=8)


@pytest.mark.parametrize("d,longest", [(64, 17001), (128, 9001), (256, 4500)])
@pytest.mark.parametrize("q,group", [(1, 3), (2, 16), (6, 8)])
def test_attention_shares_that_cut_jobs(d, longest, q, group):
    """Too many jobs for clusters and one long sequence: blocks take equal shares
    of the tiles, and jobs cut between blocks are joined (16, 32 and 64 rows)."""
    run_attention([q] * 20, [longest] + [50 + 37 * i for i in range(19)], 2, group, d, 64, seed=d + q)


@pytest.mark.parametrize("d,kv", [(64, 17001), (128, 9001), (256, 4500)])
def test_attention_shares_repeat_bit_for_bit(d, kv):
    n = 20
    kv_lens = [kv] + [70] * (n - 1)
    kp, vp, table, _, _ = make_cache(kv_lens, 2, d, 128, 2)
    q = randn(n, 8, d, seed=1).to(DEV)
    pool = hq.Pages(kp.to(DEV), vp.to(DEV))
    ws = hq.alloc_paged_attention_workspace(n, n, 1, kv, 2, 4, d)
    got = []
    for fill in (0, 255, None, None):
        if fill is not None:
            ws.fill_(fill)
        out, lse = torch.empty_like(q), torch.empty(n, 8, device=DEV)
        hq.hq_paged_attention(q, starts([1] * n).to(DEV), i32(*kv_lens), pool, table.to(DEV), 0.09, out, ws, max_q=1,
                              max_kv=kv, lse=lse)
        got.append((out, lse))
    assert all(torch.equal(o, got[0][0]) and torch.equal(s, got[0][1]) for o, s in got)


def test_attention_many_sequences():
    """More sequences than one pass of the plan counts, lengths 0 to 40."""
    n = 1500
    run_attention([1] * n, [i % 41 for i in range(n)], 1, 2, 64, 16, max_kv=40)


def test_attention_bounds_wider_than_the_lengths():
    run_attention([3, 1], [50, 20], 2, 4, 128, 16, max_q=100, max_kv=48 + 16)
    run_attention([130, 1], [150, 20], 2, 4, 128, 16, max_q=2000, max_kv=160)


@pytest.mark.parametrize("d,q_lens", [(128, [1, 9]), (64, [200, 3]), (128, [200, 3]), (256, [200, 3])])
def test_attention_strided_rows(d, q_lens):
    """Queries inside a fused projection, outputs by head."""
    kv_lens = [300, 77]
    kp, vp, table, K, V = make_cache(kv_lens, 2, d, 16, 1)
    n, heads = sum(q_lens), 6
    fused = randn(n, (heads + 4) * d, seed=8).to(DEV)
    q = fused[:, 2 * d:(heads + 2) * d].view(n, heads, d)
    by_head = torch.zeros(heads, n, d, dtype=BF, device=DEV)
    ws = hq.alloc_paged_attention_workspace(2, n, max(q_lens), 300, 2, 3, d)
    hq.hq_paged_attention(q, starts(q_lens).to(DEV), i32(*kv_lens), hq.Pages(kp.to(DEV), vp.to(DEV)), table.to(DEV),
                          d ** -0.5, by_head.transpose(0, 1), ws, max_q=max(q_lens), max_kv=300)
    ref, _, tol, _, _ = attend(q, K, V, q_lens, d ** -0.5)
    assert_within(by_head.transpose(0, 1), ref, tol)


@pytest.mark.parametrize("q_lens", [[1, 1], [150, 130]])
def test_attention_shared_pages(q_lens):
    """Two sequences over the same pages (a common prefix) get the rows of one each."""
    kp, vp, table, K, V = make_cache([320], 2, 128, 16, 4)
    table = table.repeat(2, 1)
    q = randn(sum(q_lens), 4, 128, seed=2)
    kv = [320, 200]
    out = torch.empty_like(q, device=DEV)
    ws = hq.alloc_paged_attention_workspace(2, q.shape[0], max(q_lens), 320, 2, 2, 128)
    hq.hq_paged_attention(q.to(DEV), starts(q_lens).to(DEV), i32(*kv), hq.Pages(kp.to(DEV), vp.to(DEV)), table.to(DEV),
                          0.1, out, ws, max_q=max(q_lens), max_kv=320)
    ref, _, tol, _, _ = attend(q, [K[0], K[0][:200]], [V[0], V[0][:200]], q_lens, 0.1)
    assert_within(out, ref, tol)


@pytest.mark.parametrize("d,q_lens", [(128, [1, 1]), (64, [150, 2]), (256, [150, 2])])
@pytest.mark.parametrize("bad", [-1, 1 << 30, 1000])
def test_attention_page_outside_the_pool_counts_as_zeros(d, q_lens, bad):
    """The kernel checks every page index; the call reports the bad one."""
    kv_lens = [200, 60]
    kp, vp, table, K, V = make_cache(kv_lens, 2, d, 16, 6)
    table[0, 3] = bad
    K[0][48:64] = 0
    V[0][48:64] = 0
    q = randn(sum(q_lens), 4, d, seed=2)
    out, lse = torch.empty_like(q, device=DEV), torch.empty(q.shape[:2], device=DEV)
    ws = hq.alloc_paged_attention_workspace(2, q.shape[0], max(q_lens), 200, 2, 2, d)
    st = new_status()
    hq.hq_paged_attention(q.to(DEV), starts(q_lens).to(DEV), i32(*kv_lens), hq.Pages(kp.to(DEV), vp.to(DEV)),
                          table.to(DEV), 0.1, out, ws, max_q=max(q_lens), max_kv=200, lse=lse, status=st)
    assert int(st) == hq.HQ_ST_INDEX
    ref, ref_lse, tol, _, tol_l = attend(q, K, V, q_lens, 0.1)
    assert_within(out, ref, tol)
    assert_within(lse, ref_lse, tol_l)


@pytest.mark.parametrize("start,kv,max_q", [([0, 2, 1, 4], [20, 20, 20], 4), ([0, 2, 3, 99], [20, 20, 20], 4),
                                            ([0, 1, 2, 4], [20, -3, 20], 4), ([0, 1, 2, 4], [20, 1000, 20], 4),
                                            ([0, 1, 2, 4], [20, 20, 20], 1), ([-1, 1, 2, 4], [20, 20, 20], 4)])
def test_attention_skips_an_inconsistent_sequence(start, kv, max_q):
    """Others are computed; the skipped one's rows are left, the status says so.
    (Offsets out of order can give a row to two sequences: it holds either's.)"""
    kp, vp, table, K, V = make_cache([20, 20, 20], 1, 64, 16, 2)
    q = randn(4, 2, 64, seed=1)
    out = torch.full((4, 2, 64), 9.0, dtype=BF, device=DEV)
    ws = hq.alloc_paged_attention_workspace(3, 4, 4, 32, 1, 2, 64)
    st = new_status()
    hq.hq_paged_attention(q.to(DEV), i32(*start), i32(*kv), hq.Pages(kp.to(DEV), vp.to(DEV)), table.to(DEV), 0.1, out,
                          ws, max_q=max_q, max_kv=32, status=st)
    assert int(st) == hq.HQ_ST_INDEX
    fine = [0 <= start[b] <= start[b + 1] <= 4 and start[b + 1] - start[b] <= max_q and 0 <= kv[b] <= 32
            for b in range(3)]
    owners = torch.tensor([sum(fine[b] and start[b] <= t < start[b + 1] for b in range(3)) for t in range(4)])
    assert (out.cpu()[owners == 0] == 9.0).all()
    for b in range(3):
        a, e = start[b], start[b + 1]
        if fine[b]:
            ref, _, tol, _, _ = attend(q[a:e], [K[b][:kv[b]]], [V[b][:kv[b]]], [e - a], 0.1)
            one = owners[a:e] == 1
            assert_within(out[a:e].cpu()[one], ref[one], tol[one])


@pytest.mark.parametrize("d,q_lens,kv_lens", [(128, [1, 1, 1], [7000, 30, 900]), (64, [300, 40], [2500, 100]),
                                              (128, [300, 1], [2500, 100]), (256, [300, 1], [900, 100])])
def test_attention_repeats_bit_for_bit_on_any_workspace_contents(d, q_lens, kv_lens):
    kp, vp, table, _, _ = make_cache(kv_lens, 2, d, 16, 2)
    q = randn(sum(q_lens), 8, d, seed=1).to(DEV)
    pool = hq.Pages(kp.to(DEV), vp.to(DEV))
    ws = hq.alloc_paged_attention_workspace(len(q_lens), q.shape[0], max(q_lens), max(kv_lens), 2, 4, d)
    got = []
    for fill in (0, 255, 1, None, None):
        if fill is not None:
            ws.fill_(fill)
        out = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], device=DEV)
        hq.hq_paged_attention(q, starts(q_lens).to(DEV), i32(*kv_lens), pool, table.to(DEV), 0.09, out, ws,
                              max_q=max(q_lens), max_kv=max(kv_lens), lse=lse)
        got.append((out, lse))
    assert all(torch.equal(o, got[0][0]) and torch.equal(s, got[0][1]) for o, s in got)


@pytest.mark.parametrize("d,max_q", [(128, 1), (128, 160), (256, 160)])
def test_attention_and_append_in_a_graph(d, max_q):
    """Captured once, replayed with other lengths, positions and values; two
    graphs share one workspace and run in turn."""
    kvh, group, page, width = 2, 2, 16, 30
    pool = hq.Pages(*[torch.zeros(2 * width, kvh, page, d, dtype=BF, device=DEV) for _ in range(2)])
    table = torch.arange(2 * width, dtype=torch.int32, device=DEV).view(2, width)
    n = 2 * max_q
    k, v, q = (torch.zeros(n, h, d, dtype=BF, device=DEV) for h in (kvh, kvh, kvh * group))
    slots, pos = torch.full((n,), -1, dtype=torch.int64, device=DEV), torch.zeros(n, dtype=torch.int64, device=DEV)
    start, kv_len = i32(0, 0, 0), i32(0, 0)
    q_rot = torch.zeros_like(q)
    rope = hq.rope_table(d)
    ws = hq.alloc_paged_attention_workspace(2, n, max_q, width * page, kvh, group, d)
    out = [torch.zeros_like(q) for _ in range(2)]

    def step(o):
        hq.hq_kv_append(k, v, slots, pool, positions=pos, rope=rope, q=q, q_out=q_rot)
        hq.hq_paged_attention(q_rot, start, kv_len, pool, table, d ** -0.5, o, ws, max_q=max_q, max_kv=width * page)

    s = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        for o in out:
            step(o)
            g = torch.cuda.CUDAGraph()
            s.synchronize()
            with torch.cuda.graph(g, stream=s):
                step(o)
            graphs.append(g)
    torch.cuda.synchronize()
    theta, amp = theta_of(d, 10000.0)
    dense = [[torch.zeros(0, kvh, d, dtype=BF)] * 2 for _ in range(2)]  # K, V per sequence
    for turn, lens in enumerate([(min(3, max_q), 1), (1, min(7, max_q)), (max_q, max_q), (1, 1)]):
        m = sum(lens)
        kk, vv, qq = (randn(m, h, d, seed=10 * turn + i) for i, h in enumerate((kvh, kvh, kvh * group)))
        begin = [dense[0][b].shape[0] for b in range(2)]
        p = torch.cat([begin[b] + torch.arange(lens[b]) for b in range(2)])
        which = torch.cat([torch.full((lens[b],), b) for b in range(2)])
        slots.fill_(-1)
        for dst, src in ((k, kk), (v, vv), (q, qq), (pos, p), (slots, which * width * page + p)):
            dst[:m].copy_(src)
        start.copy_(starts(lens))
        kv_len.copy_(torch.tensor([begin[b] + lens[b] for b in range(2)], dtype=torch.int32))
        graphs[turn % 2].replay()
        torch.cuda.synchronize()
        stored = hq.Pages(pool.k.cpu(), pool.v.cpu())
        for b in range(2):
            new = begin[b] + lens[b]
            for j, t in enumerate((stored.k, stored.v)):
                flat = t[b * width:(b + 1) * width].transpose(1, 2).reshape(-1, kvh, d)[:new]
                dense[j][b] = flat
        ref_k = rotate(kk, p, theta, amp, "half")
        got_k = torch.cat([dense[0][b][begin[b]:] for b in range(2)])
        assert_within(got_k, ref_k, rotate_tolerance(kk, ref_k, theta, amp, "half", p, BF))
        ref, _, tol, _, _ = attend(q_rot[:m], dense[0], dense[1], lens, d ** -0.5)
        assert_within(out[turn % 2][:m], ref, tol)


@pytest.mark.parametrize("max_q", [1, 140])
def test_attention_on_two_streams_with_their_own_workspaces(max_q):
    kv_lens = [3000, 500]
    kp, vp, table, _, _ = make_cache(kv_lens, 2, 128, 64, 2)
    pool, table = hq.Pages(kp.to(DEV), vp.to(DEV)), table.to(DEV)
    qs = [randn(2 * max_q, 8, 128, seed=i).to(DEV) for i in range(2)]
    start, kv = starts([max_q] * 2).to(DEV), i32(*kv_lens)
    ws = [hq.alloc_paged_attention_workspace(2, 2 * max_q, max_q, 3000, 2, 4, 128) for _ in range(2)]
    want = [torch.empty_like(q) for q in qs]
    for i in range(2):
        hq.hq_paged_attention(qs[i], start, kv, pool, table, 0.1, want[i], ws[i], max_q=max_q, max_kv=3000)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[torch.empty_like(q) for _ in range(6)] for q in qs]
    for rep in range(6):
        for i in range(2):
            hq.hq_paged_attention(qs[i], start, kv, pool, table, 0.1, got[i][rep], ws[i], max_q=max_q, max_kv=3000,
                                  stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i]) for i in range(2) for g in got[i])


# ----------------------------------------------------------------- join
@pytest.mark.parametrize("da,db,do", [(BF, BF, BF), (F32, BF, BF), (F32, F32, F32), (BF, F32, F32)])
@pytest.mark.parametrize("tokens,heads,d", [(1, 1, 8), (5, 3, 72), (130, 8, 128)])
def test_merge(da, db, do, tokens, heads, d):
    a, b = randn(tokens, heads, d, seed=1, dtype=da), randn(tokens, heads, d, seed=2, dtype=db)
    la, lb = randn(tokens, heads, seed=3, dtype=F32, scale=4.0), randn(tokens, heads, seed=4, dtype=F32, scale=4.0)
    la[0, 0], lb[-1, -1] = -math.inf, -math.inf  # one part empty (both, for one row)
    a[0, 0], b[-1, -1] = math.nan, math.inf      # and what it holds is not used
    if heads > 2:
        la[0, 1] = lb[0, 1] = -math.inf
        a[0, 1] = math.nan
        la[0, 2], lb[0, 2] = 300.0, -300.0       # far apart: one part counts
    out, lse = torch.empty(tokens, heads, d, dtype=do, device=DEV), torch.empty(tokens, heads, device=DEV)
    hq.hq_attention_merge(a.to(DEV), la.to(DEV), b.to(DEV), lb.to(DEV), out, lse)
    L = torch.logaddexp(la.double(), lb.double())
    wa, wb = (torch.where(l == -math.inf, 0.0, torch.exp(l.double() - L)) for l in (la, lb))
    za, zb = (torch.where((l == -math.inf)[..., None], 0.0, x.double()) for l, x in ((la, a), (lb, b)))
    ref = wa[..., None] * za + wb[..., None] * zb
    # the difference of the logs rounds once (U32 of it), expf is within 2 ulp,
    # division, two products and the sum round once each
    gap = (la - lb).double().abs().nan_to_num(posinf=0.0)
    rel = (2 * gap + 16) * U32
    tol = rel[..., None] * (wa[..., None] * za.abs() + wb[..., None] * zb.abs())
    tol = tol + (2.0 ** -8 if do == BF else U32) * (ref.abs() + tol)
    assert_within(out, ref, tol)
    assert_within(lse, L, rel + 4 * U32 * L.abs().nan_to_num(posinf=0.0))


def test_merge_in_place_and_strided():
    a, b = randn(9, 4, 64, seed=1).to(DEV), randn(4, 9, 64, seed=2).to(DEV).transpose(0, 1)
    la, lb = randn(9, 4, seed=3, dtype=F32).to(DEV), randn(9, 4, seed=4, dtype=F32).to(DEV)
    out = torch.empty_like(a)
    hq.hq_attention_merge(a, la, b, lb, out)
    hq.hq_attention_merge(a, la, b, lb, a)
    assert torch.equal(a, out)


# ----------------------------------------------------------------- together
@pytest.mark.parametrize("d,group", [(64, 1), (128, 4), (256, 2)])
@pytest.mark.parametrize("heads,tokens", [(2, 700), (1, 1), (3, 0)])
def test_compressed_attention_with_lse(d, group, heads, tokens):
    """The same output bit for bit, and the log of the weights' sum over the
    oracle's decoded keys: scores move by at most what attention_tolerance
    allows them (a rotation and a dot in binary32), here 2^-18 of sum |q||k|."""
    K, V = randn(heads * tokens, d, seed=1), randn(heads * tokens, d, seed=2)
    st = new_status()
    streams = []
    for i, x in enumerate((K, V)):
        s = hq.alloc_stream(heads * tokens, d, d, "E8", 4.0)
        hq.hq_kv_encode(x.to(DEV), d, "E8", 4.0, 30 + i, s, hq.alloc_workspace(heads * tokens, d, d), st)
        streams.append(s)
    q = randn(heads * group, d, seed=5).to(DEV)
    ws = hq.alloc_attention_workspace(heads, tokens, d, group)
    args = (streams[0], streams[1], heads, tokens, d, "E8", 4.0, 4.0, 30, 31, q, 0.125)
    plain = hq.hq_kv_attention(*args, torch.empty(heads * group, d, device=DEV), ws, group=group)
    lse = torch.empty(heads * group, device=DEV)
    both = hq.hq_kv_attention(*args, torch.empty(heads * group, d, device=DEV), ws, group=group, lse=lse)
    assert torch.equal(plain, both)
    if tokens == 0:
        assert (lse == -math.inf).all() and (both == 0).all()
        return
    kd = torch.empty(heads * tokens, d, device=DEV)
    hq.hq_kv_decode(streams[0], heads * tokens, d, d, "E8", 4.0, 30, kd)
    k = kd.double().cpu().view(heads, 1, tokens, d)
    x = q.double().cpu().view(heads, group, d, 1)
    s = 0.125 * (k @ x).squeeze(-1)
    off = 0.125 * (k.abs() @ x.abs()).squeeze(-1).max(-1).values * 2.0 ** -18
    ref = torch.logsumexp(s, -1)
    assert_within(lse.view(heads, group), ref, off + 1e-5 + 4 * U32 * ref.abs())


def test_a_model_step_from_compressed_weights_to_the_joined_cache():
    """Compressed projections -> rotation and append -> attention in chunks and
    token by token -> full pages compressed where they lie -> attention over the
    compressed history joined with the recent pages."""
    kvh, group, d, page, hidden = 2, 2, 128, 64, 512
    heads, n = kvh * group, 200
    rows = (heads + 2 * kvh) * d
    w = randn(rows, hidden, seed=1, scale=0.05)
    st = new_status()
    ws_stream = hq.alloc_stream(rows, hidden, 256, "E8", 4.0)
    hq.hq_encode(w.to(DEV), 256, "E8", 4.0, 7, ws_stream, hq.alloc_workspace(rows, hidden, 256), st)
    x = randn(n, hidden, seed=2).to(DEV)
    qkv = torch.empty(n, rows, device=DEV)
    hq.hq_decode_gemm(ws_stream, rows, hidden, 256, "E8", 4.0, 7, x, qkv, hq.alloc_gemm_workspace(rows, hidden, n), st)
    pool = hq.alloc_pages(6, page, kvh, d)
    pool.k.fill_(math.nan)
    pool.v.fill_(math.nan)
    table = i32(4, 1, 5, 2).view(1, 4)
    rope = hq.rope_table(d, 500000.0, BANDS)
    split = lambda t: (t[:, :heads * d].view(-1, heads, d), t[:, heads * d:(heads + kvh) * d].view(-1, kvh, d),  # noqa: E731
                       t[:, (heads + kvh) * d:].view(-1, kvh, d))
    out = torch.empty(n, heads, d, dtype=BF, device=DEV)
    q_rot = torch.empty_like(out)
    lse = torch.empty(n, heads, device=DEV)
    ws = hq.alloc_paged_attention_workspace(1, n, n, 256, kvh, group, d)
    scale = d ** -0.5
    at = 0
    for m in (150, 7, 1, 1, 41):
        q, k, v = split(qkv[at:at + m])
        pos = torch.arange(at, at + m, device=DEV)
        slots = table[0, pos // page].long() * page + pos % page
        hq.hq_kv_append(k, v, slots, pool, positions=pos, rope=rope, q=q, q_out=q_rot[at:at + m], status=st)
        hq.hq_paged_attention(q_rot[at:at + m], i32(0, m), i32(at + m), pool, table, scale, out[at:at + m], ws, max_q=m,
                              max_kv=256, lse=lse[at:at + m], status=st)
        at += m
    assert int(st) == 0
    q, k, v = split(qkv.cpu())
    theta, amp = theta_of(d, 500000.0, BANDS)
    pos = torch.arange(n)
    ref_q, ref_k = rotate(q, pos, theta, amp, "half"), rotate(k, pos, theta, amp, "half")
    assert_within(q_rot, ref_q, rotate_tolerance(q, ref_q, theta, amp, "half", pos, BF))
    stored_k = torch.cat([pool.k[int(p)].transpose(0, 1) for p in table[0]])[:n].cpu()
    stored_v = torch.cat([pool.v[int(p)].transpose(0, 1) for p in table[0]])[:n].cpu()
    assert_within(stored_k, ref_k, rotate_tolerance(k, ref_k, theta, amp, "half", pos, BF))
    assert torch.equal(stored_v, v.to(BF))
    ref, ref_lse, tol, _, tol_l = attend(q_rot, [stored_k], [stored_v], [n], scale)
    assert_within(out, ref, tol)
    assert_within(lse, ref_lse, tol_l)

    # the first three pages (192 tokens) become the compressed history, page by
    # page, each a slab of the pool; the last token attends over both parts
    hist = 3 * page
    parts = []
    for p in table[0, :3].tolist():
        streams = []
        for i, pl in enumerate((pool.k, pool.v)):
            s = hq.alloc_stream(kvh * page, d, d, "E8", 4.0)
            hq.hq_kv_encode(pl[p].reshape(kvh * page, d), d, "E8", 4.0, 100 * p + i, s, hq.alloc_workspace(kvh * page, d, d), st)
            streams.append(s)
        o, l = torch.empty(1, heads, d, device=DEV), torch.empty(1, heads, device=DEV)
        hq.hq_kv_attention(*streams, kvh, page, d, "E8", 4.0, 4.0, 100 * p, 100 * p + 1, q_rot[-1], scale, o,
                           hq.alloc_attention_workspace(kvh, page, d, group), group=group, lse=l, status=st)
        dec = torch.empty(2, kvh * page, d, device=DEV)
        for i in range(2):
            hq.hq_kv_decode(streams[i], kvh * page, d, d, "E8", 4.0, 100 * p + i, dec[i])
        parts.append((o, l, dec.view(2, kvh, page, d).transpose(1, 2).double().cpu()))
    recent, rl = torch.empty(1, heads, d, device=DEV), torch.empty(1, heads, device=DEV)
    hq.hq_paged_attention(q_rot[-1:], i32(0, 1), i32(n - hist), pool, table[:, 3:], scale, recent, ws, max_q=1, max_kv=64,
                          lse=rl, status=st)
    for o, l, _ in parts:
        joined, jl = torch.empty_like(recent), torch.empty_like(rl)
        hq.hq_attention_merge(o, l, recent, rl, joined, jl)
        recent, rl = joined, jl
    assert int(st) == 0
    K = torch.cat([p[2][0] for p in parts] + [stored_k[hist:].double()])
    V = torch.cat([p[2][1] for p in parts] + [stored_v[hist:].double()])
    ref, ref_lse, _, tol, tol_l = attend(q_rot[-1:], [K], [V], [1], scale)
    # the compressed scores go through a binary32 rotation: 2^-18 of sum |q||k|
    s_off = scale * (q_rot[-1:].double().cpu().abs().view(kvh, group, 1, d) @ K.abs().permute(1, 2, 0)[:, None]).max() * 2.0 ** -18
    mean = V.abs().max()
    assert_within(recent, ref, tol + 2 * s_off * mean + 64 * U32 * mean)
    assert_within(rl, ref_lse, tol_l + s_off + 64 * U32 * (1 + ref_lse.abs()))
