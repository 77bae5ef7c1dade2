"""The serving operators at the shapes where their kernels take other ways: many
jobs and long walks per block of the chunk kernel, every row tile of the kernel
for few rows, scales and masks at each head size, blocks of four tokens of the
rotation and the append, every type of the join, values at the end of their
range.  Against the binary64 forms and bounds of serving_util."""
import math

import pytest
import torch

from kv_quantization_tile_b200 import hq
from serving_util import (U32, UB, assert_within, attend, gen, make_cache, randn, rotate, rotate_tolerance, starts,
                          theta_of)
from test_gpu_serving import run_attention

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32
YARN = {"kind": "yarn", "factor": 16.0, "slow": 1.0, "fast": 32.0, "original": 4096}


# ----------------------------------------------------------------- attention
def uneven(n):
    """Chunks of 0 to 150 new tokens over up to 500 cached ones; some empty, some
    of one token, some with more new tokens than cached ones."""
    q_lens = [0 if i % 17 == 3 else 1 if i % 13 == 5 else 40 + 53 * i % 111 for i in range(n)]
    kv_lens = [0 if i % 29 == 7 else 20 + 97 * i % 481 for i in range(n)]
    return q_lens, kv_lens


@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("d,kvh,group", [(64, 8, 4), (128, 8, 2), (256, 4, 2)])
def test_many_jobs_in_a_block(d, kvh, group, window):
    """150 sequences: 5 to 18 jobs in each block of the chunk kernel, so its
    ring of segments, its queries, scores and outputs serve one job after another."""
    q_lens, kv_lens = uneven(150)
    run_attention(q_lens, kv_lens, kvh, group, d, 32, window=window, seed=d + window)


@pytest.mark.parametrize("d,q_len,kv_len,group", [(64, 512, 16391, 4), (128, 512, 16391, 4), (256, 300, 8200, 4)])
def test_long_walks_and_their_repetition(d, q_len, kv_len, group):
    """More than 50 tiles in each block: its ring of tiles wraps many times.  Two
    of the 8 KV heads are held to the binary64 form, all to their repetition."""
    kvh, page = 8, 64
    kp, vp, table, K, V = make_cache([kv_len], kvh, d, page, 7)
    q = randn(q_len, kvh * group, d, seed=8)
    pool, qd = hq.Pages(kp.to(DEV), vp.to(DEV)), q.to(DEV)
    ws = hq.alloc_paged_attention_workspace(1, q_len, q_len, kv_len, kvh, group, d)
    got = []
    for fill in (255, 0, None):
        if fill is not None:
            ws.fill_(fill)
        out, lse = torch.empty_like(qd), torch.empty(q_len, kvh * group, device=DEV)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        hq.hq_paged_attention(qd, starts([q_len]).to(DEV), torch.tensor([kv_len], dtype=torch.int32, device=DEV), pool,
                              table.to(DEV), d ** -0.5, out, ws, max_q=q_len, max_kv=kv_len, lse=lse, status=st)
        assert int(st) == 0
        got.append((out, lse))
    assert all(torch.equal(o, got[0][0]) and torch.equal(s, got[0][1]) for o, s in got)
    for h in (0, 5):
        own = slice(h * group, (h + 1) * group)
        ref, ref_lse, tol, _, tol_l = attend(q[:, own], [K[0][:, h:h + 1]], [V[0][:, h:h + 1]], [q_len], d ** -0.5)
        assert_within(got[0][0][:, own], ref, tol, h)
        assert_within(got[0][1][:, own], ref_lse, tol_l, h)


@pytest.mark.parametrize("d,group", [(64, 3), (128, 4), (256, 2)])
def test_uneven_chunks_repeat_bit_for_bit(d, group):
    q_lens, kv_lens = uneven(100)
    kp, vp, table, _, _ = make_cache(kv_lens, 4, d, 16, 2)
    q = randn(sum(q_lens), 4 * group, d, seed=1).to(DEV)
    pool = hq.Pages(kp.to(DEV), vp.to(DEV))
    ws = hq.alloc_paged_attention_workspace(100, q.shape[0], max(q_lens), max(kv_lens), 4, group, d)
    got = []
    for fill in (0, 255, None, None):
        if fill is not None:
            ws.fill_(fill)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
        hq.hq_paged_attention(q, starts(q_lens).to(DEV), torch.tensor(kv_lens, dtype=torch.int32, device=DEV), pool,
                              table.to(DEV), 0.09, out, ws, max_q=max(q_lens), max_kv=max(kv_lens), lse=lse)
        got.append((out, lse))
    assert all(torch.equal(o, got[0][0]) and torch.equal(s, got[0][1]) for o, s in got)


@pytest.mark.parametrize("d,n", [(64, 120), (128, 80), (256, 40)])
@pytest.mark.parametrize("q,group", [(1, 5), (3, 8), (6, 8), (15, 8)])
def test_shares_of_few_rows_at_every_row_tile(d, n, q, group):
    """More jobs than clusters can take (4 KV heads of up to 120 sequences): 16, 32
    and 64 rows, and two tiles of 64, by shares, over at most 1024 tokens."""
    run_attention([q] * n, [1024] + [30 + 41 * i % 700 for i in range(n - 1)], 4, group, d, 32, seed=d + q)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2], [300, 70]), ([140], [300])])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1e-6, 3.0])
def test_scales_at_the_other_head_sizes(d, q_lens, kv_lens, scale):
    run_attention(q_lens, kv_lens, 2, 2, d, 32, scale=scale)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,scale", [(100, -0.1), (60, 0.0)])
def test_scales_over_many_jobs_in_a_block(d, n, scale):
    """The sign is turned in the queries copied ahead for the next job."""
    q_lens, kv_lens = uneven(n)
    run_attention(q_lens, kv_lens, 4, 2, d, 64, scale=scale)


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 4], [90, 33]), ([100, 70], [300, 20]), ([300, 0, 5], [650, 9, 0])])
@pytest.mark.parametrize("window", [0, 40])
def test_no_causal_mask_at_the_other_head_sizes(d, q_lens, kv_lens, window):
    run_attention(q_lens, kv_lens, 2, 2, d, 16, causal=False, window=window, max_kv=max(kv_lens) + 3)


@pytest.mark.parametrize("out_dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 4], [1500, 33]), ([150], [1500])])
def test_values_at_the_end_of_their_range(d, q_lens, kv_lens, out_dtype):
    """|v| up to 2^69, and scores that stay 16 to 23 powers of two above the first
    tile's: with the first tile's maximum kept, weights reach 2^23."""
    kvh, group, page, n = 2, 4, 64, sum(q_lens)
    kp, vp, table, K, V = make_cache(kv_lens, kvh, d, page, 3)
    for b, kv in enumerate(kv_lens):
        K[b] = (0.01 * K[b].float() + (torch.arange(kv) >= 128).float()[:, None, None] * 14.0 / (d * 0.25)).to(BF)
        V[b] = torch.clamp(V[b].float() * 2.0 ** 67, -(2.0 ** 69), 2.0 ** 69).to(BF)
        for i in range(-(-kv // page)):
            m = min(page, kv - i * page)
            for pool, x in ((kp, K[b]), (vp, V[b])):
                pool[int(table[b, i]), :, :m] = x[i * page:i * page + m].transpose(0, 1)
    q = torch.ones(n, kvh * group, d, dtype=BF)
    out = torch.empty(n, kvh * group, d, dtype=out_dtype, device=DEV)
    ws = hq.alloc_paged_attention_workspace(len(q_lens), n, max(q_lens), max(kv_lens), kvh, group, d)
    hq.hq_paged_attention(q.to(DEV), starts(q_lens).to(DEV), torch.tensor(kv_lens, dtype=torch.int32, device=DEV),
                          hq.Pages(kp.to(DEV), vp.to(DEV)), table.to(DEV), 0.25, out, ws, max_q=max(q_lens),
                          max_kv=max(kv_lens))
    ref, _, tol_b, tol_f, _ = attend(q, K, V, q_lens, 0.25)
    assert_within(out, ref, tol_b if out_dtype == BF else tol_f)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_len", [1, 512])
def test_rows_that_one_token_dominates(d, q_len):
    """A token 22 to 23 powers of two above all others is its row's output, but
    for their share S of the weights: that weight's rounding to bf16 (2^-8 of it at
    most) is in numerator and denominator alike, also where the running maximum
    was taken from earlier tiles.  What is left: the others' roundings and score
    errors, (UB + e) S each, e as in attend() below 2^-8, and 4 (n + 512) U32 of
    the sums."""
    kvh, group, page, kv, at = 8, 4, 64, 2048, 1500
    kp, vp, table, K, V = make_cache([kv], kvh, d, page, 3)
    K[0] = torch.zeros(kv, kvh, d, dtype=BF)
    K[0][at] = 1.0
    V[0][at] = torch.where(torch.arange(d) % 2 == 0, 4.0, -4.0).to(BF)
    for pool, x in ((kp, K[0]), (vp, V[0])):
        for i in range(kv // page):
            pool[int(table[0, i])] = x[i * page:(i + 1) * page].transpose(0, 1)
    # scores of 15.5 to 16 at the token, 0 elsewhere
    q = (torch.linspace(15.5, 16, q_len * kvh * group).view(q_len, kvh * group, 1) * torch.ones(d)).to(BF)
    scale = 1.0 / d
    out, lse = torch.empty(q.shape, dtype=F32, device=DEV), torch.empty(q.shape[:2], device=DEV)
    ws = hq.alloc_paged_attention_workspace(1, q_len, q_len, kv, kvh, group, d)
    hq.hq_paged_attention(q.to(DEV), starts([q_len]).to(DEV), torch.tensor([kv], dtype=torch.int32, device=DEV),
                          hq.Pages(kp.to(DEV), vp.to(DEV)), table.to(DEV), scale, out, ws, max_q=q_len, max_kv=kv,
                          causal=False, lse=lse)
    ref, ref_lse, _, _, tol_l = attend(q, K, V, [q_len], scale, causal=False)
    share = (kv - 1) / (torch.exp(q[..., 0].double()) + kv - 1)
    big = V[0].double().abs().max()
    tol = (2 * (UB + 2.0 ** -8) * share + 4 * (kv + 512) * U32) * big
    assert_within(out, ref, tol[..., None].expand_as(ref))
    assert_within(lse, ref_lse, tol_l)


# ----------------------------------------------------------------- rotation
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("din,dout", [(BF, BF), (F32, F32), (F32, BF), (BF, F32)])
@pytest.mark.parametrize("d,r", [(64, 64), (128, 48), (256, 256), (16, 16)])
@pytest.mark.parametrize("inverse", [False, True])
def test_rotation_in_blocks_of_four_tokens(layout, din, dout, d, r, inverse):
    """From 16 tokens per SM on; the last block is not full."""
    tokens, heads = 2401, 3
    x = randn(tokens, heads, d, seed=d + r, dtype=din)
    pos = torch.randint(-1000, 200000, (tokens,), generator=gen(3))
    y = torch.full((tokens, heads, d), float("nan"), dtype=dout, device=DEV)
    hq.hq_rope(x.to(DEV), pos.to(DEV), hq.rope_table(r, 500000.0, YARN, layout), y, inverse=inverse)
    theta, amp = theta_of(r, 500000.0, YARN)
    ref = rotate(x, pos, theta, amp, layout, inverse)
    assert_within(y, ref, rotate_tolerance(x, ref, theta, amp, layout, pos, dout))


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d,r,page,qh", [(64, 64, 16, 4), (128, 64, 64, 0), (256, 256, 128, 3)])
def test_append_in_blocks_of_four_tokens(layout, dtype, d, r, page, qh):
    tokens, kvh = 2403, 2
    pages = tokens // page + 5
    q, k, v = (randn(tokens, h, d, seed=i, dtype=dtype) for i, h in enumerate((max(qh, 1), kvh, kvh)))
    kp, vp = (torch.full((pages, kvh, page, d), 3.0, dtype=BF) for _ in range(2))
    slots = torch.randperm(pages * page, generator=gen(4))[:tokens]
    slots[::7] = -1                        # padding
    slots[5::101] = pages * page           # past the pool
    slots[tokens - 1] = -(1 << 62)
    pos = torch.randint(0, 131072, (tokens,), generator=gen(5))
    pool = hq.Pages(kp.to(DEV), vp.to(DEV))
    q_out = torch.full((tokens, max(qh, 1), d), 7.0, dtype=BF, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    hq.hq_kv_append(k.to(DEV), v.to(DEV), slots.to(DEV), pool, positions=pos.to(DEV),
                    rope=hq.rope_table(r, 500000.0, YARN, layout), q=q.to(DEV) if qh else None,
                    q_out=q_out if qh else None, status=st)
    assert int(st) == hq.HQ_ST_INDEX
    theta, amp = theta_of(r, 500000.0, YARN)
    kept = (slots >= 0) & (slots < pages * page)
    at = slots[kept]
    for got, base, x, turn in ((pool.k, kp, k, True), (pool.v, vp, v, False)):
        ref = rotate(x, pos, theta, amp, layout) if turn else x.double()
        tol = rotate_tolerance(x, ref, theta, amp, layout, pos, BF) if turn else UB * ref.abs()
        want, off = base.double(), torch.zeros(base.shape, dtype=torch.float64)
        want[at // page, :, at % page], off[at // page, :, at % page] = ref[kept], tol[kept]
        assert_within(got, want, off)
    if qh:
        ref = rotate(q, pos, theta, amp, layout)
        tol = rotate_tolerance(q, ref, theta, amp, layout, pos, BF)
        assert_within(q_out[kept.to(DEV)], ref[kept], tol[kept])
        assert (q_out[~kept.to(DEV)] == 7.0).all()


# ----------------------------------------------------------------- join
@pytest.mark.parametrize("da", [BF, F32])
@pytest.mark.parametrize("db", [BF, F32])
@pytest.mark.parametrize("do", [BF, F32])
@pytest.mark.parametrize("tokens,heads,d", [(3, 5, 1024), (37, 33, 264), (4099, 32, 128), (2, 1, 24)])
def test_join_of_every_type_and_more_rows_than_one_wave(da, db, do, tokens, heads, d):
    """Bounds as in the smaller join: the difference of the logs rounds once (U32
    of it), expf is within 2 ulp, division, two products and the sum round once
    each, then half a step of the output type."""
    a, b = randn(tokens, heads, d, seed=1, dtype=da), randn(tokens, heads, d, seed=2, dtype=db)
    la, lb = randn(tokens, heads, seed=3, dtype=F32, scale=4.0), randn(tokens, heads, seed=4, dtype=F32, scale=4.0)
    la[::3, 0], lb[1::3, -1] = -math.inf, -math.inf
    a[::3, 0], b[1::3, -1] = math.nan, math.inf
    out, lse = torch.empty(tokens, heads, d, dtype=do, device=DEV), torch.empty(tokens, heads, device=DEV)
    hq.hq_attention_merge(a.to(DEV), la.to(DEV), b.to(DEV), lb.to(DEV), out, lse)
    L = torch.logaddexp(la.double(), lb.double())
    wa, wb = (torch.where(l == -math.inf, 0.0, torch.exp(l.double() - L)) for l in (la, lb))
    za, zb = (torch.where((l == -math.inf)[..., None], 0.0, x.double()) for l, x in ((la, a), (lb, b)))
    ref = wa[..., None] * za + wb[..., None] * zb
    rel = (2 * (la - lb).double().abs().nan_to_num(posinf=0.0) + 16) * U32
    tol = rel[..., None] * (wa[..., None] * za.abs() + wb[..., None] * zb.abs())
    assert_within(out, ref, tol + (UB if do == BF else U32) * (ref.abs() + tol))
    assert_within(lse, L, rel + 4 * U32 * L.abs().nan_to_num(posinf=0.0))
