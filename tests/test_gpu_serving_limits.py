"""The serving operators far out in their documented ranges: work that lasts longer
than the limit of a single wait inside a block (0.5 s) is not taken for a stall,
offsets pass 32 bits, one KV head serves hundreds of query heads."""
import numpy as np
import pytest
import torch

from kv_quantization_tile_b200 import hq
from serving_util import assert_within, attend, make_cache, randn, rotate, rotate_tolerance, starts, theta_of
from test_gpu_serving import run_attention

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16


def test_a_segment_longer_than_any_wait():
    """147 jobs of 56 million cached tokens each, 0.7 s for a block, and six of a
    hundred: the last of 148 blocks has one long segment and then the short ones.
    All tokens but those of one page lie far below it in score (2^-90 of its
    weights, 56 million times: nothing), so the result is that page's."""
    d, group, q_len, page, long, short = 128, 8, 32, 1024, 147, 6
    width = 56_000_000 // page
    k = randn(2, 1, page, d, seed=1, scale=0.1)
    k[0] = -0.5
    v = randn(2, 1, page, d, seed=2)
    batch = long + short
    table = torch.zeros(batch, width, dtype=torch.int32)
    place = np.random.default_rng(3).integers(0, width, long)
    table[torch.arange(long), torch.as_tensor(place)] = 1
    table[long:] = 1
    kv_len = torch.tensor([width * page] * long + [100] * short, dtype=torch.int32)
    q = 1 + randn(batch * q_len, group, d, seed=3, scale=0.02)
    out = torch.empty_like(q, device=DEV)
    lse = torch.empty(batch * q_len, group, device=DEV)
    ws = hq.alloc_paged_attention_workspace(batch, batch * q_len, q_len, width * page, 1, group, d)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    hq.hq_paged_attention(q.to(DEV), starts([q_len] * batch).to(DEV), kv_len.to(DEV), hq.Pages(k.to(DEV), v.to(DEV)),
                          table.to(DEV), 1.0, out, ws, max_q=q_len, max_kv=width * page, causal=False, lse=lse,
                          status=status)
    assert int(status) == 0
    n = [page] * long + [100] * short
    ref, ref_lse, tol, _, tol_l = attend(q, [k[1, 0, :m, None] for m in n], [v[1, 0, :m, None] for m in n], [q_len] * batch,
                                         1.0, causal=False)
    assert_within(out, ref, tol)
    assert_within(lse, ref_lse, tol_l)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_millions_of_empty_sequences_between_prompts(d):
    """The block that goes from the 20th prompt to the next passes 12 million
    sequences without new tokens (the shares cut neither place)."""
    kvh, group, page, gap = 2, 4, 1024, 12_000_000
    q_lens = [200 + 37 * i % 120 for i in range(48)]
    kv_lens = [300 + 17 * i for i in range(48)]
    kp, vp, table, K, V = make_cache(kv_lens, kvh, d, page, 5)
    at = np.arange(48) + gap * (np.arange(48) >= 20)
    batch = 48 + gap
    new, kv = np.zeros(batch, dtype=np.int64), np.zeros(batch, dtype=np.int32)
    new[at], kv[at] = q_lens, kv_lens
    wide = torch.full((batch, table.shape[1]), -1, dtype=torch.int32)
    wide[torch.as_tensor(at)] = table
    n = sum(q_lens)
    q = randn(n, kvh * group, d, seed=6)
    out, lse = torch.empty_like(q, device=DEV), torch.empty(n, kvh * group, device=DEV)
    ws = hq.alloc_paged_attention_workspace(batch, n, max(q_lens), max(kv_lens), kvh, group, d)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    hq.hq_paged_attention(q.to(DEV), starts(new).to(DEV), torch.as_tensor(kv).to(DEV), hq.Pages(kp.to(DEV), vp.to(DEV)),
                          wide.to(DEV), d ** -0.5, out, ws, max_q=max(q_lens), max_kv=max(kv_lens), lse=lse, status=status)
    assert int(status) == 0
    ref, ref_lse, tol, _, tol_l = attend(q, K, V, q_lens, d ** -0.5)
    assert_within(out, ref, tol)
    assert_within(lse, ref_lse, tol_l)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens,group", [([1, 1], [300, 5], 71), ([1], [4500], 128), ([2, 1, 5], [700, 90, 5], 129),
                                                  ([1, 1, 1], [1, 0, 2000], 300)])
def test_one_kv_head_serves_many_query_heads(d, q_lens, kv_lens, group):
    run_attention(q_lens, kv_lens, 1, group, d, 64, seed=group)


def far(shape, strides, dtype=BF):
    """A tensor of these strides in memory of its own, whose last elements lie past 2^32 bytes."""
    span = 1 + sum((n - 1) * s for n, s in zip(shape, strides))
    return torch.empty(span, dtype=dtype, device=DEV).as_strided(shape, strides)


def test_rows_past_32_bits():
    """Token strides of 1.1e9 elements: rotation, join and attention of three tokens."""
    d, heads, step = 64, 4, (1 << 30) + (1 << 26)
    pos = torch.tensor([3, 70000, 9])
    x = randn(3, heads, d, seed=1)
    xs, y = far(x.shape, (step, d, 1)), far(x.shape, (step, d, 1))
    xs.copy_(x)
    hq.hq_rope(xs, pos.to(DEV), hq.rope_table(d), y)
    theta, amp = theta_of(d, 10000.0)
    ref = rotate(x, pos, theta, amp, "half")
    assert_within(y, ref, rotate_tolerance(x, ref, theta, amp, "half", pos, BF))
    for q_lens, kv_lens in (([1, 2], [90, 40]), ([3], [500])):
        kp, vp, table, K, V = make_cache(kv_lens, 1, d, 16, 3)
        ws = hq.alloc_paged_attention_workspace(len(q_lens), 3, 3, max(kv_lens), 1, heads, d)
        hq.hq_paged_attention(xs, starts(q_lens).to(DEV), torch.tensor(kv_lens, dtype=torch.int32, device=DEV),
                              hq.Pages(kp.to(DEV), vp.to(DEV)), table.to(DEV), 0.1, y, ws, max_q=3, max_kv=max(kv_lens))
        ref, _, tol, _, _ = attend(x, K, V, q_lens, 0.1)
        assert_within(y, ref, tol)
    lse = torch.zeros(3, heads, device=DEV)
    other = torch.zeros(3, heads, d, dtype=BF, device=DEV)
    hq.hq_attention_merge(xs, lse, other, lse, y)
    assert torch.equal(y.cpu(), (0.5 * x.float()).to(BF))


@pytest.mark.parametrize("q_len", [1, 150])
def test_chunk_rows_past_32_bits(q_len):
    """Heads 1.1e9 elements apart, in both attention kernels."""
    d, heads, kv, step = 128, 4, 300, (1 << 30) + (1 << 26)
    x = randn(q_len, heads, d, seed=1)
    xs, y = far(x.shape, (d, step, 1)), far(x.shape, (d, step, 1))
    xs.copy_(x)
    kp, vp, table, K, V = make_cache([kv], 1, d, 16, 3)
    ws = hq.alloc_paged_attention_workspace(1, q_len, q_len, kv, 1, heads, d)
    hq.hq_paged_attention(xs, starts([q_len]).to(DEV), torch.tensor([kv], dtype=torch.int32, device=DEV),
                          hq.Pages(kp.to(DEV), vp.to(DEV)), table.to(DEV), 0.1, y, ws, max_q=q_len, max_kv=kv)
    ref, _, tol, _, _ = attend(x, K, V, [q_len], 0.1)
    assert_within(y, ref, tol)


def test_a_pool_past_32_bits():
    """70,000 pages of 65,536 elements in K and in V: tokens appended to the first,
    middle and last of them, then attended over by one token and by a chunk."""
    d, kvh, heads, page, pages, n = 128, 8, 16, 64, 70_000, 300
    pool = hq.alloc_pages(pages, page, kvh, d)
    table = torch.tensor([[pages - 1, 0, 32768, 65536, pages - 2]], dtype=torch.int32)
    k, v, q = randn(n, kvh, d, seed=1), randn(n, kvh, d, seed=2), randn(n, heads, d, seed=3)
    t = torch.arange(n)
    slots = table[0, t // page].long() * page + t % page
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    hq.hq_kv_append(k.to(DEV), v.to(DEV), slots.to(DEV), pool, status=status)
    for q_len in (1, n):
        out = torch.empty(q_len, heads, d, dtype=BF, device=DEV)
        ws = hq.alloc_paged_attention_workspace(1, q_len, q_len, n, kvh, heads // kvh, d)
        hq.hq_paged_attention(q[n - q_len:].to(DEV), starts([q_len]).to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV),
                              pool, table.to(DEV), d ** -0.5, out, ws, max_q=q_len, max_kv=n, status=status)
        assert int(status) == 0
        ref, _, tol, _, _ = attend(q[n - q_len:], [k], [v], [q_len], d ** -0.5)
        assert_within(out, ref, tol)
