"""Paged attention far out in its documented ranges: work that lasts longer than
the limit of a single wait inside a block (0.5 s) is not taken for a stall."""
import numpy as np
import pytest
import torch

from kv_quantization_tile_b200 import hq
from serving_util import assert_within, attend, make_cache, randn, starts

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
