"""Waits of the paged attention kernels that run out, without a fault, trap or
hang: a testing hook withholds one hand-over inside a block, the bounded waits
for it (0.5 s each) give up, the call returns with HQ_ST_TIMEOUT, and the device
and the workspace stay usable -- the same call right after gives the bits it gave
before."""
import time

import pytest
import torch

from kv_quantization_tile_b200 import hq
from serving_util import make_cache, randn, starts

pytestmark = pytest.mark.gpu
DEV = "cuda"
COPY, PRODUCT = 1, 2


def run_stalled(q_lens, kv_lens, kvh, group, d, kind, stalled, grow=False):
    kp, vp, table, _, _ = make_cache(kv_lens, kvh, d, 64, 1, stale=0.0)
    n = sum(q_lens)
    q = randn(n, kvh * group, d, seed=2)
    if grow:  # each tile's scores pass the ones before by hundreds of powers of two
        for b, kv in enumerate(kv_lens):
            for i in range(-(-kv // 64)):
                ramp = (64 * i + torch.arange(64)) * 0.02
                kp[int(table[b, i])] = ramp[:, None].to(torch.bfloat16)
        q = torch.ones_like(q)
    args = (q.to(DEV), starts(q_lens).to(DEV), torch.tensor(kv_lens, dtype=torch.int32, device=DEV),
            hq.Pages(kp.to(DEV), vp.to(DEV)), table.to(DEV), 0.5 if grow else d ** -0.5)
    ws = hq.alloc_paged_attention_workspace(len(q_lens), n, max(q_lens), max(kv_lens), kvh, group, d)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)

    def call():
        out = torch.zeros_like(args[0])
        hq.hq_paged_attention(*args, out, ws, max_q=max(q_lens), max_kv=max(kv_lens), status=status)
        torch.cuda.synchronize()
        assert int(status) == 0
        return out

    want = call()
    assert torch.isfinite(want).all()
    for _ in range(2):
        t0 = time.time()
        hq.hq_test_paged_attention_stalled(*args, torch.zeros_like(args[0]), ws, max_q=max(q_lens), max_kv=max(kv_lens),
                                           kind=kind, stalled=stalled, status=status)
        torch.cuda.synchronize()
        assert time.time() - t0 < 10.0
        assert int(status) == hq.HQ_ST_TIMEOUT
        status.zero_()
        assert torch.equal(call(), want)


@pytest.mark.parametrize("stalled", [0, 2])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_page_copy_that_never_lands_one_launch_of_clusters(d, stalled):
    run_stalled([1], [4096], 2, 4, d, COPY, stalled)


@pytest.mark.parametrize("stalled", [0, 7])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_page_copy_that_never_lands_shares_of_few_rows(d, stalled):
    run_stalled([1] * 60, [600] * 60, 8, 2, d, COPY, stalled)


@pytest.mark.parametrize("stalled", [0, 1, 12])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_a_page_copy_that_never_lands_chunks(d, stalled):
    run_stalled([1021], [2043], 8, 4, d, COPY, stalled)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens,kvh,group,last", [([1], [4096], 2, 4, 3), ([1] * 60, [600] * 60, 8, 2, 9),
                                                           ([1021], [2043], 8, 4, 17)])
def test_a_last_page_copy_that_never_lands(d, q_lens, kv_lens, kvh, group, last):
    """The load warp has issued all its copies when the others give up: it still
    stays until they have landed."""
    run_stalled(q_lens, kv_lens, kvh, group, d, COPY, last)


@pytest.mark.parametrize("grow", [False, True])
@pytest.mark.parametrize("d,stalled", [(64, 0), (64, 4), (128, 0), (128, 4), (256, 0), (256, 5), (128, 8)])
def test_products_whose_notices_never_come(d, stalled, grow):
    """Waited for where the output is rescaled (keys that grow), or at the end of
    the job (nine tiles); a failure in the first place holds until the warps next vote."""
    run_stalled([1021], [2043], 8, 4, d, PRODUCT, stalled, grow)
