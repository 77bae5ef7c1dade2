"""Host side of the serving operators (CPU): rotation tables against their
definitions, workspace sizing, and the refusal of every bad argument before
anything is launched."""
import ctypes
import math

import numpy as np
import pytest
import torch

from kv_quantization_tile_b200 import hq
from serving_util import theta_of

SCALINGS = [None, {"kind": "linear", "factor": 4.0}, {"kind": "ntk", "factor": 8.0},
            {"kind": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "original": 8192},
            {"kind": "yarn", "factor": 16.0, "slow": 1.0, "fast": 32.0, "original": 4096}]


@pytest.mark.parametrize("scaling", SCALINGS, ids=lambda s: s["kind"] if s else "plain")
@pytest.mark.parametrize("r", [16, 64, 80, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies_follow_their_definition(r, base, scaling):
    theta, amp = hq.hq_rope_frequencies(r, base, scaling)
    ref, ref_amp = theta_of(r, base, scaling)
    assert np.allclose(theta, ref, rtol=1e-12, atol=0)
    assert amp == pytest.approx(ref_amp, rel=2.0 ** -24)


def test_turns_are_the_exact_fraction_of_a_turn():
    """turns = theta / 2 pi mod 1 in 2^-64: against 60-digit arithmetic, within
    the rounding of a 64-bit significand (2^-64 of theta / 2 pi, times 4)."""
    import mpmath
    mpmath.mp.dps = 60
    theta = np.concatenate([theta_of(128, 500000.0)[0], [0.0, 2 * math.pi, 7.5, -0.25, 1e-9]])
    turns = hq.hq_rope_table(theta)
    for t, n in zip(theta, turns):
        exact = mpmath.mpf(float(t)) / (2 * mpmath.pi)
        frac = (exact - mpmath.floor(exact)) * mpmath.mpf(2) ** 64
        off = abs(frac - int(n))
        off = min(off, mpmath.mpf(2) ** 64 - off)
        assert off <= 1 + 4 * abs(exact), (t, n, off)


@pytest.mark.parametrize("r,base,scaling", [(8, 1e4, None), (24, 1e4, None), (272, 1e4, None), (64, 1.0, None),
                                            (64, math.inf, None), (64, 1e4, {"kind": "linear", "factor": 0.0}),
                                            (64, 1e4, {"kind": "linear", "factor": math.nan}),
                                            (64, 1e4, {"kind": "yarn", "factor": 0.5, "slow": 1, "fast": 32, "original": 4096}),
                                            (64, 1e4, {"kind": "bands", "factor": 8, "low": 4, "high": 1, "original": 8192}),
                                            (64, 1e4, {"kind": "bands", "factor": 8, "low": 1, "high": 4})])
def test_frequencies_refuse(r, base, scaling):
    with pytest.raises(hq.HQError) as e:
        hq.hq_rope_frequencies(r, base, scaling)
    assert e.value.code == hq.HQ_ERR_ARG


def test_unknown_names_are_refused():
    with pytest.raises(ValueError):
        hq.hq_rope_frequencies(64, 1e4, {"kind": "other", "factor": 2.0})
    with pytest.raises(ValueError):
        hq.rope_table(64, layout="other", device="cpu")
    with pytest.raises(hq.HQError):
        hq.hq_rope_table([math.inf])


# Device pointers that are never followed: every call below is refused on the host.
A = 1 << 20
LIB = hq.library()


def rows(p=A, dtype=hq.HQ_BF16, ts=1024, hs=128):
    return hq.hq_rows(p, dtype, ts, hs)


def pages(**kw):
    d = dict(k=A, v=A, pages=8, page_size=16, heads=2, head_dim=128, page_stride=4096, head_stride=2048, slot_stride=128)
    d.update(kw)
    return hq.hq_pages(*[d[n] for n, _ in hq.hq_pages._fields_])


BAD_ROWS = [dict(p=0), dict(p=A + 8), dict(dtype=7), dict(ts=1020), dict(hs=4), dict(ts=-1024),
            dict(dtype=hq.HQ_F32, ts=1022)]
BAD_PAGES = [(dict(k=0), 1), (dict(v=A + 2), 1), (dict(page_size=24), 2), (dict(page_size=8), 2), (dict(page_size=2048), 2),
             (dict(head_dim=96), 1), (dict(heads=0), 1), (dict(slot_stride=64), 1), (dict(slot_stride=132), 1),
             (dict(page_stride=2048), 1), (dict(pages=1 << 28), 2), (dict(pages=-1), 1)]


def rope(x=None, y=None, tokens=4, heads=8, d=128, pos=A, turns=A, r=128, layout=0, amp=1.0):
    x, y = x or rows(), y or rows()
    return LIB.hq_rope(ctypes.byref(x), ctypes.byref(y), tokens, heads, d, pos, turns, r, layout, amp, 0, None)


@pytest.mark.parametrize("bad", BAD_ROWS)
def test_rope_refuses_rows(bad):
    assert rope(x=rows(**bad)) == hq.HQ_ERR_ARG
    assert rope(y=rows(**bad)) == hq.HQ_ERR_ARG


@pytest.mark.parametrize("kw,code", [(dict(tokens=-1), 1), (dict(heads=-1), 1), (dict(d=120), 1), (dict(d=512), 1),
                                     (dict(pos=0), 1), (dict(pos=A + 4), 1), (dict(turns=0), 1), (dict(r=0), 1),
                                     (dict(r=24), 1), (dict(r=256), 1), (dict(layout=2), 1), (dict(amp=math.nan), 1),
                                     (dict(heads=70000), 2), (dict(tokens=1 << 31), 2), (dict(y=rows(ts=0)), 1),
                                     (dict(y=rows(ts=512)), 1), (dict(y=rows(ts=128, hs=128)), 1)])
def test_rope_refuses(kw, code):
    assert rope(**kw) == code


def test_rope_of_nothing_is_ok():
    assert rope(tokens=0, pos=0) == 0 and rope(heads=0, turns=0) == 0


def append(q=None, q_out=None, qh=0, k=None, v=None, tokens=4, pos=A, turns=A, r=128, layout=0, slots=A, pg=None):
    k, v, pg = k or rows(ts=256), v or rows(ts=256), pg or pages()
    by = lambda s: ctypes.byref(s) if s is not None else None  # noqa: E731
    return LIB.hq_kv_append(by(q), by(q_out), qh, by(k), by(v), tokens, pos, turns, r, layout, 1.0, slots, by(pg), None, None)


@pytest.mark.parametrize("bad,code", BAD_PAGES)
def test_append_refuses_pages(bad, code):
    assert append(pg=pages(**bad)) == code


@pytest.mark.parametrize("kw", [dict(k=rows(p=0)), dict(v=rows(hs=4)), dict(slots=0), dict(slots=A + 4), dict(tokens=-1),
                                dict(q=rows()), dict(q=rows(), q_out=rows()), dict(qh=8), dict(q=rows(), qh=8),
                                dict(q=rows(), q_out=rows(ts=0), qh=8), dict(r=64, turns=0), dict(r=0), dict(pos=0),
                                dict(layout=3), dict(r=256)])
def test_append_refuses(kw):
    assert append(**kw) == hq.HQ_ERR_ARG


def attention(q=None, out=None, batch=2, tokens=4, max_q=4, max_kv=64, group=4, pg=None, table=A, width=4, stride=4,
              scale=0.1, window=0, start=A, kv=A, lse=A, ws=A, ws_bytes=1 << 40):
    q, out, pg = q or rows(), out or rows(), pg or pages()
    by = ctypes.byref
    return LIB.hq_paged_attention(by(q), start, kv, batch, tokens, max_q, max_kv, group, by(pg), table, width, stride,
                                  scale, 1, window, by(out), lse, ws, ws_bytes, None, None)


@pytest.mark.parametrize("bad,code", BAD_PAGES)
def test_attention_refuses_pages(bad, code):
    assert attention(pg=pages(**bad)) == code


@pytest.mark.parametrize("bad", BAD_ROWS)
def test_attention_refuses_rows(bad):
    assert attention(q=rows(**bad)) == hq.HQ_ERR_ARG
    assert attention(out=rows(**bad)) == hq.HQ_ERR_ARG


@pytest.mark.parametrize("kw,code", [(dict(batch=-1), 1), (dict(max_q=-1), 1), (dict(max_kv=-1), 1), (dict(group=0), 1),
                                     (dict(q=rows(dtype=hq.HQ_F32)), 1), (dict(out=rows(ts=0)), 1), (dict(table=0), 1),
                                     (dict(table=A + 2), 1), (dict(stride=3), 1), (dict(scale=math.inf), 1),
                                     (dict(scale=math.nan), 1), (dict(window=-1), 1), (dict(start=0), 1), (dict(kv=A + 1), 1),
                                     (dict(lse=A + 2), 1), (dict(ws=0), 4), (dict(ws=A + 8), 4), (dict(ws_bytes=64), 4),
                                     (dict(batch=1 << 24), 2), (dict(tokens=1 << 31), 2), (dict(group=40000), 2),
                                     (dict(max_q=1 << 29), 2), (dict(max_kv=(1 << 30) + 1), 2)])
def test_attention_refuses(kw, code):
    assert attention(**kw) == code


def test_attention_of_nothing_is_ok():
    assert attention(batch=0) == 0 and attention(tokens=0) == 0 and attention(max_q=0) == 0


def merge(a=None, b=None, out=None, la=A, lb=A + 4096, lse=A + 8192, tokens=4, heads=8, d=128):
    a, b, out = a or rows(), b or rows(), out or rows()
    by = ctypes.byref
    return LIB.hq_attention_merge(by(a), la, by(b), lb, tokens, heads, d, by(out), lse, None)


@pytest.mark.parametrize("bad", BAD_ROWS)
def test_merge_refuses_rows(bad):
    for name in ("a", "b", "out"):
        assert merge(**{name: rows(**bad)}) == hq.HQ_ERR_ARG


@pytest.mark.parametrize("kw,code", [(dict(la=0), 1), (dict(lb=0), 1), (dict(lse=A), 1), (dict(lse=A + 4096), 1),
                                     (dict(lse=A + 2), 1), (dict(d=12), 1), (dict(d=2048), 1), (dict(tokens=-1), 1),
                                     (dict(tokens=1 << 31), 2), (dict(out=rows(ts=0)), 1)])
def test_merge_refuses(kw, code):
    assert merge(**kw) == code


def test_workspace_sizes():
    small = hq.hq_paged_attention_workspace_bytes(1, 1, 1, 128, 8, 128, 4)
    many = hq.hq_paged_attention_workspace_bytes(100000, 1, 1, 128, 8, 128, 4)
    assert 0 < small < many
    for bad in [(-1, 1, 1, 1, 1, 128, 1), (1, 1, 1, 1, 0, 128, 1), (1, 1, 1, 1, 1, 96, 1), (1, 1, 1, 1, 1, 128, 0)]:
        with pytest.raises(hq.HQError):
            hq.hq_paged_attention_workspace_bytes(*bad)


def test_a_workspace_for_larger_bounds_serves_smaller_calls():
    rng = np.random.default_rng(0)
    for _ in range(3000):
        d, heads, group = int(rng.choice([64, 128, 256])), int(rng.integers(1, 33)), int(rng.integers(1, 9))
        big = [int(2 ** rng.uniform(0, 8)), 0, int(2 ** rng.uniform(0, 9)), int(2 ** rng.uniform(0, 16))]
        small = [max(1, int(v * rng.uniform(0, 1))) for v in big]
        size = lambda b: hq.hq_paged_attention_workspace_bytes(b[0], b[0] * b[2], b[2], b[3], heads, d, group)  # noqa: E731
        assert size(small) <= size(big), (small, big, d, heads, group)


@pytest.mark.skipif(torch.cuda.is_available(), reason="ends at the launch, which has to fail")
def test_any_window_fits_the_workspace_of_the_bounds():
    rng = np.random.default_rng(1)
    for n in range(6000):
        d, heads, group = int(rng.choice([64, 128, 256])), int(rng.integers(1, 33)), int(rng.integers(1, 9))
        batch, max_q = int(2 ** rng.uniform(0, 6)), int(2 ** rng.uniform(0, 7))
        max_kv = int(2 ** rng.integers(8, 17)) if n % 2 else int(2 ** rng.uniform(0, 17))
        size = hq.hq_paged_attention_workspace_bytes(batch, batch * max_q, max_q, max_kv, heads, d, group)
        hs, ts = d, d * heads * group
        by = dict(q=rows(ts=ts, hs=hs), out=rows(ts=ts, hs=hs), batch=batch, tokens=batch * max_q, max_q=max_q, max_kv=max_kv,
                  group=group, ws_bytes=size, pg=pages(heads=heads, head_dim=d, page_stride=16 * d * heads, head_stride=16 * d,
                                                       slot_stride=d))
        for window in (1, max_kv // 2, max_kv - max_q, max_kv - max_q - 1, max_kv, 1 << 31, (1 << 63) - 1):
            if window >= 0:
                assert attention(window=window, **by) == hq.HQ_ERR_CUDA, (batch, max_q, max_kv, heads, group, d, window)


def test_cpu_tensors_and_wrong_shapes_are_refused():
    """The binding refuses what it could only turn into a bad device access."""
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    table = hq.rope_table(64, device="cpu")
    pos = torch.arange(2)
    with pytest.raises(ValueError, match="CUDA"):
        hq.hq_rope(x, pos, table, x)
    with pytest.raises(ValueError):
        hq.hq_rope(x, pos.int(), table, x)
    with pytest.raises(ValueError):
        hq.hq_rope(x, pos[:1], table, x)
    with pytest.raises(ValueError):
        hq.hq_rope(x, pos, table, x[:1])
    pool = hq.alloc_pages(4, 16, 4, 64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        hq.hq_kv_append(x, x, pos, pool)
    with pytest.raises(ValueError):
        hq.hq_kv_append(x, x[:, :2], pos, pool)
    with pytest.raises(ValueError):
        hq.hq_kv_append(x, x, pos, pool, q=x)
    with pytest.raises(ValueError):
        hq.Pages(pool.k, pool.v.float())
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(16, dtype=torch.uint8)
    args = dict(max_q=1, max_kv=16)
    with pytest.raises(ValueError, match="CUDA"):
        hq.hq_paged_attention(x, i32(0, 1, 2), i32(1, 1), pool, i32(0, 1).view(2, 1), 0.1, x, ws, **args)
    with pytest.raises(ValueError):
        hq.hq_paged_attention(x, i32(0, 2), i32(1, 1), pool, i32(0, 1).view(2, 1), 0.1, x, ws, **args)
    with pytest.raises(ValueError):
        hq.hq_paged_attention(x[:, :3], i32(0, 1, 2), i32(1, 1), pool, i32(0, 1).view(2, 1), 0.1, x[:, :3], ws, **args)
    with pytest.raises(ValueError):
        hq.hq_attention_merge(x, torch.zeros(2, 4), x, torch.zeros(2, 3), x)


@pytest.mark.parametrize("scale", [2.4e38, -3.4e38])
def test_attention_refuses_scales_past_the_range_of_its_exponents(scale):
    """The kernels work in powers of two: scale log2 e has to be finite too."""
    assert attention(scale=scale) == hq.HQ_ERR_ARG


@pytest.mark.parametrize("lse", [A + 4, A + 124, A + 4096 - 4, A + 4096 + 124])
def test_merge_refuses_an_lse_that_overlaps_those_it_reads(lse):
    """4 x 8 rows: 128 bytes from A and from A + 4096 are read."""
    assert merge(lse=lse) == hq.HQ_ERR_ARG
