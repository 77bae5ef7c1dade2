"""Plain binary64 forms of the serving operators (rotary positions, paged
append, paged attention, join of partial results) and the error bounds their
kernels are held to."""
import math

import numpy as np
import torch

U32, UB = 2.0 ** -24, 2.0 ** -8  # half a step of binary32 and of bf16, relative


def half_step(dtype):
    return UB if dtype == torch.bfloat16 else U32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(*shape, seed=0, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=gen(seed)) * scale).to(dtype)


# ----------------------------------------------------------------- rotation
def theta_of(r, base, scaling=None):
    """(theta, amplitude) by the definitions, scalar by scalar."""
    out, amp = [], 1.0
    for i in range(r // 2):
        t = base ** (-2 * i / r)
        if scaling:
            f, kind = scaling["factor"], scaling["kind"]
            if kind == "linear":
                t /= f
            elif kind == "ntk":
                t = (base * f ** (r / (r - 2))) ** (-2 * i / r)
            elif kind == "bands":
                n = scaling["original"] * t / (2 * math.pi)
                if n < scaling["low"]:
                    t = t / f
                elif n <= scaling["high"]:
                    s = (n - scaling["low"]) / (scaling["high"] - scaling["low"])
                    t = (1 - s) * t / f + s * t
            elif kind == "yarn":
                def pair(n):
                    return r * math.log(scaling["original"] / (2 * math.pi * n)) / (2 * math.log(base))
                lo, hi = max(math.floor(pair(scaling["fast"])), 0), min(math.ceil(pair(scaling["slow"])), r - 1)
                ramp = min(max((i - lo) / max(hi - lo, 1e-3), 0.0), 1.0)
                t = t / f * ramp + t * (1 - ramp)
                amp = 0.1 * math.log(f) + 1
        out.append(t)
    return np.array(out), amp


def rotate(x, positions, theta, amp, layout, inverse=False):
    """x [tokens, heads, d] -> binary64 rotation (torch double, CPU)."""
    x = x.double().cpu()
    r = 2 * len(theta)
    a = positions.double().cpu()[:, None, None] * torch.as_tensor(theta)
    if inverse:
        a = -a
    c, s = amp * torch.cos(a), amp * torch.sin(a)
    y = x.clone()
    i1, i2 = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i2] * c + x[..., i1] * s
    return y


def rotate_tolerance(x, ref, theta, amp, layout, positions, dtype):
    """cos and sin are each within 2 binary32 steps (sincospif, 2 ulp = 4 U32)
    after one rounding of their argument (U32 of at most pi/4) and one of the
    amplitude product; two products and a sum round once each: under 10 U32 of
    amp (|x1| + |x2|).  The reference's own angle, a binary64 product, is off by
    2^-53 of itself.  Then half a step of the output type."""
    x = x.double().cpu().abs()
    r = 2 * len(theta)
    tol = torch.zeros_like(x)
    i1, i2 = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    ang = positions.double().cpu().abs()[:, None, None] * torch.as_tensor(theta) * 2.0 ** -52
    tol[..., i1] = tol[..., i2] = amp * (x[..., i1] + x[..., i2]) * (10 * U32 + ang)
    return tol + half_step(dtype) * (ref.abs() + tol)


# ----------------------------------------------------------------- pages
def make_cache(kv_lens, kvh, d, page, seed=0, spare=2, stale=float("nan"), slot_major=False, k_scale=1.0):
    """(k pool, v pool, table, dense K, dense V): pages in shuffled order, slots
    past a sequence's length and unused pages hold `stale`, unused table
    entries -1.  Pools are [pages, kvh, page, d] (views if slot_major)."""
    rng = np.random.default_rng(seed)
    counts = [-(-n // page) for n in kv_lens]
    total = sum(counts) + spare
    shape = (total, page, kvh, d) if slot_major else (total, kvh, page, d)
    kp, vp = (torch.full(shape, stale, dtype=torch.bfloat16) for _ in range(2))
    if slot_major:
        kp, vp = kp.permute(0, 2, 1, 3), vp.permute(0, 2, 1, 3)
    order = rng.permutation(total)
    width = max(max(counts, default=0), 1)
    table = torch.full((len(kv_lens), width), -1, dtype=torch.int32)
    K, V, at = [], [], 0
    for b, n in enumerate(kv_lens):
        k = randn(n, kvh, d, seed=seed * 1000 + 2 * b, scale=k_scale)
        v = randn(n, kvh, d, seed=seed * 1000 + 2 * b + 1)
        for i in range(counts[b]):
            p = int(order[at])
            at += 1
            table[b, i] = p
            m = min(page, n - i * page)
            kp[p, :, :m] = k[i * page:i * page + m].transpose(0, 1)
            vp[p, :, :m] = v[i * page:i * page + m].transpose(0, 1)
        K.append(k)
        V.append(v)
    return kp, vp, table, K, V


def starts(q_lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(q_lens)]), dtype=torch.int32)


def attend(q, K, V, q_lens, scale, causal=True, window=0):
    """(out, lse, tolerance of a bf16 out, of an fp32 out, of lse) in binary64.
    q [tokens, heads, d] bf16, K[b], V[b] [kv, kvh, d].

    Bound.  The bf16 products of a score are exact in binary32; its d sums are
    each off by at most a binary32 step of the running absolute sum (2 U32: the
    tensor cores may truncate), so a score moves by ds <= 2 (d + 4) U32 |scale|
    sum |q k|, and the exponent's argument and ex2 (2^-22) by 8 U32 (|s| + max)
    + 4 U32: a weight changes by the factor 1 + e, e = expm1 of their sum, in
    numerator and denominator.  The weight's rounding to bf16 (UB) is in the
    numerator alone.  n + 512 binary32 additions (tokens, joins) add
    2 (n + 512) U32.  So |d out| <= (UB (1 + e) + 2 e / (1 - e) + 4 (n + 512) U32)
    sum w|v| / sum w, then half a step of the output type."""
    q = q.double().cpu()
    tokens, heads, d = q.shape
    out = torch.zeros(tokens, heads, d, dtype=torch.float64)
    lse = torch.full((tokens, heads), -math.inf, dtype=torch.float64)
    tol, tol_lse = torch.zeros_like(out), torch.zeros_like(lse)
    at = 0
    for b, nq in enumerate(q_lens):
        kv, kvh = K[b].shape[:2]
        g = heads // kvh
        pos = kv - nq + torch.arange(nq)[:, None]
        t = torch.arange(kv)[None]
        seen = torch.ones(nq, kv, dtype=torch.bool)
        if causal:
            seen &= t <= pos
        if window:
            seen &= t > pos - window
        for h in range(heads):
            if nq == 0 or kv == 0:
                continue
            k, v = K[b][:, h // g].double(), V[b][:, h // g].double()
            x = q[at:at + nq, h]
            s = scale * x @ k.T
            ds = 2 * (d + 4) * U32 * abs(scale) * (x.abs() @ k.abs().T)
            s, ds = s.masked_fill(~seen, -math.inf), ds.masked_fill(~seen, 0.0)
            any_ = seen.any(1)
            top = torch.where(any_, s.max(1).values, torch.zeros(()).double())
            w = torch.exp(s - top[:, None])
            total = w.sum(1)
            safe = torch.where(any_, total, torch.ones(()).double())
            big = s.masked_fill(~seen, 0.0).abs().max(1).values
            e = torch.expm1(ds.max(1).values + 8 * U32 * (big + top.abs()) + 4 * U32)
            out[at:at + nq, h] = (w @ v) / safe[:, None]
            lse[at:at + nq, h] = torch.where(any_, top + torch.log(safe), torch.full((), -math.inf).double())
            mean = (w @ v.abs()) / safe[:, None]
            acc = 4 * (kv + 512) * U32
            tol[at:at + nq, h] = (UB * (1 + e) + 2 * e / (1 - e) + acc)[:, None] * mean
            tol_lse[at:at + nq, h] = e + acc + 8 * U32 * (1 + lse[at:at + nq, h].nan_to_num(neginf=0.0).abs())
        at += nq
    return out, lse, tol + UB * (out.abs() + tol), tol + U32 * (out.abs() + tol), tol_lse


def assert_within(got, ref, tol, what=""):
    got = got.double().cpu()
    off = (got - ref).abs()
    same = (got == ref)  # infinities
    bad = ~(same | (off <= tol))
    assert not bad.any(), (what, int(bad.sum()), got[bad][:4], ref[bad][:4], tol.expand_as(ref)[bad][:4])
