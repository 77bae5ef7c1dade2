"""The serving operators beside the codec, as they are measured: rotary positions, the append to a paged
KV cache with the rotation on the way, attention of new tokens over that cache, and the join of two partial
attention results.  `run` computes each in plain torch operations (own = False) or through the package's
entry points (own = True); `exact` computes it again from its definition in binary64.

Shapes: 8 KV heads of 128 with 4 query heads each and up to 32768 cached tokens are the package's own KV
workload; other head sizes (64, 256) and groups are those its attention accepts.  Sequence lengths of a
ragged batch follow from the case alone, every value and page order from the seed."""
import math

import torch

own = False

DEV = "cuda"
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of 32 sequences: the queries alone are rotated; a few microseconds of work
        _rope("rope_step", 32, 32, 128, 128, "half", "plain", 8192, "bf16"),
        # a long prompt far into an extended context: half of each head rotated, binary32 in and out
        _rope("rope_prompt_far", 8191, 32, 128, 64, "interleaved", "yarn", 1 << 20, "f32"),
        # one decoding step of 64 sequences: queries rotated, keys rotated into their pages, values beside them
        _append("append_step", 64, 8, 4, 128, 128, "half", "bands", 131072, "bf16", 64),
        # a prompt's projections as the compressed products leave them (binary32), into small pages
        _append("append_prompt", 8192, 8, 4, 128, 128, "half", "linear", 32768, "f32", 16),
        # few short sequences, one token each: latency
        _attend("decode_short", 4, 1, 700, 8, 8, 64, 16, 0.8, 0, True),
        # one sequence over the package's full KV workload
        _attend("decode_long", 1, 1, 32768, 8, 4, 128, 64, 0.0, 0, False),
        # a full batch of uneven lengths, one token each
        _attend("decode_batch", 64, 1, 8192, 8, 4, 128, 16, 0.9, 0, True),
        # a few drafted tokens per sequence, wide heads, a sliding window
        _attend("draft_window", 16, 7, 6001, 4, 2, 256, 32, 0.7, 1024, False),
        # prompts of uneven lengths, some of them continued
        _attend("prompt_ragged", 8, 1021, 4093, 8, 4, 128, 64, 0.8, 0, True),
        # a chunk of a long prompt: the last 2048 of 32768 tokens
        _attend("chunk_long", 1, 2048, 32768, 8, 4, 128, 64, 0.0, 0, False),
        # one token: the compressed history's binary32 result joined with the recent pages' bf16 one
        _merge("merge_step", 1, 32, 128, "f32", "bf16", "bf16"),
        # a chunk's two partial results
        _merge("merge_chunk", 4099, 32, 128, "bf16", "bf16", "f32"),
    ]


def _rope(name, tokens, heads, d, r, layout, scaling, far, dtype):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "d": d, "r": r, "layout": layout,
            "scaling": scaling, "far": far, "dtype": dtype}


def _append(name, tokens, kvh, group, d, r, layout, scaling, far, dtype, page):
    return {"name": name, "op": "append", "tokens": tokens, "kvh": kvh, "group": group, "d": d, "r": r,
            "layout": layout, "scaling": scaling, "far": far, "dtype": dtype, "page": page}


def _attend(name, batch, q, kv, kvh, group, d, page, spread, window, lse):
    return {"name": name, "op": "attend", "batch": batch, "q": q, "kv": kv, "kvh": kvh, "group": group, "d": d,
            "page": page, "spread": spread, "window": window, "lse": lse}


def _merge(name, tokens, heads, d, a, b, out):
    return {"name": name, "op": "merge", "tokens": tokens, "heads": heads, "d": d, "a": a, "b": b, "out": out}


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    c = _draw(rng)
    c.pop("name")
    return c


def _draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "attend", "attend", "merge"])
    d = rng.choice([64, 128, 128, 256])
    if op == "rope":
        r = rng.choice([d, d // 2, d // 4])
        tokens = _log(rng, 1, 8191 * 128 // max(d, 128))
        return _rope("", tokens, rng.choice([1, 5, 8, 32]), d, r, rng.choice(["half", "interleaved"]),
                     rng.choice(["plain", "linear", "ntk", "bands", "yarn"]), _log(rng, 8192, 1 << 20),
                     rng.choice(["bf16", "f32"]))
    if op == "append":
        r = rng.choice([d, d, d // 2])
        tokens = _log(rng, 1, 8192 * 128 // max(d, 128))
        return _append("", tokens, rng.choice([1, 2, 5, 8]), rng.choice([1, 2, 4]), d, r,
                       rng.choice(["half", "interleaved"]), rng.choice(["plain", "linear", "ntk", "bands", "yarn"]),
                       _log(rng, 8192, 1 << 20), rng.choice(["bf16", "f32"]), rng.choice([16, 32, 64, 128]))
    if op == "merge":
        return _merge("", _log(rng, 1, 4099 * 128 // max(d, 128)), rng.choice([1, 8, 20, 32]), d,
                      rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"]))
    kind = rng.choice(["decode", "decode", "draft", "prompt"])
    kvh, group = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 8])
    batch = _log(rng, 1, 64) if kind != "prompt" else _log(rng, 1, 8)
    q = 1 if kind == "decode" else rng.randint(2, 16) if kind == "draft" else _log(rng, 17, 2048)
    kv = max(q, _log(rng, 1, 32768))
    # no dearer than the dearest listed case, and the plain form's scores fit beside three states
    while batch > 1 and (batch * kv * kvh * d > 64 * 8192 * 8 * 128 // 2 or batch * q * kv * kvh * group > 2048 * 32768 * 32):
        batch -= 1
    while batch * q * kv * kvh * group * d > 2048 * 32768 * 32 * 128:
        kv = max(q, kv // 2) if kv > q else kv
        q = q if kv > q else q // 2
    return _attend("", batch, q, kv, kvh, group, d, rng.choice([16, 32, 64, 128, 256]), rng.choice([0.0, 0.5, 0.9]),
                   rng.choice([0, 0, 0, 100, 1024]), rng.random() < 0.5)


def _lengths(c):
    """(new tokens, cached tokens) of each sequence: the first at the stated lengths, the others up to `spread` shorter."""
    part = [0.0] + [math.modf(i * 0.6180339887498949)[0] for i in range(1, c["batch"])]
    kv = [max(1, int(c["kv"] * (1 - c["spread"] * p))) for p in part]
    q = [max(1, min(n, int(c["q"] * (1 - c["spread"] * math.modf(3 * p)[0])))) for n, p in zip(kv, part)]
    return q, kv


def work(case):
    c = case
    if c["op"] == "rope":
        n = c["tokens"] * c["heads"] * c["d"]
        return {"bytes": 2 * n * _TYPES[c["dtype"]].itemsize + 8 * c["tokens"],
                "flops": 3 * c["tokens"] * c["heads"] * c["r"]}
    if c["op"] == "append":
        rows = c["tokens"] * c["kvh"] * (c["group"] + 2)
        return {"bytes": rows * c["d"] * (_TYPES[c["dtype"]].itemsize + 2) + 16 * c["tokens"],
                "flops": 3 * c["tokens"] * c["kvh"] * (c["group"] + 1) * c["r"]}
    if c["op"] == "merge":
        n, rows = c["tokens"] * c["heads"] * c["d"], c["tokens"] * c["heads"]
        return {"bytes": n * sum(_TYPES[c[k]].itemsize for k in ("a", "b", "out")) + 12 * rows, "flops": 3 * n}
    pairs = read = rows = 0
    for nq, nk in zip(*_lengths(c)):
        w = c["window"] or nk
        first = nk - nq  # the first new token's position
        pairs += sum(min(p + 1, w) for p in range(first, nk))
        read += nk - max(0, first + 1 - w)
        rows += nq
    heads = c["kvh"] * c["group"]
    return {"bytes": 4 * read * c["kvh"] * c["d"] + 4 * rows * heads * c["d"] + (4 * rows * heads if c["lse"] else 0),
            "flops": 4 * pairs * heads * c["d"]}


# ------------------------------------------------------------------ inputs
def _inputs(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)

    if c["op"] == "rope":
        first = int(torch.randint(0, max(1, c["far"] - c["tokens"]), (1,), generator=g, device=DEV))
        return {"x": normal(c["tokens"], c["heads"], c["d"], dtype=_TYPES[c["dtype"]]),
                "positions": first + torch.arange(c["tokens"], device=DEV),
                "y": torch.empty(c["tokens"], c["heads"], c["d"], dtype=_TYPES[c["dtype"]], device=DEV)}
    if c["op"] == "append":
        t, kvh, qh, d = c["tokens"], c["kvh"], c["kvh"] * c["group"], c["d"]
        qkv = normal(t, (qh + 2 * kvh) * d, dtype=_TYPES[c["dtype"]])  # one fused projection's rows
        pages = (t + t // 4) // c["page"] + 2
        return {"q": qkv[:, :qh * d].view(t, qh, d), "k": qkv[:, qh * d:(qh + kvh) * d].view(t, kvh, d),
                "v": qkv[:, (qh + kvh) * d:].view(t, kvh, d),
                "q_out": torch.empty(t, qh, d, dtype=torch.bfloat16, device=DEV),
                "positions": torch.randint(0, c["far"], (t,), generator=g, device=DEV),
                "slots": torch.randperm(pages * c["page"], generator=g, device=DEV)[:t],
                "kp": normal(pages, kvh, c["page"], d, dtype=torch.bfloat16),
                "vp": normal(pages, kvh, c["page"], d, dtype=torch.bfloat16)}
    if c["op"] == "merge":
        shape = (c["tokens"], c["heads"], c["d"])
        return {"a": normal(*shape, dtype=_TYPES[c["a"]]), "b": normal(*shape, dtype=_TYPES[c["b"]]),
                "lse_a": 8 + 2 * normal(*shape[:2]), "lse_b": 8 + 2 * normal(*shape[:2]),
                "out": torch.empty(*shape, dtype=_TYPES[c["out"]], device=DEV),
                "lse": torch.empty(*shape[:2], device=DEV)}
    nq, nk = _lengths(c)
    page, kvh, d, heads = c["page"], c["kvh"], c["d"], c["kvh"] * c["group"]
    count = [-(-n // page) for n in nk]
    kp = normal(sum(count) + 3, kvh, page, d, dtype=torch.bfloat16)
    vp = normal(sum(count) + 3, kvh, page, d, dtype=torch.bfloat16)
    # keys with a spread of scales over the channels, as in key caches
    kp.mul_(torch.exp2(5 * torch.rand(kvh, 1, d, generator=g, device=DEV) - 2).to(torch.bfloat16))
    order = torch.randperm(sum(count) + 3, generator=g, device=DEV).to(torch.int32)
    table = torch.zeros(c["batch"], max(count), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(count):
        table[b, :n] = order[at:at + n]
        at += n
    start = torch.zeros(c["batch"] + 1, dtype=torch.int32)
    start[1:] = torch.cumsum(torch.tensor(nq), 0)
    return {"q": normal(sum(nq), heads, d, dtype=torch.bfloat16), "kp": kp, "vp": vp, "table": table,
            "start": start.to(DEV), "kv_len": torch.tensor(nk, dtype=torch.int32, device=DEV),
            "out": torch.empty(sum(nq), heads, d, dtype=torch.bfloat16, device=DEV),
            "lse": torch.empty(sum(nq), heads, device=DEV) if c["lse"] else None}


_BASE = 500000.0
_SCALING = {"plain": None, "linear": {"kind": "linear", "factor": 4.0}, "ntk": {"kind": "ntk", "factor": 8.0},
            "bands": {"kind": "bands", "factor": 8.0, "low": 1.0, "high": 4.0, "original": 8192},
            "yarn": {"kind": "yarn", "factor": 32.0, "fast": 32.0, "slow": 1.0, "original": 32768}}


def prepare(case, seed):
    c = case
    s = {"case": c, **_inputs(c, seed)}
    if c["op"] in ("rope", "append"):
        s["theta"], s["amplitude"] = _frequencies(c["r"], _SCALING[c["scaling"]])
    if own:
        from kv_quantization_tile_b200 import hq
        if c["op"] in ("rope", "append"):
            s["rope"] = hq.rope_table(c["r"], _BASE, _SCALING[c["scaling"]], layout=c["layout"], device=DEV)
        if c["op"] in ("append", "attend"):
            s["pages"] = hq.Pages(s["kp"], s["vp"])
        if c["op"] == "attend":
            s["workspace"] = hq.alloc_paged_attention_workspace(c["batch"], s["q"].shape[0], c["q"], c["kv"],
                                                                c["kvh"], c["group"], c["d"], device=DEV)
    return s


def _frequencies(r, scaling):
    """Angle per position of each rotated pair (binary64, on the GPU), and the amplitude of the rotation."""
    i = torch.arange(0, r, 2, dtype=torch.float64, device=DEV)
    theta, amplitude = _BASE ** (-i / r), 1.0
    if scaling is None:
        return theta, amplitude
    f = scaling["factor"]
    if scaling["kind"] == "linear":
        theta = theta / f
    elif scaling["kind"] == "ntk":
        theta = (_BASE * f ** (r / (r - 2))) ** (-i / r)
    elif scaling["kind"] == "bands":  # long wavelengths stretched, short ones kept, a blend between
        wave = 2 * math.pi / theta
        blend = (scaling["original"] / wave - scaling["low"]) / (scaling["high"] - scaling["low"])
        blend = blend.clamp(0, 1)
        theta = theta * blend + theta / f * (1 - blend)
    else:  # stretched where the original context holds fewer than `slow` turns, kept above `fast`
        at = [r * math.log(scaling["original"] / (2 * math.pi * n)) / (2 * math.log(_BASE))
              for n in (scaling["fast"], scaling["slow"])]
        lo, hi = max(math.floor(at[0]), 0), min(math.ceil(at[1]), r - 1)
        ramp = ((i / 2 - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        theta = theta / f * ramp + theta * (1 - ramp)
        amplitude = 0.1 * math.log(f) + 1
    return theta, amplitude


# ------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if own:
        return _OWN[c["op"]](s, c)
    return _PLAIN[c["op"]](s, c)


def _own_rope(s, c):
    from kv_quantization_tile_b200 import hq
    return hq.hq_rope(s["x"], s["positions"], s["rope"], s["y"])


def _own_append(s, c):
    from kv_quantization_tile_b200 import hq
    hq.hq_kv_append(s["k"], s["v"], s["slots"], s["pages"], positions=s["positions"], rope=s["rope"], q=s["q"],
                    q_out=s["q_out"])
    return s["q_out"], s["kp"], s["vp"]


def _own_attend(s, c):
    from kv_quantization_tile_b200 import hq
    hq.hq_paged_attention(s["q"], s["start"], s["kv_len"], s["pages"], s["table"], c["d"] ** -0.5, s["out"],
                          s["workspace"], max_q=c["q"], max_kv=c["kv"], window=c["window"], lse=s["lse"])
    return s["out"], s["lse"]


def _own_merge(s, c):
    from kv_quantization_tile_b200 import hq
    hq.hq_attention_merge(s["a"], s["lse_a"], s["b"], s["lse_b"], s["out"], s["lse"])
    return s["out"], s["lse"]


def _rotated(x, positions, theta, amplitude, layout):
    angle = positions.to(torch.float64)[:, None] * theta
    cos = (torch.cos(angle) * amplitude).float()[:, None, :]
    sin = (torch.sin(angle) * amplitude).float()[:, None, :]
    r, x = 2 * theta.numel(), x.float()
    if layout == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        return torch.cat((a * cos - b * sin, b * cos + a * sin, x[..., r:]), -1)
    a, b = x[..., 0:r:2], x[..., 1:r:2]
    return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2), x[..., r:]), -1)


def _plain_rope(s, c):
    return _rotated(s["x"], s["positions"], s["theta"], s["amplitude"], c["layout"]).to(s["x"].dtype)


def _plain_append(s, c):
    turn = lambda x: _rotated(x, s["positions"], s["theta"], s["amplitude"], c["layout"]).to(torch.bfloat16)  # noqa: E731
    page, offset = s["slots"] // c["page"], s["slots"] % c["page"]
    s["kp"][page, :, offset] = turn(s["k"])
    s["vp"][page, :, offset] = s["v"].to(torch.bfloat16)
    return turn(s["q"]), s["kp"], s["vp"]


def _plain_attend(s, c):
    kvh, group, d, q, start = c["kvh"], c["group"], c["d"], s["q"], s["start"].long()
    table, kv_len = s["table"].long(), s["kv_len"].long()
    batch, width = table.shape

    def cached(pool):  # [batch, kv head, token, d], the pages' order undone
        return pool[table].transpose(1, 2).reshape(batch, kvh, width * c["page"], d).float()

    # the new tokens of each sequence, side by side and padded to the longest
    j = torch.arange(c["q"], device=DEV)
    nq = start[1:] - start[:-1]
    row = (start[:-1, None] + j).clamp(max=q.shape[0] - 1)
    x = q[row].view(batch, c["q"], kvh, group, d).permute(0, 2, 3, 1, 4).reshape(batch, kvh, group * c["q"], d).float()
    scores = torch.matmul(x, cached(s["kp"]).transpose(-1, -2)).mul_(d ** -0.5).view(batch, kvh, group, c["q"], -1)
    t = torch.arange(width * c["page"], device=DEV)
    position = (kv_len - nq)[:, None] + j
    seen = (t <= position[..., None]) & (t < kv_len[:, None, None])
    if c["window"]:
        seen &= t > position[..., None] - c["window"]
    scores.masked_fill_(~seen[:, None, None], float("-inf"))
    top = scores.amax(-1, keepdim=True).clamp(min=-1e30)
    scores.sub_(top).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores.view(batch, kvh, group * c["q"], -1), cached(s["vp"])).view(batch, kvh, group, c["q"], d)
    out = (out / total.clamp(min=1e-38)).permute(0, 3, 1, 2, 4).reshape(batch * c["q"], kvh * group, d)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(batch * c["q"], kvh * group)
    # back to packed rows: row r of sequence b is token r - start[b]
    r = torch.arange(q.shape[0], device=DEV)
    b = torch.searchsorted(start[1:], r, right=True)
    pick = b * c["q"] + r - start[b]
    return out[pick].to(torch.bfloat16), lse[pick] if c["lse"] else None


def _plain_merge(s, c):
    top = torch.maximum(s["lse_a"], s["lse_b"])
    wa, wb = torch.exp(s["lse_a"] - top), torch.exp(s["lse_b"] - top)
    out = (wa[..., None] * s["a"].float() + wb[..., None] * s["b"].float()) / (wa + wb)[..., None]
    return out.to(s["out"].dtype), top + torch.log(wa + wb)


_OWN = {"rope": _own_rope, "append": _own_append, "attend": _own_attend, "merge": _own_merge}
_PLAIN = {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend, "merge": _plain_merge}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    c = case
    s = _inputs(c, seed)
    with torch.no_grad():
        if c["op"] == "rope":
            return _turned(s["x"], s["positions"], c)
        if c["op"] == "append":
            kp, vp = s["kp"].double(), s["vp"].double()
            k = _turned(s["k"], s["positions"], c)
            for h in range(c["kvh"]):
                for pool, rows in ((kp, k), (vp, s["v"].double())):
                    flat = pool[:, h].reshape(-1, c["d"])
                    flat[s["slots"]] = rows[:, h]
                    pool[:, h] = flat.view(-1, c["page"], c["d"])
            return _turned(s["q"], s["positions"], c), kp, vp
        if c["op"] == "merge":
            lse = torch.logaddexp(s["lse_a"].double(), s["lse_b"].double())
            out = torch.exp(s["lse_a"].double() - lse)[..., None] * s["a"].double()
            return out + torch.exp(s["lse_b"].double() - lse)[..., None] * s["b"].double(), lse
        return _attended(s, c)


def _turned(x, positions, c):
    """Each pair as a complex number times amplitude * exp(i * position * theta)."""
    r, z = c["r"], x.double()
    theta, amplitude = [], 1.0
    for n in range(r // 2):
        one = math.exp(-2 * n / r * math.log(_BASE))
        if c["scaling"] == "linear":
            one /= 4.0
        elif c["scaling"] == "ntk":
            one = math.exp(-2 * n / r * (math.log(_BASE) + r / (r - 2) * math.log(8.0)))
        elif c["scaling"] == "bands":
            turns = 8192 * one / (2 * math.pi)  # whole turns within the original context
            if turns <= 1.0:
                one /= 8.0
            elif turns < 4.0:
                one = one / 8.0 + (one - one / 8.0) * (turns - 1.0) / 3.0
        elif c["scaling"] == "yarn":
            lo, hi = (r * math.log(32768 / (2 * math.pi * k)) / (2 * math.log(_BASE)) for k in (32.0, 1.0))
            lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), r - 1)
            kept = 1 - min(max((n - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            one = one * kept + one / 32.0 * (1 - kept)
            amplitude = 1 + 0.1 * math.log(32.0)
        theta.append(one)
    angle = positions.double()[:, None, None] * torch.tensor(theta, dtype=torch.float64, device=x.device)
    turn = torch.polar(torch.full_like(angle, amplitude), angle)
    half = c["layout"] == "half"
    pair = torch.complex(z[..., :r // 2], z[..., r // 2:r]) if half else torch.complex(z[..., 0:r:2], z[..., 1:r:2])
    pair = pair * turn
    front = torch.cat((pair.real, pair.imag), -1) if half else torch.view_as_real(pair).flatten(-2)
    return torch.cat((front, z[..., r:]), -1)


def _attended(s, c):
    nq, nk = _lengths(c)
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    at = 0
    for b in range(c["batch"]):
        pages = s["table"][b, :-(-nk[b] // c["page"])].long()
        ages = torch.arange(nk[b] - nq[b], nk[b], device=DEV)[:, None] - torch.arange(nk[b], device=DEV)
        hidden = (ages < 0) | (ages >= (c["window"] or nk[b] + 1))
        for h in range(c["kvh"]):
            k = s["kp"][pages, h].reshape(-1, c["d"])[:nk[b]].double()
            v = s["vp"][pages, h].reshape(-1, c["d"])[:nk[b]].double()
            for g in range(h * c["group"], (h + 1) * c["group"]):
                score = s["q"][at:at + nq[b], g].double() @ k.T / math.sqrt(c["d"])
                score[hidden] = -math.inf
                lse[at:at + nq[b], g] = torch.logsumexp(score, -1)
                out[at:at + nq[b], g] = torch.softmax(score, -1) @ v
        at += nq[b]
    return out, lse if c["lse"] else None
