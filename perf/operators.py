"""Attention operators that a decoder layer runs in front of its routed-expert
layer, as they are measured: rotary positions, appending rotated keys and
values to a paged cache, and attention of new tokens over that cache.

Each case has a plain form in elementary torch operations and the call a user
makes of the framework's operator; ``own`` selects which of the two ``run``
makes. ``exact`` gives the operators' definitions in 64 bits.

Definitions. Positions p are integers; freq[i] is the rotation speed of pair i
as a fraction of a turn per position in units of 2^-64, so the angle is
2 pi frac(p freq[i] / 2^64) and p freq[i] may wrap as a 64-bit integer.

- rotary: pair (a, b) -> magnitude (a cos - b sin, b cos + a sin); the pairs of
  the first ``rot`` values of a head are (i, i + rot/2) in the half layout and
  (2i, 2i + 1) interleaved; the other values are copied. ``inverse`` turns the
  other way: the gradient with respect to the input.
- append: q is rotated; k is rotated and written with v to the slots of a
  cache [pages, kv_heads, page, head_dim]; slot = page id * page + offset.
- attention: sequence s has its last n_s tokens in q rows cu_q[s]..cu_q[s+1],
  its kv_len_s keys in the pages of its table row. Query i stands at
  p = kv_len_s - n_s + i and sees key j where j < kv_len_s and (j <= p and
  (window == 0 or j > p - window), or j < prefix_s). The score is
  cap tanh(scale q.k / cap) (or scale q.k) - slope_h |p - j|; outputs are the
  softmax-weighted values and the natural logarithm of the softmax's sum.
"""
import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases
def _rope(tokens, heads, head_dim, rot, layout, dtype, first, inverse=False, factor=1.0,
          fused=False):
    return {"op": "rope", "tokens": tokens, "heads": heads, "head_dim": head_dim, "rot": rot,
            "layout": layout, "dtype": dtype, "first": first, "inverse": inverse,
            "factor": factor, "fused": fused}


def _append(tokens, q_heads, kv_heads, head_dim, rot, page, pool, layout, dtype, prefill):
    return {"op": "append", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rot": rot, "page": page, "pool": pool, "layout": layout,
            "dtype": dtype, "prefill": prefill}


def _attend(batch, new, context, mix, q_heads, kv_heads, head_dim, page, dtype, softcap=0.0,
            window=0, slopes=False, prefix=0):
    return {"op": "attend", "batch": batch, "new": new, "context": context, "mix": mix,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "dtype": dtype, "softcap": softcap, "window": window, "slopes": slopes,
            "prefix": prefix}


def listed():
    cases = {
        # one token of one user: the call's latency
        "rope_one_token": _rope(1, 40, 128, 128, "half", "bf16", 131071),
        # a prefill batch, q inside a fused q/k/v projection, half of each head
        # turned, frequencies stretched eight times for a long context
        "rope_prefill_partial": _rope(8192, 32, 128, 64, "interleaved", "bf16", 0, factor=8.0,
                                      fused=True),
        # a training step's gradient of the keys, an odd number of tokens
        "rope_gradient": _rope(2047, 8, 64, 64, "half", "fp16", 0, inverse=True),
        # the decode step of 64 users
        "append_decode64": _append(64, 32, 8, 128, 128, 16, 65536, "half", "bf16", False),
        # a prefill batch written to large pages
        "append_prefill8192": _append(8192, 32, 8, 128, 128, 64, 16384, "interleaved", "bf16",
                                      True),
        # the next token of one user after 4095: latency, one sequence over the GPU
        "attend_decode1": _attend(1, 1, 4096, "even", 32, 8, 128, 16, "bf16"),
        # the next token of 64 users with contexts of up to 16384: cache bandwidth
        "attend_decode64": _attend(64, 1, 16384, "ragged", 32, 8, 128, 16, "bf16"),
        # four drafted tokens of 33 users to verify, small heads
        "attend_verify4": _attend(33, 4, 4001, "ragged", 16, 4, 64, 32, "fp16"),
        # a chunk of a long prompt over what is cached already
        "attend_chunk_long": _attend(1, 1000, 65536, "even", 32, 8, 128, 64, "bf16"),
        # a whole prompt
        "attend_prefill8192": _attend(1, 8192, 8192, "even", 32, 8, 128, 64, "bf16"),
        # chunks and single tokens in one batch, capped scores, a window
        "attend_mixed_capped": _attend(16, 512, 4096, "mixed", 32, 8, 128, 16, "bf16",
                                       softcap=50.0, window=1024),
        # distance bias and a prefix that all tokens see, an odd head size
        "attend_bias_prefix": _attend(3, 777, 2011, "ragged", 12, 12, 96, 16, "fp16",
                                      slopes=True, prefix=300),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "rope":
        d = rng.choice([64, 96, 128, 256])
        return _rope(_log_int(rng, 1, 8192), rng.randint(1, 40), d,
                     rng.choice([d, d // 2, d // 4]), rng.choice(["half", "interleaved"]), dtype,
                     rng.randint(0, 200000), rng.random() < 0.5, rng.choice([1.0, 8.0]),
                     rng.random() < 0.5)
    d = rng.choice([64, 80, 96, 128, 128])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        tokens = _log_int(rng, 1, 8192)
        return _append(tokens, kv * group, kv, d, rng.choice([d, d // 2]), page,
                       (tokens + page - 1) // page * page * 2 + 16 * page,
                       rng.choice(["half", "interleaved"]), dtype, rng.random() < 0.5)
    limit = {k: max(work(c)[k] for c in listed()) for k in ("flops", "bytes")}
    while True:
        kind = rng.choice(["decode", "chunk", "chunk"])
        context = _log_int(rng, 1, 65536)
        new = rng.randint(1, 4) if kind == "decode" else _log_int(rng, 1, 8192)
        new = min(new, context)
        case = _attend(_log_int(rng, 1, 64), new, context,
                       rng.choice(["even", "ragged", "mixed"]), kv * group, kv, d, page, dtype,
                       rng.choice([0.0, 0.0, 30.0]), rng.choice([0, 0, _log_int(rng, 16, 4096)]),
                       rng.random() < 0.25, rng.choice([0, 0, 0, rng.randint(1, 512)]))
        w = work(case)
        padded = case["batch"] * new * context * case["q_heads"]
        if (padded <= 2 ** 31 and case["batch"] * context * kv * d <= 2 ** 30 and
                w["flops"] <= limit["flops"] / 2 and w["bytes"] <= limit["bytes"] / 2):
            return case


def _lengths(case):
    """New tokens and keys of each sequence: numpy int64 arrays, fixed by the case."""
    rng = random.Random("%(batch)d %(new)d %(context)d %(mix)s" % case)
    n, kv = [], []
    for b in range(case["batch"]):
        new, length = case["new"], case["context"]
        if b and case["mix"] != "even":
            length = rng.randint(max(1, length // 16), length)
            new = rng.randint(1, min(new, length))
            if case["mix"] == "mixed" and b % 4:
                new = 1
        n.append(new)
        kv.append(length)
    return np.array(n, dtype=np.int64), np.array(kv, dtype=np.int64)


# ------------------------------------------------------------------ inputs
def _frequencies(rot, factor, base=10000.0, original=4096):
    """Turns per position in units of 2^-64 of each pair, and the magnitude.
    factor > 1: the pairs that make fewer than one turn within the original
    context are slowed by it, those with more than 32 are not, linearly between."""
    freq = []
    for i in range(rot // 2):
        theta = base ** (-2.0 * i / rot)
        if factor != 1.0:
            keep = min(1.0, max(0.0, (original * theta / (2 * math.pi) - 1.0) / 31.0))
            theta = theta * keep + theta / factor * (1.0 - keep)
        freq.append(int(theta / (2 * math.pi) * 2.0 ** 64))
    return freq, 1.0 if factor == 1.0 else 1.0 + 0.1 * math.log(factor)


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]
    s = {"case": case, "dtype": dtype}
    if case["op"] != "attend":
        freq, s["magnitude"] = _frequencies(case["rot"], case.get("factor", 1.0))
        s["freq"] = torch.tensor(freq, dtype=torch.int64, device="cuda")
    if case["op"] == "rope":
        t, h, d = case["tokens"], case["heads"], case["head_dim"]
        wide = h + (16 if case["fused"] else 0)
        s["x"] = _normal(gen, (t, wide, d), dtype)[:, :h]
        s["positions"] = torch.arange(case["first"], case["first"] + t, dtype=torch.int32,
                                      device="cuda")
        return s
    hq, hk, d, page = case["q_heads"], case["kv_heads"], case["head_dim"], case["page"]
    if case["op"] == "append":
        t = case["tokens"]
        qkv = _normal(gen, (t, hq + 2 * hk, d), dtype)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        pages = -(-case["pool"] // page)
        if case["prefill"]:  # consecutive positions over shuffled pages
            order = torch.randperm(pages, generator=gen, device="cuda")
            pos = torch.arange(t, device="cuda")
            s["slots"] = order[pos // page] * page + pos % page
        else:                # one token of each of many sequences
            s["slots"] = torch.randperm(pages * page, generator=gen, device="cuda")[:t]
            pos = torch.randint(0, 131072, (t,), generator=gen, device="cuda")
        s["positions"] = pos.to(torch.int32)
        max_tokens, max_seqs = t, 1
    else:
        n, kv = _lengths(case)
        s["max_q"] = int(n.max())
        max_tokens, max_seqs = int(n.sum()), len(n)
        s["q"] = _normal(gen, (max_tokens, hq, d), dtype)
        columns = -(-int(kv.max()) // page)
        used = -(-kv // page)
        pages = int(used.sum()) + 1
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        first = torch.from_numpy(np.concatenate([[0], np.cumsum(used)[:-1]])).cuda()
        index = first[:, None] + torch.arange(columns, device="cuda")
        s["page_table"] = order[index.clamp(max=pages - 1)]
        s["cu_q"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).to("cuda", torch.int32)
        s["kv_len"] = torch.from_numpy(kv).to("cuda", torch.int32)
        s["slopes"] = s["prefix"] = None
        if case["slopes"]:
            s["slopes"] = torch.pow(2.0, -8.0 / hq * torch.arange(1, hq + 1, device="cuda",
                                                                  dtype=torch.float32))
        if case["prefix"]:
            s["prefix"] = torch.full((len(n),), case["prefix"], dtype=torch.int32, device="cuda")
    s["k_pages"] = _normal(gen, (pages, hk, page, d), dtype)
    s["v_pages"] = _normal(gen, (pages, hk, page, d), dtype)
    if own:  # the handle a program keeps for its layers
        import w4a16_routed_expert_router_gb300 as moe
        s["layer"] = moe.PagedAttention(hq, hk, d, page, max_tokens, max_seqs, dtype=dtype)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        return _RUN_OWN[case["op"]](s, case)
    return _RUN_PLAIN[case["op"]](s, case)


def _own_rope(s, case):
    import w4a16_routed_expert_router_gb300 as moe
    return moe.moe_attn_rope(s["x"], s["positions"], s["freq"], layout=case["layout"],
                             magnitude=s["magnitude"], inverse=case["inverse"])


def _own_append(s, case):
    q = s["layer"].append(s["q"], s["k"], s["v"], s["positions"], s["slots"], s["k_pages"],
                          s["v_pages"], s["freq"], layout=case["layout"],
                          magnitude=s["magnitude"])
    return q, s["k_pages"], s["v_pages"]


def _own_attend(s, case):
    return s["layer"].forward(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["cu_q"],
                              s["kv_len"], s["max_q"], softcap=case["softcap"],
                              window=case["window"], slopes=s["slopes"], prefix=s["prefix"],
                              return_lse=True)


def _turn(x, positions, freq, layout, magnitude, inverse):
    """Rotary positions of x [tokens, heads, head_dim] in 32 bits."""
    phase = positions.to(torch.int64)[:, None] * freq[None, :]       # wraps: whole turns drop out
    angle = phase.to(torch.float32) * (2.0 * math.pi / 2.0 ** 64)
    cos, sin = angle.cos()[:, None] * magnitude, angle.sin()[:, None] * magnitude
    if inverse:
        sin = -sin
    half = freq.numel()
    f = x.to(torch.float32)
    turned, rest = f[..., :2 * half], f[..., 2 * half:]
    if layout == "half":
        a, b = turned[..., :half], turned[..., half:]
        out = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = turned[..., 0::2], turned[..., 1::2]
        out = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([out, rest], dim=-1).to(x.dtype)


def _plain_rope(s, case):
    return _turn(s["x"], s["positions"], s["freq"], case["layout"], s["magnitude"],
                 case["inverse"])


def _plain_append(s, case):
    args = s["positions"], s["freq"], case["layout"], s["magnitude"], False
    page = torch.div(s["slots"], case["page"], rounding_mode="floor")
    offset = s["slots"] - page * case["page"]
    s["k_pages"][page, :, offset] = _turn(s["k"], *args)
    s["v_pages"][page, :, offset] = s["v"]
    return _turn(s["q"], *args), s["k_pages"], s["v_pages"]


def _plain_attend(s, case):
    """All sequences padded to the longest one."""
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    group, n_max = hq // hk, s["max_q"]
    table, kv_len = s["page_table"].to(torch.int64), s["kv_len"].to(torch.int64)
    cu = s["cu_q"].to(torch.int64)
    batch, n, tokens = kv_len.numel(), cu[1:] - cu[:-1], s["q"].shape[0]

    row = torch.arange(n_max, device="cuda")
    index = (cu[:-1, None] + row).clamp(max=tokens - 1)
    q = s["q"][index].to(torch.float32).view(batch, n_max, hk, group, d)
    q = q.permute(0, 2, 3, 1, 4).reshape(batch, hk, group * n_max, d)
    k = s["k_pages"][table].to(torch.float32).transpose(1, 2).reshape(batch, hk, -1, d)
    v = s["v_pages"][table].to(torch.float32).transpose(1, 2).reshape(batch, hk, -1, d)
    key = torch.arange(k.shape[2], device="cuda")

    x = torch.matmul(q, k.transpose(2, 3)).view(batch, hk, group, n_max, -1)
    x *= 1.0 / math.sqrt(d)
    if case["softcap"]:
        x = (x / case["softcap"]).tanh_() * case["softcap"]
    p = (kv_len - n)[:, None] + row                                   # position of each query
    away = p[:, :, None] - key                                        # [batch, n_max, keys]
    if s["slopes"] is not None:
        x -= s["slopes"].view(1, hk, group, 1, 1) * away.abs()[:, None, None].to(torch.float32)
    seen = away >= 0
    if case["window"]:
        seen &= away < case["window"]
    if s["prefix"] is not None:
        seen |= key < s["prefix"].view(-1, 1, 1)
    seen &= key < kv_len.view(-1, 1, 1)
    x.masked_fill_(~seen[:, None, None], -math.inf)
    top = x.amax(dim=-1, keepdim=True).clamp(min=-1e30)
    x = (x - top).exp_()
    total = x.sum(dim=-1, keepdim=True)
    out = torch.matmul(x.view(batch, hk, group * n_max, -1), v).view(batch, hk, group, n_max, d)
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    lse = (top + total.log()).squeeze(-1)

    token = torch.arange(tokens, device="cuda")
    seq = torch.searchsorted(cu, token, right=True) - 1
    local = token - cu[seq]
    out = out.permute(0, 3, 1, 2, 4).reshape(batch, n_max, hq, d)[seq, local]
    lse = lse.permute(0, 3, 1, 2).reshape(batch, n_max, hq)[seq, local]
    return out.to(s["dtype"]), lse


_RUN_PLAIN = {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}
_RUN_OWN = {"rope": _own_rope, "append": _own_append, "attend": _own_attend}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "rope":
        values = case["tokens"] * case["heads"] * case["head_dim"]
        pairs = case["tokens"] * case["heads"] * case["rot"] // 2
        return {"bytes": 4 * values + 4 * case["tokens"] + 4 * case["rot"], "flops": 6 * pairs}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "append":
        t = case["tokens"]
        return {"bytes": 4 * t * (hq + 2 * hk) * d + 12 * t + 4 * case["rot"],
                "flops": 3 * t * (hq + hk) * case["rot"]}
    n, kv = _lengths(case)
    pairs = keys = 0
    for new, length in zip(n, kv):
        p = np.arange(length - new, length)
        lo = np.maximum(0, p - case["window"] + 1) if case["window"] else np.zeros_like(p)
        prefix = min(case["prefix"], length)
        pairs += int((p + 1 - lo).sum() + np.minimum(prefix, lo).sum() +
                     np.maximum(0, prefix - (p + 1)).sum())
        keys += int(length - lo[0] + min(prefix, lo[0]))
    tokens = int(n.sum())
    pages = int((-(-kv // case["page"])).sum())
    return {"bytes": 4 * tokens * hq * d + 4 * tokens * hq + 4 * keys * hk * d + 4 * pages +
            8 * len(n), "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ the definitions in 64 bits
def _angles(s):
    """Angles [tokens, pairs] of the case's positions; products modulo 2^64."""
    p = s["positions"].cpu().numpy().astype(np.uint64)
    f = s["freq"].cpu().numpy().astype(np.uint64)
    turns = (p[:, None] * f[None, :]).astype(np.float64) / 2.0 ** 64
    return torch.from_numpy(2 * np.pi * turns).cuda()


def _rotated(s, x, angle, layout, sign):
    y = x.to(torch.float64).clone()
    pairs = angle.shape[1]
    if layout == "half":
        first, second = slice(0, pairs), slice(pairs, 2 * pairs)
    else:
        first, second = slice(0, 2 * pairs, 2), slice(1, 2 * pairs, 2)
    z = torch.complex(y[..., first], y[..., second])
    z = z * torch.polar(torch.full_like(angle, s["magnitude"]), sign * angle)[:, None]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _rotated(s, s["x"], _angles(s), case["layout"], -1 if case["inverse"] else 1)
    if case["op"] == "append":
        angle = _angles(s)
        kp, vp = s["k_pages"].to(torch.float64), s["v_pages"].to(torch.float64)
        k = _rotated(s, s["k"], angle, case["layout"], 1)
        for j, slot in enumerate(s["slots"].tolist()):
            kp[slot // case["page"], :, slot % case["page"]] = k[j]
            vp[slot // case["page"], :, slot % case["page"]] = s["v"][j].to(torch.float64)
        return _rotated(s, s["q"], angle, case["layout"], 1), kp, vp
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if work(case)["flops"] > 1e12:
        return None
    cu, kv_len = s["cu_q"].tolist(), s["kv_len"].tolist()
    out = torch.empty((cu[-1], hq, d), dtype=torch.float64, device="cuda")
    lse = torch.empty((cu[-1], hq), dtype=torch.float64, device="cuda")
    for b, length in enumerate(kv_len):
        ids = s["page_table"][b, :-(-length // case["page"])].to(torch.int64)
        j = torch.arange(length, device="cuda")
        for g in range(hk):
            k = s["k_pages"][ids, g].reshape(-1, d)[:length].to(torch.float64)
            v = s["v_pages"][ids, g].reshape(-1, d)[:length].to(torch.float64)
            for h in range(g * (hq // hk), (g + 1) * (hq // hk)):
                step = max(1, 2 ** 26 // length)
                for lo in range(cu[b], cu[b + 1], step):
                    hi = min(lo + step, cu[b + 1])
                    p = torch.arange(lo, hi, device="cuda")[:, None] + (length - cu[b + 1])
                    x = s["q"][lo:hi, h].to(torch.float64) @ k.T / math.sqrt(d)
                    if case["softcap"]:
                        x = case["softcap"] * torch.tanh(x / case["softcap"])
                    if s["slopes"] is not None:
                        x = x - s["slopes"][h].item() * (p - j).abs()
                    ok = j <= p
                    if case["window"]:
                        ok = ok & (j > p - case["window"])
                    if case["prefix"]:
                        ok = ok | (j < case["prefix"])
                    x = torch.where(ok, x, torch.full_like(x, -math.inf))
                    lse[lo:hi, h] = torch.logsumexp(x, dim=1)
                    out[lo:hi, h] = torch.exp(x - lse[lo:hi, h, None]) @ v
    return out, lse
