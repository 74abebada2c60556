"""More operators that a decoder layer runs in front of its routed-expert layer,
as they are measured: norms of queries and keys for each head with the rotary
positions in the same pass, and their gradient; a paged cache of 8-bit keys and
values, quantised as it is written and read back; attention over that cache; and
attention with a sliding window and a few first tokens that stay visible.

Each case has a plain form in elementary torch operations and the call a user
makes of the framework's operator; ``own`` selects which of the two ``run``
makes. ``exact`` gives the operators' definitions in 64 bits.

Definitions.

- norm: y = R_p((x / sqrt(mean(x^2) + eps)) * (weight + offset)) for each head of
  each token, R_p the rotary positions of perf/operators.py: a pair's angle at
  position p is 2 pi frac(p freq / 2^64). The weight is one per value of a head,
  for all heads or for each. Gradients, with u = R_p^T dy and n the normed x:
  dweight = sum of u n over what shares it, dx = (h - n mean(h n)) / sqrt(mean(x^2)
  + eps) with h = u (weight + offset).
- 8-bit cache: e4m3 codes [pages, kv_heads, page, head_dim] and a scale for each
  16 tokens (a block) and head, a power of two: a value is code * scale. A token
  with the value x raises its block's scale to the least power of two s with
  |x| <= 448 s, at least 2^-64 and at most 2^64, and is held as x / s rounded to
  the nearest code; codes that the block held go by the new scale, rounded again.
  The first token of a block begins it: what its scale was does not count.
  Reading back gives code * scale.
- attention: as in perf/operators.py, over either cache; query i of a sequence,
  at p = kv_len - n + i, sees key j where j < kv_len and j <= p and (window == 0
  or j > p - window or j < sinks).
"""
import math
import random

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_BLOCK, _TOP, _EXP = 16, 448.0, 64


# ------------------------------------------------------------------ cases
def _norm(tokens, q_heads, kv_heads, head_dim, rot, layout, dtype, wide, each, offset, gradient):
    return {"op": "norm", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads,
            "head_dim": head_dim, "rot": rot, "layout": layout, "dtype": dtype,
            "wide_weight": wide, "weight_each_head": each, "offset": offset,
            "gradient": gradient}


def _cache(batch, new, context, mix, q_heads, kv_heads, head_dim, page, layout, dtype, back):
    return {"op": "cache", "batch": batch, "new": new, "context": context, "mix": mix,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "layout": layout, "dtype": dtype, "back": back}


def _attend(batch, new, context, mix, q_heads, kv_heads, head_dim, page, dtype, bits=8,
            softcap=0.0, window=0, sinks=0):
    return {"op": "attend", "batch": batch, "new": new, "context": context, "mix": mix,
            "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim, "page": page,
            "dtype": dtype, "bits": bits, "softcap": softcap, "window": window, "sinks": sinks}


def listed():
    cases = {
        # one token of one user: the call's latency
        "norm_one_token": _norm(1, 32, 8, 128, 128, "half", "bf16", False, False, 0.0, False),
        # a prefill batch out of a fused projection, weights around zero, half of a head turned
        "norm_prefill8192": _norm(8192, 32, 8, 128, 64, "interleaved", "bf16", True, False, 1.0,
                                  False),
        # a training step's gradients, an odd number of tokens, a weight for each head
        "norm_gradient2047": _norm(2047, 16, 4, 64, 64, "half", "fp16", False, True, 0.0, True),
        # the gradients of a batch of long sequences
        "norm_gradient16384": _norm(16384, 32, 8, 128, 128, "half", "bf16", True, False, 0.0,
                                    True),
        # the decode step of 64 users: a token appended to each, its block read back
        "cache_decode64": _cache(64, 1, 4096, "ragged", 32, 8, 128, 16, "half", "bf16", "block"),
        # a chunk of a prompt behind an odd number of cached tokens, read back whole
        "cache_prefill8191": _cache(1, 8191, 9000, "even", 32, 8, 128, 64, "interleaved", "bf16",
                                    "new"),
        # caches of several users read back for a move to another place
        "cache_read_long": _cache(16, 0, 16384, "ragged", 32, 8, 128, 32, "half", "fp16", "all"),
        # the next token of one user after 4095: latency, one sequence over the GPU
        "attend8_decode1": _attend(1, 1, 4096, "even", 32, 8, 128, 16, "bf16"),
        # the next token of 64 users with contexts of up to 16384: cache bandwidth
        "attend8_decode64": _attend(64, 1, 16384, "ragged", 32, 8, 128, 16, "bf16"),
        # chunks and single tokens over what is cached already, an odd number of keys
        "attend8_chunk_long": _attend(4, 1000, 32767, "mixed", 32, 8, 128, 64, "bf16"),
        # four drafted tokens of 48 users that keep a window and the first tokens, small heads
        "attend_sinks_decode": _attend(48, 4, 30011, "ragged", 16, 4, 64, 32, "fp16",
                                       window=4096, sinks=4),
        # a prompt under a window and the first tokens, 16-bit cache
        "attend_sinks_prompt": _attend(2, 8192, 8192, "even", 16, 4, 128, 16, "bf16", bits=16,
                                       window=1024, sinks=5),
    }
    return [dict(c, name=n) for n, c in cases.items()]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "cache", "attend", "attend"])
    dtype = rng.choice(["bf16", "fp16"])
    kv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 7, 8])
    layout = rng.choice(["half", "interleaved"])
    if op == "norm":
        d = rng.choice([64, 80, 96, 128, 256])
        while kv * group * d > 4096:
            group -= 1
        return _norm(_log_int(rng, 1, 8192), kv * group, kv, d, rng.choice([d, d // 2, d // 4]),
                     layout, dtype, rng.random() < 0.5, rng.random() < 0.3, rng.choice([0.0, 1.0]),
                     rng.random() < 0.6)
    d = rng.choice([64, 80, 96, 128, 128])
    page = rng.choice([16, 32, 64, 128, 256])
    limit = {k: max(work(c)[k] for c in listed() if c["op"] == op) for k in ("flops", "bytes")}
    while True:
        context = _log_int(rng, 1, 32768)
        mix = rng.choice(["even", "ragged", "mixed"])
        batch = _log_int(rng, 1, 64)
        if rng.random() < 0.5:
            new = min(context, rng.randint(1, 4))
        else:
            new = min(context, _log_int(rng, 1, 8192))
        if op == "cache":
            back = rng.choice(["block", "new", "all"])
            case = _cache(batch, new, context, mix, kv * group, kv, d, page, layout, dtype, back)
        else:
            case = _attend(batch, new, context, mix, kv * group, kv, d, page, dtype,
                           rng.choice([8, 8, 8, 16]), rng.choice([0.0, 0.0, 0.0, 30.0]))
            if case["bits"] == 16 or rng.random() < 0.4:
                case["window"] = _log_int(rng, 16, 4096)
                case["sinks"] = rng.randint(1, 64)
        w = work(case)
        padded = batch * new * context * kv * group
        if (padded <= 2 ** 31 and batch * context * kv * d <= 2 ** 30 and
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
            new = rng.randint(min(1, new), min(new, length))
            if case["mix"] == "mixed" and b % 4:
                new = min(new, 1)
        n.append(new)
        kv.append(length)
    return np.array(n, dtype=np.int64), np.array(kv, dtype=np.int64)


def _read_from(case, n, kv):
    """First position that is read back of each sequence: its last block, its new tokens, or all."""
    if case["back"] == "block":
        return np.maximum(kv - 1, 0) // _BLOCK * _BLOCK
    return kv - n if case["back"] == "new" else np.zeros_like(kv)


# ------------------------------------------------------------------ inputs
def _frequencies(rot, base=10000.0):
    return [int(base ** (-2.0 * i / rot) / (2 * math.pi) * 2.0 ** 64) for i in range(rot // 2)]


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _codes(gen, shape):
    """e4m3 codes as a block has them: normal values under a scale that leaves room above."""
    flat = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
    for page in flat.view(torch.uint8).split(max(1, 2 ** 26 // math.prod(shape[1:]))):
        x = torch.randn(page.shape, generator=gen, device="cuda") * 100.0
        page.copy_(x.clamp_(-_TOP, _TOP).to(torch.float8_e4m3fn).view(torch.uint8))
    return flat


def _scales(gen, shape):
    return torch.pow(2.0, torch.randint(-9, -5, shape, generator=gen, device="cuda").float())


def _weights(gen, case, heads, dtype):
    shape = (heads, case["head_dim"]) if case["weight_each_head"] else (case["head_dim"],)
    w = torch.randn(shape, generator=gen, device="cuda") * 0.2 + (1.0 - case["offset"])
    return w if case["wide_weight"] else w.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = _DTYPES[case["dtype"]]
    s = {"case": case, "dtype": dtype, "eps": 1e-6}
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] != "attend":
        s["freq"] = torch.tensor(_frequencies(case.get("rot", d)), dtype=torch.int64,
                                 device="cuda")
    if case["op"] == "norm":
        t = case["tokens"]
        qkv = _normal(gen, (t, hq + 2 * hk, d), dtype)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        s["q_weight"], s["k_weight"] = (_weights(gen, case, h, dtype) for h in (hq, hk))
        first = int(torch.randint(0, 100000, (), generator=gen, device="cuda"))
        s["positions"] = torch.arange(first, first + t, dtype=torch.int32, device="cuda")
        if case["gradient"]:
            s["dq"], s["dk"] = _normal(gen, (t, hq, d), dtype), _normal(gen, (t, hk, d), dtype)
        return s
    page = case["page"]
    n, kv = _lengths(case)
    s["max_q"], tokens = int(n.max()), int(n.sum())
    columns = -(-int(kv.max()) // page)
    used = -(-kv // page)
    pages = int(used.sum()) + 1
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    first = torch.from_numpy(np.concatenate([[0], np.cumsum(used)[:-1]])).cuda()
    index = first[:, None] + torch.arange(columns, device="cuda")
    s["page_table"] = order[index.clamp(max=pages - 1)]
    s["cu_q"] = torch.from_numpy(np.concatenate([[0], np.cumsum(n)])).to("cuda", torch.int32)
    s["kv_len"] = torch.from_numpy(kv).to("cuda", torch.int32)
    shape = (pages, hk, page, d)
    if case.get("bits", 8) == 8:
        s["k_pages"], s["v_pages"] = _codes(gen, shape), _codes(gen, shape)
        s["k_scales"], s["v_scales"] = (_scales(gen, (pages, hk, page // _BLOCK))
                                        for _ in range(2))
    else:
        s["k_pages"], s["v_pages"] = _normal(gen, shape, dtype), _normal(gen, shape, dtype)
        s["k_scales"] = s["v_scales"] = None
    if case["op"] == "cache":
        qkv = _normal(gen, (tokens, hq + 2 * hk, d), dtype)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        s["q_weight"], s["k_weight"] = ((torch.rand(d, generator=gen, device="cuda") + 0.5)
                                        .to(dtype) for _ in range(2))
        seq = np.repeat(np.arange(len(n)), n)
        at = np.arange(tokens) - np.repeat(np.cumsum(n) - n, n) + np.repeat(kv - n, n)
        s["positions"] = torch.from_numpy(at).to("cuda", torch.int32)
        ids = s["page_table"][torch.from_numpy(seq).cuda(), torch.from_numpy(at // page).cuda()]
        s["slots"] = ids.to(torch.int64) * page + torch.from_numpy(at % page).cuda()
        # blocks that hold tokens from before: a sequence's first new token is not its block's
        entered = [i for i in np.flatnonzero(at == np.repeat(kv - n, n)) if at[i] % _BLOCK]
        s["entered"] = s["slots"][torch.tensor(entered, dtype=torch.int64, device="cuda")] // _BLOCK
        lo = _read_from(case, n, kv)
        s["read_first"] = torch.from_numpy(lo).to("cuda", torch.int32)
        s["rows"] = int((kv - lo).sum())
        s["read_cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(kv - lo)])).to(
            "cuda", torch.int32)
    else:
        s["q"] = _normal(gen, (tokens, hq, d), dtype)
    if own:  # the handle a program keeps for its layers
        import w4a16_routed_expert_router_gb300 as moe
        s["layer"] = moe.PagedAttention(hq, hk, d, page, max(tokens, 1), len(n), dtype=dtype)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    if own:
        return _RUN_OWN[case["op"]](s, case)
    return _RUN_PLAIN[case["op"]](s, case)


def _own_norm(s, case):
    import w4a16_routed_expert_router_gb300 as moe
    norm = moe.HeadNorm(s["q_weight"], s["k_weight"], s["eps"], case["offset"])
    if case["gradient"]:
        return moe.moe_attn_norm_rope_backward(s["dq"], s["dk"], s["q"], s["k"], s["positions"],
                                               s["freq"], norm, layout=case["layout"])
    return moe.moe_attn_norm_rope(s["q"], s["k"], s["positions"], s["freq"], norm,
                                  layout=case["layout"])


def _own_cache(s, case):
    import w4a16_routed_expert_router_gb300 as moe
    cache = s["k_pages"], s["v_pages"]
    scales = {"k_scales": s["k_scales"], "v_scales": s["v_scales"]}
    q = None
    if case["new"]:
        norm = moe.HeadNorm(s["q_weight"], s["k_weight"], s["eps"], 0.0)
        q = s["layer"].append(s["q"], s["k"], s["v"], s["positions"], s["slots"], *cache,
                              s["freq"], layout=case["layout"], norm=norm, **scales)
    k, v = s["layer"].read(*cache, s["page_table"], s["read_cu"], s["read_first"], s["rows"],
                           **scales)
    return q, k, v, s["k_scales"], s["v_scales"]


def _own_attend(s, case):
    return s["layer"].forward(s["q"], s["k_pages"], s["v_pages"], s["page_table"], s["cu_q"],
                              s["kv_len"], s["max_q"], softcap=case["softcap"],
                              window=case["window"], sinks=case["sinks"],
                              k_scales=s["k_scales"], v_scales=s["v_scales"], return_lse=True)


def _turn(f, positions, freq, layout, inverse=False):
    """Rotary positions of f [tokens, heads, head_dim], in 32 bits."""
    phase = positions.to(torch.int64)[:, None] * freq[None, :]       # wraps: whole turns drop out
    angle = phase.to(torch.float32) * (2.0 * math.pi / 2.0 ** 64)
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    if inverse:
        sin = -sin
    half = freq.numel()
    turned, rest = f[..., :2 * half], f[..., 2 * half:]
    if layout == "half":
        a, b = turned[..., :half], turned[..., half:]
        out = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = turned[..., 0::2], turned[..., 1::2]
        out = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([out, rest], dim=-1)


def _norm_turn(s, x, weight, offset, layout):
    f = x.to(torch.float32)
    f = f * (f.square().mean(dim=-1, keepdim=True) + s["eps"]).rsqrt()
    return _turn(f * (weight.to(torch.float32) + offset), s["positions"], s["freq"], layout)


def _norm_gradient(s, case, dy, x, weight):
    f = x.to(torch.float32)
    r = (f.square().mean(dim=-1, keepdim=True) + s["eps"]).rsqrt()
    n = f * r
    u = _turn(dy.to(torch.float32), s["positions"], s["freq"], case["layout"], inverse=True)
    h = u * (weight.to(torch.float32) + case["offset"])
    dx = (h - n * (h * n).mean(dim=-1, keepdim=True)) * r
    dw = (u * n).sum(dim=0 if weight.dim() == 2 else (0, 1), dtype=torch.float64)
    return dx.to(x.dtype), dw.to(torch.float32)


def _plain_norm(s, case):
    if case["gradient"]:
        dq, dq_weight = _norm_gradient(s, case, s["dq"], s["q"], s["q_weight"])
        dk, dk_weight = _norm_gradient(s, case, s["dk"], s["k"], s["k_weight"])
        return dq, dk, dq_weight, dk_weight
    return tuple(_norm_turn(s, s[n], s[n + "_weight"], case["offset"],
                            case["layout"]).to(s["dtype"]) for n in ("q", "k"))


def _power_of_two(top):
    """The least power of two s with top <= 448 s, within 2^-64 .. 2^64."""
    m, e = torch.frexp(top / _TOP)
    e = torch.where(m > 0.5, e, e - 1).clamp(-_EXP, _EXP)
    return torch.ldexp(torch.ones_like(top), torch.where(top > 0, e, torch.full_like(e, -_EXP)))


def _to_code(x):
    return x.clamp(-_TOP, _TOP).to(torch.float8_e4m3fn).view(torch.uint8)


def _put(s, f, pages, scales):
    """Values f [tokens, kv_heads, head_dim] to their slots of one half of the cache."""
    page = pages.shape[2]
    block, offset = s["slots"] // _BLOCK, s["slots"] % _BLOCK
    rows = scales.transpose(1, 2).flatten(0, 1).clone()               # [blocks, kv_heads]
    keep = torch.where(offset == 0, 0.0, 1.0)[:, None]
    least = torch.full_like(rows, 2.0 ** -_EXP)
    old = torch.ones_like(rows[:, :1]).index_reduce_(0, block, keep.to(rows.dtype), "amin")
    old = torch.where(old > 0, rows, least)
    top = torch.zeros_like(rows).index_reduce_(0, block, f.abs().amax(dim=-1), "amax")
    now = torch.maximum(old, _power_of_two(top))
    codes = pages.view(torch.uint8)
    e, per = s["entered"], page // _BLOCK
    at = (e // per)[:, None], slice(None), (e % per * _BLOCK)[:, None] + torch.arange(
        _BLOCK, device="cuda")
    held = codes[at].view(torch.float8_e4m3fn).to(torch.float32)     # [blocks, 16, kv_heads, d]
    codes[at] = _to_code(held * (old[e] / now[e])[:, None, :, None])
    codes[s["slots"] // page, :, s["slots"] % page] = _to_code(f / now[block][..., None])
    rows[block] = now[block]
    scales.copy_(rows.view(scales.shape[0], per, -1).transpose(1, 2))


def _read(s, pages, scales, dtype):
    """The rows that are read back, [rows, kv_heads, head_dim]."""
    page, row = pages.shape[2], torch.arange(s["rows"], device="cuda")
    cu = s["read_cu"].to(torch.int64)
    seq = torch.searchsorted(cu, row, right=True) - 1
    at = row - cu[seq] + s["read_first"][seq]
    ids, offset = s["page_table"][seq, at // page].to(torch.int64), at % page
    f = pages.view(torch.uint8)[ids, :, offset].view(torch.float8_e4m3fn).to(torch.float32)
    return (f * scales[ids, :, offset // _BLOCK][..., None]).to(dtype)


def _plain_cache(s, case):
    q = None
    if case["new"]:
        q = _norm_turn(s, s["q"], s["q_weight"], 0.0, case["layout"]).to(s["dtype"])
        _put(s, _norm_turn(s, s["k"], s["k_weight"], 0.0, case["layout"]), s["k_pages"],
             s["k_scales"])
        _put(s, s["v"].to(torch.float32), s["v_pages"], s["v_scales"])
    return (q, _read(s, s["k_pages"], s["k_scales"], s["dtype"]),
            _read(s, s["v_pages"], s["v_scales"], s["dtype"]), s["k_scales"], s["v_scales"])


def _gathered(pages, scales, table):
    """Keys or values of all sequences, [batch, kv_heads, keys, head_dim] in 32 bits."""
    if scales is None:
        f = pages[table].to(torch.float32)
    else:
        f = pages.view(torch.uint8)[table].view(torch.float8_e4m3fn).to(torch.float32)
        b, c, h, p, d = f.shape
        f = f.view(b, c, h, p // _BLOCK, _BLOCK, d).mul_(scales[table][..., None, None])
        f = f.view(b, c, h, p, d)
    return f.transpose(1, 2).reshape(table.shape[0], pages.shape[1], -1, pages.shape[3])


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
    k = _gathered(s["k_pages"], s["k_scales"], table)
    v = _gathered(s["v_pages"], s["v_scales"], table)
    key = torch.arange(k.shape[2], device="cuda")

    x = torch.matmul(q, k.transpose(2, 3)).view(batch, hk, group, n_max, -1)
    x *= 1.0 / math.sqrt(d)
    if case["softcap"]:
        x = (x / case["softcap"]).tanh_() * case["softcap"]
    p = (kv_len - n)[:, None] + row                                   # position of each query
    away = p[:, :, None] - key                                        # [batch, n_max, keys]
    seen = away >= 0
    if case["window"]:
        seen &= (away < case["window"]) | (key < case["sinks"])
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


_RUN_PLAIN = {"norm": _plain_norm, "cache": _plain_cache, "attend": _plain_attend}
_RUN_OWN = {"norm": _own_norm, "cache": _own_cache, "attend": _own_attend}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    hq, hk, d = case["q_heads"], case["kv_heads"], case["head_dim"]
    if case["op"] == "norm":
        t, each = case["tokens"], case["weight_each_head"]
        values = t * (hq + hk) * d
        weights = d * ((hq + hk) if each else 2) * (4 if case["wide_weight"] else 2)
        small = 4 * t + 4 * case["rot"] + weights
        if case["gradient"]:
            return {"bytes": 6 * values + small + 4 * d * ((hq + hk) if each else 2),
                    "flops": 16 * values}
        return {"bytes": 4 * values + small, "flops": 8 * values}
    n, kv = _lengths(case)
    tokens = int(n.sum())
    if case["op"] == "cache":
        lo = _read_from(case, n, kv)
        rows, blocks = int((kv - lo).sum()), int((-(-kv // _BLOCK) - lo // _BLOCK).sum())
        pages = int((-(-kv // case["page"]) - lo // case["page"]).sum())
        written = int((-(-kv // _BLOCK) - (kv - n) // _BLOCK)[n > 0].sum())
        append = tokens * (4 * hq * d + 6 * hk * d + 12) + 8 * written * hk
        read = rows * 6 * hk * d + 8 * blocks * hk + 4 * pages + 8 * len(n)
        return {"bytes": append + 4 * d * (tokens > 0) + read,
                "flops": 8 * tokens * (hq + hk) * d + 4 * (tokens + rows) * hk * d}
    pairs = keys = 0
    for new, length in zip(n, kv):
        p = np.arange(length - new, length)
        lo = np.maximum(0, p - case["window"] + 1) if case["window"] else np.zeros_like(p)
        pairs += int((p + 1 - lo).sum() + np.minimum(case["sinks"], lo).sum())
        keys += int(length - lo[0] + min(case["sinks"], lo[0]))
    pages = int((-(-kv // case["page"])).sum())
    a_key = 4 * d if case["bits"] == 16 else 2 * d + 8 / _BLOCK
    return {"bytes": 4 * tokens * hq * d + 4 * tokens * hq + int(a_key * keys * hk) + 4 * pages +
            8 * len(n), "flops": 4 * pairs * hq * d}


# ------------------------------------------------------------------ the definitions in 64 bits
def _rotated(s, y, layout):
    """Rotary positions in fp64 by complex numbers; angles by products modulo 2^64."""
    p = s["positions"].cpu().numpy().astype(np.uint64)
    f = s["freq"].cpu().numpy().astype(np.uint64)
    turns = torch.from_numpy((p[:, None] * f[None, :]).astype(np.float64) / 2.0 ** 64).cuda()
    unit = torch.polar(torch.ones_like(turns), 2 * math.pi * turns)[:, None]
    rot = 2 * f.size
    if layout == "half":
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * unit
        turned = torch.cat([z.real, z.imag], dim=-1)
    else:
        z = torch.view_as_complex(y[..., :rot].unflatten(-1, (-1, 2)).contiguous()) * unit
        turned = torch.view_as_real(z).flatten(-2)
    return torch.cat([turned, y[..., rot:]], dim=-1)


def _normed(s, x, weight, offset):
    length = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
    return x / torch.sqrt(length ** 2 / x.shape[-1] + s["eps"]) * (weight + offset)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        results, gradients = [], ([], [])
        for n in ("q", "k"):
            x = s[n].to(torch.float64).requires_grad_(case["gradient"])
            w = s[n + "_weight"].to(torch.float64).requires_grad_(case["gradient"])
            y = _rotated(s, _normed(s, x, w, case["offset"]), case["layout"])
            if case["gradient"]:
                y.backward(s["d" + n].to(torch.float64))
                gradients[0].append(x.grad)
                gradients[1].append(w.grad)
            else:
                results.append(y)
        return tuple(results) or (*gradients[0], *gradients[1])
    if case["op"] == "cache":
        return _exact_cache(s, case)
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
            k, v = (_head64(s, half, ids, g)[:length] for half in ("k", "v"))
            for h in range(g * (hq // hk), (g + 1) * (hq // hk)):
                step = max(1, 2 ** 26 // length)
                for lo in range(cu[b], cu[b + 1], step):
                    hi = min(lo + step, cu[b + 1])
                    p = torch.arange(lo, hi, device="cuda")[:, None] + (length - cu[b + 1])
                    x = s["q"][lo:hi, h].to(torch.float64) @ k.T / math.sqrt(d)
                    if case["softcap"]:
                        x = case["softcap"] * torch.tanh(x / case["softcap"])
                    ok = j <= p
                    if case["window"]:
                        ok = ok & ((j > p - case["window"]) | (j < case["sinks"]))
                    x = torch.where(ok, x, torch.full_like(x, -math.inf))
                    lse[lo:hi, h] = torch.logsumexp(x, dim=1)
                    out[lo:hi, h] = torch.exp(x - lse[lo:hi, h, None]) @ v
    return out, lse


def _nearest(x):
    """x rounded to the nearest e4m3 value, of two as near to the one with the even code."""
    code = torch.arange(127, device="cuda")
    exponent, fraction = (code >> 3).to(torch.float64), (code & 7).to(torch.float64)
    value = torch.where(code < 8, fraction / 512, (1 + fraction / 8) * torch.exp2(exponent - 7))
    middle = (value[1:] + value[:-1]) / 2
    below, above = (torch.bucketize(x.abs(), middle, right=r) for r in (False, True))
    return value[torch.where(below % 2 == 0, below, above)] * x.sign()


def _exact_cache(s, case):
    page, (n, kv) = case["page"], _lengths(case)
    lo, cu = _read_from(case, n, kv), s["cu_q"].tolist()
    q, new = None, {"v": s["v"].to(torch.float64)}
    if case["new"]:
        q, new["k"] = (_rotated(s, _normed(s, s[h].to(torch.float64),
                                           s[h + "_weight"].to(torch.float64), 0.0),
                                case["layout"]) for h in ("q", "k"))
    values, scales = {"k": [], "v": []}, {h: s[h + "_scales"].to(torch.float64) for h in "kv"}
    for half in "kv":
        for b, length in enumerate(kv.tolist()):
            at = torch.arange(length, device="cuda")
            ids, block = s["page_table"][b, at // page].to(torch.int64), at % page // _BLOCK
            f = s[half + "_pages"].view(torch.uint8)[ids, :, at % page].view(
                torch.float8_e4m3fn).to(torch.float64)
            f = f * scales[half][ids, :, block][..., None]
            if n[b]:
                old = length - int(n[b])
                begin = old // _BLOCK * _BLOCK
                f[old:] = new[half][cu[b]:cu[b + 1]]
                top = f.abs().amax(dim=-1)
                top[begin:old] = 0
                top = torch.nn.functional.pad(top[begin:], (0, 0, 0, -length % _BLOCK))
                top = top.view(-1, _BLOCK, top.shape[1]).amax(dim=1)
                scale = torch.exp2(torch.ceil(torch.log2(top / _TOP)).clamp(-_EXP, _EXP))
                if old % _BLOCK:
                    scale[0] = torch.maximum(scale[0], scales[half][ids[begin], :, block[begin]])
                each = scale.repeat_interleave(_BLOCK, 0)[:length - begin, :, None]
                f[begin:] = _nearest((f[begin:] / each).clamp(-_TOP, _TOP)) * each
                scales[half][ids[begin::_BLOCK], :, block[begin::_BLOCK]] = scale
            values[half].append(f[int(lo[b]):])
    # Keys are rounded to 8 bits behind the norm and the rotation, whose last bits
    # in 32 decide next to a code's border: they are compared with the plain form's.
    return q, None, torch.cat(values["v"]), scales["k"], scales["v"]


def _head64(s, half, ids, g):
    """One sequence's keys or values of kv head g, [keys, head_dim] in fp64."""
    pages, scales = s[half + "_pages"], s[half + "_scales"]
    if scales is None:
        return pages[ids, g].reshape(-1, pages.shape[3]).to(torch.float64)
    f = pages.view(torch.uint8)[ids, g].view(torch.float8_e4m3fn).to(torch.float64)
    f = f.reshape(-1, pages.shape[3])
    return f * scales[ids, g].to(torch.float64).reshape(-1, 1).repeat_interleave(_BLOCK, 0)
