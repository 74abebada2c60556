"""The attention operators' definitions in fp64 on the CPU, written out for the
tests: rotary positions, one sequence's attention, and the bounds the kernels'
results have to keep.

Bounds, with u the unit roundoff of the 16-bit type (2^-8 bf16, 2^-11 fp16):
- rotary: |out - ref| <= u |ref| + 2^-20 (|a| + |b|): one rounding of the
  result, and fp32 angles, sines and products on the pair (a, b);
- attention: |out - ref| <= (u |ref| + (u + 1e-4) A) + 2^-24, A the softmax of
  the same scores applied to |v|: one rounding of the result, one of each
  softmax numerator, and fp32 scores (error below 1e-4 / 2 at the sizes and
  values of the tests: 128 products of standard normal values);
  |lse - ref| <= 1e-4 + 2^-22 |ref|, the second term for fp32 scores and sums
  whose own spacing is more than that (up to 2^-23 |ref| each).
fp16 adds 2^-24 per value for results below the normal range.
"""
import math

import numpy as np
import torch

ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def frequencies(rot, base=10000.0):
    return torch.tensor([int(base ** (-2.0 * i / rot) / (2 * math.pi) * 2.0 ** 64)
                         for i in range(rot // 2)], dtype=torch.int64)


def rotary(x, positions, freq, layout, magnitude=1.0, inverse=False):
    """(result, bound without the rounding) in fp64 of x [tokens, heads, dim]."""
    x = x.detach().cpu().double()
    half = freq.numel()
    turns = [[((int(p) * int(f)) % 2 ** 64) / 2.0 ** 64 for f in freq.tolist()]
             for p in positions.tolist()]
    ang = 2 * math.pi * torch.tensor(turns, dtype=torch.float64).reshape(len(turns), half)
    c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None] * (-1 if inverse else 1)
    idx = torch.arange(half)
    ia, ib = (idx, idx + half) if layout == "half" else (2 * idx, 2 * idx + 1)
    a, b = x[..., ia], x[..., ib]
    out, slack = x.clone(), torch.zeros_like(x)
    out[..., ia] = magnitude * (a * c - b * s)
    out[..., ib] = magnitude * (b * c + a * s)
    slack[..., ia] = slack[..., ib] = 2.0 ** -20 * abs(magnitude) * (a.abs() + b.abs())
    return out, slack


def check_rotary(got, want, slack, dtype):
    bound = ROUND[dtype] * want.abs() + slack + 2.0 ** -24
    err = (got.detach().cpu().double() - want).abs()
    assert bool((err <= bound).all()), float((err - bound).max())


def seen_mask(n, kv, window=0, prefix=0):
    p = torch.arange(n)[:, None] + (kv - n)
    j = torch.arange(kv)[None, :]
    ok = j <= p
    if window:
        ok = ok & (j > p - window)
    return ok | (j < prefix)


def sequence(q, k, v, scale, softcap=0.0, window=0, slopes=None, prefix=0):
    """q [n, hq, d], k and v [kv, hk, d] (any type): (out, A, lse) in fp64."""
    q, k, v = q.double(), k.double(), v.double()
    n, hq, d = q.shape
    kv, hk = k.shape[0], k.shape[1]
    head = torch.arange(hq) // (hq // hk)
    x = torch.einsum("nhd,jhd->hnj", q, k[:, head]) * scale
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    p = torch.arange(n)[:, None] + (kv - n)
    j = torch.arange(kv)[None, :]
    if slopes is not None:
        x = x - slopes.double()[:, None, None] * (p - j).abs()
    x = x.masked_fill(~seen_mask(n, kv, window, prefix), -math.inf)
    if kv == 0:
        return (torch.zeros(n, hq, d, dtype=torch.float64),) * 2 + (
            torch.full((n, hq), -math.inf, dtype=torch.float64),)
    lse = torch.logsumexp(x, dim=-1)
    w = torch.exp(x - torch.where(lse.isinf(), torch.zeros_like(lse), lse)[..., None])
    out = torch.einsum("hnj,jhd->nhd", w, v[:, head])
    a = torch.einsum("hnj,jhd->nhd", w, v[:, head].abs())
    return out, a, lse.T


def check_attention(got, lse, want, a, want_lse, dtype):
    u = ROUND[dtype]
    got = got.detach().cpu().double()
    bound = u * want.abs() + (u + 1e-4) * a + 2.0 ** -24
    err = (got - want).abs()
    assert bool(torch.isfinite(got).all())
    assert bool((err <= bound).all()), (float((err - bound).max()), int((err > bound).sum()))
    if lse is not None:
        lse = lse.detach().cpu().double()
        empty = want_lse.isinf()
        assert bool((lse.isinf() == empty).all()) and bool((lse[empty] < 0).all())
        gap = (lse - want_lse)[~empty].abs()
        assert bool((gap <= 1e-4 + 2.0 ** -22 * want_lse[~empty].abs()).all()), float(gap.max())


class Batch:
    """A ragged batch on the device with its fp64 results."""

    def __init__(self, lens, hq, hk, d, page, dtype, seed=0, device="cuda:0", softcap=0.0,
                 window=0, slopes=False, prefix=None, poison=True, heads_inner=True, scale=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.dtype, self.device, self.page = lens, dtype, device, page
        n = [a for a, _ in lens]
        kv = [b for _, b in lens]
        used = [-(-b // page) for b in kv]
        pages = sum(used) + 3
        self.tokens = sum(n)
        q = torch.randn(self.tokens, hq, d, generator=g).to(dtype)
        # pages nothing uses, and rows behind a sequence's end, hold NaN
        kp = torch.full((pages, hk, page, d), math.nan if poison else 0.0).to(dtype)
        vp = kp.clone()
        order = torch.randperm(pages, generator=g)[:sum(used)].tolist()
        columns = max(used + [1]) + 1
        table = torch.full((len(lens), columns), 2 ** 31 - 1, dtype=torch.int32)
        self.scale = d ** -0.5 if scale is None else scale
        self.softcap, self.window = softcap, window
        sl = torch.rand(hq, generator=g) * 0.1 if slopes else None
        pre = prefix if prefix is not None else [0] * len(lens)
        outs, bounds, lses = [], [], []
        row = 0
        for s, (a, b) in enumerate(lens):
            k = torch.randn(b, hk, d, generator=g).to(dtype)
            v = torch.randn(b, hk, d, generator=g).to(dtype)
            for c in range(used[s]):
                pid = order.pop()
                table[s, c] = pid
                m = min(page, b - c * page)
                kp[pid, :, :m] = k[c * page:c * page + m].transpose(0, 1)
                vp[pid, :, :m] = v[c * page:c * page + m].transpose(0, 1)
            o, bound, l = sequence(q[row:row + a], k, v, self.scale, softcap, window, sl,
                                   max(0, pre[s]))
            outs.append(o)
            bounds.append(bound)
            lses.append(l)
            row += a
        self.want, self.bound, self.want_lse = torch.cat(outs), torch.cat(bounds), torch.cat(lses)
        cu = np.concatenate([[0], np.cumsum(n)])
        self.q = q.to(device)
        if heads_inner:
            self.k_pages, self.v_pages = kp.to(device), vp.to(device)
        else:  # [pages, page, heads, dim] in memory
            self.k_pages = kp.transpose(1, 2).contiguous().to(device).transpose(1, 2)
            self.v_pages = vp.transpose(1, 2).contiguous().to(device).transpose(1, 2)
        self.table = table.to(device)
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device=device)
        self.kv_len = torch.tensor(kv, dtype=torch.int32, device=device)
        self.max_q = max(n)
        self.slopes = None if sl is None else sl.to(device)
        self.prefix = None if prefix is None else torch.tensor(prefix, dtype=torch.int32,
                                                               device=device)

    def run(self, layer, **kw):
        args = dict(softcap=self.softcap, window=self.window, slopes=self.slopes,
                    prefix=self.prefix, scale=self.scale, return_lse=True)
        args.update(kw)
        return layer.forward(self.q, self.k_pages, self.v_pages, self.table, self.cu_q,
                             self.kv_len, self.max_q, **args)

    def check(self, out, lse):
        check_attention(out, lse, self.want, self.bound, self.want_lse, self.dtype)
