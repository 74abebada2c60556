"""The definitions of include/moe_attn8.h in fp64 on the CPU, written out for the
tests, and the bounds the kernels' results have to keep.

Bounds, with u the unit roundoff of the 16-bit type:
- norm and rotation: |y - ref| <= u |ref| + 2^-19 (|a| + |b|), (a, b) the normed
  pair: one rounding of the result; in fp32 a sum of squares of up to 256 values (at
  most 21 roundings one after the other, half of which the root keeps: 2^-20.6), its
  root (2^-22), the products, cosines and sines (2^-22 each);
- gradient: |dx - ref| <= u |ref| + 2^-18 r (H + |n| mean(H |n|)), H the sum of |dy|
  over the pair times the weight: twice the chain above; |dw - ref| <= 2^-16 sum
  |u n|: the same and at most 200 additions one after the other;
- cache: a value held is the nearest code times the scale, where the value is exact
  (V); where it comes out of a norm and a rotation (K) it is off by half a step of
  the codes there plus the fp32 error above;
- attention as in attn_cases.py, with k and v = code * scale exact.
"""
import math

import torch

from tests import attn_cases as ac

BLOCK, TOP, EXP = 16, 448.0, 64
F8 = torch.float8_e4m3fn

_CODE = torch.arange(127)
VALUE = torch.where(_CODE < 8, _CODE / 512.0,
                    (1 + (_CODE & 7) / 8.0) * torch.exp2((_CODE >> 3).double() - 7)).double()


def nearest(x):
    """fp64 x rounded to the nearest e4m3 value (ties to the even code), saturating."""
    mid = (VALUE[1:] + VALUE[:-1]) / 2
    a = x.abs().clamp(max=TOP)
    below, above = torch.bucketize(a, mid), torch.bucketize(a, mid, right=True)
    return torch.copysign(VALUE[torch.where(below % 2 == 0, below, above)], x)


def half_step(x):
    """Half the distance of the codes around |x| (below 448)."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))).clamp(-6, 8)
    return torch.exp2(e - 4)


def scale_for(top):
    """The least power of two s with top <= 448 s, within 2^-64 .. 2^64 (fp64)."""
    m, e = torch.frexp(top.double() / TOP)
    e = torch.where(m > 0.5, e, e - 1)
    e = torch.where(top > 0, e, torch.full_like(e, -EXP)).clamp(-EXP, EXP)
    return torch.ldexp(torch.ones_like(top, dtype=torch.float64), e)


def normed(x, weight, offset, eps):
    """(n (weight + offset), n, r) in fp64 of x [tokens, heads, dim]."""
    x = x.detach().cpu().double()
    r = 1.0 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    return x * r * (weight.detach().cpu().double() + offset), x * r, r


def norm_rope(x, weight, offset, eps, pos, freq, layout, magnitude=1.0):
    """(result, slack)."""
    y = normed(x, weight, offset, eps)[0]
    out, slack = ac.rotary(y, pos, freq, layout, magnitude)
    rest = torch.where(slack > 0, torch.zeros_like(y), y.abs())
    return out, 2 * slack + 2.0 ** -19 * rest


def norm_rope_gradient(dy, x, weight, offset, eps, pos, freq, layout, magnitude=1.0):
    """(dx, its slack, dw, its slack), dw for each head."""
    w = weight.detach().cpu().double() + offset
    _, n, r = normed(x, weight, offset, eps)
    u, slack = ac.rotary(dy, pos, freq, layout, magnitude, inverse=True)
    pair = torch.where(slack > 0, slack * 2.0 ** 20, u.abs())
    h, big = u * w, pair * w.abs()
    dx = r * (h - n * (h * n).mean(-1, keepdim=True))
    bound = 2.0 ** -18 * r * (big + n.abs() * (big * n.abs()).mean(-1, keepdim=True))
    return dx, bound, (u * n).sum(0), 2.0 ** -16 * (pair * n.abs()).sum(0)


class Cache:
    """A cache in plain fp64 and the rule by which it is written."""

    def __init__(self, pages, heads, page, dim, g, fill=True):
        self.page, self.heads, self.dim = page, heads, dim
        shape = (pages, heads, page, dim)
        blocks = (pages, heads, page // BLOCK)
        self.values, self.scales = {}, {}
        for half in "kv":
            code = torch.randint(0, 127, shape, generator=g) if fill else torch.full(shape, 127)
            code = code + 128 * torch.randint(0, 2, shape, generator=g)
            self.values[half] = code.to(torch.uint8).view(F8)
            self.scales[half] = torch.pow(2.0, torch.randint(-9, -3, blocks, generator=g).float())
            if not fill:
                self.scales[half].fill_(math.nan)

    def held(self, half):
        """code * scale in fp64, [pages, heads, page, dim]."""
        s = self.scales[half].double().repeat_interleave(BLOCK, 2)[..., None]
        return self.values[half].float().double() * s

    def append(self, half, x, slots):
        """x [tokens, heads, dim] fp64 to their slots, one block after the other."""
        t = 0
        while t < len(slots):
            n = 1
            while (t + n < len(slots) and slots[t + n] // BLOCK == slots[t] // BLOCK and
                   slots[t + n] > slots[t + n - 1] >= 0):
                n += 1
            if slots[t] >= 0:
                page, at = slots[t] // self.page, slots[t] % self.page
                block, first = at // BLOCK, at % BLOCK
                finite = torch.where(x[t:t + n].isfinite(), x[t:t + n], torch.zeros(()).double())
                s = scale_for(finite.abs().amax((0, 2)))
                old = self.scales[half][page, :, block].double()
                rows = self.values[half][page, :, block * BLOCK:(block + 1) * BLOCK]
                if first:
                    grown = s > old
                    again = nearest(rows.float().double() * (old / s)[:, None, None])
                    again = torch.where(grown[:, None, None], again, rows.float().double())
                    rows.copy_(again.float().to(F8))
                    s = torch.maximum(s, old)
                for i in range(n):
                    code = nearest(x[t + i] / s[:, None])
                    code = torch.where(x[t + i].isnan(), x[t + i], code)
                    rows[:, slots[t + i] % BLOCK] = code.float().to(F8)
                self.scales[half][page, :, block] = s.float()
            t += n

    def on(self, device):
        return ([self.values[h].to(device) for h in "kv"] +
                [self.scales[h].to(device) for h in "kv"])


def quantised(x):
    """(codes, scales, values fp64) of x [keys, heads, dim] in blocks of 16 keys."""
    keys, heads, dim = x.shape
    pad = -keys % BLOCK
    p = torch.cat([x.double(), torch.zeros(pad, heads, dim, dtype=torch.float64)])
    p = p.view(-1, BLOCK, heads, dim)
    s = scale_for(p.abs().amax((1, 3)))
    code = nearest(p / s[:, None, :, None])
    return (code.view(-1, heads, dim)[:keys], s,
            (code * s[:, None, :, None]).view(-1, heads, dim)[:keys])


class Batch8:
    """A ragged batch over an 8-bit cache with its fp64 results."""

    def __init__(self, lens, hq, hk, d, page, dtype, seed=0, device="cuda:0", softcap=0.0,
                 window=0, slopes=False, prefix=None, sinks=0, heads_inner=True, scale=None,
                 gains=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.dtype, self.device, self.page = lens, dtype, device, page
        self.softcap, self.window, self.sinks = softcap, window, sinks
        self.scale = d ** -0.5 if scale is None else scale
        n, kv = [a for a, _ in lens], [b for _, b in lens]
        used = [-(-b // page) for b in kv]
        pages = sum(used) + 3
        self.tokens = sum(n)
        q = torch.randn(self.tokens, hq, d, generator=g).to(dtype)
        # pages nothing uses, and rows and scales behind a sequence's end, hold NaN
        codes = [torch.full((pages, hk, page, d), math.nan) for _ in "kv"]
        scales = [torch.full((pages, hk, page // BLOCK), math.nan) for _ in "kv"]
        order = torch.randperm(pages, generator=g)[:sum(used)].tolist()
        columns = max(used + [1]) + 1
        table = torch.full((len(lens), columns), 2 ** 31 - 1, dtype=torch.int32)
        sl = torch.rand(hq, generator=g) * 0.1 if slopes else None
        pre = prefix if prefix is not None else [0] * len(lens)
        outs, bounds, lses = [], [], []
        row = 0
        for s, (a, b) in enumerate(lens):
            halves = []
            for half in range(2):
                x = torch.randn(b, hk, d, generator=g).to(dtype)
                if gains is not None:   # blocks of very different sizes
                    each = torch.pow(2.0, torch.randint(*gains[half], (-(-b // BLOCK), 1, 1),
                                                        generator=g).float())
                    x = x * each.repeat_interleave(BLOCK, 0)[:b]
                halves.append(quantised(x))
            for c in range(used[s]):
                pid = order.pop()
                table[s, c] = pid
                m = min(page, b - c * page)
                blocks = -(-m // BLOCK)
                for half in range(2):
                    code, sc, _ = halves[half]
                    codes[half][pid, :, :m] = code[c * page:c * page + m].transpose(0, 1).float()
                    at = c * page // BLOCK
                    scales[half][pid, :, :blocks] = sc[at:at + blocks].T.float()
            o, bound, lse = sequence(q[row:row + a], halves[0][2], halves[1][2], self.scale,
                                     softcap, window, sl, max(0, pre[s]), sinks)
            outs.append(o)
            bounds.append(bound)
            lses.append(lse)
            row += a
        self.want, self.bound, self.want_lse = torch.cat(outs), torch.cat(bounds), torch.cat(lses)
        self.q = q.to(device)
        f8 = [c.to(F8) for c in codes]
        if heads_inner:
            self.k_pages, self.v_pages = (c.to(device) for c in f8)
        else:  # [pages, page, heads, dim] in memory
            self.k_pages, self.v_pages = (
                c.view(torch.uint8).transpose(1, 2).contiguous().to(device).transpose(1, 2).view(F8)
                for c in f8)
        self.k_scales, self.v_scales = (x.to(device) for x in scales)
        self.table = table.to(device)
        cu = torch.tensor([0] + n, dtype=torch.int32).cumsum(0, dtype=torch.int32)
        self.cu_q = cu.to(device)
        self.kv_len = torch.tensor(kv, dtype=torch.int32, device=device)
        self.max_q = max(n)
        self.slopes = None if sl is None else sl.to(device)
        self.prefix = None if prefix is None else torch.tensor(prefix, dtype=torch.int32,
                                                               device=device)

    def run(self, layer, **kw):
        args = dict(softcap=self.softcap, window=self.window, slopes=self.slopes,
                    prefix=self.prefix, scale=self.scale, sinks=self.sinks, return_lse=True,
                    k_scales=self.k_scales, v_scales=self.v_scales)
        args.update(kw)
        return layer.forward(self.q, self.k_pages, self.v_pages, self.table, self.cu_q,
                             self.kv_len, self.max_q, **args)

    def check(self, out, lse):
        ac.check_attention(out, lse, self.want, self.bound, self.want_lse, self.dtype)


def sequence(q, k, v, scale, softcap=0.0, window=0, slopes=None, prefix=0, sinks=0):
    """attn_cases.sequence with first tokens that stay visible."""
    q, k, v = q.double(), k.double(), v.double()
    n, hq, _ = q.shape
    kv, hk = k.shape[0], k.shape[1]
    if kv == 0 or not window or not sinks:
        return ac.sequence(q, k, v, scale, softcap, window, slopes, prefix)
    head = torch.arange(hq) // (hq // hk)
    x = torch.einsum("nhd,jhd->hnj", q, k[:, head]) * scale
    if softcap:
        x = softcap * torch.tanh(x / softcap)
    p = torch.arange(n)[:, None] + (kv - n)
    j = torch.arange(kv)[None, :]
    if slopes is not None:
        x = x - slopes.double()[:, None, None] * (p - j).abs()
    ok = ((j <= p) & ((j > p - window) | (j < sinks))) | (j < prefix)
    x = x.masked_fill(~ok, -math.inf)
    lse = torch.logsumexp(x, dim=-1)
    w = torch.exp(x - lse[..., None])
    out = torch.einsum("hnj,jhd->nhd", w, v[:, head])
    return out, torch.einsum("hnj,jhd->nhd", w, v[:, head].abs()), lse.T
