"""One decoder layer served with the framework: attention over a paged cache,
then the routed-expert layer.

    python examples/decoder_layer.py [--config tiny16|decode64] [--steps 8]
        [--norm] [--cache8] [--window N --sinks M]

Prompts of different lengths are prefilled in chunks, single tokens of some
sequences beside chunks of others in one batch, then every sequence decodes.
--norm puts norms of the heads in front of their rotation, --cache8 holds keys and
values in 8 bits, --window and --sinks hide what lies between a sequence's first
tokens and its last ones.
Weights are random, projections are plain matrix products; the cache, the
rotary positions, the attention and the experts are the framework's kernels.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import moe_synth as ms  # noqa: E402
import w4a16_routed_expert_router_gb300 as moe  # noqa: E402
from moe_synth.device import upload_layer  # noqa: E402


def rms_norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.pow(2).mean(-1, keepdim=True) + 1e-6)).to(x.dtype)


class DecoderLayer:
    """x + attention(norm(x)), then x + experts(norm(x))."""

    def __init__(self, shape: ms.MoeShape, q_heads, kv_heads, head_dim, page_size=16,
                 num_pages=1024, max_tokens=2048, max_seqs=64, device="cuda:0", seed=0,
                 norm=False, cache8=False, window=0, sinks=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        hidden, self.q_heads, self.kv_heads, self.dim = shape.hidden, q_heads, kv_heads, head_dim
        self.device = torch.device(device)

        def weight(rows, cols):
            w = torch.randn(rows, cols, generator=gen, device=device) * cols ** -0.5
            return w.to(torch.bfloat16)

        self.w_qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.w_out = weight(hidden, q_heads * head_dim)
        self.norm = None
        if norm:
            self.norm = moe.HeadNorm(*(1 + 0.1 * torch.randn(head_dim, generator=gen, device=device)
                                       for _ in range(2)))
        self.window, self.sinks = window, sinks
        self.freq, self.magnitude = moe.moe_attn_rope_frequencies(head_dim, device=device)
        dtype = torch.float8_e4m3fn if cache8 else torch.bfloat16
        self.cache = moe.PagedKvCache(num_pages, kv_heads, page_size, head_dim, dtype=dtype,
                                      device=device)
        self.attention_op = moe.PagedAttention(q_heads, kv_heads, head_dim, page_size, max_tokens,
                                               max_seqs, device=device)
        layer = ms.make_layer(shape)
        self.experts = moe.MoeLayer(hidden, shape.experts, shape.top_k, shape.inter,
                                    shape.shared_inter, max_tokens,
                                    upload_layer(layer, device)[0], device=self.device.index)

    def close(self):
        self.attention_op.close()
        self.experts.close()

    def attention(self, x, seqs, counts):
        """x [tokens, hidden]: counts[i] new tokens of sequence seqs[i], in order."""
        positions, slots = [], []
        for s, n in zip(seqs, counts):
            p, where = self.cache.extend(s, n)
            positions += p
            slots += where
        to = dict(device=self.device)
        table, kv_len = self.cache.tables(seqs)
        cu_q = torch.tensor([0] + list(counts), dtype=torch.int32).cumsum(0, dtype=torch.int32)
        qkv = (rms_norm(x) @ self.w_qkv.T).view(len(x), -1, self.dim)
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)
        k_pages, v_pages = self.cache.k_pages, self.cache.v_pages
        q = self.attention_op.append(q, k, v, torch.tensor(positions, dtype=torch.int32, **to),
                                     torch.tensor(slots, dtype=torch.int64, **to), k_pages,
                                     v_pages, self.freq, magnitude=self.magnitude,
                                     norm=self.norm, **self.cache.scales)
        out = self.attention_op.forward(q, k_pages, v_pages, table, cu_q.to(self.device), kv_len,
                                        max(counts), window=self.window, sinks=self.sinks,
                                        **self.cache.scales)
        return x + out.view(len(x), -1) @ self.w_out.T

    def forward(self, x, seqs, counts):
        x = self.attention(x, seqs, counts)
        y = self.experts.forward(rms_norm(x).contiguous().view(torch.int16))
        return x + y.view(torch.bfloat16)

    def check(self):
        """Device errors of both halves (0: none)."""
        return (self.attention_op.check_device_errors() |
                moe.moe_w4a16_check_device_errors(self.experts.handle))


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--config", default="tiny16", choices=["tiny16", "decode64"])
    p.add_argument("--steps", type=int, default=8)
    p.add_argument("--norm", action="store_true", help="norms of the heads of q and k")
    p.add_argument("--cache8", action="store_true", help="keys and values in 8 bits")
    p.add_argument("--window", type=int, default=0, help="last keys that a token sees (0: all)")
    p.add_argument("--sinks", type=int, default=0, help="first keys that it sees all the same")
    args = p.parse_args(argv)
    shape = ms.CONFIGS[args.config]
    heads = (32, 8, 128) if shape.hidden == 4096 else (4, 2, 64)
    layer = DecoderLayer(shape, *heads, norm=args.norm, cache8=args.cache8, window=args.window,
                         sinks=args.sinks)
    gen = torch.Generator(device="cuda:0").manual_seed(1)

    def tokens(n):
        return torch.randn(n, shape.hidden, generator=gen, device="cuda:0").to(torch.bfloat16)

    prompts = {"a": 700, "b": 33, "c": 1}
    layer.forward(tokens(512 + 33), ["a", "b"], [512, 33])           # a chunk of a, all of b
    layer.forward(tokens(188 + 1 + 1), ["a", "b", "c"], [188, 1, 1])  # the rest, and a token of b
    layer.forward(tokens(len(prompts)), list(prompts), [1] * len(prompts))  # the first decode step
    torch.cuda.synchronize()
    begin = time.perf_counter()
    for _ in range(args.steps):
        y = layer.forward(tokens(len(prompts)), list(prompts), [1] * len(prompts))
    torch.cuda.synchronize()
    ms_step = (time.perf_counter() - begin) / max(args.steps, 1) * 1e3
    flags = layer.check()
    lengths = {s: layer.cache.length(s) for s in prompts}
    layer.close()
    print(f"{args.config}: keys {lengths}, {ms_step:.3f} ms a decode step, device errors {flags:#x}")
    return 0 if flags == 0 and bool(torch.isfinite(y.float()).all()) else 1


if __name__ == "__main__":
    sys.exit(main())
