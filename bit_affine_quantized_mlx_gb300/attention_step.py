"""Greedy decoding through the library's kernels, attention included: a prompt, then steps.

A small stack of layers, each an attention block and a mixture-of-experts layer, on random
weights:

    h -> norm -> q, k, v projections -> lily_qk_norm_rope -> lily_kv8_append
      -> lily_kv8_attention -> output projection -> + h
      -> norm -> lily_q4_moe_prefill / lily_q4_moe_decode -> + h

and lily_q4_gemv_argmax on the last token.  The projections are plain matrix products; everything
else of a layer runs in the library.  Sequences of different lengths share one paged 8-bit cache;
the prompt is one ragged call, each step one token a sequence.

    python -m bit_affine_quantized_mlx_gb300.attention_step [--steps 16] [--prompts 300 77 1]
"""
from __future__ import annotations

import argparse
import os
import sys

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


class Stack:
    """Layers on random weights: hidden width, heads, and a cache of `capacity` tokens a sequence."""

    def __init__(self, hidden=256, q_heads=8, kv_heads=2, head_dim=64, layers=2, experts=16, vocab=4096,
                 sequences=3, capacity=1024, page=64, max_tokens=1024, seed=0):
        import torch
        import bit_affine_quantized_mlx_gb300 as q4
        from bit_affine_quantized_mlx_gb300 import synth
        self.torch, self.q4 = torch, q4
        self.hidden, self.q_heads, self.kv_heads, self.head_dim = hidden, q_heads, kv_heads, head_dim
        self.sequences, self.page, self.pages = sequences, page, -(-capacity // page)
        g = torch.Generator().manual_seed(seed)
        rand = lambda *s: (torch.randn(s, generator=g) * s[-1] ** -0.5).bfloat16().cuda()
        # half of each head is rotated, for contexts four times the original 256 positions
        turns = q4.to_device(q4.lily_rope_turns(head_dim // 2, 10000.0, "yarn", factor=4.0, original_len=256))
        one = lambda: (1 + 0.1 * torch.randn(head_dim, generator=g)).bfloat16().cuda()
        self.layers = []
        for i in range(layers):
            moe = synth.draw_layer(hidden, experts, 2, 128, shared=True, router_std=0.05, router_bias=False,
                                   key=(70 + seed, i))
            self.layers.append({
                "qkv": rand((q_heads + 2 * kv_heads) * head_dim, hidden), "out": rand(hidden, q_heads * head_dim),
                "rope": q4.QKNormRope(head_dim, head_dim // 2, turns, one(), one(),
                                      rope_scale=0.1 * np.log(4.0) + 1.0),
                "cache": q4.KV8Cache.new(sequences * self.pages, kv_heads, page, head_dim),
                "moe": q4.DeviceLayer.upload(moe)})
        self.embed = rand(vocab, hidden)
        self.head = q4.DeviceQ4.upload(synth.draw_q4(vocab, hidden, 71 + seed, 0))
        # pages of a sequence need not be neighbours
        table = torch.randperm(sequences * self.pages, generator=g).reshape(sequences, self.pages)
        self.table = table.to(torch.int32).cuda()
        self.max_tokens = max(max_tokens, 16)
        moe0 = self.layers[0]["moe"]
        self.ws_moe = q4.new_workspace(max(q4.lily_q4_moe_workspace_bytes(moe0, self.max_tokens, prefill=True),
                                           q4.lily_q4_moe_workspace_bytes(moe0, 16)))
        self.ws_head = q4.new_workspace(q4.lily_q4_gemv_argmax_workspace_bytes(vocab, hidden))
        largest = q4.KV8Batch(self.table, torch.zeros(sequences + 1, dtype=torch.int32, device="cuda"),
                              torch.zeros(sequences, dtype=torch.int32, device="cuda"), self.max_tokens, capacity)
        self.ws_kv = q4.new_workspace(q4.lily_kv8_attention_workspace_bytes(
            self.layers[0]["cache"], largest, self.max_tokens, q_heads))

    def _norm(self, x):
        y = x.float()
        return (y * self.torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()

    def forward(self, tokens, counts, lengths):
        """Hidden states of `tokens` (the sequences' new tokens, end to end, counts[b] of each); the
        sequences hold lengths[b] tokens once they are in the cache."""
        torch, q4 = self.torch, self.q4
        T, D = int(tokens.numel()), self.head_dim
        start = np.concatenate([[0], np.cumsum(counts)])
        dev = lambda a: torch.from_numpy(np.asarray(a, np.int32)).cuda()
        batch = q4.KV8Batch(self.table, dev(start), dev(lengths), int(max(counts)), int(max(lengths)))
        pos = dev(np.concatenate([np.arange(n - c, n) for c, n in zip(counts, lengths)]))
        h = self.embed[tokens]
        for layer in self.layers:
            rows = (self._norm(h) @ layer["qkv"].T).view(T, -1, D)
            q, k, v = rows.split([self.q_heads, self.kv_heads, self.kv_heads], 1)
            q4.lily_qk_norm_rope(layer["rope"], q, k, pos, q, k)
            q4.lily_kv8_append(layer["cache"], batch, k, v, ws=self.ws_kv)
            out = torch.empty((T, self.q_heads, D), dtype=torch.bfloat16, device="cuda")
            q4.lily_kv8_attention(layer["cache"], batch, q, out, D ** -0.5, ws=self.ws_kv)
            h = h + out.view(T, -1) @ layer["out"].T
            x = self._norm(h).view(torch.int16)
            y = torch.empty_like(x)
            moe = q4.lily_q4_moe_decode if T <= 16 else q4.lily_q4_moe_prefill
            moe(layer["moe"], x, y, ws=self.ws_moe)
            h = h + y.view(torch.bfloat16)
        return h

    def next_tokens(self, h, counts):
        """The greedy token after each sequence's last row."""
        torch, q4 = self.torch, self.q4
        last = np.cumsum(counts) - 1
        token = torch.empty(len(counts), dtype=torch.int32, device="cuda")
        x = self._norm(h).view(torch.int16)
        for b, row in enumerate(last):
            q4.lily_q4_gemv_argmax(self.head, x[row], token[b:b + 1], ws=self.ws_head)
        return token.long()

    def check(self):
        for ws in (self.ws_kv, self.ws_moe, self.ws_head):
            status = self.q4.lily_q4_workspace_status(ws)
            if status != self.q4.OK:
                raise self.q4.Q4Error(status, "attention_step")


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--prompts", type=int, nargs="*", default=[300, 77, 1], help="prompt lengths")
    ap.add_argument("--steps", type=int, default=16)
    args = ap.parse_args(argv)

    from bit_affine_quantized_mlx_gb300 import build
    build.build()
    import torch
    stack = Stack(sequences=len(args.prompts), capacity=max(args.prompts) + args.steps + 1,
                  max_tokens=sum(args.prompts))
    tokens = torch.randint(0, 4096, (sum(args.prompts),), generator=torch.Generator().manual_seed(1)).cuda()
    counts, lengths = list(args.prompts), list(args.prompts)
    said = []
    for _ in range(args.steps):
        token = stack.next_tokens(stack.forward(tokens, counts, lengths), counts)
        said.append(token)
        tokens, counts, lengths = token, [1] * len(lengths), [n + 1 for n in lengths]
    torch.cuda.synchronize()
    stack.check()
    for b, n in enumerate(args.prompts):
        print(f"sequence {b} ({n} prompt tokens):", " ".join(str(int(t[b])) for t in said))


if __name__ == "__main__":
    main()
