"""Decoder blocks behind a shared prompt: paged attention next to the routed-expert layer.

A batch of sequences continues one common prompt. Each block is

    x = x + attention(rmsnorm(x))      append + forward of PagedAttention
    x = x + experts(rmsnorm(x))        MoELayer

The prompt's keys and values are computed once and stand in pages that every
sequence's attention reads as one prefix; each sequence's own tokens go to
pages of its own. Weights are random: the example shows the calls and their
order, not a trained model. The dense projections are plain torch products.

    python examples/shared_prefix_decode.py --seqs 16 --prompt 1000 --steps 8
"""
import argparse
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from w4a16_routed_expert_gb300 import synth  # noqa: E402
from w4a16_routed_expert_gb300.attention import PagedAttention  # noqa: E402
from w4a16_routed_expert_gb300.layer import MoELayer  # noqa: E402

PAGE = 16


class Block:
    """One decoder block over its own paged cache."""

    def __init__(self, shape, *, q_heads, kv_heads, head_dim, num_pages, max_tokens, max_seqs, seed):
        dev, H = torch.device("cuda"), shape.hidden
        gen = torch.Generator(device=dev).manual_seed(seed)

        def weight(rows, cols):
            return (torch.randn(rows, cols, generator=gen, device=dev) * rows ** -0.5).half()

        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.w_qkv = weight(H, (q_heads + 2 * kv_heads) * head_dim)
        self.w_out = weight(q_heads * head_dim, H)
        self.cache = torch.zeros(2, num_pages, PAGE, kv_heads, head_dim, dtype=torch.float16, device=dev)
        self.attn = PagedAttention(num_q_heads=q_heads, num_kv_heads=kv_heads, head_dim=head_dim, max_tokens=max_tokens,
                                   max_seqs=max_seqs, k_cache=self.cache[0], v_cache=self.cache[1], rotary_dim=head_dim,
                                   q_norm=torch.ones(head_dim, device=dev), k_norm=torch.ones(head_dim, device=dev))
        lay = synth.make_layer(shape, seed=seed)
        self.experts = MoELayer(hidden=H, intermediate=shape.intermediate, num_experts=shape.num_experts,
                                top_k=shape.top_k, group_size=shape.group_size, renormalize=shape.renormalize,
                                max_tokens=max_tokens, router_w=torch.from_numpy(lay.router_w).to(dev),
                                pool=torch.from_numpy(lay.records).to(dev),
                                expert_to_slot=torch.from_numpy(lay.expert_to_slot).to(dev))

    @staticmethod
    def norm(x):
        return torch.nn.functional.rms_norm(x.float(), (x.shape[1],)).half()

    def forward(self, x, positions, slots, batch):
        """x [T][H]: T query tokens at these positions, their keys and values
        to these cache slots, attention over the batch (PagedAttention.forward's
        arguments)."""
        qkv = (self.norm(x) @ self.w_qkv).view(x.shape[0], -1, self.head_dim)
        q, k, v = qkv.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)
        q = self.attn.append(q, k, v, positions, slots)
        x = x + self.attn.forward(q, **batch).flatten(1) @ self.w_out
        return x + self.experts.forward(self.norm(x))


class SharedPrefixDecoder:
    """Blocks and the bookkeeping of their pages: a prompt read by all
    sequences (share=True) or by each from pages of its own (share=False, the
    same numbers computed the long way)."""

    def __init__(self, shape, *, n_blocks, q_heads, kv_heads, head_dim, seqs, prompt_len, max_new, share=True, seed=0):
        self.seqs, self.prompt_len, self.share = seqs, prompt_len, share
        self.own_pages = -(-(max_new + (0 if share else prompt_len)) // PAGE)
        prefix_pages = -(-prompt_len // PAGE)
        num_pages = prefix_pages + seqs * self.own_pages
        dev = torch.device("cuda")
        order = torch.randperm(num_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32)
        self.prefix = order[:prefix_pages].to(dev)
        self.table = order[prefix_pages:].view(seqs, self.own_pages).to(dev)
        self.blocks = [Block(shape, q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, num_pages=num_pages,
                             max_tokens=max(prompt_len, seqs), max_seqs=seqs, seed=seed + i) for i in range(n_blocks)]
        self.offsets = torch.arange(seqs + 1, dtype=torch.int32, device=dev)
        self.new = 0  # tokens each sequence has of its own

    @staticmethod
    def _slots(pages, at):
        return (pages.gather(-1, (at // PAGE).long()) * PAGE + at % PAGE).to(torch.int32)

    def prefill(self, x):
        """The prompt's hidden states x [prompt_len][H], once; returns the
        last block's output."""
        n, dev = self.prompt_len, x.device
        at = torch.arange(n, device=dev, dtype=torch.int32)
        slots = self._slots(self.prefix, at)
        ends = torch.tensor([0, n], dtype=torch.int32, device=dev)
        batch = dict(q_offsets=ends, max_q_len=n, seq_lens=ends[1:], max_seq_len=n, block_table=self.prefix[None])
        for blk in self.blocks:
            x = blk.forward(x, at, slots, batch)
            if not self.share:  # every sequence's own copy of the prompt
                for b in range(self.seqs):
                    own = self._slots(self.table[b], at).long()
                    flat = blk.cache.flatten(1, 2)
                    flat[:, own] = flat[:, slots.long()]
        return x

    def step(self, x):
        """One token of every sequence: hidden states x [seqs][H]."""
        dev = x.device
        before = 0 if self.share else self.prompt_len
        at = torch.full((self.seqs, 1), before + self.new, device=dev, dtype=torch.int32)
        slots = self._slots(self.table, at)[:, 0]
        positions = torch.full((self.seqs,), self.prompt_len + self.new, dtype=torch.int32, device=dev)
        lens = before + self.new + 1
        batch = dict(q_offsets=self.offsets, max_q_len=1, max_seq_len=lens, block_table=self.table,
                     seq_lens=torch.full((self.seqs,), lens, dtype=torch.int32, device=dev),
                     prefix_len=self.prompt_len if self.share else 0, prefix_pages=self.prefix)
        for blk in self.blocks:
            x = blk.forward(x, positions, slots, batch)
        self.new += 1
        return x

    def sync(self):
        for blk in self.blocks:
            blk.attn.sync()
            blk.experts.sync()


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seqs", type=int, default=16)
    ap.add_argument("--prompt", type=int, default=1000)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--blocks", type=int, default=2)
    args = ap.parse_args()
    shape = synth.OLMOE
    gen = torch.Generator(device="cuda").manual_seed(1)
    prompt = torch.randn(args.prompt, shape.hidden, generator=gen, device="cuda").half()
    token = torch.randn(args.seqs, shape.hidden, generator=gen, device="cuda").half()
    for share in (True, False):
        d = SharedPrefixDecoder(shape, n_blocks=args.blocks, q_heads=16, kv_heads=16, head_dim=128, seqs=args.seqs,
                                prompt_len=args.prompt, max_new=args.steps + 1, share=share)
        d.prefill(prompt)
        x = Block.norm(d.step(token))
        d.sync()
        t0 = time.perf_counter()
        for _ in range(args.steps):
            x = Block.norm(d.step(x))
        d.sync()
        ms = (time.perf_counter() - t0) / args.steps * 1e3
        print(f"prompt {'shared' if share else 'copied'}: {ms:.3f} ms a step of {args.seqs} sequences, "
              f"{args.seqs / ms * 1e3:.0f} tokens/s, |x| {float(x.float().abs().mean()):.4f}")


if __name__ == "__main__":
    main()
