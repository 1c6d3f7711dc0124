"""One decoder attention block on 4-bit weights and a 4-bit key/value cache.

The block of a 7B-shaped decoder (4096 wide, 32 heads of 128): the fused q|k|v
projection and the o projection are QLoRA NF4 linears; keys and values go to a
paged cache in NF4 codes as they are made, and attention reads them back from
there.  A prompt of each sequence is taken in one call, then tokens one at a
time; every step's output is compared with that of the whole sequence taken as
one prompt, which sees the same codes.  A sequence can also be forked: its tokens
are read back and stored again in another one's pages, and both go on from there.

    python examples/decode_attention.py [--seqs 3] [--prompt 300] [--steps 8]
"""

from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

WIDTH, HEADS, DIM, PAGE, RANK = 4096, 32, 128, 64, 16


class Block:
    """The linears, the cache and each sequence's pages."""

    def __init__(self, seqs: int, max_len: int, generator):
        import torch

        import bit_nf4_quantized_quant_amd as qa
        self.qa = qa
        dev = generator.device

        def draw(*shape, std, dtype=torch.bfloat16):
            return (torch.randn(shape, generator=generator, device=dev) * std).to(dtype)
        self.qkv = qa.quantize(draw(3 * WIDTH, WIDTH, std=0.02, dtype=torch.float32))
        self.o = qa.quantize(draw(WIDTH, WIDTH, std=0.02, dtype=torch.float32))
        self.A, self.B = draw(RANK, WIDTH, std=1 / WIDTH), draw(3 * WIDTH, RANK, std=0.01)
        per_seq = -(-max_len // PAGE)
        self.cache = qa.kv_cache(seqs * per_seq, PAGE, HEADS, DIM, dev)
        self.pages = torch.randperm(seqs * per_seq, generator=generator, device=dev).int().view(seqs, per_seq)
        self.lengths = torch.zeros(seqs, dtype=torch.int32, device=dev)
        self.max_len = max_len

    def step(self, x):
        """x [seqs, n, WIDTH] bf16: n new tokens of each sequence -> the block's output, same shape."""
        import torch
        seqs, n, _ = x.shape
        position = self.lengths[:, None] + torch.arange(n, device=x.device)               # of the new tokens
        slots = self.pages.gather(1, position // PAGE).int() * PAGE + (position % PAGE).int()
        self.lengths += n
        qkv, _ = self.qa.linear_fwd(x.reshape(seqs * n, WIDTH).contiguous(), self.qkv, self.A, self.B, alpha=16.0, want_h=False)
        q, k, v = qkv.view(seqs * n, 3, HEADS, DIM).unbind(1)
        self.qa.kv_write(k, v, self.cache, slots.flatten())
        out, _ = self.qa.kv_attention(q, self.cache, self.pages, self.lengths, max_len=self.max_len)
        y, _ = self.qa.linear_fwd(out.view(seqs * n, WIDTH), self.o, None, None, alpha=0.0)
        return y.view(seqs, n, WIDTH)


    def fork(self, source: int, target: int):
        """Sequence `target` becomes a copy of `source`.  Storing what was read back gives the same values: the largest
        magnitude of a run reads back as its scale."""
        import torch
        position = torch.arange(int(self.lengths[source]), device=self.lengths.device)
        slots = self.pages[:, position // PAGE] * PAGE + (position % PAGE).int()
        k, v = self.qa.kv_read(self.cache, slots[source].contiguous(), torch.float32)
        self.qa.kv_write(k, v, self.cache, slots[target].contiguous())
        self.lengths[target] = self.lengths[source]


def run(seqs: int = 3, prompt: int = 300, steps: int = 8, seed: int = 0) -> float:
    """The largest relative difference (2-norm over a token's output) of the stepwise run from the one-prompt run."""
    import torch
    total = prompt + steps
    x = torch.randn((seqs, total, WIDTH), generator=torch.Generator("cuda").manual_seed(seed + 1), device="cuda").bfloat16()
    stepwise = Block(seqs, total, torch.Generator("cuda").manual_seed(seed))
    parts = [stepwise.step(x[:, :prompt])] + [stepwise.step(x[:, t:t + 1]) for t in range(prompt, total)]
    whole = Block(seqs, total, torch.Generator("cuda").manual_seed(seed)).step(x)
    got, ref = torch.cat(parts, 1).float(), whole.float()
    return float(((got - ref).norm(dim=-1) / ref.norm(dim=-1)).max())


def run_forked(prompt: int = 300, steps: int = 4, seed: int = 0) -> float:
    """The largest difference between a sequence's and its copy's outputs on the same further tokens."""
    import torch
    g = torch.Generator("cuda").manual_seed(seed)
    block = Block(2, prompt + steps, g)
    block.step(torch.randn((2, prompt, WIDTH), generator=g, device="cuda").bfloat16())
    block.fork(0, 1)
    off = 0.0
    for _ in range(steps):
        y = block.step(torch.randn((1, 1, WIDTH), generator=g, device="cuda").bfloat16().expand(2, 1, WIDTH)).float()
        off = max(off, float((y[0] - y[1]).abs().max()))
    return off


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--seqs", type=int, default=3)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=8)
    a = ap.parse_args()
    off = run(a.seqs, a.prompt, a.steps)
    print(f"{a.seqs} sequences, prompt of {a.prompt}, {a.steps} single tokens: largest difference from one prompt {off:.2e}")
    print(f"a copy of a sequence after {a.prompt} tokens: largest difference {run_forked(a.prompt, a.steps):.2e}")


if __name__ == "__main__":
    main()
