"""A tensor-parallel attention block that serves, on one GPU standing in for its D ranks.

Each step takes one new token of every sequence through the block as a server would:

  1. AgMatmul: every rank gathers the tokens' rows from the D row shards and multiplies them by its
     columns of the fused q/k/v projection;
  2. PagedCache.append_rope: q and k are rotated, k and v written to the rank's paged cache;
  3. DecodeAttention: the new tokens attend over everything cached so far;
  4. GemmAllReduceFlags: the ranks' heads times their rows of the output projection, summed.

    python examples/decode_block.py [16bit|mxfp8|mxfp4]

runs some steps and compares the last one with the block computed in 32 bits without a cache.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import all_gather_gemm_amd as A  # noqa: E402
from all_gather_gemm_amd import attention as T  # noqa: E402


class DecodeBlock:
    """The block's weights, handles and caches for `batch` sequences of up to `most` tokens."""

    def __init__(self, ranks=4, hidden=1024, q_heads=16, kv_heads=4, head_dim=64, batch=8, most=512,
                 page=16, storage="16bit", dtype="bf16", seed=0):
        g = torch.Generator().manual_seed(seed)
        td = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
        self.ranks, self.batch, self.page = ranks, batch, page
        self.q, self.kv, self.dim = q_heads // ranks, kv_heads // ranks, head_dim
        columns = (self.q + 2 * self.kv) * head_dim
        draw = lambda *s: (torch.randn(s, generator=g) / math.sqrt(s[0])).to(td).to("cuda")  # noqa: E731
        self.w_in = [draw(hidden, columns) for _ in range(ranks)]
        self.w_out = [draw(self.q * head_dim, hidden) for _ in range(ranks)]
        self.project = [A.AgMatmul(ranks, batch, columns, hidden, dtype=dtype, rank=r)
                        for r in range(ranks)]
        self.reduce = A.GemmAllReduceFlags(ranks, batch, hidden, self.q * head_dim, dtype=dtype)
        self.rope = T.Rope(head_dim, dtype=dtype)
        each = -(-most // page)
        self.caches = [T.PagedCache.empty(batch * each, page, self.kv, head_dim, dtype=dtype,
                                          storage=storage) for _ in range(ranks)]
        self.attend = [T.DecodeAttention(self.q, self.kv, head_dim, dtype=dtype, storage=storage)
                       for _ in range(ranks)]
        # the pages of a sequence lie anywhere in the pool
        self.table = torch.randperm(batch * each, generator=g).view(batch, each).int().to("cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def step(self, x):
        """x [batch, hidden]: the new token of every sequence. Returns the block's output."""
        positions = self.lens.long()
        slots = self.table.gather(1, (positions // self.page)[:, None])[:, 0].long() * self.page + \
            positions % self.page
        self.lens += 1
        shards = [s.contiguous() for s in x.chunk(self.ranks)]
        heads = []
        for r in range(self.ranks):
            qkv = self.project[r].run(shards, self.w_in[r]).view(self.batch, -1, self.dim)
            q, k, v = qkv.split([self.q, self.kv, self.kv], dim=1)
            q = self.caches[r].append_rope(self.rope, q, k, v, positions, slots)
            out = self.attend[r].run(q, self.caches[r], self.table, self.lens)
            heads.append(out.view(self.batch, -1))
        return self.reduce.run(heads, self.w_out)

    def reference(self, xs):
        """The last step's output in 32 bits, from all tokens [steps, batch, hidden] at once."""
        steps, batch = xs.shape[:2]
        at = torch.arange(steps, device=xs.device, dtype=torch.float64)
        a = at[:, None] * torch.tensor(self.rope.thetas(), dtype=torch.float64, device=xs.device)
        cos, sin = (f(a).float()[:, None, None] for f in (torch.cos, torch.sin))
        y = 0
        for r in range(self.ranks):
            qkv = (xs.float() @ self.w_in[r].float()).view(steps, batch, -1, self.dim)
            q, k, v = qkv.split([self.q, self.kv, self.kv], dim=2)
            turn = lambda z: torch.cat((  # noqa: E731
                z[..., :self.dim // 2] * cos - z[..., self.dim // 2:] * sin,
                z[..., self.dim // 2:] * cos + z[..., :self.dim // 2] * sin), -1)
            q, k = turn(q)[-1], turn(k).repeat_interleave(self.q // self.kv, 2)
            v = v.repeat_interleave(self.q // self.kv, 2)
            p = torch.softmax((k * q).sum(-1) / math.sqrt(self.dim), 0)
            y = y + (p[..., None] * v).sum(0).view(batch, -1) @ self.w_out[r].float()
        return y


def main(storage="16bit", steps=100, **sizes):
    """Runs `steps` steps; returns how far the last is from the reference, relative."""
    block = DecodeBlock(storage=storage, **sizes)
    g = torch.Generator().manual_seed(1)
    w = block.w_in[0]
    xs = torch.randn((steps, block.batch, w.shape[0]), generator=g).to(w.dtype).to("cuda")
    for x in xs:
        y = block.step(x)
    want = block.reference(xs)
    return float((y.float() - want).norm() / want.norm())


if __name__ == "__main__":
    kind = sys.argv[1] if len(sys.argv) > 1 else "16bit"
    print(f"{kind} cache: the last of 100 steps is {main(kind):.2g} off (relative, 2-norm)")
