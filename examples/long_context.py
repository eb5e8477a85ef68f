"""Long contexts on one rank of a tensor-parallel attention block, as a server runs them.

  shared   conversations behind one system prompt: the prompt's keys and values are in the cache once, and
           PrefixAttention reads them once for all conversations;
  selected one long document: PageIndex bounds the keys of its pages, and each step attends to the pages with the
           highest scores alone;
  evicted  endless conversations: AttentionMass adds up the weights that tokens get, and when a conversation has
           grown past a limit Evictor keeps those with the most, in fresh pages; the old ones are free again.

    python examples/long_context.py

runs all three with random projections and prints how far each is from attention in 32 bits over the tokens
that it attends to (the first and the last), or over all tokens (the second: what selecting leaves out).
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from all_gather_gemm_amd import attention as T  # noqa: E402
from all_gather_gemm_amd import long_context as L  # noqa: E402


class Rank:
    """The heads of one rank, a paged cache and the pages that are free in it."""

    def __init__(self, pages, q_heads=8, kv_heads=2, dim=64, page=16, storage="16bit", dtype="bf16", seed=0):
        self.q_heads, self.kv_heads, self.dim, self.page = q_heads, kv_heads, dim, page
        self.geometry = dict(dtype=dtype, storage=storage)
        self.cache = T.PagedCache.empty(pages, page, kv_heads, dim, **self.geometry)
        self.rope = T.Rope(dim, dtype=dtype)
        self.g = torch.Generator().manual_seed(seed)
        self.free = torch.randperm(pages, generator=self.g).tolist()
        self.td = self.cache.torch_dtype

    def take(self, *shape):
        """A page table of free pages."""
        n = math.prod(shape)
        taken, self.free = self.free[:n], self.free[n:]
        return torch.tensor(taken, dtype=torch.int32).view(shape).to("cuda")

    def give(self, table):
        self.free += table.flatten().tolist()

    def slots(self, table, positions):
        """The slots of tokens at these places of each row of a page table."""
        return table.gather(1, positions // self.page).long() * self.page + positions % self.page

    def projected(self, tokens):
        """q, k and v of `tokens` tokens, as a projection would give them."""
        heads = self.q_heads + 2 * self.kv_heads
        qkv = torch.randn((tokens, heads, self.dim), generator=self.g).to(self.td).to("cuda")
        return qkv.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)

    def append(self, table, first, count):
        """`count` new tokens of each row's sequence from position `first` (int32 [batch]) on; returns the rotated
        q of the last one of each."""
        batch = table.shape[0]
        at = first.long()[:, None] + torch.arange(count, device="cuda")
        q, k, v = self.projected(batch * count)
        q = self.cache.append_rope(self.rope, q, k, v, at.flatten(), self.slots(table, at).flatten())
        return q.view(batch, count, self.q_heads, self.dim)[:, -1]

    def reference(self, q, slots):
        """Attention of one q [q_heads, dim] in 32 bits over the tokens in these slots [kv_heads, tokens]."""
        out = []
        for h in range(self.kv_heads):
            k, v = (x[:, h].float() for x in self.cache.read(slots[h].contiguous()))
            mine = q[h * (self.q_heads // self.kv_heads):(h + 1) * (self.q_heads // self.kv_heads)].float()
            out.append(torch.softmax(mine @ k.t().contiguous() / math.sqrt(self.dim), -1) @ v)
        return torch.cat(out)


def off(got, want):
    return float((got.float() - want).norm() / want.norm())


def shared(batch=12, prompt=300, steps=6, **kw):
    r = Rank(64 + 4 * batch, **kw)
    prefix = r.take(1, -(-prompt // r.page))
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    r.append(prefix, zero, prompt)
    prefix_lens = zero + prompt
    own = r.take(batch, 4)
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    attend = L.PrefixAttention(r.q_heads, r.kv_heads, r.dim, **r.geometry)
    for _ in range(steps):
        at = lens.long()[:, None]                      # positions go on behind the prompt's
        q, k, v = r.projected(batch)
        q = r.cache.append_rope(r.rope, q, k, v, at[:, 0] + prompt, r.slots(own, at)[:, 0])
        lens += 1
        out = attend.run(q, r.cache, prefix, prefix_lens, own, lens)
    first = r.slots(prefix, torch.arange(prompt, device="cuda")[None])
    mine = r.slots(own, torch.arange(steps, device="cuda")[None].expand(batch, -1))
    want = [r.reference(q[b], torch.cat((first[0], mine[b])).expand(r.kv_heads, -1)) for b in range(batch)]
    return off(out, torch.stack(want))


def selected(tokens=1500, budget=24, steps=4, **kw):
    pages = -(-(tokens + steps) // kw.get("page", 16))
    r = Rank(pages + 8, **kw)
    table = r.take(1, pages)
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    r.append(table, lens, tokens)
    lens += tokens
    index = L.PageIndex(r.cache)
    index.update(table, lens)                          # the document's pages, once
    attend = T.DecodeAttention(r.q_heads, r.kv_heads, r.dim, **r.geometry)
    for _ in range(steps):
        q = r.append(table, lens, 1)
        lens += 1
        index.update(table, lens, lens - 1)            # the page that has the new token
        pages, n = index.select(q, table, lens, budget)
        out = attend.run(q, r.cache, pages, n)
    at = torch.arange(int(n[0]), device="cuda").expand(r.kv_heads, -1)
    chosen = r.reference(q[0], r.slots(pages[0], at))
    whole = r.reference(q[0], r.slots(table, torch.arange(int(lens[0]), device="cuda")[None]).expand(r.kv_heads, -1))
    return off(out[0], chosen), off(out[0], whole)


def evicted(batch=4, limit=128, keep=64, steps=200, **kw):
    each = -(-limit // kw.get("page", 16))
    r = Rank(2 * batch * each + 4, **kw)
    attend = T.DecodeAttention(r.q_heads, r.kv_heads, r.dim, **r.geometry)
    adder = L.AttentionMass(r.q_heads, r.kv_heads, r.dim, **r.geometry)
    evictor = L.Evictor(keep, sink=4, recent=16)
    table = r.take(batch, each)
    lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
    mass = torch.zeros((batch, r.kv_heads, limit), device="cuda")
    for step in range(steps):
        at = lens.long()[:, None]
        q, k, v = r.projected(batch)
        position = torch.full((batch,), step, dtype=torch.int64, device="cuda")
        q = r.cache.append_rope(r.rope, q, k, v, position, r.slots(table, at)[:, 0])
        lens += 1
        out, lse = attend.run(q, r.cache, table, lens, return_lse=True)
        adder.add(mass, q, lse, r.cache, table, lens, decay=0.99, out=mass)
        if step + 1 < steps and int(lens[0]) == limit:
            fresh = r.take(batch, each)
            lens, _, kept = evictor.run(r.cache, table, lens, mass, fresh)
            r.give(table)
            table, mass = fresh, torch.zeros_like(mass)
            mass[:, :, :keep] = kept
    at = torch.arange(int(lens[0]), device="cuda")[None].expand(batch, -1)
    s = r.slots(table, at)
    want = [r.reference(q[b], s[b].expand(r.kv_heads, -1)) for b in range(batch)]
    return off(out, torch.stack(want)), int(lens[0])


if __name__ == "__main__":
    print(f"shared prompt: {shared():.2g} off")
    chosen, whole = selected()
    print(f"selected pages: {chosen:.2g} off over them, {whole:.2g} over all tokens")
    print("evicted: {:.2g} off over the {} tokens held".format(*evicted()))
