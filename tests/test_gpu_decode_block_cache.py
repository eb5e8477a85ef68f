"""The example's attention block against what its caches hold: its last step from the keys and values as
the caches give them back, so that the bounds of 16 bits hold for coded caches too.

Tolerances (relative, 2-norm of all outputs): q, the heads and the result are each rounded to 16 bits, 2^-9
(bf16) or 2^-12 (f16) of their norm at most, q twice and what that moves in the scores (of magnitude 1)
as much again: under 8 such roundings, 2^-6 and 2^-9."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def last_step(block, x):
    """The step of x [batch, hidden] in 64 bits, from the caches."""
    batch, y = block.batch, 0
    lens = block.lens.tolist()
    position = block.lens.double() - 1
    a = position[:, None] * torch.tensor(block.rope.thetas(), dtype=torch.float64, device=x.device)
    cos, sin = torch.cos(a)[:, None], torch.sin(a)[:, None]
    for r in range(block.ranks):
        q = (x.double() @ block.w_in[r].double()).view(batch, -1, block.dim)[:, :block.q]
        q1, q2 = q.chunk(2, -1)
        q = torch.cat((q1 * cos - q2 * sin, q2 * cos + q1 * sin), -1)
        heads = torch.empty_like(q)
        for b in range(batch):
            t = torch.arange(lens[b], device=x.device)
            slots = block.table[b].long()[t // block.page] * block.page + t % block.page
            k, v = (z.double().repeat_interleave(block.q // block.kv, 1) for z in block.caches[r].read(slots))
            p = torch.softmax((k * q[b]).sum(-1) / math.sqrt(block.dim), 0)
            heads[b] = (p[..., None] * v).sum(0)
        y = y + heads.view(batch, -1) @ block.w_out[r].double()
    return y


@pytest.mark.parametrize("storage", ["16bit", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("dtype,most", [("bf16", 2.0 ** -6), ("f16", 2.0 ** -9)])
@pytest.mark.parametrize("sizes", [{}, dict(ranks=2, hidden=512, q_heads=6, kv_heads=2, head_dim=128, batch=6,
                                            page=8, most=64)])
def test_last_step_from_the_cache(storage, dtype, most, sizes):
    spec = importlib.util.spec_from_file_location(
        "decode_block", os.path.join(ROOT, "examples", "decode_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    block = mod.DecodeBlock(storage=storage, dtype=dtype, **sizes)
    g = torch.Generator().manual_seed(3)
    w = block.w_in[0]
    for _ in range(40):
        x = torch.randn((block.batch, w.shape[0]), generator=g).to(w.dtype).to("cuda")
        y = block.step(x)
    want = last_step(block, x)
    assert float((y.double() - want).norm() / want.norm()) < most
