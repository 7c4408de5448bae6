"""The decoder example: its attention against plain attention over what the cache holds, and its graph of a step."""
import math
import os
import sys

import pytest

import bit_moe_expert_routing_gb300 as moe
from bit_moe_expert_routing_gb300 import build, synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def plain_attend(layer, x, batch, pos, lengths, off):
    """attend() in 64 bits over the cache's own values."""
    import decoder
    d = layer.cache.head_dim
    h = torch.nn.functional.rms_norm(x, x.shape[-1:]) @ layer.qkv.T
    q = decoder.rotate(h.view(len(x), -1, d)[:, :layer.heads], pos).double()
    kv = moe.KVBatch(torch.tensor([0] + lengths).cumsum(0).int().cuda(), torch.tensor(lengths).int().cuda(), batch._t[2],
                     sum(lengths), max(lengths), max(lengths))
    keys, vals = (t.double().split(lengths) for t in layer.cache.read(kv))
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lengths):
        rows = slice(off[b], off[b + 1])
        k, v = (t[b].repeat_interleave(layer.heads // layer.kv_heads, 1) for t in (keys, vals))
        s = torch.einsum("thd,khd->htk", q[rows], k) / math.sqrt(d)
        at, key = pos[rows][:, None], torch.arange(n, device="cuda")[None]
        seen = key <= at
        if layer.window:
            seen &= (key > at - layer.window) | (key < layer.sinks)
        out[rows] = torch.einsum("htk,khd->thd", s.masked_fill(~seen, -math.inf).softmax(-1), v)
    return x.double() + out.flatten(1) @ layer.proj.T.double()


def test_the_decoder_serves_ragged_prompts_and_single_tokens():
    import decoder
    build.build()
    D, lengths, steps = 256, [70, 1, 33], 4
    make = lambda i: synth.make_layer(i, D, 16, 4, 128)  # noqa: E731
    dec = decoder.build(2, lengths, steps, 8, 2, 64, 16, make, window=24, sinks=2)
    x = torch.randn(sum(lengths), D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    seen = []
    for layer in dec.layers:
        attend = layer.attend
        layer.attend = lambda x, batch, pos, ws, attend=attend: seen.append((x, batch, pos, attend(x, batch, pos, ws))) or seen[-1][3]
    y = dec.prompt(x)
    assert y.shape == (3, D) and torch.isfinite(y).all()
    # x + o W^T: bf16 roundings of o (bounded by 2^-8 of the values it averages), of the product (2^-9 of a sum over 512
    # of them, once more for a split sum) and of the sum itself; values are of order 4: 2^-5 absolute, 2^-7 relative
    close = dict(atol=2.0 ** -5, rtol=2.0 ** -7)
    off = [0, 70, 71, 104]
    for layer, (xi, batch, pos, got) in zip(dec.layers, seen):
        torch.testing.assert_close(got.double(), plain_attend(layer, xi, batch, pos, lengths, off), **close)
    for t in range(steps):
        seen.clear()
        y = dec.step(y.clone())
        lengths = [n + 1 for n in lengths]
        assert dec.kv_len.tolist() == lengths and torch.isfinite(y).all()
        dec.check()
        if t == 0:
            # the captured step's tensors, filled by the replay: the two calls before were the one outside the capture
            for layer, (xi, batch, pos, got) in zip(dec.layers, seen[2:]):
                torch.testing.assert_close(got.double(), plain_attend(layer, xi, batch, pos, lengths, [0, 1, 2, 3]), **close)
