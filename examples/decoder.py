"""A small decoder that serves ragged prompts: every layer is attention over a
4-bit paged key/value cache followed by a 4-bit mixture-of-experts layer.

The prompts go through in one ragged step; after that a step takes one token
per sequence and is one CUDA graph, replayed with the lengths and positions
advanced on the device. Weights are random, and a sequence's next input is its
last output, so the example shows the calls and their cost, not text.

    python examples/decoder.py [--layers 2] [--seqs 4] [--prompt 1500] [--steps 64]
"""
import argparse
import ctypes
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402
import torch.nn.functional as F  # noqa: E402

import bit_moe_expert_routing_gb300 as moe  # noqa: E402
from bit_moe_expert_routing_gb300 import synth  # noqa: E402


def rotate(x, pos):
    """Rotary position embedding of x [tokens, heads, head dim] at pos [tokens]."""
    half = x.shape[-1] // 2
    freq = 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float32) / half)
    angle = (pos[:, None].float() * freq)[:, None]
    a, b = x.float().chunk(2, dim=-1)
    return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], dim=-1).to(x.dtype)


class Layer:
    def __init__(self, seed, experts, heads, kv_heads, head_dim, n_pages, page, window=0, sinks=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.experts = experts  # a DeviceLayer
        self.heads, self.kv_heads, self.window, self.sinks = heads, kv_heads, window, sinks
        D, qd, kd = experts.D, heads * head_dim, kv_heads * head_dim
        self.qkv = (torch.randn(qd + 2 * kd, D, generator=g, device="cuda") * D ** -0.5).bfloat16()
        self.proj = (torch.randn(D, qd, generator=g, device="cuda") * qd ** -0.5).bfloat16()
        self.cache = moe.KVCache.empty(n_pages, page, kv_heads, head_dim)

    def attend(self, x, batch, pos, ws):
        """x + attention of x's tokens over the cache, after their keys and values are appended to it."""
        h = F.rms_norm(x, x.shape[-1:]) @ self.qkv.T
        h = h.view(len(x), self.heads + 2 * self.kv_heads, -1)
        q, k, v = h.split([self.heads, self.kv_heads, self.kv_heads], dim=1)
        self.cache.append(rotate(k, pos), v, batch)  # v is a slice of the fused projection
        o = self.cache.attention(rotate(q, pos), batch, window=self.window, sinks=self.sinks, workspace=ws)
        return x + o.flatten(1) @ self.proj.T

    def forward(self, x, batch, pos, attn_ws, moe_ws):
        x = self.attend(x, batch, pos, attn_ws)
        return x + self.experts.forward(F.rms_norm(x, x.shape[-1:]), workspace=moe_ws)


class Decoder:
    def __init__(self, layers, lengths, steps, page):
        """Room for prompts of the given lengths and `steps` tokens more each, every sequence's pages in one table."""
        self.layers, self.lengths, self.room = layers, list(lengths), max(lengths) + steps
        cols = -(-self.room // page)
        self.table = torch.arange(len(lengths) * cols, dtype=torch.int32, device="cuda").view(len(lengths), cols)
        self.kv_len = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.graph = None

    def workspaces(self, batch, T):
        """One workspace each for the attention and the experts of all layers: they run one after the other."""
        return (max((l.cache.attention_workspace(l.heads, batch, l.window, l.sinks) for l in self.layers),
                    key=lambda w: w.numel()), self.layers[0].experts.workspace(T))

    def prompt(self, x):
        """x bf16 [sum of lengths, D], the prompts one after the other; returns each one's last output."""
        off = torch.tensor([0] + self.lengths).cumsum(0)
        batch = moe.KVBatch(off.int().cuda(), self.kv_len, self.table, len(x), max(self.lengths), max(self.lengths))
        pos = torch.cat([torch.arange(n) for n in self.lengths]).cuda()
        ws = self.workspaces(batch, len(x))
        for layer in self.layers:
            x = layer.forward(x, batch, pos, *ws)
        return x[(off[1:] - 1).cuda()]

    def one(self, x):
        """A token of every sequence, at the lengths the device holds."""
        self.kv_len += 1
        for layer in self.layers:
            x = layer.forward(x, self.batch, self.kv_len - 1, *self.ws)
        return x

    def step(self, x):
        if self.graph is None:
            n = len(self.lengths)
            q_off = torch.arange(n + 1, dtype=torch.int32, device="cuda")
            self.batch = moe.KVBatch(q_off, self.kv_len, self.table, n, 1, self.room)  # max_kv bounds every later step
            self.ws = self.workspaces(self.batch, n)
            self.x, lengths = x.clone(), self.kv_len.clone()
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                self.one(self.x)  # first use of the libraries, outside the capture; the real step writes the same slots
            torch.cuda.current_stream().wait_stream(s)
            self.kv_len.copy_(lengths)
            self.graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(self.graph):
                self.y = self.one(self.x)
        self.x.copy_(x)
        self.graph.replay()
        return self.y

    def check(self):
        for layer in self.layers:
            layer.cache.check()
        if self.graph is not None:
            st = moe.moe_get_device_status(ctypes.c_void_p(self.ws[1].data_ptr()), None)
            assert st == moe.MOE_OK, moe.moe_status_string(st)


def build(layers, lengths, steps, heads, kv_heads, head_dim, page, experts, window=0, sinks=0):
    """Layers in turn see everything and a sliding window with sinks; `experts(i)` is layer i's synth layer."""
    n_pages = len(lengths) * -(-(max(lengths) + steps) // page)
    return Decoder([Layer(i, moe.DeviceLayer(experts(i)), heads, kv_heads, head_dim, n_pages, page,
                          window if i % 2 else 0, sinks if i % 2 else 0) for i in range(layers)], lengths, steps, page)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--seqs", type=int, default=4)
    p.add_argument("--prompt", type=int, default=1500, help="tokens of the longest prompt")
    p.add_argument("--steps", type=int, default=64)
    a = p.parse_args()
    lengths = [max(1, a.prompt * (i + 1) // a.seqs) for i in range(a.seqs)]
    D = 2048
    dec = build(a.layers, lengths, a.steps, 16, 2, 128, 64, lambda i: synth.make_layer(i, D, 256, 8, 512), 512, 4)
    x = torch.randn(sum(lengths), D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    dec.prompt(x)  # warm up: the same slots are written again
    ev[0].record()
    y = dec.prompt(x)
    ev[1].record()
    for i in range(a.steps):
        if i == 1:
            ev[2].record()
        y = dec.step(y)
    ev[3].record()
    torch.cuda.synchronize()
    dec.check()
    assert torch.isfinite(y).all()
    held = sum(t.numel() * t.element_size() for l in dec.layers for t in (
        l.cache.k_codes, l.cache.k_scales, l.cache.k_biases, l.cache.v_codes, l.cache.v_scales, l.cache.v_biases))
    print(f"prompts: {sum(lengths)} tokens of {a.seqs} sequences in {ev[0].elapsed_time(ev[1]):.3f} ms")
    if a.steps > 1:
        t = ev[2].elapsed_time(ev[3]) / (a.steps - 1)
        print(f"decode: {t * 1000:.1f} us per step of {a.seqs} tokens ({a.seqs / t * 1000:.0f} tokens/s)")
    print(f"cache: {held / 2**20:.1f} MiB of 4-bit keys and values ({a.layers} layers)")


if __name__ == "__main__":
    main()
