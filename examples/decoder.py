"""A small decoder that serves ragged prompts: every layer is attention over a
4-bit paged key/value cache followed by a 4-bit mixture-of-experts layer.

The prompts go through in one ragged step. Each is then continued a number of
times: the continuations share the prompt's pages, and attend to them once for
all of them where that pays. After that a step takes one token per sequence and
is one CUDA graph, replayed with the lengths, positions and pages advanced on
the device. Weights are random, and a sequence's next input is its last output,
so the example shows the calls and their cost, not text.

    python examples/decoder.py [--layers 2] [--seqs 4] [--prompt 1500] [--steps 64] [--continuations 1]
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
    """Rotary position embedding of x [tokens, heads, head dim] at pos [tokens]: in plain form what the layers' Rotary
    does to queries and keys (heads without norms)."""
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
        half = head_dim // 2
        self.rotary = moe.Rotary([10000.0 ** (-i / half) for i in range(half)])
        self.prefix = None  # what groups of the step's sequences share (a KVPrefix)

    def attend(self, x, batch, pos, ws):
        """x + attention of x's tokens over the cache, after their keys and values are appended to it."""
        h = F.rms_norm(x, x.shape[-1:]) @ self.qkv.T
        h = h.view(len(x), self.heads + 2 * self.kv_heads, -1)
        q, k, v = h.split([self.heads, self.kv_heads, self.kv_heads], dim=1)  # slices of the fused projection
        q = self.cache.append_rotary(q, k, v, batch, self.rotary, positions=pos)
        o = self.cache.attention(q, batch, window=self.window, sinks=self.sinks, workspace=ws, prefix=self.prefix)
        return x + o.flatten(1) @ self.proj.T

    def forward(self, x, batch, pos, attn_ws, moe_ws):
        x = self.attend(x, batch, pos, attn_ws)
        return x + self.experts.forward(F.rms_norm(x, x.shape[-1:]), workspace=moe_ws)


class Decoder:
    def __init__(self, layers, lengths, steps, page, continuations=1):
        """Room for prompts of the given lengths, each continued `continuations` times by `steps` tokens: prompt i and
        its continuations are sequences i * continuations and on."""
        self.layers, self.lengths, self.n, self.page = layers, list(lengths), continuations, page
        self.room = max(lengths) + steps
        self.pages = moe.KVPages([l.cache for l in layers], len(lengths) * continuations, -(-self.room // page))
        self.kv_len = torch.zeros(self.pages.n_seqs, dtype=torch.int32, device="cuda")
        self.kv_len[::continuations] = torch.tensor(lengths, dtype=torch.int32)
        self.graph = None

    def workspaces(self, batch, T):
        """One workspace each for the attention and the experts of all layers: they run one after the other."""
        return (max((l.cache.attention_workspace(l.heads, batch, l.window, l.sinks, l.prefix) for l in self.layers),
                    key=lambda w: w.numel()), self.layers[0].experts.workspace(T))

    def prompt(self, x):
        """x bf16 [sum of lengths, D], the prompts one after the other; returns each one's last output."""
        new = torch.zeros(self.pages.n_seqs, dtype=torch.int64)
        new[::self.n] = torch.tensor(self.lengths)
        off = torch.cat([new[:1] * 0, new.cumsum(0)])
        batch = self.pages.batch(off.int().cuda(), self.kv_len, len(x), max(self.lengths), max(self.lengths))
        pos = torch.cat([torch.arange(n) for n in self.lengths]).int().cuda()
        ws = self.workspaces(batch, len(x))
        self.pages.update(batch)
        for layer in self.layers:
            x = layer.forward(x, batch, pos, *ws)
        return x[(off[1:][::self.n] - 1).cuda()]

    def fork(self):
        """Lets every prompt's other continuations share its pages."""
        i = torch.arange(self.pages.n_seqs, dtype=torch.int32)
        src, dst = (i // self.n * self.n)[i % self.n > 0].cuda(), i[i % self.n > 0].cuda()
        self.pages.fork(src, dst)
        self.kv_len.copy_(self.kv_len[::self.n].repeat_interleave(self.n))
        # the first positions of all of a group are the prompt's
        off = torch.arange(0, self.pages.n_seqs + 1, self.n, dtype=torch.int32, device="cuda")
        own = max(self.room - n // self.page * self.page for n in self.lengths)
        prefix = moe.KVPrefix(off, torch.tensor(self.lengths, dtype=torch.int32, device="cuda"), self.n, max(self.lengths), own)
        for layer in self.layers:
            layer.prefix = prefix

    def one(self, x):
        """A token of every sequence, at the lengths the device holds."""
        self.kv_len += 1
        self.pages.update(self.batch)  # a page for those that have filled theirs, copies of shared ones
        for layer in self.layers:
            x = layer.forward(x, self.batch, self.kv_len - 1, *self.ws)
        return x

    def step(self, x):
        if self.graph is None:
            n = self.pages.n_seqs
            q_off = torch.arange(n + 1, dtype=torch.int32, device="cuda")
            self.batch = self.pages.batch(q_off, self.kv_len, n, 1, self.room)  # max_kv bounds every later step
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
        self.pages.check()
        for layer in self.layers:
            layer.cache.check()
        if self.graph is not None:
            st = moe.moe_get_device_status(ctypes.c_void_p(self.ws[1].data_ptr()), None)
            assert st == moe.MOE_OK, moe.moe_status_string(st)


def build(layers, lengths, steps, heads, kv_heads, head_dim, page, experts, window=0, sinks=0, continuations=1):
    """Layers in turn see everything and a sliding window with sinks; `experts(i)` is layer i's synth layer."""
    n_pages = sum(-(-n // page) + continuations * (steps // page + 2) for n in lengths)
    return Decoder([Layer(i, moe.DeviceLayer(experts(i)), heads, kv_heads, head_dim, n_pages, page,
                          window if i % 2 else 0, sinks if i % 2 else 0) for i in range(layers)], lengths, steps, page, continuations)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--layers", type=int, default=2)
    p.add_argument("--seqs", type=int, default=4)
    p.add_argument("--prompt", type=int, default=1500, help="tokens of the longest prompt")
    p.add_argument("--steps", type=int, default=64)
    p.add_argument("--continuations", type=int, default=1, help="of each prompt, sharing its pages")
    a = p.parse_args()
    lengths = [max(1, a.prompt * (i + 1) // a.seqs) for i in range(a.seqs)]
    D = 2048
    dec = build(a.layers, lengths, a.steps, 16, 2, 128, 64, lambda i: synth.make_layer(i, D, 256, 8, 512), 512, 4, a.continuations)
    x = torch.randn(sum(lengths), D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    ev = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
    dec.prompt(x)  # warm up: the same slots are written again
    ev[0].record()
    y = dec.prompt(x)
    ev[1].record()
    if a.continuations > 1:
        dec.fork()
        y = y.repeat_interleave(a.continuations, 0)
        y = y + 0.1 * torch.randn(y.shape, generator=torch.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
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
        print(f"decode: {t * 1000:.1f} us per step of {len(y)} tokens ({len(y) / t * 1000:.0f} tokens/s)")
    print(f"cache: {held / 2**20:.1f} MiB of 4-bit keys and values ({a.layers} layers)")


if __name__ == "__main__":
    main()
