"""A plain 64-bit implementation of the 4-bit key/value cache and its
attention, and the inputs of their tests (not a test module)."""
from __future__ import annotations

import math

import numpy as np
import torch

GROUP = 64
LIMIT = 65536.0


def bf16_round(x: np.ndarray) -> np.ndarray:
    """Doubles to the nearest bf16 (ties to even), as doubles: the fraction keeps seven bits."""
    bits = np.ascontiguousarray(x, dtype=np.float64).view(np.int64)
    return ((bits + (1 << 44) - 1 + ((bits >> 45) & 1)) & ~((1 << 45) - 1)).view(np.float64)


def quantise(x: np.ndarray):
    """x (doubles) [..., D] -> codes [..., D], scales, biases [..., D / 64], from the definition."""
    x = np.where(np.isnan(x), 0.0, np.clip(x, -LIMIT, LIMIT))
    g = x.reshape(*x.shape[:-1], x.shape[-1] // GROUP, GROUP)
    b = g.min(-1, keepdims=True)
    s = bf16_round((g.max(-1, keepdims=True) - b) / 15.0)
    q = np.where(s > 0, np.clip(np.rint((g - b) / np.where(s > 0, s, 1.0)), 0, 15), 0)
    return q.reshape(x.shape).astype(np.int64), s[..., 0], b[..., 0]


def values(codes, scales, biases):
    g = codes.reshape(*codes.shape[:-1], codes.shape[-1] // GROUP, GROUP)
    return bf16_round(g * scales[..., None] + biases[..., None]).reshape(codes.shape)


def pack(codes: np.ndarray) -> np.ndarray:
    w = (codes.reshape(*codes.shape[:-1], codes.shape[-1] // 8, 8).astype(np.uint64) << (4 * np.arange(8, dtype=np.uint64))).sum(-1)
    return w.astype(np.uint32).view(np.int32)


def unpack(words: np.ndarray) -> np.ndarray:
    w = words.view(np.uint32).astype(np.int64)
    return ((w[..., None] >> (4 * np.arange(8))) & 15).reshape(*words.shape[:-1], words.shape[-1] * 8)


def bf16_bits(x: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


class Batch:
    """Sequences with `new` step tokens and `kv` positions (step tokens
    included), their pages dealt out in a shuffled order, unused table entries
    invalid and a few pages left over."""

    def __init__(self, new, kv, page, seed=0, spare=3):
        r = np.random.RandomState(seed)
        self.new, self.kv, self.page = list(new), list(kv), page
        need = [-(-max(0, l) // page) for l in kv]
        self.n_pages = max(1, sum(need) + spare)
        order = r.permutation(self.n_pages)
        self.table = np.full((len(new), max(need + [1])), -7, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.q_off = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.n_tokens = int(self.q_off[-1])

    def places(self, b):
        """(page, slot) of every position of sequence b."""
        p = np.arange(self.kv[b])
        return self.table[b, p // self.page], p % self.page

    def device(self, moe, max_new=None, max_kv=None):
        c = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        return moe.KVBatch(c(self.q_off), c(np.array(self.kv, dtype=np.int32)), c(self.table), self.n_tokens,
                           max_new or max(self.new + [1]), max_kv or max(self.kv + [1]))


def junk_cache(moe, n_pages, page, kv_heads, dim, seed=1):
    """A cache whose every slot holds garbage: random codes, NaN and infinite scales and biases."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = moe.KVCache.empty(n_pages, page, kv_heads, dim)
    for name in ("k", "v"):
        getattr(c, name + "_codes").random_(generator=g)
        getattr(c, name + "_scales").fill_(float("nan"))
        getattr(c, name + "_biases").fill_(float("inf"))
    return c


def fill(cache, batch: Batch, seed=2, spread=1.0, outliers=False):
    """Puts random keys and values at every position of the batch (packed here, not by the library) and returns them as
    the cache holds them: per sequence doubles [kv, kv heads, dim] (on the GPU)."""
    r = np.random.RandomState(seed)
    held = []
    for name in ("k", "v"):
        codes, scales, biases = (getattr(cache, f"{name}_{a}") for a in ("codes", "scales", "biases"))
        per_seq = []
        for b in range(len(batch.new)):
            n = max(0, batch.kv[b])
            x = r.randn(n, cache.kv_heads, cache.head_dim) * (spread if name == "k" else 1.0)
            if outliers:
                x *= np.exp(r.randn(1, 1, cache.head_dim))
            x = bf16_bits(x).double().numpy()
            q, s, z = quantise(x)
            if n:
                pg, sl = (torch.from_numpy(a.astype(np.int64)).cuda() for a in batch.places(b))
                codes[pg, :, sl] = torch.from_numpy(pack(q)).cuda()
                scales[pg, :, sl] = bf16_bits(s).cuda()
                biases[pg, :, sl] = bf16_bits(z).cuda()
            per_seq.append(torch.from_numpy(values(q, s, z)).cuda())
        held.append(per_seq)
    return held


def attention_reference(q, batch: Batch, keys, vals, scale, window=0, sinks=0):
    """(out, lse, size) in 64 bits, row by row from the definition; size is sum_j p_j |v_j|, what the error bounds scale with."""
    heads, dim = q.shape[1], q.shape[2]
    out = torch.zeros(batch.n_tokens, heads, dim, dtype=torch.float64, device="cuda")
    size = torch.zeros_like(out)
    lse = torch.full((batch.n_tokens, heads), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(len(batch.new)):
        n, kv, t0 = batch.new[b], max(0, batch.kv[b]), int(batch.q_off[b])
        if n == 0 or kv == 0:
            continue
        pos = torch.arange(n, device="cuda")[:, None] + (batch.kv[b] - n)
        j = torch.arange(kv, device="cuda")[None, :]
        sees = j <= pos
        if window:
            sees = sees & ((j > pos - window) | (j < sinks))
        some = sees.any(1)
        for h in range(heads):
            k, v = keys[b][:, h * keys[b].shape[1] // heads], vals[b][:, h * keys[b].shape[1] // heads]
            s = (q[t0:t0 + n, h].double() @ k.T) * scale
            s = torch.where(sees, s, -math.inf)
            top = torch.where(some, s.amax(1), 0.0)
            p = torch.exp(s - top[:, None])
            tot = p.sum(1)
            p = p / torch.where(some, tot, 1.0)[:, None]
            out[t0:t0 + n, h] = p @ v
            size[t0:t0 + n, h] = p @ v.abs()
            lse[t0:t0 + n, h] = torch.where(some, top + torch.log(torch.where(some, tot, 1.0)), -math.inf)
    return out, lse, size


def check_attention(out, lse, ref, what=""):
    """The bound of every output value: the output is rounded to bf16 once (2^-9 of it), each probability at most once
    (2^-9 of sum p |v|), and the fp32 sums and exponentials of 2^-20 relative are far below; doubled, 2^-8 of both.
    The log-sum-exp is computed in fp32 from fp32 sums of exact products: 2^-16 absolute covers sums of 256 products
    of a few units, 2^-18 relative the larger scores."""
    r_out, r_lse, size = ref
    out = out.double()
    assert torch.equal(torch.isfinite(out), torch.isfinite(r_out)), what
    d = (out - r_out).abs()
    bound = 2.0 ** -8 * (r_out.abs() + size) + 1e-30
    worst = (d / bound).max().item() if d.numel() else 0.0
    assert worst <= 1.0, (what, worst)
    if lse is not None:
        lse = lse.double()
        empty = r_lse == -math.inf
        assert torch.equal(lse == -math.inf, empty), what
        e = (lse - r_lse).abs()[~empty]
        if e.numel():
            tol = 2.0 ** -16 + 2.0 ** -18 * r_lse.abs()[~empty]
            assert (e <= tol).all(), (what, (e / tol).max().item())
    return worst
