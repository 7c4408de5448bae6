"""The attention operators of the serving path: their cases, inputs, plain form and exact values.

A 4-bit paged key/value cache in the library's number format (groups of 64
along the head, 4-bit codes, one bf16 scale and bias per group) and the
attention that reads it. Three operations:

  append   quantises a step's new keys and values into the cache's pages and
           reads the new tokens back as the values the cache now holds
  read     reads a range of every sequence back as bf16
  attend   causal grouped-query attention of the new tokens over the cache,
           optionally with a sliding window and a few first tokens that stay
           visible; returns the output and each row's log-sum-exp

A value of the cache is bf16(scale * code + bias), rounded once.
"""
import math

import torch

own = False

GROUP = 64
LIMIT = 65536.0  # the cache holds magnitudes up to 2^16


def listed():
    return [
        # a decode step of a few requests: one new token each, latency
        dict(name="append_b8", op="append", heads=16, kv_heads=2, dim=256, page=64, seqs=8, new_lo=1, new_hi=1,
             kv_lo=300, kv_hi=2000, window=0, sinks=0),
        # prompts of five requests written in one call, odd lengths, small pages
        dict(name="append_prompts", op="append", heads=32, kv_heads=8, dim=128, page=16, seqs=5, new_lo=2001, new_hi=4100,
             kv_lo=0, kv_hi=0, window=0, sinks=0),
        # a few short odd histories read back with small heads
        dict(name="read_ragged", op="read", heads=8, kv_heads=4, dim=64, page=32, seqs=3, new_lo=601, new_hi=2333,
             kv_lo=0, kv_hi=900, window=0, sinks=0),
        # one long context read back whole
        dict(name="read_128k", op="read", heads=16, kv_heads=2, dim=256, page=64, seqs=1, new_lo=131072, new_hi=131072,
             kv_lo=0, kv_hi=0, window=0, sinks=0),
        # the first tokens of an answer to a short prompt: the smallest call
        dict(name="decode_b1_short", op="attend", heads=16, kv_heads=2, dim=128, page=16, seqs=1, new_lo=1, new_hi=1,
             kv_lo=77, kv_hi=77, window=0, sinks=0),
        # one request deep in a long context: few rows, a long axis to split
        dict(name="decode_b1_64k", op="attend", heads=16, kv_heads=2, dim=256, page=64, seqs=1, new_lo=1, new_hi=1,
             kv_lo=65537, kv_hi=65537, window=0, sinks=0),
        # a full serving batch of ragged contexts
        dict(name="decode_b64", op="attend", heads=32, kv_heads=8, dim=128, page=64, seqs=64, new_lo=1, new_hi=1,
             kv_lo=700, kv_hi=8191, window=0, sinks=0),
        # a batch with a sliding window and four sink tokens, one query head per cached head
        dict(name="decode_window", op="attend", heads=8, kv_heads=8, dim=64, page=32, seqs=32, new_lo=1, new_hi=1,
             kv_lo=500, kv_hi=16000, window=1024, sinks=4),
        # four drafted tokens of each request verified at once
        dict(name="verify_4", op="attend", heads=16, kv_heads=2, dim=128, page=32, seqs=16, new_lo=4, new_hi=4,
             kv_lo=1000, kv_hi=6000, window=0, sinks=0),
        # a prompt's first chunk
        dict(name="prefill_4k", op="attend", heads=16, kv_heads=2, dim=128, page=64, seqs=1, new_lo=4096, new_hi=4096,
             kv_lo=0, kv_hi=0, window=0, sinks=0),
        # a later chunk of a long prompt, wide heads: the largest
        dict(name="chunk_at_32k", op="attend", heads=16, kv_heads=2, dim=256, page=64, seqs=1, new_lo=1024, new_hi=1024,
             kv_lo=31744, kv_hi=31744, window=0, sinks=0),
        # ragged prompts of a sliding-window layer with sinks, small heads
        dict(name="prefill_window", op="attend", heads=16, kv_heads=4, dim=64, page=16, seqs=3, new_lo=1100, new_hi=4001,
             kv_lo=0, kv_hi=700, window=512, sinks=4),
    ]


def draw(rng):
    """One more case: sizes spread over the logarithm of their ranges."""
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["append", "read", "attend", "attend", "attend", "attend"])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 6, 8])
    case = dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]), window=0, sinks=0)
    if op != "attend":
        seqs = log_int(1, 64)
        new = log_int(1, max(2, 2 ** 25 // (kv_heads * dim * seqs)))
        return dict(case, seqs=seqs, new_lo=max(1, new // 2), new_hi=new, kv_lo=0, kv_hi=log_int(1, 3000))
    kind = rng.choice(["decode", "decode", "draft", "prefill", "chunk"])
    if kind in ("decode", "draft"):
        seqs = log_int(1, 64)
        kv = log_int(16, max(32, min(65536, 2 ** 28 // (kv_heads * dim * seqs))))
        new = 1 if kind == "decode" else rng.randint(2, 5)
        case.update(seqs=seqs, new_lo=new, new_hi=new, kv_lo=kv // 3, kv_hi=kv)
    elif kind == "prefill":
        seqs = log_int(1, 6)
        new = log_int(17, 4096 // seqs)
        case.update(seqs=seqs, new_lo=max(1, new // 2), new_hi=new, kv_lo=0, kv_hi=0)
    else:
        seqs = log_int(1, 4)
        new = log_int(17, 900 // seqs)
        kv = log_int(200, 16000)
        case.update(seqs=seqs, new_lo=max(1, new // 2), new_hi=new, kv_lo=kv // 2, kv_hi=kv)
    if rng.random() < 0.35:
        case.update(window=log_int(16, 4096), sinks=rng.choice([0, 1, 4, 17]))
    return case


def lengths(case):
    """New tokens and cached tokens before them, per sequence: a fixed spread over the case's ranges."""
    n = case["seqs"]
    spread = [(i * 0.6180339887498949) % 1.0 for i in range(n)]
    new = [case["new_lo"] + int(round(f * (case["new_hi"] - case["new_lo"]))) for f in spread]
    old = [case["kv_lo"] + int(round((1 - f) * (case["kv_hi"] - case["kv_lo"]))) for f in spread]
    return new, old


def work(case):
    new, old = lengths(case)
    w, s, d = case["window"], case["sinks"], case["dim"]
    row = case["kv_heads"] * d
    if case["op"] in ("append", "read"):
        n = sum(new) * row * 2  # keys and values
        moved = n * 0.5625 + n * 2  # codes with their scales, and bf16, one read and the other written
        if case["op"] == "append":
            moved += n * 2  # the values read back
        return {"bytes": moved, "flops": 0}
    # visible keys summed over the tokens, and the keys that at least one of a sequence's tokens sees
    pairs = keys = 0
    for m, o in zip(new, old):
        if w:
            pairs += sum(min(p + 1, w + min(s, max(0, p + 1 - w))) for p in range(o, o + m))
            below = max(0, o - w + 1)
            keys += o + m - below + min(s, below)
        else:
            pairs += m * o + m * (m + 1) // 2
            keys += o + m
    n = sum(new)
    return {"bytes": keys * row * 2 * 0.5625 + 2 * n * case["heads"] * d * 2 + 4 * n * case["heads"],
            "flops": 4 * pairs * case["heads"] * d}


def quantise(x):
    """x [..., D] -> codes (int32 0..15), scales, biases (bf16) per group of 64."""
    g = torch.nan_to_num(x.float(), nan=0.0, posinf=LIMIT, neginf=-LIMIT).clamp(-LIMIT, LIMIT)
    g = g.reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = g.amin(-1, keepdim=True), g.amax(-1, keepdim=True)
    s = torch.div(hi - lo, torch.full_like(lo, 15.0)).to(torch.bfloat16)
    b = lo.to(torch.bfloat16)
    sf = s.float()
    q = torch.round(torch.div(g - b.float(), torch.where(sf > 0, sf, torch.ones_like(sf)))).clamp(0, 15)
    q = torch.where(sf > 0, q, torch.zeros_like(q)).to(torch.int32)
    return q.reshape(x.shape), s.squeeze(-1), b.squeeze(-1)


def values(codes, scales, biases):
    """What codes, scales and biases stand for: bf16(scale * code + bias)."""
    g = codes.reshape(*codes.shape[:-1], -1, GROUP).float()
    return (g * scales.float().unsqueeze(-1) + biases.float().unsqueeze(-1)).to(torch.bfloat16).reshape(codes.shape)


def pack(codes):
    """Codes [..., D] -> int32 words [..., D / 8], code j in bits 4j .. 4j + 3."""
    w = codes.reshape(*codes.shape[:-1], -1, 8).long() << torch.arange(0, 32, 4, device=codes.device)
    w = w.sum(-1)
    return torch.where(w >= 1 << 31, w - (1 << 32), w).to(torch.int32)


def unpack(words):
    c = (words.unsqueeze(-1) >> torch.arange(0, 32, 4, dtype=torch.int32, device=words.device)) & 15
    return c.reshape(*words.shape[:-1], -1)


def inputs(case, seed):
    new, old = lengths(case)
    dev = "cuda"
    r = torch.Generator(device=dev)
    r.manual_seed(seed)
    page, kvh, d, n = case["page"], case["kv_heads"], case["dim"], case["seqs"]
    total = [a + b for a, b in zip(new, old)]
    most = max(-(-t // page) for t in total)
    need = [-(-t // page) for t in total]
    pages = sum(need) + 3
    # pages are handed out in no order; entries past a sequence's length name no page
    order = torch.randperm(pages, generator=r, device=dev).to(torch.int32)
    table = torch.full((n, most), -1, dtype=torch.int32, device=dev)
    slot = torch.arange(most, device=dev)
    starts = torch.tensor([sum(need[:i]) for i in range(n)], device=dev)
    held = slot[None, :] < torch.tensor(need, device=dev)[:, None]
    table[held] = order[(starts[:, None] + slot[None, :])[held]]

    def bf16(*shape):
        return torch.randn(*shape, generator=r, device=dev).to(torch.bfloat16)

    # keys have channels of different size, as trained models' keys do
    size = torch.exp(0.5 * torch.randn(kvh, 1, d, generator=r, device=dev))
    st = dict(case=case, new=new, old=old, table=table,
              q_off=torch.tensor([sum(new[:i]) for i in range(n + 1)], dtype=torch.int32, device=dev),
              kv_len=torch.tensor(total, dtype=torch.int32, device=dev))
    for name, scale in (("k", size), ("v", 1.0)):
        c, s, b = quantise((torch.randn(pages, kvh, page, d, generator=r, device=dev) * scale).to(torch.bfloat16))
        st[name + "_codes"], st[name + "_scales"], st[name + "_biases"] = pack(c), s, b
    if case["op"] == "append":
        st["k"], st["v"] = bf16(sum(new), kvh, d) * size[:, 0].to(torch.bfloat16), bf16(sum(new), kvh, d)
    if case["op"] == "attend":
        st["q"] = bf16(sum(new), case["heads"], d)
    return st


def prepare(case, seed):
    st = inputs(case, seed)
    if own:  # the cache and batch handles over the same tensors that a serving loop keeps
        import bit_moe_expert_routing_gb300 as moe
        st["cache"] = moe.KVCache(*(st[a + b] for a in ("k", "v") for b in ("_codes", "_scales", "_biases")))
        st["batch"] = moe.KVBatch(st["q_off"], st["kv_len"], st["table"], sum(st["new"]), max(st["new"]),
                                  max(a + b for a, b in zip(st["new"], st["old"])))
        if case["op"] == "attend":
            st["workspace"] = st["cache"].attention_workspace(case["heads"], st["batch"], case["window"], case["sinks"])
    return st


def run(st):
    case = st["case"]
    if own:
        cache, batch = st["cache"], st["batch"]
        if case["op"] == "append":
            cache.append(st["k"], st["v"], batch)
        if case["op"] in ("append", "read"):
            k, v = cache.read(batch)
            return {"k": k, "v": v}
        out, lse = cache.attention(st["q"], batch, window=case["window"], sinks=case["sinks"], lse=True,
                                   workspace=st["workspace"])
        return {"out": out, "lse": lse}
    if case["op"] == "append":
        return plain_append(st)
    if case["op"] == "read":
        return plain_read(st)
    return plain_attend(st)


def token_places(st):
    """Page and slot of every new token."""
    n = int(st["q"].shape[0]) if "q" in st else int(st["k"].shape[0]) if "k" in st else sum(st["new"])
    tok = torch.arange(n, device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(st["q_off"], tok, right=True) - 1
    pos = st["kv_len"][seq] - st["q_off"][seq + 1] + tok
    page = st["case"]["page"]
    return seq, pos, st["table"][seq, (pos // page).long()].long(), (pos % page).long()


def plain_append(st):
    _, _, page, slot = token_places(st)
    for_kv = {}
    for name in ("k", "v"):
        c, s, b = quantise(st[name])
        st[name + "_codes"][page, :, slot] = pack(c)
        st[name + "_scales"][page, :, slot] = s
        st[name + "_biases"][page, :, slot] = b
        for_kv[name] = values(c, s, b)
    return for_kv


def plain_read(st):
    _, _, page, slot = token_places(st)
    return {name: values(unpack(st[name + "_codes"][page, :, slot]), st[name + "_scales"][page, :, slot],
                         st[name + "_biases"][page, :, slot]) for name in ("k", "v")}


def plain_attend(st):
    case, kv_len, q_off, q = st["case"], st["kv_len"], st["q_off"], st["q"]
    n, page, d, kvh, heads = case["seqs"], case["page"], case["dim"], case["kv_heads"], case["heads"]
    most, longest = max(st["new"]), max(a + b for a, b in zip(st["new"], st["old"]))
    # padded to the longest sequence: [sequence, kv head, position, dim]
    at = st["table"].clamp(min=0).long()
    keys = torch.arange(longest, device=q.device)

    def cached(name):
        x = values(unpack(st[name + "_codes"][at]), st[name + "_scales"][at], st[name + "_biases"][at])
        return x.transpose(1, 2).reshape(n, kvh, -1, d)[:, :, :longest].float()

    i = torch.arange(most, device=q.device)
    new = (q_off[1:] - q_off[:-1])
    valid = i[None, :] < new[:, None]                                         # [sequence, new token]
    rows = torch.where(valid, q_off[:-1, None] + i[None, :], 0).long()
    pos = (kv_len - new)[:, None] + i[None, :]
    sees = keys[None, None, :] <= pos[:, :, None]
    if case["window"]:
        sees &= (keys[None, None, :] > pos[:, :, None] - case["window"]) | (keys < case["sinks"])[None, None, :]
    sees &= valid[:, :, None]
    qs = q[rows].reshape(n, most, kvh, heads // kvh, d).permute(0, 2, 3, 1, 4).float()  # [seq, kv head, head, token, d]
    k = cached("k")
    s = torch.matmul(qs.reshape(n, kvh, -1, d), k.transpose(2, 3)).reshape(n, kvh, -1, most, longest)
    del k
    s = (s * d ** -0.5).masked_fill_(~sees[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = torch.exp(s.sub_(top))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(n, kvh, -1, longest), cached("v")).reshape(n, kvh, -1, most, d)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n, most, heads, d)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(n, most, heads)
    return {"out": o[valid].to(q.dtype), "lse": lse[valid]}


def exact(case, seed):
    """The definition, sequence by sequence, in 64 bits."""
    st = inputs(case, seed)
    page, d, kvh, heads = case["page"], case["dim"], case["kv_heads"], case["heads"]
    nib = 4 * torch.arange(8, device="cuda")

    def bf16(x):  # the nearest bf16, ties to even: the 45 low bits of the double's fraction go
        bits = x.contiguous().view(torch.int64)
        return ((bits + (1 << 44) - 1 + ((bits >> 45) & 1)) & ~((1 << 45) - 1)).view(torch.float64)

    def held(name, b, lo, hi):
        """Positions lo .. hi - 1 of sequence b, [hi - lo, kv head, dim], as doubles."""
        p = torch.arange(lo, hi, device="cuda")
        pg, sl = st["table"][b].long()[p // page], p % page
        w = st[name + "_codes"][pg, :, sl].long() & 0xFFFFFFFF
        c = ((w[..., None] >> nib) & 15).double().flatten(-2).unflatten(-1, (-1, GROUP))
        x = c * st[name + "_scales"][pg, :, sl].double()[..., None] + st[name + "_biases"][pg, :, sl].double()[..., None]
        return bf16(x).flatten(-2)

    if case["op"] == "append":
        got = {}
        for name in ("k", "v"):
            x = st[name].double().unflatten(-1, (-1, GROUP))
            b = x.min(-1, keepdim=True).values
            s = bf16((x.max(-1, keepdim=True).values - b) / 15.0)
            c = torch.where(s > 0, torch.round((x - b) / torch.where(s > 0, s, 1.0)).clamp(0, 15), 0.0)
            got[name] = bf16(c * s + b).flatten(-2)
        return got
    if case["op"] == "read":
        return {name: torch.cat([held(name, b, o, o + m) for b, (m, o) in enumerate(zip(st["new"], st["old"]))])
                for name in ("k", "v")}
    outs, lses, at, g = [], [], 0, heads // kvh
    for b, (m, o) in enumerate(zip(st["new"], st["old"])):
        pos, keys = torch.arange(o, o + m, device="cuda")[:, None], torch.arange(o + m, device="cuda")[None, :]
        hidden = keys > pos
        if case["window"]:
            hidden |= (keys <= pos - case["window"]) & (keys >= case["sinks"])
        k, v = held("k", b, 0, o + m), held("v", b, 0, o + m)
        out = torch.empty(m, heads, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(m, heads, dtype=torch.float64, device="cuda")
        for h in range(heads):
            s = (st["q"][at:at + m, h].double() @ k[:, h // g].T) / math.sqrt(d)
            s[hidden] = -math.inf
            lse[:, h] = torch.logsumexp(s, -1)
            out[:, h] = torch.exp(s - lse[:, h, None]) @ v[:, h // g]
        outs.append(out)
        lses.append(lse)
        at += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
