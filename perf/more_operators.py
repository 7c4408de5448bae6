"""Operators of a serving step around the 4-bit key/value cache: their cases, inputs, plain form and exact values.

The cache's format is the library's: groups of 64 along the head, 4-bit codes,
one bf16 scale and bias per group; a cached value is bf16(scale * code + bias),
rounded once. Three families:

  rotary  norms every query and key head, rotates them to their positions (one
          axis, or time, height and width) and quantises the keys and values
          into the cache; the cached tokens are then read back
  pages   gives sequences their pages, forks them, takes pages back, copies
          what is written while shared, and moves pages together
  prefix  attention of a step whose sequences, group by group, share their
          first positions
"""
import math

import torch

own = False

GROUP = 64
LIMIT = 65536.0  # the cache holds magnitudes up to 2^16


def listed():
    return [
        # a decode step of a few requests, a quarter of each wide head rotated: latency
        dict(name="rotary_b8", op="rotary", heads=16, kv_heads=2, dim=256, rot=64, pairs="halves", axes=1, norm=True,
             page=64, seqs=8, new_lo=1, new_hi=1, old_lo=300, old_hi=2000),
        # five prompts of odd lengths in one call, whole heads rotated, small pages
        dict(name="rotary_prompts", op="rotary", heads=32, kv_heads=8, dim=128, rot=128, pairs="halves", axes=1, norm=True,
             page=16, seqs=5, new_lo=2001, new_hi=4100, old_lo=0, old_hi=0),
        # prompts with an image each: time, height and width turn their own frequencies of small heads
        dict(name="rotary_images", op="rotary", heads=8, kv_heads=4, dim=64, rot=64, pairs="neighbours", axes=3, norm=False,
             page=32, seqs=3, new_lo=601, new_hi=2333, old_lo=0, old_hi=900),
        # a chunk of a very long prompt: angles of far positions
        dict(name="rotary_far", op="rotary", heads=16, kv_heads=2, dim=256, rot=256, pairs="halves", axes=1, norm=True,
             page=64, seqs=1, new_lo=4096, new_hi=4096, old_lo=1000003, old_hi=1000003),
        # a speculative step's bookkeeping: last step's rejected drafts give their pages back, new drafts get theirs
        dict(name="pages_drafts", op="pages", kind="drafts", kv_heads=2, dim=256, page=16, layers=1, seqs=64, len_lo=300,
             len_hi=4000, draft=5, parents=0, spare=300),
        # several continuations of each of a few prompts, over and over: the last, part-filled page of each is copied
        dict(name="pages_fork", op="pages", kind="fork", kv_heads=8, dim=128, page=64, layers=2, seqs=36, len_lo=700,
             len_hi=5001, draft=1, parents=4, spare=40),
        # half of the requests end and the cache of four layers is moved together
        dict(name="pages_compact", op="pages", kind="compact", kv_heads=8, dim=128, page=64, layers=4, seqs=48, len_lo=900,
             len_hi=6000, draft=1, parents=0, spare=100),
        # a few requests with one system prompt: the smallest call
        dict(name="prefix_b8", op="prefix", heads=16, kv_heads=2, dim=128, page=16, groups=1, seqs=8, prefix_lo=2000,
             prefix_hi=2000, own_lo=1, own_hi=200, new_lo=1, new_hi=1),
        # a full serving batch with one long document, one token each
        dict(name="prefix_b64_32k", op="prefix", heads=16, kv_heads=2, dim=256, page=64, groups=1, seqs=64, prefix_lo=32768,
             prefix_hi=32768, own_lo=40, own_hi=1500, new_lo=1, new_hi=1),
        # six prompts with four continuations each, four drafted tokens at once, ragged
        dict(name="prefix_drafts", op="prefix", heads=32, kv_heads=8, dim=128, page=32, groups=6, seqs=24, prefix_lo=1000,
             prefix_hi=8000, own_lo=4, own_hi=700, new_lo=4, new_hi=4),
        # a dozen questions on one document, small heads
        dict(name="prefix_questions", op="prefix", heads=16, kv_heads=4, dim=64, page=16, groups=1, seqs=12, prefix_lo=16001,
             prefix_hi=16001, own_lo=60, own_hi=301, new_lo=60, new_hi=301),
        # longer tails of two long documents, wide heads: the largest
        dict(name="prefix_chunks", op="prefix", heads=16, kv_heads=2, dim=256, page=64, groups=2, seqs=8, prefix_lo=12000,
             prefix_hi=20001, own_lo=130, own_hi=400, new_lo=130, new_hi=260),
    ]


def draw(rng):
    """One more case: sizes spread over the logarithm of their ranges."""
    def log_int(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["rotary", "pages", "prefix", "prefix"])
    dim = rng.choice([64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    heads = kv_heads * rng.choice([1, 2, 4, 5, 6, 8])
    page = rng.choice([16, 32, 64, 128])
    if op == "rotary":
        seqs = log_int(1, 64)
        new = log_int(1, max(2, 2 ** 25 // ((heads + 2 * kv_heads) * dim * seqs)))
        return dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, rot=rng.choice([r for r in (16, 32, 64, 96, 128, 256) if r <= dim]),
                    pairs=rng.choice(["halves", "halves", "neighbours"]), axes=rng.choice([1, 1, 3]), norm=rng.random() < 0.7,
                    page=page, seqs=seqs, new_lo=max(1, new // 2), new_hi=new, old_lo=0, old_hi=log_int(1, 200000 // seqs + 1))
    if op == "pages":
        kind = rng.choice(["drafts", "fork", "compact"])
        seqs = log_int(2, 64)
        length = log_int(20, max(40, min(30000, 2 ** 27 // (kv_heads * dim * seqs))))
        return dict(op=op, kind=kind, kv_heads=kv_heads, dim=dim, page=page, layers=rng.randint(1, 3), seqs=seqs,
                    len_lo=max(1, length // 3), len_hi=length, draft=rng.randint(1, 9),
                    parents=rng.randint(1, max(1, seqs // 3)) if kind == "fork" else 0, spare=rng.randint(0, 200))
    groups = log_int(1, 8)
    seqs = groups + log_int(1, 64) - 1
    prefix = log_int(64, max(128, min(40000, 2 ** 24 // (kv_heads * dim))))
    if rng.random() < 0.6:
        new = rng.choice([1, 1, 1, 2, 4, 5])
        old = log_int(1, max(2, min(2000, 2 ** 25 // (kv_heads * dim * seqs))))
    else:
        new = log_int(2, max(3, min(400, 2 ** 36 // (4 * heads * dim * prefix * seqs))))
        old = 0
    return dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, page=page, groups=groups, seqs=seqs, prefix_lo=max(1, prefix // 2),
                prefix_hi=prefix, own_lo=new + old // 8, own_hi=new + old, new_lo=max(1, new // 2) if old == 0 else new, new_hi=new)


def spread(n, lo, hi, at=0):
    """n numbers of [lo, hi], always the same ones."""
    return [lo + int(round(((i + at) * 0.6180339887498949) % 1.0 * (hi - lo))) for i in range(n)]


def lengths(case):
    """Step tokens and cached positions of every sequence (these tokens included), and the shared positions of each group."""
    n = case["seqs"]
    if case["op"] == "rotary":
        new = spread(n, case["new_lo"], case["new_hi"])
        return new, [a + b for a, b in zip(new, spread(n, case["old_lo"], case["old_hi"], 3))], []
    shared = spread(case["groups"], case["prefix_lo"], case["prefix_hi"])
    new = spread(n, case["new_lo"], case["new_hi"])
    tail = [max(a, b) for a, b in zip(new, spread(n, case["own_lo"], case["own_hi"]))]
    return new, [shared[g] // case["page"] * case["page"] + t for g, t in zip(group_of(case), tail)], shared


def group_of(case):
    """The group of every sequence: as equal as they go."""
    return [i * case["groups"] // case["seqs"] for i in range(case["seqs"])]


def page_lengths(case):
    """The rounds of one pass: each a list of (positions, step tokens) per sequence."""
    n, draft = case["seqs"], case["draft"]
    base = spread(n, case["len_lo"], case["len_hi"])
    if case["kind"] == "drafts":  # the last step's drafts are dropped, but for one; then new ones
        return [[(l, 1) for l in base], [(l + draft, draft) for l in base]]
    if case["kind"] == "fork":  # the continuations before end; the new ones go on from their parents
        p = case["parents"]
        of = [i if i < p else (i - p) % p for i in range(n)]
        return [[(base[i], 0) if i < p else (0, 0) for i in range(n)],
                [(base[of[i]], 0) if i < p else (base[of[i]] + draft, draft) for i in range(n)]]
    return [[(0, 0)] * n, [(l, 0) for l in base], [(l, 0) if i % 2 else (0, 0) for i, l in enumerate(base)]]


def page_room(case):
    """Table columns and pages of the cache."""
    size = case["page"]
    most = [max(r[i][0] for r in page_lengths(case)) for i in range(case["seqs"])]
    return -(-max(most) // size) + 1, sum(-(-l // size) for l in most) + case["spare"] + 1


def work(case):
    if case["op"] == "pages":
        size = case["page"]
        columns, pages = page_room(case)
        rounds = page_lengths(case)
        moved = 0
        if case["kind"] == "fork":  # the part-filled page of every continuation
            moved = sum(1 for a in rounds[1][case["parents"]:] if (a[0] - a[1]) % size)
        if case["kind"] == "compact":  # what lies past the pages in use
            held = [-(-l // size) for l, _ in rounds[1]]
            live, at = sum(h for i, h in enumerate(held) if i % 2), 0
            for i, h in enumerate(held):
                moved += max(0, at + h - max(at, live)) if i % 2 else 0
                at += h
        entries = sum(-(-l // size) for l, _ in rounds[-1])
        # tables, counts and references once, and the pages' bytes read and written
        return {"bytes": 4 * (2 * entries + 4 * case["seqs"] + 2 * pages) +
                2 * moved * case["layers"] * case["kv_heads"] * size * case["dim"] * 2 * 0.5625, "flops": 0}
    new, total, shared = lengths(case)
    d, row, n = case["dim"], case["kv_heads"] * case["dim"], sum(new)
    if case["op"] == "rotary":  # queries read and written; keys and values read, held in the cache, and read back
        return {"bytes": n * case["heads"] * d * 4 + n * row * 2 * (2 + 0.5625 + 2) + 4 * n * (case["axes"] > 1) * case["axes"],
                "flops": 0}
    of, pairs, keys = group_of(case), 0, sum(s // case["page"] * case["page"] for s in shared)
    for i, (m, t) in enumerate(zip(new, total)):
        pairs += m * (t - m) + m * (m + 1) // 2
        keys += t - shared[of[i]] // case["page"] * case["page"]
    return {"bytes": keys * row * 2 * 0.5625 + 2 * n * case["heads"] * d * 2 + 4 * n * case["heads"],
            "flops": 4 * pairs * case["heads"] * d}


# ---- the cache's format ----------------------------------------------------------------------------------------------

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


NAMES = [a + b for a in ("k", "v") for b in ("_codes", "_scales", "_biases")]


# ---- inputs ----------------------------------------------------------------------------------------------------------

def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def offsets(counts):
    return ints([sum(counts[:i]) for i in range(len(counts) + 1)])


def inputs(case, seed):
    r = torch.Generator(device="cuda")
    r.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=r, device="cuda")

    kvh, d, page, n = case["kv_heads"], case["dim"], case["page"], case["seqs"]
    st = dict(case=case)

    def random_pages(count):
        c = torch.randint(0, 2 ** 32, (count, kvh, page, d // 8), generator=r, device="cuda") - 2 ** 31
        s = (torch.rand(count, kvh, page, d // GROUP, generator=r, device="cuda") + 0.1).to(torch.bfloat16)
        b = normal(count, kvh, page, d // GROUP).to(torch.bfloat16)
        return [c.to(torch.int32), s, b]

    if case["op"] == "pages":
        columns, pages = page_room(case)
        st["table"] = torch.full((n, columns), -1, dtype=torch.int32, device="cuda")
        st["held"], st["refs"] = ints([0] * n), ints([0] * pages)
        st["layers"] = [random_pages(pages) + random_pages(pages) for _ in range(case["layers"])]
        # which pages the sequences of the first round start from is of no matter but for the parents'
        st["rounds"] = [(ints([l for l, _ in x]), offsets([m for _, m in x]), sum(m for _, m in x)) for x in page_lengths(case)]
        if case["kind"] == "fork":
            p = case["parents"]
            st["src"], st["dst"] = ints([(i - p) % p for i in range(p, n)]), ints(list(range(p, n)))
            # the parents hold pages in no order
            lens = [page_lengths(case)[0][i][0] for i in range(p)]
            order = torch.randperm(pages, generator=r, device="cuda").to(torch.int32)
            at = 0
            for i, l in enumerate(lens):
                need = -(-l // page)
                st["table"][i, :need] = order[at:at + need]
                st["held"][i] = need
                at += need
            st["refs"][order[:at].long()] = 1
        return st

    new, total, shared = lengths(case)
    st.update(new=new, total=total, q_off=offsets(new), kv_len=ints(total))
    # pages are handed out in no order; entries past a sequence's length name no page
    need = [-(-t // page) for t in total]
    pages = sum(need) + 3 + sum(-(-s // page) for s in shared)
    order = torch.randperm(pages, generator=r, device="cuda").to(torch.int32)
    st["table"] = torch.full((n, max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at, common = 0, {}
    for i in range(n):
        k = 0
        if case["op"] == "prefix":  # whole pages of the group's prefix are the same ones
            g = group_of(case)[i]
            k = shared[g] // page
            if g not in common:
                common[g] = order[at:at + k]
                at += k
            st["table"][i, :k] = common[g]
        st["table"][i, k:need[i]] = order[at:at + need[i] - k]
        at += need[i] - k
    # keys have channels of different size, as trained models' keys do
    size = torch.exp(0.5 * normal(kvh, 1, d))
    heads = case["heads"]
    if case["op"] == "rotary":
        # one projection's output: queries, keys and values side by side; a position past 2^20 keeps no pages before it
        st["qkv"] = normal(sum(new), heads + 2 * kvh, d)
        st["qkv"][:, heads:heads + kvh] *= size[:, 0]
        st["qkv"] = st["qkv"].to(torch.bfloat16)
        st["freq"] = torch.exp(-math.log(1e6) * torch.arange(case["rot"] // 2, dtype=torch.float64) / (case["rot"] // 2))
        st["axis"], st["positions"] = None, None
        if case["axes"] > 1:
            half = case["rot"] // 2
            st["axis"] = [0 if i < half // 4 else 1 + (i % 2) for i in range(half)]
            st["positions"] = image_positions(new, total)
        st["q_weight"] = st["k_weight"] = None
        if case["norm"]:
            st["q_weight"], st["k_weight"] = 1 + 0.3 * normal(d), 1 + 0.3 * normal(d)
        for i in range(n):  # pages of positions before the step are other programs' business here
            st["table"][i, :(total[i] - new[i]) // page] = -1
        used = st["table"] >= 0
        pages = int(used.sum()) + 3
        st["table"][used] = torch.randperm(pages, generator=r, device="cuda").to(torch.int32)[:int(used.sum())]
        for a in ("k", "v"):
            for b, x in zip(("_codes", "_scales", "_biases"), random_pages(pages)):
                st[a + b] = x
        return st
    for name, scale in (("k", size), ("v", 1.0)):
        c, s, b = quantise((normal(pages, kvh, page, d) * scale).to(torch.bfloat16))
        st[name + "_codes"], st[name + "_scales"], st[name + "_biases"] = pack(c), s, b
    st["q"] = normal(sum(new), heads, d).to(torch.bfloat16)
    of = group_of(case)
    st["seq_off"] = offsets([of.count(g) for g in range(case["groups"])])
    st["length"] = ints(shared)
    return st


def image_positions(new, total):
    """[3, tokens]: text at equal positions on all axes, and in the middle of each sequence an image's rows and columns."""
    out = []
    for m, t in zip(new, total):
        p = [[], [], []]
        at, side = t - m, int(math.sqrt(m // 2))
        for i in range(m):
            j = i - m // 4
            if 0 <= j < side * side:
                here = (at, at + j // side, at + j % side)
                if j == side * side - 1:
                    at += side
            else:
                here = (at, at, at)
                at += 1
            for a in range(3):
                p[a].append(here[a])
        out.append(p)
    return ints([sum((p[a] for p in out), []) for a in range(3)])


def prepare(case, seed):
    st = inputs(case, seed)
    if not own:
        return st
    # the handles over the same tensors that a serving loop keeps
    import bit_moe_expert_routing_gb300 as moe
    if case["op"] == "pages":
        pages = moe.KVPages([moe.KVCache(*a) for a in st["layers"]], case["seqs"], st["table"].shape[1])
        for name in ("table", "held", "refs"):
            getattr(pages, name).copy_(st[name])
        most = max(m for x in page_lengths(case) for _, m in x)
        st["pages"], st["batches"] = pages, [pages.batch(q_off, kv_len, n, most, st["table"].shape[1] * case["page"])
                                             for kv_len, q_off, n in st["rounds"]]
        return st
    st["cache"] = moe.KVCache(*(st[a] for a in NAMES))
    st["batch"] = moe.KVBatch(st["q_off"], st["kv_len"], st["table"], sum(st["new"]), max(st["new"]), max(st["total"]))
    if case["op"] == "rotary":
        st["rotary"] = moe.Rotary(st["freq"], axis=st["axis"], interleaved=case["pairs"] == "neighbours",
                                  q_weight=st["q_weight"], k_weight=st["k_weight"], eps=1e-6)
        return st
    of, size = group_of(case), case["page"]
    shared = st["length"].tolist()
    own_most = max(t - shared[g] // size * size for t, g in zip(st["total"], of))
    st["prefix"] = moe.KVPrefix(st["seq_off"], st["length"], max(sum(m for m, h in zip(st["new"], of) if h == g) for g in set(of)),
                                max(shared), own_most)
    st["workspace"] = st["cache"].attention_workspace(case["heads"], st["batch"], prefix=st["prefix"])
    return st


def run(st):
    case = st["case"]
    if case["op"] == "rotary":
        q, k, v = st["qkv"].split([case["heads"], case["kv_heads"], case["kv_heads"]], dim=1)
        if not own:
            return plain_rotary(st, q, k, v)
        q = st["cache"].append_rotary(q, k, v, st["batch"], st["rotary"], positions=st["positions"])
        k, v = st["cache"].read(st["batch"])
        return {"q": q, "k": k, "v": v}
    if case["op"] == "prefix":
        if not own:
            return plain_prefix(st)
        out, lse = st["cache"].attention(st["q"], st["batch"], lse=True, prefix=st["prefix"], workspace=st["workspace"])
        return {"out": out, "lse": lse}
    if own:
        pages = st["pages"]
        for i, batch in enumerate(st["batches"]):
            if case["kind"] == "fork" and i == 1:
                pages.fork(st["src"], st["dst"])
            pages.update(batch)
        if case["kind"] == "compact":
            pages.compact()
        table, held, refs = pages.table, pages.held, pages.refs
    else:
        for i, (kv_len, q_off, _) in enumerate(st["rounds"]):
            if case["kind"] == "fork" and i == 1:
                plain_fork(st)
            plain_update(st, kv_len, q_off)
        if case["kind"] == "compact":
            plain_compact(st)
        table, held, refs = st["table"], st["held"], st["refs"]
    # pages are moved as they are: code words, and scales and biases as their bits, are whole numbers here, not values
    return {"table": table, "held": held, "refs": refs,
            "layers": [[a if a.dtype == torch.int32 else a.view(torch.int16) for a in layer] for layer in st["layers"]]}


# ---- plain forms -----------------------------------------------------------------------------------------------------

def token_places(st):
    """Sequence, position, page and slot of every step token."""
    tok = torch.arange(sum(st["new"]), device="cuda", dtype=torch.int32)
    seq = torch.searchsorted(st["q_off"], tok, right=True) - 1
    pos = st["kv_len"][seq] - st["q_off"][seq + 1] + tok
    page = st["case"]["page"]
    return seq, pos, st["table"][seq, (pos // page).long()].long(), (pos % page).long()


def plain_rotary(st, q, k, v):
    case, rot = st["case"], st["case"]["rot"]
    _, pos, page, slot = token_places(st)
    at = pos[:, None] if st["positions"] is None else st["positions"][st["axis"]].T
    angle = at.double() * st["freq"].to(pos.device)  # far positions need every bit of it
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turned(x, weight):
        x = x.float()
        if weight is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight
        a, rest = x[..., :rot], x[..., rot:]
        if case["pairs"] == "halves":
            a, b = a.chunk(2, dim=-1)
            y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
        else:
            a, b = a[..., 0::2], a[..., 1::2]
            y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
        return torch.cat([y, rest], dim=-1).to(torch.bfloat16)

    got = {"q": turned(q, st["q_weight"])}
    for name, x in (("k", turned(k, st["k_weight"])), ("v", v)):
        c, s, b = quantise(x)
        st[name + "_codes"][page, :, slot] = pack(c)
        st[name + "_scales"][page, :, slot] = s
        st[name + "_biases"][page, :, slot] = b
        got[name] = values(c, s, b)
    return got


def plain_update(st, kv_len, q_off):
    """Every sequence holds the pages of its positions, and those of its step tokens alone."""
    table, refs, size = st["table"], st["refs"], st["case"]["page"]
    new = q_off[1:] - q_off[:-1]
    need = (kv_len + size - 1) // size
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    drop = (table >= 0) & (col >= need[:, None])
    refs.index_add_(0, table[drop], torch.full_like(table[drop], -1))
    table[drop] = -1
    held = torch.minimum(st["held"], need)
    # pages to be written that others hold too, and those that are not there yet, sequence by sequence
    first = torch.where(new > 0, (kv_len - new).clamp(min=0) // size, table.shape[1])
    twice = (col >= first[:, None]) & (col < held[:, None]) & (table >= 0) & (refs[table.clamp(min=0).long()] > 1)
    more = (col >= held[:, None]) & (col < need[:, None])
    want = (twice | more).flatten()
    free = torch.nonzero(refs == 0).flatten().to(torch.int32)
    place = torch.nonzero(want).flatten()
    page = free[:len(place)]  # lowest first (the cases have enough)
    before = table.flatten()[place]
    copied = twice.flatten()[place]
    src, dst = before[copied].long(), page[copied].long()
    for layer in st["layers"]:
        for a in layer:
            a[dst] = a[src]
    refs.index_add_(0, before[copied], torch.full_like(before[copied], -1))
    refs[page.long()] = 1
    table.view(-1)[place] = page
    st["held"].copy_(need)


def plain_fork(st):
    src, dst = st["src"].long(), st["dst"].long()
    rows = st["table"][src]
    st["refs"].index_add_(0, rows[rows >= 0], torch.ones_like(rows[rows >= 0]))
    st["table"][dst] = rows
    st["held"][dst] = st["held"][src]


def plain_compact(st):
    """Pages in use past their number move, in order, to the free ones below it."""
    refs, table = st["refs"], st["table"]
    live = int((refs > 0).sum())
    src, dst = torch.nonzero(refs[live:] > 0).flatten() + live, torch.nonzero(refs[:live] == 0).flatten()
    for layer in st["layers"]:
        for a in layer:
            a[dst] = a[src]
    to = torch.arange(len(refs), device=refs.device, dtype=torch.int32)
    to[src] = dst.to(torch.int32)
    refs[dst] = refs[src]
    refs[src] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], table))


def plain_prefix(st):
    case, d, size = st["case"], st["case"]["dim"], st["case"]["page"]
    kvh, heads = case["kv_heads"], case["heads"]

    def cached(name, pages):  # [kv head, position, dim]
        at = pages.long()
        x = values(unpack(st[name + "_codes"][at]), st[name + "_scales"][at], st[name + "_biases"][at])
        return x.transpose(0, 1).reshape(kvh, -1, d).float()

    outs, lses, first, common = [], [], 0, {}
    shared = [s // size for s in spread(case["groups"], case["prefix_lo"], case["prefix_hi"])]
    for i, (m, t) in enumerate(zip(st["new"], st["total"])):
        g, row = group_of(case)[i], st["table"][i]
        if g not in common:
            common = {g: [cached(name, row[:shared[g]]) for name in ("k", "v")]}
        k, v = (torch.cat([common[g][j], cached(name, row[shared[g]:-(-t // size)])], dim=1)[:, :t]
                for j, name in enumerate(("k", "v")))
        q = st["q"][first:first + m].float().reshape(m, kvh, -1, d).permute(1, 2, 0, 3).reshape(kvh, -1, d)
        s = torch.matmul(q, k.transpose(1, 2)).reshape(kvh, -1, m, t) * d ** -0.5
        hidden = torch.arange(t, device=q.device)[None, :] > torch.arange(t - m, t, device=q.device)[:, None]
        s.masked_fill_(hidden, -math.inf)
        top = s.amax(-1, keepdim=True)
        p = torch.exp(s.sub_(top))
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.reshape(kvh, -1, t), v).reshape(kvh, -1, m, d) / total
        outs.append(o.permute(2, 0, 1, 3).reshape(m, heads, d).to(torch.bfloat16))
        lses.append((top + torch.log(total)).squeeze(-1).permute(2, 0, 1).reshape(m, heads))
        first += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


# ---- exact values ----------------------------------------------------------------------------------------------------

def nearest_bf16(x):
    """The nearest bf16, ties to even, as doubles: the 45 low bits of the double's fraction go."""
    bits = x.contiguous().view(torch.int64)
    return ((bits + (1 << 44) - 1 + ((bits >> 45) & 1)) & ~((1 << 45) - 1)).view(torch.float64)


def exact(case, seed):
    """The definitions in 64 bits: whole numbers have none but themselves."""
    if case["op"] == "pages":
        return None
    st = inputs(case, seed)
    return exact_rotary(st) if case["op"] == "rotary" else exact_prefix(st)


def exact_rotary(st):
    case, n, half = st["case"], sum(st["new"]), st["case"]["rot"] // 2
    pos = torch.cat([torch.arange(t - m, t, device="cuda") for m, t in zip(st["new"], st["total"])])
    halves = case["pairs"] == "halves"
    x = st["qkv"].double()
    got = {}
    for name, lo, hi, w in (("q", 0, case["heads"], st["q_weight"]),
                            ("k", case["heads"], case["heads"] + case["kv_heads"], st["k_weight"])):
        y = x[:, lo:hi].clone()
        if w is not None:
            y = y / torch.sqrt(torch.sum(y ** 2, -1, keepdim=True) / case["dim"] + 1e-6) * w.double()
        z = y.clone()
        for i in range(half):
            a, b = (i, i + half) if halves else (2 * i, 2 * i + 1)
            p = pos if st["positions"] is None else st["positions"][st["axis"][i]]
            turn = torch.polar(torch.ones(n, dtype=torch.float64, device="cuda"), p.double() * float(st["freq"][i]))
            c = torch.complex(y[:, :, a], y[:, :, b]) * turn[:, None]
            z[:, :, a], z[:, :, b] = c.real, c.imag
        got[name] = z
    held = {"q": got["q"]}
    for name, y in (("k", nearest_bf16(got["k"])), ("v", x[:, case["heads"] + case["kv_heads"]:])):
        g = y.unflatten(-1, (-1, GROUP))
        b = g.min(-1, keepdim=True).values
        s = nearest_bf16((g.max(-1, keepdim=True).values - b) / 15.0)
        c = torch.where(s > 0, torch.round((g - b) / torch.where(s > 0, s, 1.0)).clamp(0, 15), 0.0)
        held[name] = nearest_bf16(c * s + b).flatten(-2)
    return held


def exact_prefix(st):
    case = st["case"]
    page, d, heads = case["page"], case["dim"], case["heads"]
    g = heads // case["kv_heads"]
    nib = 4 * torch.arange(8, device="cuda")

    def held(name, b, n):
        """Positions 0 .. n - 1 of sequence b, [n, kv head, dim], as doubles."""
        p = torch.arange(n, device="cuda")
        pg, sl = st["table"][b].long()[p // page], p % page
        w = st[name + "_codes"][pg, :, sl].long() & 0xFFFFFFFF
        c = ((w[..., None] >> nib) & 15).double().flatten(-2).unflatten(-1, (-1, GROUP))
        x = c * st[name + "_scales"][pg, :, sl].double()[..., None] + st[name + "_biases"][pg, :, sl].double()[..., None]
        return nearest_bf16(x).flatten(-2)

    outs, lses, at = [], [], 0
    for b, (m, t) in enumerate(zip(st["new"], st["total"])):
        k, v = held("k", b, t), held("v", b, t)
        later = torch.arange(t, device="cuda")[None, :] > torch.arange(t - m, t, device="cuda")[:, None]
        out = torch.empty(m, heads, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(m, heads, dtype=torch.float64, device="cuda")
        for h in range(heads):
            s = (st["q"][at:at + m, h].double() @ k[:, h // g].T) / math.sqrt(d)
            s[later] = -math.inf
            lse[:, h] = torch.logsumexp(s, -1)
            out[:, h] = torch.exp(s - lse[:, h, None]) @ v[:, h // g]
        outs.append(out)
        lses.append(lse)
        at += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
