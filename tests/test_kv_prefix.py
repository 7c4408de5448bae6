"""Attention of sequences that share their first positions: the same values as without sharing, from the definition in 64 bits."""
import ctypes
import math

import numpy as np
import pytest

import bit_moe_expert_routing_gb300 as moe
from bit_moe_expert_routing_gb300 import build

torch = pytest.importorskip("torch")

from kv_util import Batch, attention_reference, check_attention, fill, junk_cache  # noqa: E402

P = 1 << 20  # a well-aligned address that nothing reads


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moe.lib()


# --- refusals and sizes, on the CPU -------------------------------------------------------------------

def c_args(n_seqs=8, n_tokens=8, max_new=1, max_kv=1000, heads=16, window=0, **prefix):
    x = moe.moe_kv_prefix(2, 4, 500, 600, P, P)
    for name, v in prefix.items():
        setattr(x, name, v)
    return (moe.moe_kv_cache(10, 16, 2, 128, P, P, P, P, P, P, P), moe.moe_kv_batch(n_seqs, n_tokens, max_new, max_kv, P, P, P, 64),
            x, moe.moe_attention(heads, window, 0, 0.1))


def size(*a, **kw):
    return moe.moe_attention_prefix_workspace_size(*c_args(*a, **kw))


def forward(args, q=P, qs=2048, out=2 * P, lse=None, ws=P, nbytes=1 << 40):
    return moe.moe_attention_prefix_forward(*args, q, qs, out, lse, ws, nbytes, None)


@pytest.mark.parametrize("prefix", [dict(n_groups=-1), dict(n_groups=65536), dict(max_tokens=-1), dict(max_len=-1),
                                    dict(max_len=2 ** 24 + 1), dict(max_own=-1), dict(max_own=2 ** 24 + 1), dict(seq_off=None),
                                    dict(length=None), dict(seq_off=P + 2), dict(length=P + 1)])
def test_bad_groups_are_refused(prefix):
    assert size(**prefix) == 0
    assert forward(c_args(**prefix)) == moe.MOE_ERR_ARG
    assert moe.moe_last_launch_count() == 0


def test_what_the_attention_refuses_is_refused():
    a = c_args()
    for kw in (dict(q=None), dict(q=P + 2), dict(qs=2047), dict(out=None), dict(out=2 * P + 8), dict(out=P), dict(lse=2 * P + 2)):
        assert forward(a, **kw) == moe.MOE_ERR_ARG, kw
    n = size()
    for kw in (dict(ws=None), dict(ws=P + 16), dict(nbytes=n - 1)):
        assert forward(a, **kw) == moe.MOE_ERR_WORKSPACE
    assert forward(c_args(heads=7)) == moe.MOE_ERR_SHAPE and forward(c_args(window=-1)) == moe.MOE_ERR_ARG
    assert moe.lib().moe_attention_prefix_forward(*(ctypes.byref(x) for x in a[:2]), None, ctypes.byref(a[3]), P, 2048, 2 * P,
                                                  None, P, 1 << 40, None) == moe.MOE_ERR_ARG
    assert forward(c_args(n_tokens=0), q=None, out=None, ws=None) == moe.MOE_OK
    assert moe.moe_last_launch_count() == 0


@pytest.mark.parametrize("window", [0, 512])
def test_a_larger_steps_workspace_serves_a_smaller_one(window):
    """No bound of the step or of its groups lowers the size."""
    seqs, tokens, kv = [1, 2, 8, 33, 64, 300], [1, 8, 64, 600, 4000], [100, 448, 900, 2048, 2100, 40000]
    groups, most, lens, own = [0, 1, 2, 7, 64], [0, 1, 8, 17, 64, 600], [0, 15, 16, 896, 2100, 33000], [1, 447, 900, 2050, 9000]
    got = {}
    grid = (seqs, tokens, kv, groups, most, lens, own)
    for i in np.ndindex(*(len(g) for g in grid)):
        s, t, v, g, m, l, o = (x[k] for x, k in zip(grid, i))
        n = got[i] = size(s, t, min(t, 17), v, window=window, n_groups=g, max_tokens=m, max_len=l, max_own=o)
        for a in range(7):
            below = i[:a] + (i[a] - 1,) + i[a + 1:]
            assert got.get(below, 1) <= n, (s, t, v, g, m, l, o, a)


# --- results ----------------------------------------------------------------------------------------

class Shared(Batch):
    """Groups of sequences: `groups` has (shared positions, [(step tokens, positions past them)]). The shared whole pages
    are the same ones in all of a group's rows."""

    def __init__(self, groups, page, seed=0):
        new = [n for _, s in groups for n, _ in s]
        kv = [length // page * page + own for length, s in groups for _, own in s]
        super().__init__(new, kv, page, seed)
        self.seq_off = np.cumsum([0] + [len(s) for _, s in groups]).astype(np.int32)
        self.length = np.array([length for length, _ in groups], dtype=np.int32)
        for g, (length, s) in enumerate(groups):
            first = self.seq_off[g]
            for b in range(first + 1, self.seq_off[g + 1]):
                self.table[b, :length // page] = self.table[first, :length // page]

    def prefix(self, **over):
        groups = range(len(self.length))
        tokens = [sum(self.new[self.seq_off[g]:self.seq_off[g + 1]]) for g in groups]
        own = [self.kv[b] - self.length[g] // self.page * self.page for g in groups
               for b in range(self.seq_off[g], self.seq_off[g + 1])]
        kw = dict(max_tokens=max(tokens), max_len=int(max(self.length)), max_own=int(max(own)))
        kw.update(over)
        return moe.KVPrefix(torch.from_numpy(self.seq_off).cuda(), torch.from_numpy(self.length).cuda(), **kw)


def share(cache, batch, held):
    """fill() gave every sequence its own values, the later ones over the earlier in shared pages: what is there is what
    the last sequence of a group put there."""
    for per_seq in held:
        for g in range(len(batch.length)):
            n = int(batch.length[g]) // batch.page * batch.page
            last = per_seq[batch.seq_off[g + 1] - 1] if batch.seq_off[g + 1] > batch.seq_off[g] else None
            for b in range(batch.seq_off[g], batch.seq_off[g + 1]):
                per_seq[b][:n] = last[:min(n, len(per_seq[b]))]
    return held


def rows(n, heads, dim, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, heads, dim, generator=g, device="cuda").to(torch.bfloat16)


@pytest.fixture
def each_path():
    def paths():
        for path in (0, 1, 2):
            moe.moe_set_option(moe.MOE_OPT_FORCE_PATH, path)
            yield path
    yield paths
    moe.moe_set_option(moe.MOE_OPT_FORCE_PATH, 0)


GROUPS = [
    [(100, [(1, 1), (1, 30), (1, 7)])],
    [(16, [(1, 1)] * 2), (0, [(1, 5), (2, 2)]), (333, [(1, 50)]), (15, [(3, 9), (1, 1)])],
    [(700, [(4, 4 + 9 * i) for i in range(9)]), (64, [(5, 5), (1, 300)])],
    [(257, [(40, 40), (1, 2), (130, 160), (17, 17)])],
    [(1200, [(0, 3), (1, 10), (0, 0), (1, 1)]), (50, [(0, 0), (0, 1)])],
    [(2500, [(1, 1 + 13 * i) for i in range(20)])],
    [(130, [(70, 70), (33, 64), (0, 5), (90, 300)]), (16, [(129, 200), (128, 128), (1, 1)]), (0, [(40, 41)])],
    [(1000, [(256, 256)] * 3 + [(1, 129)] + [(300, 512)])],
]


@pytest.mark.gpu
@pytest.mark.parametrize("dim,heads,kv_heads,page", [(64, 8, 8, 16), (128, 16, 2, 16), (256, 6, 2, 64), (64, 20, 4, 32),
                                                    (128, 64, 1, 128)])
@pytest.mark.parametrize("groups", GROUPS, ids=range(len(GROUPS)))
def test_sharing_changes_no_value(groups, dim, heads, kv_heads, page, each_path):
    batch = Shared(groups, page)
    cache = junk_cache(moe, batch.n_pages, page, kv_heads, dim)
    held = share(cache, batch, fill(cache, batch, outliers=True))
    q = rows(batch.n_tokens, heads, dim)
    ref = attention_reference(q, batch, *held, float(np.float32(dim ** -0.5)))
    dev, prefix = batch.device(moe), batch.prefix()
    for path in each_path():
        ws = cache.attention_workspace(heads, dev, prefix=prefix)
        ws.fill_(0xFF)
        out, lse = cache.attention(q, dev, lse=True, prefix=prefix, workspace=ws)
        cache.check()
        check_attention(out, lse, ref, path)
        # bounds far above the lengths
        wide = batch.prefix(max_tokens=batch.n_tokens, max_len=6000, max_own=7000)
        out = cache.attention(q, batch.device(moe, max_kv=9000), prefix=wide)
        cache.check()
        check_attention(out, None, ref, path)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("scale", [0.0, -0.05, 3.0])
def test_other_scales(dim, scale, each_path):
    batch = Shared([(300, [(2, 20), (1, 1), (9, 40)])], 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, dim)
    held = share(cache, batch, fill(cache, batch, spread=0.3))
    q = rows(batch.n_tokens, 8, dim)
    ref = attention_reference(q, batch, *held, float(np.float32(scale)))
    for path in each_path():
        out, lse = cache.attention(q, batch.device(moe), scale=scale, lse=True, prefix=batch.prefix())
        cache.check()
        check_attention(out, lse, ref, path)


@pytest.mark.gpu
def test_long_prefixes_and_many_rows():
    """The part that is shared on the tensor cores, divided over the GPU; the sequences' own parts of a few rows and of many."""
    for dim, heads, kv_heads, groups in ((256, 16, 2, [(20000, [(1, 1 + 29 * i) for i in range(40)])]),
                                         (128, 16, 2, [(9000, [(1, 60)] * 17), (4000, [(70, 90), (200, 300)])]),
                                         (64, 16, 4, [(6000, [(90, 90), (301, 301), (2, 2)])])):
        batch = Shared(groups, 64)
        cache = junk_cache(moe, batch.n_pages, 64, kv_heads, dim)
        held = share(cache, batch, fill(cache, batch))
        q = rows(batch.n_tokens, heads, dim)
        ref = attention_reference(q, batch, *held, float(np.float32(dim ** -0.5)))
        out, lse = cache.attention(q, batch.device(moe), lse=True, prefix=batch.prefix())
        cache.check()
        check_attention(out, lse, ref, dim)


@pytest.mark.gpu
def test_several_passes():
    """More expanded keys than one pass has room for, group by group and head by head; against the same without sharing."""
    dim, kvh, page, shared, seqs, new = 256, 8, 256, 131072, 8, 70
    pages = 4 * shared // page
    cache = moe.KVCache.empty(pages + 2 * seqs, page, kvh, dim)
    g = torch.Generator(device="cuda").manual_seed(4)
    for t in (cache.k_codes, cache.v_codes):
        t.random_(generator=g)
    for name, scale in (("k", 2.0 ** -6), ("v", 2.0 ** -3)):  # values of +-1: a score of a few units
        getattr(cache, name + "_scales").fill_(scale)
        getattr(cache, name + "_biases").fill_(-8 * scale)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.cat([torch.arange(pages).view(4, -1).repeat_interleave(2, 0), pages + torch.arange(2 * seqs).view(seqs, 2)], 1)
    batch = moe.KVBatch(i([new * b for b in range(seqs + 1)]), i([shared + new + 31 * b for b in range(seqs)]),
                        table.int().cuda().contiguous(), seqs * new, new, shared + 512)
    q = rows(seqs * new, 8, dim)
    prefix = moe.KVPrefix(i([0, 2, 4, 6, 8]), i([shared] * 4), 2 * new, shared, 512)
    ref, ref_lse = cache.attention(q, batch, lse=True)
    out, lse = cache.attention(q, batch, lse=True, prefix=prefix)
    cache.check()
    # both are within 2^-8 (|o| + sum p |v|) of the value, |v| at most 1
    assert ((out.double() - ref.double()).abs() <= 2.0 ** -7 * (ref.double().abs() + 1)).all()
    torch.testing.assert_close(lse, ref_lse, atol=2.0 ** -15, rtol=2.0 ** -17)
    assert ref.float().std() > 0.001


@pytest.mark.gpu
def test_a_window_reads_near_positions_only(each_path):
    batch = Shared([(300, [(2, 20), (1, 1)])], 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, 128)
    held = share(cache, batch, fill(cache, batch))
    q = rows(batch.n_tokens, 8, 128)
    for window, sinks in ((40, 3), (2 ** 31 - 1, 0)):
        ref = attention_reference(q, batch, *held, float(np.float32(128 ** -0.5)), window, sinks)
        for path in each_path():
            out, lse = cache.attention(q, batch.device(moe), window=window, sinks=sinks, lse=True, prefix=batch.prefix())
            cache.check()
            check_attention(out, lse, ref, (window, path))


@pytest.mark.gpu
@pytest.mark.parametrize("heads,new", [(8, [1, 3, 1]), (16, [40, 30, 60])])
def test_sequences_that_begin_inside_the_shared_part_are_on_their_own(heads, new, each_path):
    """Lengths larger than what a sequence has behind its step tokens: it is attended to whole; the others share."""
    batch = Shared([(160, [(n, n + 8) for n in new])], 16)
    batch.kv[1] = 90  # within the shared pages
    cache = junk_cache(moe, batch.n_pages, 16, 2, 64)
    held = share(cache, batch, fill(cache, batch))
    q = rows(batch.n_tokens, heads, 64)
    ref = attention_reference(q, batch, *held, 0.125)
    for path in each_path():
        out, lse = cache.attention(q, batch.device(moe), lse=True, prefix=batch.prefix(max_own=100))
        cache.check()
        check_attention(out, lse, ref, path)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("heads,new", [(8, [1, 3, 1]), (16, [70, 60, 90])])
def test_sequences_that_ended_and_groups_of_which_nobody_shares(dim, heads, new, each_path):
    """A group's first sequence has ended and its pages are gone, or is there without step tokens, or all begin inside."""
    groups = [(160, [(0, 0), (new[0], new[0] + 8), (new[1], new[1])]), (96, [(0, 7), (0, 3), (new[2], 99)]),
              (400, [(new[0], new[0]), (new[1], new[1])]), (64, [(0, 0), (0, 0)])]
    batch = Shared(groups, 16)
    batch.kv[6], batch.kv[7] = 70, 90  # inside the shared 400
    cache = junk_cache(moe, batch.n_pages, 16, 2, dim)
    held = share(cache, batch, fill(cache, batch))
    table = batch.table.copy()
    batch.kv[0] = batch.kv[3] = batch.kv[8] = batch.kv[9] = 0
    table[[0, 3, 8, 9]] = -1
    dev = batch.device(moe, max_kv=1000)
    dev._t[2].copy_(torch.from_numpy(table))
    for per_seq in held:
        for b in (0, 3, 8, 9):
            per_seq[b] = per_seq[b][:0]
    q = rows(batch.n_tokens, heads, dim)
    ref = attention_reference(q, batch, *held, float(np.float32(dim ** -0.5)))
    for path in each_path():
        out, lse = cache.attention(q, dev, lse=True, prefix=batch.prefix(max_own=600))
        cache.check()
        check_attention(out, lse, ref, path)


@pytest.mark.gpu
@pytest.mark.parametrize("heads,new", [(8, [1, 3, 1]), (16, [40, 30, 60])])
def test_groups_out_of_order_or_past_their_bounds_share_nothing(heads, new, each_path):
    batch = Shared([(160, [(new[0], new[0] + 8), (new[1], new[1])]), (64, [(new[2], 99)])], 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, 64)
    held = share(cache, batch, fill(cache, batch))
    q = rows(batch.n_tokens, heads, 64)
    ref = attention_reference(q, batch, *held, 0.125)
    dev = batch.device(moe)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    good = dict(max_tokens=max(new[0] + new[1], new[2]), max_len=160, max_own=260)
    for path in each_path():
        for seq_off, length, over in ((i(0, 2, 4), i(160, 64), {}), (i(1, 2, 3), i(160, 64), {}), (i(0, 4, 3), i(160, 64), {}),
                                      (i(0, -1, 3), i(160, 64), {}), (i(0, 2, 2), i(160, 64), {}), (i(0, 2, 3), i(161, 64), {}),
                                      (i(0, 2, 3), i(-1, 64), {}), (i(0, 2, 3), i(160, 64), dict(max_tokens=new[0]))):
            out, lse = cache.attention(q, dev, lse=True, prefix=moe.KVPrefix(seq_off, length, **dict(good, **over)))
            if path:  # (by its size, this step is taken whole)
                with pytest.raises(moe.MoEError):
                    cache.check()
            check_attention(out, lse, ref, (path, seq_off.tolist(), length.tolist()))
        if not path:
            continue
        # one past max_own: recorded, and its rows stay as they are
        out = torch.full_like(q, 7.0)
        cache.attention(q, dev, out=out, prefix=batch.prefix(max_own=50))
        with pytest.raises(moe.MoEError):
            cache.check()
        n = new[0] + new[1]
        assert (out[n:] == 7.0).all()
        check_attention(out[:n], None, tuple(r[:n] for r in ref), path)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [(1, 3), (50, 20)])
def test_missing_pages_are_left_out(new, each_path):
    """A page of the shared part that is missing: its positions are seen by none of the group, and that is recorded."""
    batch = Shared([(160, [(new[0], new[0] + 8), (new[1], 30)])], 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, 64)
    held = share(cache, batch, fill(cache, batch))
    dev = batch.device(moe)
    dev._t[2][:, 3] = -1
    q = rows(batch.n_tokens, 8, 64)
    # as if those keys were not there
    cut = lambda t: torch.cat([t[:48], t[64:]])  # noqa: E731
    short = Batch(batch.new, [k - 16 for k in batch.kv], 16)
    ref = attention_reference(q, short, *([cut(t) for t in per_seq] for per_seq in held), 0.125)
    for path in each_path():
        out, lse = cache.attention(q, dev, lse=True, prefix=batch.prefix())
        with pytest.raises(moe.MoEError):
            cache.check()
        check_attention(out, lse, ref, path)


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_captured_steps_and_a_consumer_behind_them(dim):
    """One graph per step, replayed with the lengths advanced in place, two graphs on one workspace, another stream."""
    batch = Shared([(400, [(1, 20), (1, 60), (1, 33)]), (200, [(1, 5)] * 5)], 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, dim)
    held = share(cache, batch, fill(cache, batch))
    q = rows(batch.n_tokens, 16, dim)
    dev = batch.device(moe, max_kv=2000)
    prefix = batch.prefix(max_own=1000, max_len=1500)
    ws = cache.attention_workspace(16, dev, prefix=prefix)
    out, got = torch.empty_like(q), [torch.empty_like(q) for _ in range(2)]
    cache.attention(q, dev, out=out, workspace=ws, prefix=prefix)
    torch.cuda.synchronize()
    graphs = []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out.fill_(math.nan)
            cache.attention(q, dev, out=out, workspace=ws, prefix=prefix)
            got[k].copy_(out)
        graphs.append(g)
    lens = dev._t[1]
    for back in (7, 4, 0):
        kv = [n - min(back, 4) if n - min(back, 4) > 416 or n < 300 else n for n in batch.kv]
        kv = [max(k, (400 if b < 3 else 192) + 1) for b, k in enumerate(kv)]
        lens.copy_(torch.tensor(kv, dtype=torch.int32))
        now = Batch.__new__(Batch)
        now.__dict__.update(batch.__dict__, kv=kv)
        ref = attention_reference(q, now, *([t[:k] for t, k in zip(p, kv)] for p in held), float(np.float32(dim ** -0.5)))
        for _ in range(5):
            for k, g in enumerate(graphs):
                g.replay()
        torch.cuda.synchronize()
        for o in got:
            check_attention(o, None, ref, back)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = cache.attention(q, dev, prefix=prefix, stream=s)
    s.synchronize()
    assert torch.equal(o, got[0])
    cache.check()
    cpu = torch.zeros(3, dtype=torch.int32)
    for bad in (lambda: moe.KVPrefix(cpu, cpu[:2], 1, 1, 1), lambda: moe.KVPrefix(cpu.cuda(), cpu.cuda(), 1, 1, 1),
                lambda: moe.KVPrefix(cpu.cuda().long(), cpu.cuda()[:2], 1, 1, 1),
                lambda: moe.KVPrefix(cpu.cuda(), cpu.cuda()[:2], 1, 2 ** 31, 1)):
        with pytest.raises(ValueError):
            bad()
