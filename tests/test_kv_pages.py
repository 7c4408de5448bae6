"""The pages of a set of sequences: what update, fork, compact and copy do to tables, references and contents, against a
plain model that goes through the sequences one by one."""
import ctypes

import numpy as np
import pytest

import bit_moe_expert_routing_gb300 as moe
from bit_moe_expert_routing_gb300 import build

torch = pytest.importorskip("torch")

P = 1 << 20  # a well-aligned address that nothing reads


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moe.lib()


# --- refusals, on the CPU ---------------------------------------------------------------------------

def c_pages(**kw):
    p = moe.moe_kv_pages(10, 16, 4, 8, P, P, P, P, P)
    for name, v in kw.items():
        setattr(p, name, v)
    return p


def c_cache(**kw):
    c = moe.moe_kv_cache(10, 16, 2, 128, P, P, P, P, P, P, P)
    for name, v in kw.items():
        setattr(c, name, v)
    return c


def c_batch(**kw):
    b = moe.moe_kv_batch(4, 4, 1, 100, P, P, P, 8)
    for name, v in kw.items():
        setattr(b, name, v)
    return b


@pytest.mark.parametrize("pages,want", [
    (dict(page_size=8), moe.MOE_ERR_SHAPE), (dict(page_size=24), moe.MOE_ERR_SHAPE), (dict(page_size=512), moe.MOE_ERR_SHAPE),
    (dict(n_pages=0), moe.MOE_ERR_SHAPE), (dict(n_seqs=0), moe.MOE_ERR_SHAPE), (dict(n_seqs=65536), moe.MOE_ERR_SHAPE),
    (dict(columns=0), moe.MOE_ERR_SHAPE), (dict(columns=2 ** 20 + 1), moe.MOE_ERR_SHAPE), (dict(table=None), moe.MOE_ERR_ARG),
    (dict(held=P + 4), moe.MOE_ERR_ARG), (dict(refs=P + 8), moe.MOE_ERR_ARG), (dict(scratch=None), moe.MOE_ERR_ARG),
    (dict(status=P + 16), moe.MOE_ERR_ARG)])
def test_bad_sets_are_refused(pages, want):
    p, c = c_pages(**pages), [c_cache()]
    assert moe.moe_kv_pages_update(p, c_batch(), c, None) == want
    assert moe.moe_kv_pages_fork(p, P, P, 1, None) == want
    assert moe.moe_kv_pages_compact(p, c, None) == want
    assert moe.moe_last_launch_count() == 0


def test_bad_caches_and_steps_are_refused():
    p = c_pages()
    for caches, want in (([], moe.MOE_ERR_ARG), ([c_cache(head_dim=96)], moe.MOE_ERR_SHAPE),
                         ([c_cache(k_codes=None)], moe.MOE_ERR_ARG), ([c_cache(), c_cache(kv_heads=4)], moe.MOE_ERR_SHAPE),
                         ([c_cache(), c_cache(head_dim=64)], moe.MOE_ERR_SHAPE)):
        assert moe.moe_kv_pages_update(p, c_batch(), caches, None) == want
        assert moe.moe_kv_pages_compact(p, caches, None) == want
        assert moe.moe_kv_copy_pages(caches, P, P, 1, None) == want
    for caches in ([c_cache(n_pages=11)], [c_cache(page_size=32)], [c_cache(), c_cache(n_pages=9)]):
        assert moe.moe_kv_pages_update(p, c_batch(), caches, None) == moe.MOE_ERR_SHAPE
        assert moe.moe_kv_pages_compact(p, caches, None) == moe.MOE_ERR_SHAPE
    for batch in (dict(n_seqs=3), dict(block_table=2 * P), dict(table_stride=9), dict(q_off=None), dict(kv_len=None),
                  dict(kv_len=P + 2), dict(max_new=-1), dict(max_kv=-1), dict(max_kv=2 ** 24 + 1)):
        assert moe.moe_kv_pages_update(p, c_batch(**batch), [c_cache()], None) == moe.MOE_ERR_ARG, batch
    l, ref = moe.lib(), ctypes.byref
    one = moe._caches([c_cache()])
    assert l.moe_kv_pages_update(ref(p), None, one, 1, None) == moe.MOE_ERR_ARG
    assert l.moe_kv_pages_update(ref(p), ref(c_batch()), None, 1, None) == moe.MOE_ERR_ARG
    assert l.moe_kv_pages_update(None, ref(c_batch()), one, 1, None) == moe.MOE_ERR_ARG
    assert l.moe_kv_pages_compact(ref(p), (moe._KC * 1)(), 1, None) == moe.MOE_ERR_ARG
    for src, dst, n in ((P, P, -1), (P, P, 5), (None, P, 1), (P, None, 1), (P + 2, P, 1), (P, P + 1, 1)):
        assert moe.moe_kv_pages_fork(p, src, dst, n, None) == moe.MOE_ERR_ARG
    for src, dst, n in ((P, P, -1), (None, P, 1), (P, None, 1), (P + 2, P, 1), (P, P + 1, 1)):
        assert moe.moe_kv_copy_pages([c_cache()], src, dst, n, None) == moe.MOE_ERR_ARG
    assert moe.moe_kv_pages_fork(p, None, None, 0, None) == moe.MOE_OK
    assert moe.moe_kv_copy_pages([c_cache()], None, None, 0, None) == moe.MOE_OK
    assert moe.moe_last_launch_count() == 0


def test_scratch_sizes():
    assert moe.moe_kv_pages_scratch(10, 4) > 30
    for n_pages, n_seqs in ((0, 1), (1, 0), (-1, 1), (2 ** 28 + 1, 1), (1, 65536)):
        assert moe.moe_kv_pages_scratch(n_pages, n_seqs) == 0


# --- a plain model -----------------------------------------------------------------------------------

class Model:
    """The set and a word per page for its contents."""

    def __init__(self, n_pages, size, n_seqs, columns):
        self.size, self.columns = size, columns
        self.table = np.full((n_seqs, columns), -1, dtype=np.int64)
        self.held = np.zeros(n_seqs, dtype=np.int64)
        self.refs = np.zeros(n_pages, dtype=np.int64)
        self.words = np.arange(n_pages) + 1000
        self.bad = False

    def update(self, kv, new, max_new, max_kv):
        ok = [0 <= k <= max_kv and 0 <= n <= max_new and -(-k // self.size) <= self.columns for k, n in zip(kv, new)]
        self.bad |= not all(ok)
        for b, k in enumerate(kv):
            if ok[b]:
                for j in range(-(-k // self.size), self.held[b]):
                    if self.table[b, j] >= 0:
                        self.refs[self.table[b, j]] -= 1
                    self.table[b, j] = -1
                self.held[b] = min(self.held[b], -(-k // self.size))
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        shared = self.refs > 1
        for b, (k, n) in enumerate(zip(kv, new)):
            if not ok[b] and n and k >= 0:  # what it might write leaves it, if others hold it
                for j in range(max(k - n, 0) // self.size if n > 0 else 0, self.held[b]):
                    if self.table[b, j] >= 0 and shared[self.table[b, j]]:
                        self.refs[self.table[b, j]] -= 1
                        self.table[b, j] = -1
        old, words = self.table.copy(), self.words.copy()
        out = False
        for b, (k, n) in enumerate(zip(kv, new)):
            if not ok[b]:
                continue
            first = max(k - n, 0) // self.size if n > 0 else self.columns
            copies = [j for j in range(first, self.held[b]) if old[b, j] >= 0 and shared[old[b, j]]]
            more = list(range(self.held[b], -(-k // self.size)))
            if not copies and not more:
                continue
            out |= len(copies) + len(more) > len(free)
            for j in copies:
                self.refs[old[b, j]] -= 1
                self.table[b, j] = -1
                if not out:
                    to = free.pop(0)
                    self.table[b, j], self.refs[to], self.words[to] = to, 1, words[old[b, j]]
            if not out:
                for j in more:
                    to = free.pop(0)
                    self.table[b, j], self.refs[to] = to, 1
                self.held[b] += len(more)
        self.bad |= out

    def fork(self, src, dst):
        n = len(self.held)
        held = self.held.copy()
        for i, (s, d) in enumerate(zip(src, dst)):
            if not (0 <= s < n and 0 <= d < n) or d in src or d in dst[:i] or held[d]:
                self.bad = True
                continue
            self.table[d], self.held[d] = self.table[s], self.held[s]
            for p in self.table[s, :self.held[s]]:
                if p >= 0:
                    self.refs[p] += 1

    def compact(self):
        live = int((self.refs > 0).sum())
        src = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        dst = [p for p in range(live) if self.refs[p] == 0]
        for s, d in zip(src, dst):
            self.words[d] = self.words[s]
            self.refs[d], self.refs[s] = self.refs[s], 0
            self.table[self.table == s] = d


def caches(layers, n_pages, size, kv_heads, dim):
    """Caches whose pages hold their layer's and their own number everywhere."""
    out = []
    for i in range(layers):
        c = moe.KVCache.empty(n_pages, size, kv_heads, dim)
        for a, t in enumerate((c.k_codes, c.k_scales, c.k_biases, c.v_codes, c.v_scales, c.v_biases)):
            w = torch.arange(n_pages, dtype=torch.int32, device="cuda") + 1000
            if t.dtype == torch.int32:
                t.copy_((w * 64 + i * 8 + a).view(-1, 1, 1, 1).expand_as(t))
            else:
                t.view(torch.int16).copy_((w * 8 + a).to(torch.int16).view(-1, 1, 1, 1).expand_as(t))
        out.append(c)
    return out


def check_words(cs, words):
    w = torch.from_numpy(words).to(torch.int32).cuda()
    for i, c in enumerate(cs):
        for a, t in enumerate((c.k_codes, c.k_scales, c.k_biases, c.v_codes, c.v_scales, c.v_biases)):
            if t.dtype == torch.int32:
                want = (w * 64 + i * 8 + a).view(-1, 1, 1, 1)
            else:
                t, want = t.view(torch.int16), (w * 8 + a).to(torch.int16).view(-1, 1, 1, 1)
            assert torch.equal(t, want.expand_as(t)), (i, a)


def check_same(pages, model):
    assert pages.table.cpu().tolist() == model.table.tolist()
    assert pages.held.cpu().tolist() == model.held.tolist()
    assert pages.refs.cpu().tolist() == model.refs.tolist()
    check_words(pages.caches, model.words)
    if model.bad:
        with pytest.raises(moe.MoEError):
            pages.check()
        model.bad = False
    else:
        pages.check()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def step(pages, kv, new, max_new=None, max_kv=None):
    off = np.concatenate([[0], np.cumsum(new)])
    return pages.batch(i32(*off.tolist()), i32(*kv), int(max(0, off[-1])), max_new if max_new is not None else max(1, *new),
                       max_kv if max_kv is not None else pages.columns * pages.page_size)


@pytest.mark.gpu
@pytest.mark.parametrize("n_pages,size,n_seqs,columns,kv_heads,dim,layers", [
    (40, 16, 5, 9, 1, 64, 1), (97, 32, 40, 12, 3, 128, 2), (1, 16, 2, 1, 2, 256, 1), (5003, 16, 130, 50, 1, 64, 1),
    (300, 256, 33, 40, 2, 128, 1), (200, 64, 7, 33, 8, 128, 3),
    (30001, 16, 9, 4000, 1, 64, 1), (70003, 16, 300, 300, 1, 64, 1)])
def test_a_long_random_run(n_pages, size, n_seqs, columns, kv_heads, dim, layers):
    """Steps that grow, shrink, end and fork sequences, with too few pages and bad numbers now and then."""
    r = np.random.RandomState(n_pages + n_seqs)
    pages = moe.KVPages(caches(layers, n_pages, size, kv_heads, dim), n_seqs, columns)
    m = Model(n_pages, size, n_seqs, columns)
    kv = np.zeros(n_seqs, dtype=np.int64)
    for turn in range(40):
        what = r.randint(6)
        if what == 0 and n_seqs > 1:
            n = r.randint(1, n_seqs)
            src, dst = r.randint(0, n_seqs, n), r.randint(-1, n_seqs + 1, n)
            if r.randint(3):  # mostly ones that go through
                empty = [b for b in range(n_seqs) if m.held[b] == 0]
                full = [b for b in range(n_seqs) if m.held[b] > 0]
                if not empty or not full:
                    continue
                dst = r.permutation(empty)[:r.randint(1, len(empty) + 1)]
                src = r.choice(full, len(dst))
                kv[dst] = kv[src]
            pages.fork(i32(*src.tolist()), i32(*dst.tolist()))
            m.fork(src.tolist(), dst.tolist())
        elif what == 1:
            pages.compact()
            m.compact()
        else:
            budget = n_pages * size // max(1, n_seqs) * (1 if r.randint(4) else 3)
            new = np.zeros(n_seqs, dtype=np.int64)
            for b in range(n_seqs):
                k = r.randint(8)
                if k == 0:
                    kv[b] = 0
                elif k == 1:
                    kv[b] = max(0, kv[b] - r.randint(0, 3 * size))
                elif k < 6:
                    new[b] = r.randint(1, 2 * size) if k < 4 else 1
                    kv[b] = min(kv[b] + new[b], columns * size, budget)
            asked = kv.copy()
            if r.randint(5) == 0:
                asked[r.randint(n_seqs)] = r.choice([-1, columns * size + 1, 2 ** 24])
            pages.update(step(pages, asked.tolist(), new.tolist()))
            m.update(asked.tolist(), new.tolist(), max(1, *new), columns * size)
            kv = np.minimum(kv, m.held * size)
        check_same(pages, m)


@pytest.mark.gpu
def test_forks_copy_what_they_write_and_no_more():
    cs = caches(2, 50, 16, 2, 64)
    pages, m = moe.KVPages(cs, 6, 8), Model(50, 16, 6, 8)
    moves = [([100, 0, 0, 0, 0, 0], [100, 0, 0, 0, 0, 0])]
    for kv, new in moves:
        pages.update(step(pages, kv, new)), m.update(kv, new, 100, 128)
    pages.fork(i32(0, 0, 0), i32(1, 3, 5)), m.fork([0, 0, 0], [1, 3, 5])
    check_same(pages, m)
    assert m.refs.max() == 4 and m.held.tolist() == [7, 7, 0, 7, 0, 7]
    # 1 writes into the shared last page, 3 only past a page's end, 5 nothing, and 0 goes back to 90 and on from there
    kv, new = [91, 101, 0, 113, 0, 100], [1, 1, 0, 1, 0, 0]
    pages.update(step(pages, kv, new)), m.update(kv, new, 1, 128)
    check_same(pages, m)
    assert m.table[1, 6] not in m.table[5] and m.table[3, 6] == m.table[5, 6] and m.table[0, 5] not in m.table[5]
    # chains of forks, a fork of a fork that ended
    pages.fork(i32(3), i32(2)), m.fork([3], [2])
    kv, new = [0, 101, 114, 0, 0, 100], [0, 0, 1, 0, 0, 0]
    pages.update(step(pages, kv, new)), m.update(kv, new, 1, 128)
    check_same(pages, m)
    pages.compact(), m.compact()
    check_same(pages, m)


@pytest.mark.gpu
def test_no_page_of_another_sequence_is_written_when_pages_run_out():
    pages, m = moe.KVPages(caches(1, 3, 16, 1, 64), 3, 4), Model(3, 16, 3, 4)
    for kv, new in (([40, 0, 0], [40, 0, 0]),):
        pages.update(step(pages, kv, new)), m.update(kv, new, 40, 64)
    pages.fork(i32(0), i32(1)), m.fork([0], [1])
    kv, new = [40, 41, 0], [0, 1, 0]
    pages.update(step(pages, kv, new)), m.update(kv, new, 1, 64)
    assert m.bad and m.table[1].tolist() == [m.table[0, 0], m.table[0, 1], -1, -1]
    check_same(pages, m)
    kv, new = [40, 0, 1], [0, 0, 1]  # and it can end
    pages.update(step(pages, kv, new)), m.update(kv, new, 1, 64)
    assert m.bad
    check_same(pages, m)


@pytest.mark.gpu
def test_wishes_past_32_bits():
    """2100 sequences that want 2^20 pages each, of eight: none gets any, and the last one, which wants one, neither."""
    pages = moe.KVPages(caches(1, 8, 16, 1, 64), 2100, 2 ** 20)
    q_off = torch.zeros(2101, dtype=torch.int32, device="cuda")
    kv = torch.full((2100,), 2 ** 24, dtype=torch.int32, device="cuda")
    kv[-1] = 5
    pages.update(pages.batch(q_off, kv, 0, 0, 2 ** 24))
    with pytest.raises(moe.MoEError):
        pages.check()
    assert pages.held.sum() == 0 and pages.refs.sum() == 0 and (pages.table == -1).all()
    kv[:-1] = 3
    kv[7:-1] = 0
    pages.update(pages.batch(q_off, kv, 0, 0, 2 ** 24))
    pages.check()
    assert pages.table[:7, 0].tolist() == list(range(7)) and pages.table[-1, 0] == 7


@pytest.mark.gpu
def test_a_step_past_its_bounds_writes_into_no_other_sequence():
    """Sequences that update() does not touch may still be appended to: what they share leaves them from there on."""
    cs = caches(1, 40, 16, 1, 64)
    pages, m = moe.KVPages(cs, 5, 8), Model(40, 16, 5, 8)
    kv, new = [100, 0, 0, 0, 0], [100, 0, 0, 0, 0]
    pages.update(step(pages, kv, new)), m.update(kv, new, 100, 128)
    pages.fork(i32(0, 0, 0, 0), i32(1, 2, 3, 4)), m.fork([0] * 4, [1, 2, 3, 4])
    check_same(pages, m)
    # 1: more tokens than max_new; 2: past max_kv; 3: past the table; 4: as it should be
    kv, new = [100, 103, 113, 130, 101], [0, 3, 20, 1, 1]
    b = step(pages, kv, new, max_new=2, max_kv=110)
    pages.update(b), m.update(kv, new, 2, 110)
    assert m.bad and m.table[0].tolist() == list(range(7)) + [-1] and m.table[1, 5:].tolist() == [5, -1, -1]
    assert m.table[2, 4:].tolist() == [4, -1, -1, -1] and m.table[3, 6] == 6 and m.table[4, 6] == 7
    check_same(pages, m)
    before = [t[:7].clone() for t in (cs[0].k_codes, cs[0].k_scales, cs[0].v_codes)]
    x = torch.randn(b.n_tokens, 1, 64, device="cuda").bfloat16()
    cs[0].append(x, x, b)
    for t, was in zip((cs[0].k_codes, cs[0].k_scales, cs[0].v_codes), before):
        assert torch.equal(t[:7].view(torch.int16), was.view(torch.int16))
    with pytest.raises(moe.MoEError):
        cs[0].check()


@pytest.mark.gpu
def test_bad_forks_and_copies_are_left_out():
    pages, m = moe.KVPages(caches(1, 30, 16, 1, 64), 8, 4), Model(30, 16, 8, 4)
    kv = [20, 33, 0, 0, 0, 0, 0, 0]
    pages.update(step(pages, kv, kv)), m.update(kv, kv, 33, 64)
    # twice the same destination, one that holds pages, chains, itself, out of range
    src, dst = [0, 1, 0, 2, 0, -1, 8, 1, 5, 1, 2 ** 31 - 1][:8], [2, 2, 1, 3, 4, 5, 6, 7]
    pages.fork(i32(*src), i32(*dst)), m.fork(src, dst)
    check_same(pages, m)
    pages.fork(i32(0, 1), i32(8, -1)), m.fork([0, 1], [8, -1])
    check_same(pages, m)
    pages.fork(i32(6), i32(6)), m.fork([6], [6])
    check_same(pages, m)
    pages.copy(i32(3, 7, 30, -1, 4), i32(20, 7, 21, 22, 2 ** 31 - 1))
    m.words[20] = m.words[3]
    check_words(pages.caches, m.words)
    with pytest.raises(moe.MoEError):
        pages.caches[0].check()
    for bad in (lambda: pages.copy(i32(1, 2), i32(3)), lambda: pages.fork(i32(1)[None], i32(3)),
                lambda: pages.fork(i32(1).long(), i32(3)), lambda: moe.KVPages([], 2, 2), lambda: moe.KVPages(pages.caches, 0, 2),
                lambda: moe.KVPages(pages.caches, 2, 0),
                lambda: moe.KVPages([pages.caches[0], moe.KVCache.empty(30, 16, 2, 64)], 2, 2)):
        with pytest.raises(ValueError):
            bad()
    other = moe.KVPages(pages.caches, 8, 4)
    with pytest.raises(moe.MoEError):  # another set's batch
        pages.update(step(other, kv, kv))


@pytest.mark.gpu
def test_many_layers_and_a_captured_step():
    """More caches than one launch takes, and a step replayed with the lengths advanced on the device."""
    cs = caches(67, 12, 16, 1, 64)
    pages, m = moe.KVPages(cs, 3, 6), Model(12, 16, 3, 6)
    kv = [30, 0, 0]
    pages.update(step(pages, kv, kv)), m.update(kv, kv, 30, 96)
    pages.fork(i32(0), i32(2)), m.fork([0], [2])
    check_same(pages, m)
    lens = i32(30, 0, 30)
    batch = pages.batch(i32(0, 1, 1, 2), lens, 2, 1, 96)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lens += torch.ones_like(lens)
        lens[1].zero_()
        pages.update(batch)
    kv = np.array([30, 0, 30])
    for _ in range(20):
        g.replay()
        kv += [1, 0, 1]
        m.update(kv.tolist(), [1, 0, 1], 1, 96)
    check_same(pages, m)
    pages.compact(), m.compact()
    check_same(pages, m)


@pytest.mark.gpu
def test_a_batch_of_the_set_serves_the_caches():
    """Appended through the set's table, forked, written on and compacted, every sequence reads back what it was given."""
    g = torch.Generator(device="cuda").manual_seed(0)
    cs = [moe.KVCache.empty(64, 16, 2, 128) for _ in range(2)]
    pages = moe.KVPages(cs, 4, 12)
    x = [torch.randn(100, 2, 128, generator=g, device="cuda").bfloat16() for _ in range(4)]

    def run(kv, new, rows):
        b = step(pages, kv, new)
        pages.update(b)
        for c in cs:
            c.append(rows, rows, b)
        return b

    def read(kv):
        return cs[1].read(step(pages, kv, kv))[0].split(kv)

    run([50, 0, 70, 0], [50, 0, 70, 0], torch.cat([x[0][:50], x[2][:70]]))
    first = read([50, 0, 70, 0])
    pages.fork(i32(0, 2), i32(1, 3))
    run([51, 53, 70, 90], [1, 3, 0, 20], torch.cat([x[0][50:51], x[1][50:53], x[3][70:90]]))
    pages.compact()
    got = read([51, 53, 70, 90])
    assert torch.equal(got[0][:50], first[0]) and torch.equal(got[1][:50], first[0])
    assert torch.equal(got[2], first[2]) and torch.equal(got[3][:70], first[2])
    for b, (lo, hi) in {0: (50, 51), 1: (50, 53), 3: (70, 90)}.items():
        one = moe.KVCache.empty(8, 16, 2, 128)
        t = moe.KVBatch(i32(0, hi - lo), i32(hi - lo), i32(*range(8))[None], hi - lo, hi - lo, 100)
        one.append(x[b][lo:hi], x[b][lo:hi], t)
        assert torch.equal(got[b][lo:], one.read(t)[0])
    pages.check()
    for c in cs:
        c.check()
