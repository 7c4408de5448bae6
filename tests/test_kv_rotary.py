"""The rotated append: head norms, rotation and quantisation in one pass, against the definition in 64 bits."""
import ctypes
import math

import numpy as np
import pytest

import bit_moe_expert_routing_gb300 as moe
from bit_moe_expert_routing_gb300 import build

torch = pytest.importorskip("torch")

from kv_util import Batch, bf16_bits, junk_cache  # noqa: E402

P = 1 << 20  # a well-aligned address that nothing reads


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    moe.lib()


# --- refusals, on the CPU ---------------------------------------------------------------------------

def c_args(cache=None, batch=None, **rotary):
    c = moe.moe_kv_cache(10, 16, 2, 128, P, P, P, P, P, P, P)
    b = moe.moe_kv_batch(2, 2, 1, 100, P, P, P, 8)
    r = moe.moe_rotary(64, 0, 1, 1e-6, P, P, P, P)
    for s, kw in ((c, cache or {}), (b, batch or {}), (r, rotary)):
        for name, v in kw.items():
            setattr(s, name, v)
    return c, b, r


def call(c, b, r, positions=None, heads=8, q=P, qs=1024, out=2 * P, k=P, ks=256, v=P, vs=256):
    return moe.moe_kv_append_rotary(c, b, r, positions, heads, q, qs, out, k, ks, v, vs, None)


@pytest.mark.parametrize("rotary,want", [
    (dict(rotary_dim=-16), moe.MOE_ERR_SHAPE), (dict(rotary_dim=144), moe.MOE_ERR_SHAPE), (dict(rotary_dim=24), moe.MOE_ERR_SHAPE),
    (dict(axes=0), moe.MOE_ERR_SHAPE), (dict(axes=5), moe.MOE_ERR_SHAPE), (dict(turns=None), moe.MOE_ERR_ARG),
    (dict(turns=P + 4), moe.MOE_ERR_ARG), (dict(q_weight=P + 8), moe.MOE_ERR_ARG),
    (dict(k_weight=P + 8), moe.MOE_ERR_ARG), (dict(eps=0.0), moe.MOE_ERR_ARG), (dict(eps=-1e-6), moe.MOE_ERR_ARG),
    (dict(eps=math.inf), moe.MOE_ERR_ARG), (dict(eps=math.nan), moe.MOE_ERR_ARG)])
def test_bad_rotations_are_refused(rotary, want):
    assert call(*c_args(**rotary)) == want
    assert call(*c_args(batch=dict(n_tokens=0), **rotary)) == want
    assert moe.moe_last_launch_count() == 0


def test_bad_caches_and_operands_are_refused():
    assert call(*c_args(cache=dict(head_dim=96))) == moe.MOE_ERR_SHAPE
    assert call(*c_args(batch=dict(max_kv=-1))) == moe.MOE_ERR_ARG
    assert moe.lib().moe_kv_append_rotary(*(ctypes.byref(x) for x in c_args()[:2]), None, None, 8, P, 1024, 2 * P, P, 256, P, 256,
                                          None) == moe.MOE_ERR_ARG
    for kw in (dict(heads=0), dict(heads=16385)):
        assert call(*c_args(), **kw) == moe.MOE_ERR_SHAPE
    for kw in (dict(positions=P + 2), dict(q=None), dict(q=P + 2), dict(qs=1016), dict(qs=1028), dict(out=None), dict(out=2 * P + 8), dict(out=P),
               dict(k=None), dict(ks=248), dict(v=P + 8), dict(vs=-256), dict(k=2 * P), dict(v=2 * P)):
        assert call(*c_args(), **kw) == moe.MOE_ERR_ARG, kw
    assert call(*c_args(batch=dict(n_tokens=0)), q=None, k=None, v=None, out=None) == moe.MOE_OK
    assert moe.moe_last_launch_count() == 0


def test_the_handle_checks_what_it_is_given():
    r = moe.Rotary([1.0] * 8, device="cpu")
    assert r.rotary_dim == 16 and r.axes == 1
    for kw in (dict(inv_freq=[1.0] * 7), dict(inv_freq=[math.nan] * 8), dict(inv_freq=[1.0] * 8, axis=[0] * 7),
               dict(inv_freq=[1.0] * 8, axis=[4] * 8), dict(inv_freq=[1.0] * 8, q_weight=torch.ones(64, dtype=torch.bfloat16)),
               dict(inv_freq=[1.0] * 8, k_weight=torch.ones(128)[::2])):
        with pytest.raises(ValueError):
            moe.Rotary(**kw, device="cpu")


def test_turns_are_the_frequencies_in_64_bits():
    freq = [math.pi, -math.pi, 2 * math.pi, 0.0, 1.0, 1e-6, 1e6, -1.0]
    r = moe.Rotary(freq, device="cpu")
    for f, t in zip(freq, r._turns.tolist()):
        # a double holds f / 2 pi to 2^-53 relative, twice rounded
        want = f / (2 * math.pi)
        off = (t / 2 ** 64 - want) % 1.0
        assert min(off, 1.0 - off) <= 2.0 ** -51 * max(1.0, abs(want)), f


# --- results ----------------------------------------------------------------------------------------

def reference(x, weight, eps, freq, interleaved, pos):
    """x doubles [n, heads, D], pos [half, n] -> normed and turned, with the size of what each element is a sum of."""
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    half = len(freq)
    y, size = x.clone(), x.abs()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        ang = pos[i].double() * freq[i]
        c, s = torch.cos(ang)[:, None], torch.sin(ang)[:, None]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        size[..., a] = size[..., b] = x[..., a].abs() + x[..., b].abs()
    return y, size


def check_turned(got, want, size):
    """One rounding to bf16, 2^-8 of the value at most, and what comes before in fp32: an angle off by 2^-25 turns (2^-22
    radians), cosines by 2^-22, the norm and the products by 2^-21 of their sizes; 2^-18 of the size covers them."""
    d = (got.double() - want).abs()
    bound = 2.0 ** -8 * want.abs() + 2.0 ** -18 * size + 1e-37
    assert torch.isfinite(got).all()
    assert (d <= bound).all(), (d / bound).max().item()


CASES = [
    # dim, rotary_dim, heads, kv_heads, new, kv, page, interleaved, axes, norm
    (128, 128, 8, 2, [1], [1], 16, False, 1, True),
    (256, 64, 16, 2, [1] * 8, [300, 1, 77, 2000, 5, 64, 65, 900], 64, False, 1, True),
    (64, 64, 8, 4, [37, 0, 130, 5], [37, 9, 200, 5], 32, True, 3, False),
    (64, 16, 3, 1, [17, 3], [20, 3], 16, False, 1, True),
    (128, 96, 5, 5, [33], [50], 128, True, 2, True),
    (256, 256, 4, 1, [70, 1], [70, 513], 16, False, 4, True),
    (128, 0, 6, 3, [19], [19], 16, False, 1, True),
    (64, 32, 64, 1, [301], [400], 256, False, 1, False),
    (128, 112, 2, 2, [9, 8, 7], [9, 800, 70], 16, False, 3, True),
    (256, 192, 2, 2, [600], [600], 64, True, 1, True),
    (128, 128, 32, 8, [2001, 0, 2999], [2001, 7, 3500], 16, False, 1, True),
    (256, 256, 40, 8, [1, 2], [400, 2], 32, False, 1, True),
    (64, 48, 40, 8, [1], [65], 16, True, 2, True),
    (64, 64, 7, 7, [900], [1000], 64, False, 1, True),
    (256, 16, 1, 1, [3] * 40, [3 + 5 * i for i in range(40)], 16, False, 1, False),
]


def run_case(dim, rot, heads, kvh, new, kv, page, interleaved, axes, norm, seed=0, base=1e4, positions=None, scale=1.0,
             stream=None, max_kv=None):
    r = np.random.RandomState(seed)
    batch = Batch(new, kv, page, seed)
    n = batch.n_tokens
    cache = junk_cache(moe, batch.n_pages, page, kvh, dim)
    # one projection's output, with other columns around the heads
    wide = (torch.from_numpy(r.randn(n, heads + 2 * kvh + 1, dim)).cuda() * scale).to(torch.bfloat16)
    q, k, v = wide[:, :heads], wide[:, heads:heads + kvh], wide[:, heads + kvh:heads + 2 * kvh]
    freq = [base ** (-2 * i / max(rot, 1)) for i in range(rot // 2)]
    axis = [int(a) for a in r.randint(0, axes, rot // 2)]
    if rot:
        axis[-1] = axes - 1
    qw, kw = ((1 + 0.3 * torch.from_numpy(r.randn(dim)).float().cuda()) if norm else None for _ in range(2))
    rotary = moe.Rotary(freq, axis, interleaved, qw, kw, 1e-6)
    dev = batch.device(moe, max_kv=max_kv)
    if positions is None and axes > 1:
        positions = torch.from_numpy(r.randint(-50, 100000, (axes, n)).astype(np.int32)).cuda()
    own = torch.cat([torch.arange(l - m, l) for m, l in zip(new, kv)] + [torch.zeros(0, dtype=torch.int64)]).cuda()
    at = [own if positions is None else positions[a] if positions.dim() == 2 else positions for a in axis]
    got = cache.append_rotary(q, k, v, dev, rotary, positions=positions, stream=stream)
    if stream is not None:
        stream.synchronize()
    qr = reference(q.double(), qw, 1e-6, freq, interleaved, at)
    kr = reference(k.double(), kw, 1e-6, freq, interleaved, at)
    return cache, batch, dev, wide, rotary, got, qr, kr


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}x{c[3]}-{sum(c[4])}")
def test_queries_and_cached_keys_and_values(case):
    dim, rot, heads, kvh = case[:4]
    cache, batch, dev, wide, rotary, got, (qr, qsize), (kr, ksize) = run_case(*case)
    cache.check()
    check_turned(got, qr, qsize)
    # the keys as queries would be turned are what append() quantises, bit for bit
    other = junk_cache(moe, batch.n_pages, case[6], kvh, dim)
    pos = None
    if rotary.axes > 1:
        r = np.random.RandomState(0)  # the same draws as run_case's
        r.randn(batch.n_tokens, heads + 2 * kvh + 1, dim), r.randint(0, case[8], rot // 2), r.randn(dim), r.randn(dim)
        if case[9] is False:
            r = np.random.RandomState(0)
            r.randn(batch.n_tokens, heads + 2 * kvh + 1, dim), r.randint(0, case[8], rot // 2)
        pos = torch.from_numpy(r.randint(-50, 100000, (case[8], batch.n_tokens)).astype(np.int32)).cuda()
    k, v = wide[:, heads:heads + kvh], wide[:, heads + kvh:heads + 2 * kvh]
    as_q = moe.Rotary.__new__(moe.Rotary)
    as_q.__dict__.update(rotary.__dict__, q_weight=rotary.k_weight)
    as_q.c = moe.moe_rotary.from_buffer_copy(rotary.c)
    as_q.c.q_weight = rotary.c.k_weight
    as_q._ref = ctypes.byref(as_q.c)
    turned = junk_cache(moe, batch.n_pages, case[6], kvh, dim).append_rotary(k, k, v, dev, as_q, positions=pos)
    check_turned(turned, kr, ksize)
    other.append(turned, v, dev)
    other.check()
    for name in ("k_codes", "k_scales", "k_biases", "v_codes", "v_scales", "v_biases"):
        a, b = getattr(cache, name), getattr(other, name)
        # (as bits: what was not written is NaN in both)
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)), name


@pytest.mark.gpu
def test_far_positions_keep_their_angles():
    """At 2^24 positions a frequency of one turns by 16 million radians: fp32 would be off by whole radians."""
    far = torch.tensor([2 ** 24 - 1, 12345677, 1000003, -(2 ** 31), 2 ** 31 - 1, 0], dtype=torch.int32, device="cuda")
    for interleaved in (False, True):
        cache, batch, dev, _, _, got, (qr, size), _ = run_case(128, 128, 4, 1, [6], [6], 16, interleaved, 1, True, positions=far)
        cache.check()
        # the reference's own angle, a double, is 2^31 2^-53 radians off
        check_turned(got, qr, size)
    # and in place: a sequence that long, whose earlier pages are not there
    cache = junk_cache(moe, 4, 256, 1, 64)
    table = torch.full((1, 2 ** 16), -1, dtype=torch.int32, device="cuda")
    table[0, -1] = 2
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    b = moe.KVBatch(i(0, 9), i(2 ** 24), table, 9, 9, 2 ** 24)
    x = torch.randn(9, 3, 64, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3)).bfloat16()
    freq = [1e6 ** (-i / 32) for i in range(32)]
    got = cache.append_rotary(x[:, :1], x[:, 1:2], x[:, 2:], b, moe.Rotary(freq))
    cache.check()
    pos = torch.arange(2 ** 24 - 9, 2 ** 24, device="cuda")
    check_turned(got, *reference(x[:, :1].double(), None, 0, freq, False, [pos] * 32))


@pytest.mark.gpu
def test_padding_missing_pages_and_bounds():
    """Tokens at negative positions are turned and not cached; pages that are missing and lengths past the bound are recorded."""
    case = (128, 64, 4, 2, [5, 20, 3], [2, 33, 3], 16, False, 1, True)
    cache, batch, dev, wide, rotary, got, (qr, size), _ = run_case(*case)
    cache.check()
    check_turned(got, qr, size)
    k, _ = cache.read(dev)
    assert (k[:3] == 0).all() and (k[3:].abs().amax((1, 2)) > 0).all()
    before = cache.k_codes.clone()
    dev._t[2][1, 1] = -1  # the second sequence's second page
    q, k, v = wide[:, :4], wide[:, 4:6] * 2, wide[:, 6:8] * 2
    again = cache.append_rotary(q, k, v, dev, rotary)
    assert torch.equal(again, got)
    with pytest.raises(moe.MoEError):
        cache.check()
    page = batch.table[1, 1]
    assert torch.equal(cache.k_codes[page], before[page])
    short = batch.device(moe, max_kv=20)
    again = cache.append_rotary(q, k, v, short, rotary)
    assert torch.equal(again, got)
    with pytest.raises(moe.MoEError):
        cache.check()


@pytest.mark.gpu
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_numbers_at_the_edges(dim):
    """Zeros, numbers whose squares pass fp32, NaN and infinities, head by head."""
    batch = Batch([6], [6], 16)
    x = torch.randn(6, 4, dim, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    x[0] = 0.0
    x[1] *= 2.0 ** 100
    x[2] *= 2.0 ** -100
    x[3, :, 5] = 3e38
    x = x.bfloat16()
    x[4, 1, 7], x[5, 1, 9] = math.nan, math.inf
    x[4, 2, 7], x[5, 2, 9] = math.nan, -math.inf
    w = torch.full((dim,), 1.5, device="cuda")
    freq = [0.5 ** i for i in range(dim // 2)]
    rot = moe.Rotary(freq, q_weight=w, k_weight=w, eps=1e-5)
    cache = junk_cache(moe, batch.n_pages, 16, 1, dim)
    dev = batch.device(moe)
    got = cache.append_rotary(x[:, :2], x[:, 2:3], x[:, 3:], dev, rot)
    with pytest.raises(moe.MoEError):  # NaN and infinite keys
        cache.check()
    pos = [torch.arange(6, device="cuda")] * (dim // 2)
    ref, size = reference(x[:, :2].double(), w, 1e-5, freq, False, pos)
    check_turned(got[:4], ref[:4], size[:4])
    check_turned(got[4:, 0], ref[4:, 0], size[4:, 0])
    assert got[4, 1].isnan().all() and got[5, 1].isnan().any()
    k, v = cache.read(dev)
    kr, _ = reference(x[:4, 2:3].double(), w, 1e-5, freq, False, [p[:4] for p in pos])
    # a code's half step: a fifteenth of the group's range, and the roundings of scale, bias and value
    g = kr.unflatten(-1, (-1, 64))
    step = ((g.amax(-1) - g.amin(-1)) / 15)[..., None].expand_as(g).flatten(-2)
    assert ((k[:4].double() - kr).abs() <= 0.51 * step + 2.0 ** -6 * g.abs().amax(-1)[..., None].expand_as(g).flatten(-2) + 1e-37).all()
    assert (k[4] == 0).all() and torch.isfinite(k).all() and torch.isfinite(v[:3]).all()


@pytest.mark.gpu
def test_other_streams_graphs_and_outputs():
    case = (128, 128, 8, 2, [3, 40], [100, 40], 16, False, 1, True)
    cache, batch, dev, wide, rotary, got, _, _ = run_case(*case)
    want = [t.clone() for t in (cache.k_codes, cache.v_codes)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    _, _, _, _, _, other, _, _ = run_case(*case, stream=s)
    assert torch.equal(other, got)
    q, k, v = wide[:, :8], wide[:, 8:10], wide[:, 10:12]
    out = torch.empty_like(got)
    cache.append_rotary(q, k, v, dev, rotary, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out.zero_()
        cache.append_rotary(q, k, v, dev, rotary, out=out)
    cache.k_codes.zero_(), cache.v_codes.zero_()
    junk = junk_cache(moe, batch.n_pages, 16, 2, 128)
    cache.k_codes.copy_(junk.k_codes), cache.v_codes.copy_(junk.v_codes)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, got)
    assert torch.equal(cache.k_codes, want[0]) and torch.equal(cache.v_codes, want[1])
    for bad in (dict(out=out[:, :4]), dict(out=out.float()), dict(positions=torch.zeros(42, dtype=torch.int32, device="cuda")),
                dict(positions=torch.zeros(43, dtype=torch.int64, device="cuda")),
                dict(positions=torch.zeros(2, 43, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            cache.append_rotary(q, k, v, dev, rotary, **bad)
    with pytest.raises(ValueError):
        cache.append_rotary(q, k, v, dev, moe.Rotary([1.0] * 8, q_weight=torch.ones(64, device="cuda")))
