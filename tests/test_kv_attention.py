"""The 4-bit key/value cache and its attention on the GPU, against the plain 64-bit implementation of kv_util."""
import ctypes
import math

import numpy as np
import pytest

import bit_moe_expert_routing_gb300 as moe
from bit_moe_expert_routing_gb300 import build

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from kv_util import (Batch, attention_reference, bf16_bits, check_attention, fill, junk_cache, quantise,  # noqa: E402
                     unpack, values)


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    moe.lib()


def rows(n, heads, dim, seed=5, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(n, heads, dim, generator=g, device="cuda") * spread).to(torch.bfloat16)


def cached(cache, batch, name):
    """Codes, scales and biases of the step's tokens as numpy arrays [n_tokens, kv heads, ...]."""
    got = []
    for a in ("codes", "scales", "biases"):
        t = getattr(cache, f"{name}_{a}")
        parts = []
        for b, n in enumerate(batch.new):
            pg, sl = batch.places(b)
            at = slice(batch.kv[b] - n, batch.kv[b])
            parts.append(t[torch.from_numpy(pg[at].astype(np.int64)).cuda(), :, torch.from_numpy(sl[at]).cuda()])
        x = torch.cat(parts).cpu()
        got.append(x.numpy() if a == "codes" else x.double().numpy())
    return unpack(got[0]), got[1], got[2]


# --- append and read ---------------------------------------------------------------------------

@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("page,kv_heads,new,old", [
    (16, 1, [1], [0]),                         # the first token of a sequence
    (16, 3, [1, 1, 1, 1], [15, 16, 17, 500]),  # one token before, at and after a page's end
    (64, 2, [5, 0, 131, 1], [60, 33, 1, 63]),  # odd lengths across pages, a sequence without step tokens
    (256, 8, [300], [77]),
    (32, 5, [2 ** i for i in range(9)], [31] * 9),
])
def test_append_writes_the_definition_bit_for_bit(dim, page, kv_heads, new, old):
    batch = Batch(new, [a + b for a, b in zip(new, old)], page, seed=dim)
    cache = junk_cache(moe, batch.n_pages, page, kv_heads, dim)
    before = {n: getattr(cache, n).clone() for n in ("k_codes", "v_codes")}
    k, v = rows(batch.n_tokens, kv_heads, dim, 1), rows(batch.n_tokens, kv_heads, dim, 2, spread=7.0)
    k[0, 0, :64] = 1.25  # a constant group: scale 0
    v[-1, -1, :64] = torch.arange(64, device="cuda") * 0.5 - 3  # halves of a step: ties of the code's rounding
    dev = batch.device(moe)
    cache.append(k, v, dev)
    cache.check()
    for name, x in (("k", k), ("v", v)):
        ref = quantise(x.double().cpu().numpy())
        got = cached(cache, batch, name)
        for a, b, what in zip(got, ref, ("codes", "scales", "biases")):
            assert np.array_equal(a, b), (name, what)
    # and nothing else: every other slot keeps its bits
    for name in before:
        now, was = getattr(cache, name), before[name]
        written = torch.zeros(now.shape[0], now.shape[2], dtype=torch.bool, device="cuda")
        for b, n in enumerate(batch.new):
            pg, sl = batch.places(b)
            written[torch.from_numpy(pg[len(pg) - n:].astype(np.int64)).cuda(), torch.from_numpy(sl[len(sl) - n:]).cuda()] = True
        keep = ~written[:, None, :, None].expand_as(now)
        assert torch.equal(now[keep], was[keep])
    # reading back gives the values bit for bit
    rk, rv = cache.read(dev)
    for got, x in ((rk, k), (rv, v)):
        assert np.array_equal(got.double().cpu().numpy(), values(*quantise(x.double().cpu().numpy())))
    cache.check()


def test_append_takes_slices_of_a_fused_projection():
    batch = Batch([7, 20], [40, 20], 16)
    qkv = rows(batch.n_tokens, 4 + 2 + 2, 128)  # [tokens, q heads + k heads + v heads, dim]
    a, b = (junk_cache(moe, batch.n_pages, 16, 2, 128) for _ in range(2))
    dev = batch.device(moe)
    a.append(qkv[:, 4:6], qkv[:, 6:8], dev)
    b.append(qkv[:, 4:6].contiguous(), qkv[:, 6:8].contiguous(), dev)
    for name in ("k_codes", "v_codes"):
        assert torch.equal(getattr(a, name), getattr(b, name))


def test_append_saturates_and_reports_what_it_cannot_hold():
    batch = Batch([4], [4], 16)
    cache = moe.KVCache.empty(batch.n_pages, 16, 1, 64)
    x = rows(4, 1, 64)
    x[1, 0, 3], x[1, 0, 4], x[2, 0, 0], x[3, 0, 9] = math.nan, 1.0, math.inf, -3e38
    dev = batch.device(moe)
    cache.append(x, rows(4, 1, 64), dev)
    with pytest.raises(moe.MoEError) as e:
        cache.check()
    assert e.value.status == moe.MOE_ERR_DEVICE_CHECK
    cache.check()  # reading the status clears it
    k, _ = cache.read(dev)
    assert np.array_equal(k.double().cpu().numpy(), values(*quantise(x.double().cpu().numpy())))
    assert torch.isfinite(k).all()
    # at the limits of the range nothing overflows and nothing is recorded
    x = torch.zeros(4, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[0, 0, 0], x[0, 0, 1] = 65536.0, -65536.0
    x[1] = rows(1, 1, 64)[0] * 1e-30
    x[2, 0, 5] = -1e-39
    cache.append(x, x, dev)
    cache.check()
    k, v = cache.read(dev)
    assert torch.isfinite(k).all() and torch.equal(k, v)
    assert np.array_equal(k[:2].double().cpu().numpy(), values(*quantise(x[:2].double().cpu().numpy())))


def test_padding_and_missing_pages():
    # three of five step tokens lie before position 0: not written, read as zero, and no error
    batch = Batch([5], [2], 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, 64)
    x = rows(5, 2, 64)
    dev = batch.device(moe)
    cache.append(x, x, dev)
    k, v = cache.read(dev)
    cache.check()
    assert (k[:3] == 0).all() and (v[:3] == 0).all()
    assert np.array_equal(k[3:].double().cpu().numpy(), values(*quantise(x[3:].double().cpu().numpy())))
    # a page that the table does not name: recorded, and the others are as they should be
    batch = Batch([40], [40], 16)
    batch.table[0, 1] = batch.n_pages
    cache = junk_cache(moe, batch.n_pages, 16, 2, 64)
    x = rows(40, 2, 64)
    dev = batch.device(moe)
    cache.append(x, x, dev)
    k, _ = cache.read(dev)
    with pytest.raises(moe.MoEError):
        cache.check()
    want = values(*quantise(x.double().cpu().numpy()))
    want[16:32] = 0
    assert np.array_equal(k.double().cpu().numpy(), want)


# --- attention ---------------------------------------------------------------------------------

@pytest.fixture
def forced():
    """Sets which kernels take the attention (0: by the sequences' sizes, 1: few rows, 2: many rows)."""
    yield lambda path: moe.moe_set_option(moe.MOE_OPT_FORCE_PATH, path)
    moe.moe_set_option(moe.MOE_OPT_FORCE_PATH, 0)


def run_attention(heads, kv_heads, dim, page, new, kv, window=0, sinks=0, scale=None, spread=1.0, seed=0, q=None,
                  max_new=None, max_kv=None, outliers=False):
    batch = Batch(new, kv, page, seed=seed)
    cache = junk_cache(moe, batch.n_pages, page, kv_heads, dim)
    keys, vals = fill(cache, batch, seed=seed + 1, spread=spread, outliers=outliers)
    if q is None:
        q = rows(batch.n_tokens, heads, dim, seed + 2)
    dev = batch.device(moe, max_new, max_kv)
    s = dim ** -0.5 if scale is None else scale
    s = float(np.float32(s))
    ref = attention_reference(q, batch, keys, vals, s, window, sinks)
    was = moe.moe_get_option(moe.MOE_OPT_FORCE_PATH)
    try:
        for path in [was] if was else [1, 2, 0]:  # each size through both kernels, and as it is dispatched
            moe.moe_set_option(moe.MOE_OPT_FORCE_PATH, path)
            out, lse = cache.attention(q, dev, scale=scale, window=window, sinks=sinks, lse=True)
            cache.check()
            check_attention(out, lse, ref, path)
    finally:
        moe.moe_set_option(moe.MOE_OPT_FORCE_PATH, was)
    return batch, cache, dev, q, out, lse


DECODE = [
    # heads, kv_heads, page, new, kv
    (1, 1, 16, [1], [1]),
    (8, 1, 16, [1, 1, 1], [15, 16, 17]),
    (16, 2, 64, [1] * 5, [63, 64, 65, 127, 129]),
    (16, 2, 32, [1, 1], [1000, 3]),
    (6, 3, 128, [1, 1, 1], [257, 700, 31]),
    (10, 2, 256, [1], [600]),
    (12, 4, 16, [1] * 9, [1, 2, 3, 5, 9, 33, 48, 100, 511]),
    (64, 1, 16, [1, 1], [200, 77]),
    (24, 2, 16, [2, 1, 3], [90, 5, 3]),
    (16, 2, 16, [4, 4], [300, 4]),
    (4, 4, 64, [8, 1], [2100, 1500]),
    (8, 8, 16, [0, 1, 0, 2], [10, 40, 0, 2]),
]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads,page,new,kv", DECODE)
def test_attention_few_rows(dim, heads, kv_heads, page, new, kv):
    run_attention(heads, kv_heads, dim, page, new, kv, seed=dim + len(kv))


PREFILL = [
    (2, 1, 16, [129], [129]),
    (8, 2, 64, [300], [300]),
    (16, 2, 32, [64, 200, 17], [64, 345, 1000]),
    (5, 1, 16, [97, 131], [97, 140]),
    (4, 4, 256, [255, 257], [255, 600]),
    (64, 1, 16, [40], [100]),
    (12, 2, 128, [1, 250, 0, 2], [333, 250, 20, 90]),  # one token beside a prompt
    (7, 7, 64, [260], [400]),
]


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads,page,new,kv", PREFILL)
def test_attention_many_rows(dim, heads, kv_heads, page, new, kv):
    run_attention(heads, kv_heads, dim, page, new, kv, seed=dim + len(kv))


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,kv", [([1, 1, 1], [700, 100, 5]), ([3, 2], [400, 1111]), ([290], [290]), ([70, 140], [1000, 515])])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 0), (128, 130), (5000, 2), (257, 33)])
def test_attention_window_and_sinks(dim, new, kv, window, sinks):
    run_attention(8, 2, dim, 16, new, kv, window=window, sinks=sinks, seed=window)


@pytest.mark.parametrize("dim,heads,kv_heads,kv,window", [(64, 8, 8, 20011, 0), (128, 16, 2, 33333, 0), (256, 16, 2, 16385, 0),
                                                          (128, 8, 1, 30000, 9000)])
@pytest.mark.parametrize("new", [1, 3, 150])
def test_attention_long_context(dim, heads, kv_heads, kv, window, new):
    run_attention(heads, kv_heads, dim, 64, [new], [kv], window=window, sinks=4 if window else 0, seed=3)


@pytest.mark.parametrize("dim,max_kv", [(128, 1 << 20), (64, 1 << 22)])
def test_attention_in_passes(dim, max_kv):
    """A bound on the lengths whose expanded tiles are more than one pass holds: passes over sequences and kv heads."""
    run_attention(12, 3, dim, 16, [150, 0, 90, 1], [150, 30, 300, 260], max_kv=max_kv)


def test_offsets_past_32_bits(forced):
    """Pages whose codes lie more than 2^31 words into the arrays."""
    heads, kv_heads, dim, page = 16, 8, 256, 256
    batch = Batch([3, 40], [700, 90], page, spare=46000)
    batch.table = np.where(batch.table < 0, batch.table, batch.n_pages - 1 - batch.table % 7 - 7 * np.arange(batch.table.size)
                           .reshape(batch.table.shape)).astype(np.int32)
    used = [p for b in range(2) for p in set(batch.places(b)[0].tolist())]
    assert len(set(used)) == len(used) and min(used) * kv_heads * page * (dim // 8) > 2 ** 31
    cache = moe.KVCache.empty(batch.n_pages, page, kv_heads, dim)
    fill(cache, batch)
    k, v = rows(batch.n_tokens, kv_heads, dim, 1), rows(batch.n_tokens, kv_heads, dim, 2)
    dev = batch.device(moe)
    cache.append(k, v, dev)
    for got, x in zip(cache.read(dev), (k, v)):
        assert np.array_equal(got.double().cpu().numpy(), values(*quantise(x.double().cpu().numpy())))
    # all positions of both sequences, read back, are what the attention sees
    every = Batch([700, 90], [700, 90], page)
    every.table = batch.table
    keys, vals = (t.double().split(every.new) for t in cache.read(every.device(moe)))
    q = rows(batch.n_tokens, heads, dim, 3)
    ref = attention_reference(q, batch, keys, vals, float(np.float32(dim ** -0.5)))
    for path in (1, 2):
        forced(path)
        out, lse = cache.attention(q, dev, lse=True)
        cache.check()
        check_attention(out, lse, ref, path)


@pytest.mark.parametrize("new,kv", [([1, 2], [300, 70]), ([200], [260])])
@pytest.mark.parametrize("scale,spread", [(0.0, 1.0), (-0.3, 1.0), (1.0, 6.0), (1e-4, 1000.0)])
def test_attention_scales(new, kv, scale, spread):
    """No score, negative scales, and scores so large that one key takes nearly everything."""
    run_attention(8, 2, 128, 32, new, kv, scale=scale, spread=spread, outliers=True)


@pytest.mark.parametrize("new,kv", [([3], [2]), ([2, 5, 1], [0, 3, 7]), ([200], [150]), ([130, 20], [0, 600])])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_rows_that_see_nothing_give_zero(dim, new, kv):
    batch, _, _, _, out, lse = run_attention(8, 2, dim, 16, new, kv)
    assert (lse == -math.inf).any()


@pytest.mark.parametrize("path", [0, 1, 2])
@pytest.mark.parametrize("new,kv", [([1, 1], [100, 37]), ([3, 2], [100, 37]), ([150, 90], [150, 300])])
def test_masked_places_and_other_rows_do_not_leak(new, kv, path, forced):
    """Slots past a sequence's end hold NaN and infinities (junk_cache), a query row of NaN or infinities spoils its
    own output alone, and bounds above the lengths change nothing."""
    forced(path)
    heads, dim = 8, 128
    batch, cache, dev, q, out, lse = run_attention(heads, 2, dim, 16, new, kv)
    bad = q.clone()
    bad[0, 3] = math.nan
    bad[-1, 5] = math.inf
    o2, l2 = cache.attention(bad, dev, lse=True)
    assert torch.isnan(o2[0, 3]).all() and torch.isnan(o2[-1, 5]).all() and torch.isnan(l2[0, 3])
    keep = torch.ones(batch.n_tokens, heads, dtype=torch.bool, device="cuda")
    keep[0, 3] = keep[-1, 5] = False
    assert torch.equal(o2[keep], out[keep]) and torch.equal(l2[keep], lse[keep])
    run_attention(heads, 2, dim, 16, new, kv, max_new=max(new) + 1, max_kv=5000)


@pytest.mark.parametrize("path", [0, 1, 2])
@pytest.mark.parametrize("new,kv", [([1, 1], [3000, 37]), ([4], [900]), ([150], [700])])
def test_attention_is_repeatable_and_takes_strided_queries(new, kv, path, forced):
    forced(path)
    batch, cache, dev, q, out, lse = run_attention(8, 2, 128, 32, new, kv)
    for _ in range(3):
        o, l = cache.attention(q, dev, lse=True)
        assert torch.equal(o, out) and torch.equal(l, lse)
    wide = torch.full((batch.n_tokens, 12, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:10] = q
    assert torch.equal(cache.attention(wide[:, 2:10], dev), out)
    # without lse, into a given output, with a workspace full of junk
    o = torch.full((q.numel() + 8,), math.nan, dtype=torch.bfloat16, device="cuda")[8:].view_as(q)  # 16-byte aligned, no more
    ws = cache.attention_workspace(8, dev)
    ws.fill_(0xFF)
    assert cache.attention(q, dev, out=o, workspace=ws) is o and torch.equal(o, out)


def test_attention_on_another_stream_and_in_a_graph():
    batch, cache, dev, q, out, _ = run_attention(8, 2, 128, 32, [1, 1, 1], [500, 37, 1290])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = cache.attention(q, dev, stream=s)
    s.synchronize()
    assert torch.equal(o, out)
    static, ws = torch.zeros_like(q), cache.attention_workspace(8, dev)
    with torch.cuda.stream(s):
        cache.attention(q, dev, out=static, workspace=ws)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attention(q, dev, out=static, workspace=ws)
    static.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(static, out)


@pytest.mark.parametrize("path", [0, 1, 2])
@pytest.mark.parametrize("new,kv", [([1, 1], [100, 300]), ([2], [300]), ([140], [300])])
def test_a_missing_page_is_recorded_and_left_out(new, kv, path, forced):
    forced(path)
    batch = Batch(new, kv, 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, 64)
    keys, vals = fill(cache, batch)
    q = rows(batch.n_tokens, 8, 64)
    gone = batch.table.copy()
    gone[-1, 3] = -1
    whole, batch.table = batch.table, gone
    out, lse = cache.attention(q, batch.device(moe), lse=True)
    with pytest.raises(moe.MoEError) as e:
        cache.check()
    assert e.value.status == moe.MOE_ERR_DEVICE_CHECK
    # the same sequence with those sixteen positions cut out, in the rows after them
    batch.table = whole
    left = [i for i in range(kv[-1]) if not 48 <= i < 64]
    n = new[-1]
    small = Batch([n], [kv[-1] - 16], 16)
    ref = attention_reference(q[batch.n_tokens - n:], small, [keys[-1][left]], [vals[-1][left]], float(np.float32(64 ** -0.5)))
    check_attention(out[batch.n_tokens - n:], lse[batch.n_tokens - n:], ref)


def test_a_step_through_append_and_attention():
    """Prompt, then one token at a time, against attention over all the values the cache should hold."""
    heads, kv_heads, dim, page = 8, 2, 128, 16
    prompt, steps = [37, 150], 4
    final = [p + steps for p in prompt]
    pages = Batch([1, 1], final, page)
    cache = junk_cache(moe, pages.n_pages, page, kv_heads, dim)
    held = [[], []]
    for t in range(steps + 1):
        new = prompt if t == 0 else [1, 1]
        batch = Batch(new, [p + t for p in prompt], page)
        batch.table = pages.table
        k, v, q = (rows(batch.n_tokens, h, dim, 100 * t + i) for i, h in enumerate((kv_heads, kv_heads, heads)))
        dev = batch.device(moe)
        cache.append(k, v, dev)
        out, lse = cache.attention(q, dev, lse=True)
        for which, x in enumerate((k, v)):
            x = torch.from_numpy(values(*quantise(x.double().cpu().numpy()))).cuda()
            parts = [x[batch.q_off[b]:batch.q_off[b + 1]] for b in range(2)]
            held[which] = parts if t == 0 else [torch.cat([a, b]) for a, b in zip(held[which], parts)]
        check_attention(out, lse, attention_reference(q, batch, held[0], held[1], float(np.float32(dim ** -0.5))), t)
    cache.check()


def test_launches_are_counted_and_timed():
    batch, cache, dev, q, _, _ = run_attention(8, 2, 128, 32, [1], [50])
    assert moe.moe_last_launch_count() >= 1
    moe.moe_set_option(moe.MOE_OPT_KERNEL_TIMING, 1)
    try:
        moe.moe_kernel_times()
        cache.append(rows(1, 2, 128), rows(1, 2, 128), dev)
        cache.read(dev)
        cache.attention(q, dev)
        t = moe.moe_kernel_times()
    finally:
        moe.moe_set_option(moe.MOE_OPT_KERNEL_TIMING, 0)
    assert "kv_append" in t and "kv_read" in t and any(n.startswith("attention") for n in t)
