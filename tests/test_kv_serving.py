"""The cache's attention as a serving loop calls it: bounds above the lengths, a consumer straight behind it on the stream,
many sequences, and workspaces and settings kept between steps."""
import math

import numpy as np
import pytest

import bit_moe_expert_routing_gb300 as moe
from bit_moe_expert_routing_gb300 import build

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from kv_util import (Batch, attention_reference, bf16_bits, bf16_round, check_attention, fill, junk_cache, pack,  # noqa: E402
                     quantise, values)


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    moe.lib()


def rows(n, heads, dim, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(n, heads, dim, generator=g, device="cuda").to(torch.bfloat16)


# Under a bound of 5000 positions items may be cut, but these are short: their units (10 and the tiles of 32 positions)
# are dealt out in eights at least, and the tiles of each fall to one CTA. In the last one no sequence is the few-row
# kernel's at all, beside a prompt that is long enough for the many-row kernels.
@pytest.mark.parametrize("new,kv", [([1], [100]), ([1], [190]), ([1] * 16, [50] * 16), ([1, 1500], [100, 1500]),
                                    ([1400, 1300], [1400, 1300])])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_a_kernel_behind_the_call_sees_its_output(dim, new, kv):
    batch = Batch(new, kv, 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, dim)
    keys, vals = fill(cache, batch)
    q = rows(batch.n_tokens, 16, dim)
    dev = batch.device(moe, max_new=max(new) + 1, max_kv=5000)
    ref = attention_reference(q, batch, keys, vals, float(np.float32(dim ** -0.5)))
    out, ws = torch.empty_like(q), cache.attention_workspace(16, dev)
    cache.attention(q, dev, out=out, workspace=ws)
    torch.cuda.synchronize()
    g, got = torch.cuda.CUDAGraph(), torch.empty_like(out)
    with torch.cuda.graph(g):
        out.fill_(math.nan)
        cache.attention(q, dev, out=out, workspace=ws)
        got.copy_(out)
    for _ in range(20):
        g.replay()
    torch.cuda.synchronize()
    check_attention(got, None, ref)
    for _ in range(20):  # and in a stream
        out.fill_(math.nan)
        cache.attention(q, dev, out=out, workspace=ws)
        got.copy_(out)
    check_attention(got, None, ref)
    cache.check()


@pytest.fixture
def each_path():
    """The kernels by turns: by the sequences' sizes, few rows, many rows."""
    def paths():
        for path in (0, 1, 2):
            moe.moe_set_option(moe.MOE_OPT_FORCE_PATH, path)
            yield path
    yield paths
    moe.moe_set_option(moe.MOE_OPT_FORCE_PATH, 0)


@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 2 ** 20, 4), (300, 0),
                                          (299, 2 ** 31 - 1), (17, 2 ** 31 - 1)])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_windows_past_every_position(dim, window, sinks, each_path):
    """No limit, as a number, with tokens at negative positions (padding) beside others."""
    batch = Batch([5, 290, 3, 40, 1], [2, 200, 0, 300, 260], 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, dim)
    keys, vals = fill(cache, batch)
    q = rows(batch.n_tokens, 8, dim)
    ref = attention_reference(q, batch, keys, vals, float(np.float32(dim ** -0.5)), window, sinks)
    for max_kv in (300, 5000):
        dev = batch.device(moe, max_kv=max_kv)
        for path in each_path():
            out, lse = cache.attention(q, dev, window=window, sinks=sinks, lse=True)
            cache.check()
            check_attention(out, lse, ref, (path, max_kv))


@pytest.mark.parametrize("dim,max_kv", [(128, 1500), (256, 600), (64, 1500)])
def test_the_largest_steps_workspace_serves_every_step(dim, max_kv):
    """A loop with one workspace as its sequences end: whole items with many sequences, cut ones with few."""
    ws = None
    for n in (64, 32, 3, 1):
        kv = [max_kv - 7 * i for i in range(n)]
        batch = Batch([1] * n, kv, 16)
        cache = junk_cache(moe, batch.n_pages, 16, 2, dim)
        keys, vals = fill(cache, batch)
        q = rows(n, 16, dim)
        dev = batch.device(moe, max_kv=max_kv)
        if ws is None:
            ws = cache.attention_workspace(16, dev)
        ws.fill_(0xFF)
        out, lse = cache.attention(q, dev, lse=True, workspace=ws)
        cache.check()
        check_attention(out, lse, attention_reference(q, batch, keys, vals, float(np.float32(dim ** -0.5))), n)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,kv,window,sinks", [([1], [700], 100, 0), ([2, 1], [901, 333], 50, 3), ([150], [700], 101, 5),
                                                 ([150, 40], [1000, 517], 17, 0), ([260], [420], 130, 20), ([1], [40], 7, 33)])
def test_places_that_no_row_sees_may_hold_anything(dim, new, kv, window, sinks, each_path):
    """Between the sinks and the first row's window nothing was ever written: NaN scales, infinite biases."""
    batch = Batch(new, kv, 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, dim)
    keys, vals = fill(cache, batch)
    for b, (n, end) in enumerate(zip(new, kv)):
        pg, sl = batch.places(b)
        unseen = slice(sinks, max(sinks, end - n - window + 1))
        pg, sl = torch.from_numpy(pg[unseen].astype(np.int64)).cuda(), torch.from_numpy(sl[unseen]).cuda()
        for name in ("k", "v"):
            getattr(cache, name + "_scales")[pg, :, sl] = math.nan
            getattr(cache, name + "_biases")[pg, :, sl] = math.inf
    q = rows(batch.n_tokens, 8, dim)
    ref = attention_reference(q, batch, keys, vals, float(np.float32(dim ** -0.5)), window, sinks)
    dev = batch.device(moe)
    for path in each_path():
        out, lse = cache.attention(q, dev, window=window, sinks=sinks, lse=True)
        cache.check()
        check_attention(out, lse, ref, path)


def test_handles_refuse_what_the_kernels_cannot_reach():
    """Tensors elsewhere than the cache, a workspace without memory behind all of it, numbers that a C int would cut."""
    batch = Batch([1, 2], [40, 30], 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, 64)
    fill(cache, batch)
    q, k = rows(3, 8, 64), rows(3, 2, 64)
    dev = batch.device(moe)
    n = cache.attention_workspace(8, dev).numel()
    out = cache.attention(q, dev)
    for ws in (torch.empty(n, dtype=torch.uint8), torch.empty(256, dtype=torch.uint8, device="cuda").expand(n // 256 + 1, 256),
               torch.empty(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            cache.attention(q, dev, workspace=ws)
    with pytest.raises(moe.MoEError) as e:
        cache.attention(q, dev, workspace=torch.empty(n - 256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == moe.MOE_ERR_WORKSPACE
    assert torch.equal(cache.attention(q, dev, workspace=torch.empty(n // 4 + 1, device="cuda")), out)  # bytes count, of any type
    away = batch.device(moe)
    away.device = torch.device("cuda", 1)  # as a batch made on another GPU
    for call in (lambda: cache.append(k, k, away), lambda: cache.read(away), lambda: cache.attention(q, away)):
        with pytest.raises(ValueError):
            call()
    big = 2 ** 32 + 1
    for kw in (dict(window=big), dict(sinks=big), dict(window=-big)):
        with pytest.raises(ValueError):
            cache.attention(q, dev, **kw)
        with pytest.raises(ValueError):
            cache.attention_workspace(8, dev, **kw)
    t = dev._t
    for bounds in ((3 + 2 ** 32, 2, 40), (3, big, 40), (3, 2, big)):
        with pytest.raises(ValueError):
            moe.KVBatch(*t, *bounds)
    with pytest.raises(moe.MoEError):  # (in range, and refused by the library)
        cache.attention(q, dev, window=-1)
    torch.cuda.synchronize()
    cache.check()


def coded(cache, batch, which, pick, seed=7):
    """Puts scales, biases and codes of the caller's own making at every position; returns the values they stand for.
    pick(r, n) gives the scales, biases and largest codes of n groups."""
    r = np.random.RandomState(seed)
    held = []
    for b in range(len(batch.new)):
        n, g = batch.kv[b], cache.head_dim // 64
        s, z, top = (a.reshape(n, cache.kv_heads, g) for a in pick(r, n * cache.kv_heads * g))
        s, z = bf16_round(s), bf16_round(z)
        c = r.randint(0, 1 << 30, (n, cache.kv_heads, g, 64)) % (top[..., None] + 1)
        pg, sl = (torch.from_numpy(a.astype(np.int64)).cuda() for a in batch.places(b))
        c = c.reshape(n, cache.kv_heads, cache.head_dim)
        getattr(cache, which + "_codes")[pg, :, sl] = torch.from_numpy(pack(c)).cuda()
        getattr(cache, which + "_scales")[pg, :, sl] = bf16_bits(s).cuda()
        getattr(cache, which + "_biases")[pg, :, sl] = bf16_bits(z).cuda()
        held.append(torch.from_numpy(values(c.astype(np.float64), s, z)).cuda())
    return held


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("new,kv", [([1, 3], [700, 77]), ([150], [200])])
def test_a_cache_of_the_callers_own_making(dim, new, kv, each_path):
    """Magnitudes up to 2^16 from scales up to 2^17 (append's are below 2^13.2), of either sign."""
    def pick(r, n):
        sign = r.choice([-1.0, 1.0], n)
        e = r.choice([2.0 ** 17, 2.0 ** 16, 40000.0, 2.0 ** 15, 2.0 ** 14, 8000.0, 3.0], n)
        return sign * e, -sign * 65536.0, np.minimum(15, (131072.0 // e)).astype(np.int64)
    batch = Batch(new, kv, 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, dim)
    keys, vals = (coded(cache, batch, w, pick, seed) for w, seed in (("k", 7), ("v", 8)))
    assert all(t.abs().max() <= 65536 for t in keys + vals)
    q = rows(batch.n_tokens, 8, dim)
    scale = float(np.float32(2.0 ** -17))
    ref = attention_reference(q, batch, keys, vals, scale)
    dev = batch.device(moe)
    for path in each_path():
        out, lse = cache.attention(q, dev, scale=scale, lse=True)
        cache.check()
        check_attention(out, lse, ref, path)


@pytest.mark.parametrize("dim", [64, 128, 256])
def test_small_values_keep_their_bits(dim, each_path):
    """Values about 2^-90, in units of which the bounds are as ever."""
    batch = Batch([2, 150], [300, 200], 16)
    cache = junk_cache(moe, batch.n_pages, 16, 2, dim)
    keys, _ = fill(cache, batch)
    unit = 2.0 ** -90
    vals = coded(cache, batch, "v", lambda r, n: (unit * (0.1 + r.rand(n)), -8 * unit * r.rand(n), np.full(n, 15)))
    q = rows(batch.n_tokens, 8, dim)
    out, lse, size = attention_reference(q, batch, keys, vals, float(np.float32(dim ** -0.5)))
    dev = batch.device(moe)
    for path in each_path():
        got = cache.attention(q, dev)
        check_attention(got.double() / unit, None, (out / unit, lse, size / unit), path)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [129, 257, 300])
@pytest.mark.parametrize("prompt", [False, True])
def test_many_sequences(dim, n, prompt, each_path):
    """More sequences than a CTA sums up at a time, some without step tokens at the ends of such a run, lengths that are
    cut and, with prompt, one of many rows behind the others."""
    r = np.random.RandomState(n)
    new = r.choice([0, 1, 1, 1, 3], n)
    new[120:128], new[-3:-1], new[-1], new[0] = 0, 0, 2, 0
    kv = new + np.exp(r.uniform(0, np.log(400), n)).astype(int)
    kv[[5, n // 2, n - 1]] += 1500
    if prompt:
        new[n - 2] = kv[n - 2] = 300
    batch = Batch(new.tolist(), kv.tolist(), 32)
    cache = junk_cache(moe, batch.n_pages, 32, 2, dim)
    keys, vals = fill(cache, batch)
    q = rows(batch.n_tokens, 8, dim)
    ref = attention_reference(q, batch, keys, vals, float(np.float32(dim ** -0.5)))
    dev = batch.device(moe, max_kv=5000)
    for path in each_path():
        out, lse = cache.attention(q, dev, lse=True)
        cache.check()
        check_attention(out, lse, ref, path)
    k = rows(batch.n_tokens, 2, dim, 9)
    cache.append(k, k, dev)
    got = cache.read(dev)
    cache.check()
    want = values(*quantise(k.double().cpu().numpy()))
    assert all(np.array_equal(t.double().cpu().numpy(), want) for t in got)


@pytest.mark.parametrize("dim,heads,kv_heads", [(64, 8, 8), (128, 16, 2), (256, 16, 2)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1024, 4)])
def test_a_mixed_step(dim, heads, kv_heads, window, sinks):
    """Single tokens deep in their contexts, drafted tokens and a later chunk of a prompt in one call, under
    the bound of a long capacity."""
    r = np.random.RandomState(dim)
    new = [1] * 11 + [4, 512, 1, 5]
    kv = [int(x) for x in np.exp(r.uniform(np.log(200), np.log(4000), 15))]
    kv[12] = 2300
    batch = Batch(new, kv, 64)
    cache = junk_cache(moe, batch.n_pages, 64, kv_heads, dim)
    keys, vals = fill(cache, batch)
    q = rows(batch.n_tokens, heads, dim)
    ref = attention_reference(q, batch, keys, vals, float(np.float32(dim ** -0.5)), window, sinks)
    dev = batch.device(moe, max_kv=32768)
    out, lse = cache.attention(q, dev, window=window, sinks=sinks, lse=True)
    cache.check()
    check_attention(out, lse, ref)
    again = cache.attention(q, dev, window=window, sinks=sinks)
    assert torch.equal(again, out)


def test_more_units_than_32_bits_number_are_refused():
    """The few-row kernel asked for at a size that it does not number; nothing is launched."""
    n = 1 << 17
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = moe.KVCache.empty(4, 16, 1, 64)
    q = torch.empty(n, 64, 64, dtype=torch.bfloat16, device="cuda")
    batch = moe.KVBatch(i(0, n), i(n), torch.zeros(1, n // 16, dtype=torch.int32, device="cuda"), n, n, 1 << 24)
    moe.moe_set_option(moe.MOE_OPT_FORCE_PATH, 1)
    try:
        ws = cache.attention_workspace(64, batch)
        with pytest.raises(moe.MoEError) as e:
            cache.attention(q, batch, workspace=ws)
        assert e.value.status == moe.MOE_ERR_CUDA and moe.moe_last_launch_count() == 0
    finally:
        moe.moe_set_option(moe.MOE_OPT_FORCE_PATH, 0)
