"""The key/value cache's entry points without a GPU: sizes and the refusal of bad arguments on the host."""
import ctypes

import numpy as np
import pytest

import bit_moe_expert_routing_gb300 as moe
from bit_moe_expert_routing_gb300 import build

kv_util = pytest.importorskip("kv_util")

P = 1 << 20  # a well-aligned address that nothing reads


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return moe.lib()


def cache(n_pages=10, page_size=16, kv_heads=2, head_dim=128, ptr=P, status=P, **kw):
    c = moe.moe_kv_cache(n_pages, page_size, kv_heads, head_dim, ptr, ptr, ptr, ptr, ptr, ptr, status)
    for name, v in kw.items():
        setattr(c, name, v)
    return c


def batch(n_seqs=2, n_tokens=2, max_new=1, max_kv=100, ptr=P, stride=8, **kw):
    b = moe.moe_kv_batch(n_seqs, n_tokens, max_new, max_kv, ptr, ptr, ptr, stride)
    for name, v in kw.items():
        setattr(b, name, v)
    return b


def attn(heads=8, window=0, sinks=0, scale=0.1):
    return moe.moe_attention(heads, window, sinks, scale)


BAD = [
    (dict(head_dim=96), {}, moe.MOE_ERR_SHAPE), (dict(head_dim=192), {}, moe.MOE_ERR_SHAPE),
    (dict(head_dim=512), {}, moe.MOE_ERR_SHAPE), (dict(page_size=8), {}, moe.MOE_ERR_SHAPE),
    (dict(page_size=24), {}, moe.MOE_ERR_SHAPE), (dict(page_size=512), {}, moe.MOE_ERR_SHAPE),
    (dict(kv_heads=0), {}, moe.MOE_ERR_SHAPE), (dict(kv_heads=257), {}, moe.MOE_ERR_SHAPE),
    (dict(n_pages=0), {}, moe.MOE_ERR_SHAPE),
    (dict(k_codes=None), {}, moe.MOE_ERR_ARG), (dict(v_biases=P + 8), {}, moe.MOE_ERR_ARG),
    (dict(status=None), {}, moe.MOE_ERR_ARG), (dict(status=P + 16), {}, moe.MOE_ERR_ARG),
    ({}, dict(n_seqs=-1), moe.MOE_ERR_ARG), ({}, dict(n_tokens=-1), moe.MOE_ERR_ARG),
    ({}, dict(n_tokens=(1 << 20) + 1), moe.MOE_ERR_ARG), ({}, dict(n_seqs=0), moe.MOE_ERR_ARG),
    ({}, dict(max_new=0), moe.MOE_ERR_ARG), ({}, dict(max_kv=-1), moe.MOE_ERR_ARG),
    ({}, dict(max_kv=(1 << 24) + 1), moe.MOE_ERR_ARG), ({}, dict(q_off=None), moe.MOE_ERR_ARG),
    ({}, dict(kv_len=None), moe.MOE_ERR_ARG), ({}, dict(block_table=None), moe.MOE_ERR_ARG),
    ({}, dict(table_stride=-1), moe.MOE_ERR_ARG),
]


@pytest.mark.parametrize("c,b,want", BAD)
def test_bad_caches_and_batches_are_refused(c, b, want):
    c, b = cache(**c), batch(**b)
    assert moe.moe_kv_append(c, b, P, 256, P, 256, None) == want
    assert moe.moe_kv_read(c, b, P, P, None) == want
    assert moe.moe_attention_workspace_size(c, b, attn()) == 0
    assert moe.moe_attention_forward(c, b, attn(), P, 1024, 2 * P, None, P, 1 << 40, None) == want
    assert moe.moe_last_launch_count() == 0


def test_null_structs_are_refused(lib):
    assert lib.moe_kv_append(None, ctypes.byref(batch()), P, 256, P, 256, None) == moe.MOE_ERR_ARG
    assert lib.moe_kv_read(ctypes.byref(cache()), None, P, P, None) == moe.MOE_ERR_ARG
    assert lib.moe_attention_workspace_size(ctypes.byref(cache()), ctypes.byref(batch()), None) == 0
    assert lib.moe_attention_forward(ctypes.byref(cache()), ctypes.byref(batch()), None, P, 1024, 2 * P, None, P, 1 << 40,
                                     None) == moe.MOE_ERR_ARG


def test_operands_are_checked():
    c, b, w = cache(), batch(), 1 << 40
    for k, ks, v, vs in ((None, 256, P, 256), (P, 256, None, 256), (P + 2, 256, P, 256), (P, 255, P, 256),
                         (P, 248, P, 256), (P, 256, P, 260), (P, 256, P, -256)):
        assert moe.moe_kv_append(c, b, k, ks, v, vs, None) == moe.MOE_ERR_ARG, (k, ks, v, vs)
    assert moe.moe_kv_read(c, b, P + 4, P, None) == moe.MOE_ERR_ARG
    assert moe.moe_kv_read(c, b, None, P + 4, None) == moe.MOE_ERR_ARG
    assert moe.moe_kv_read(c, b, None, None, None) == moe.MOE_OK  # nothing asked for
    for q, qs, out, lse in ((None, 1024, 2 * P, None), (P + 2, 1024, 2 * P, None), (P, 1016, 2 * P, None),
                            (P, 1025, 2 * P, None), (P, 1024, None, None), (P, 1024, 2 * P + 8, None),
                            (P, 1024, P, None), (P, 1024, 2 * P, 2 * P + 2)):
        assert moe.moe_attention_forward(c, b, attn(), q, qs, out, lse, P, w, None) == moe.MOE_ERR_ARG, (q, qs, out, lse)
    n = moe.moe_attention_workspace_size(c, b, attn())
    assert n > 0
    for ws, size in ((None, n), (P + 16, n), (P, n - 1)):
        assert moe.moe_attention_forward(c, b, attn(), P, 1024, 2 * P, None, ws, size, None) == moe.MOE_ERR_WORKSPACE


@pytest.mark.parametrize("a,want", [(dict(heads=7), moe.MOE_ERR_SHAPE), (dict(heads=1), moe.MOE_ERR_SHAPE),
                                    (dict(heads=0), moe.MOE_ERR_SHAPE), (dict(heads=130), moe.MOE_ERR_SHAPE),
                                    (dict(window=-1), moe.MOE_ERR_ARG), (dict(sinks=-1), moe.MOE_ERR_ARG),
                                    (dict(scale=float("nan")), moe.MOE_ERR_ARG),
                                    (dict(scale=float("inf")), moe.MOE_ERR_ARG)])
def test_attention_settings_are_checked(a, want):
    assert moe.moe_attention_workspace_size(cache(), batch(), attn(**a)) == 0
    assert moe.moe_attention_forward(cache(), batch(), attn(**a), P, 1 << 20, 2 * P, None, P, 1 << 40, None) == want


def test_empty_steps_are_no_ops():
    for b in (batch(n_tokens=0), batch(n_tokens=0, n_seqs=0, max_new=0, max_kv=0, q_off=None, kv_len=None, block_table=None)):
        assert moe.moe_kv_append(cache(), b, None, 0, None, 0, None) == moe.MOE_OK
        assert moe.moe_kv_read(cache(), b, P, P, None) == moe.MOE_OK
        assert moe.moe_attention_workspace_size(cache(), b, attn()) > 0
        assert moe.moe_attention_forward(cache(), b, attn(), None, 0, None, None, None, 0, None) == moe.MOE_OK
        assert moe.moe_last_launch_count() == 0


def test_workspace_grows_with_the_bounds():
    """A workspace sized for a larger step serves a smaller one."""
    size = lambda **kw: moe.moe_attention_workspace_size(cache(), batch(**kw), attn())  # noqa: E731
    last = 0
    for max_kv in (1, 100, 1000, 10000, 100000):
        n = size(max_kv=max_kv)
        assert n >= last and n % 256 == 0
        last = n
    assert size(n_seqs=8, n_tokens=8) >= size(n_seqs=2, n_tokens=2)
    assert size(n_tokens=600, max_new=300) >= size(n_tokens=600, max_new=300, max_kv=50)


def test_python_handles_check_their_tensors():
    torch = pytest.importorskip("torch")
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on a GPU
        moe.KVBatch(i, i[:2], i[:2, None], 2, 1, 10)
    with pytest.raises(ValueError):
        moe.KVCache.empty(2, 16, 2, 128, device="cpu")


# --- the plain implementation itself, against hand-worked values -----------------------------------

def test_reference_quantisation_hand_worked():
    x = np.zeros((1, 64))
    x[0, :4] = [-1.0, 0.5, 14.0, 6.5]  # range 15: scale 1, bias -1; 0.5 -> 1.5 ties to 2, 6.5 -> 7.5 to 8
    q, s, b = kv_util.quantise(x)
    assert s[0, 0] == 1.0 and b[0, 0] == -1.0
    assert list(q[0, :4]) == [0, 2, 15, 8] and q[0, 4] == 1
    v = kv_util.values(q, s, b)
    assert list(v[0, :5]) == [-1.0, 1.0, 14.0, 7.0, 0.0]
    assert kv_util.unpack(kv_util.pack(q)).tolist() == q.tolist()
    q, s, b = kv_util.quantise(np.full((1, 64), 3.25))
    assert s[0, 0] == 0 and b[0, 0] == 3.25 and (q == 0).all()


def test_reference_rounding_is_nearest_even():
    torch = pytest.importorskip("torch")
    x = np.random.RandomState(0).randn(5000).astype(np.float32)
    assert np.array_equal(kv_util.bf16_round(x.astype(np.float64)), torch.from_numpy(x).to(torch.bfloat16).double().numpy())
    assert kv_util.bf16_round(np.array([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8])).tolist() == [1.0, 1 + 2.0 ** -6]
