"""The host side of the attention's entry point without a GPU: kv_api.cu compiled with stand-ins for the kernels' launches,
which record what they are called with."""
import ctypes
import os
import subprocess

import pytest

import bit_moe_expert_routing_gb300 as moe
from bit_moe_expert_routing_gb300 import build

P = 1 << 20  # a well-aligned address that nothing reads

HARNESS = r"""
#include "kv_api.cu"

namespace moe {
static int paths[2], snapshots, used[2];  // the option's value at the first and at later looks; bytes each kind of kernel uses
static AttnArgs last;
Options options_snapshot() {
  Options o;
  o.force_path = paths[snapshots++ > 0];
  return o;
}
int num_sms() { return 152; }
void reset_launch_count() {}
void timing_begin(const Options&, cudaStream_t) {}
void launch_done(const Options&, cudaStream_t, const char*) {}
size_t attention_few_workspace(const AttnArgs&, int) { return 4096; }
size_t attention_many_workspace(const AttnArgs&) { return 1 << 20; }
long long attention_few_items(const AttnArgs&, int) { return 1 << 20; }
cudaError_t attention_few(const AttnArgs& a, int, void*, bool, const KvCall&) {
  last = a, used[0] = 4096;
  return cudaSuccess;
}
cudaError_t attention_many(const AttnArgs& a, int, void*, const KvCall&) {
  last = a, used[1] = 1 << 20;
  return cudaSuccess;
}
cudaError_t kv_append(const KvArgs&, const uint16_t*, long long, const uint16_t*, long long, const KvCall&) { return cudaSuccess; }
cudaError_t kv_read(const KvArgs&, uint16_t*, uint16_t*, const KvCall&) { return cudaSuccess; }
}  // namespace moe

extern "C" void set_paths(int first, int later) {
  moe::paths[0] = first, moe::paths[1] = later;
  moe::snapshots = moe::used[0] = moe::used[1] = 0;
}
extern "C" int bytes_used() { return moe::used[0] + moe::used[1]; }
extern "C" int last_window() { return moe::last.window; }
extern "C" int last_sinks() { return moe::last.sinks; }
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    d = tmp_path_factory.mktemp("kv_host")
    src, so = d / "harness.cu", d / "harness.so"
    src.write_text(HARNESS)
    subprocess.run([build._nvcc(), *build.ARCH, "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-shared",
                    "-Xlinker", "-Bsymbolic", "-I", build.CSRC, "-I", os.path.join(build.ROOT, "include"), str(src), "-o",
                    str(so)], check=True, capture_output=True)
    lib = ctypes.CDLL(str(so))
    for name in ("moe_attention_workspace_size", "moe_attention_forward"):
        getattr(lib, name).restype, getattr(lib, name).argtypes = moe.SIGNATURES[name]
    return lib


def step(max_kv=1000, n_tokens=300, window=0, sinks=0):
    return (moe.moe_kv_cache(10, 16, 2, 128, P, P, P, P, P, P, P), moe.moe_kv_batch(1, n_tokens, n_tokens, max_kv, P, P, P, 64),
            moe.moe_attention(16, window, sinks, 0.1))


def size(host, c, b, a):
    return host.moe_attention_workspace_size(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a))


def forward(host, c, b, a, nbytes):
    return host.moe_attention_forward(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), P, 2048, 2 * P, None, P, nbytes, None)


@pytest.mark.parametrize("first,later", [(1, 2), (2, 1), (0, 1), (1, 0), (0, 2), (2, 0)])
def test_an_option_set_during_the_call_does_not_change_its_kernels(host, first, later):
    """Another thread's change of the path between the workspace's check and the launches."""
    s = step()
    host.set_paths(first, first)
    n = size(host, *s)
    host.set_paths(first, later)
    assert forward(host, *s, n) == moe.MOE_OK
    assert 0 < host.bytes_used() <= n
    host.set_paths(first, later)
    assert forward(host, *s, n - 1) == moe.MOE_ERR_WORKSPACE
    assert host.bytes_used() == 0


INT_MAX = 2 ** 31 - 1


@pytest.mark.parametrize("window,sinks,want", [(0, 0, (0, 0)), (0, 7, (0, 0)), (1, 0, (1, 0)), (999, 4, (999, 4)),
                                               (999, INT_MAX, (999, 1000)), (1000, 4, (0, 0)), (INT_MAX, 0, (0, 0)),
                                               (INT_MAX, INT_MAX, (0, 0)), (INT_MAX - 2 ** 24, 1, (0, 0))])
def test_windows_and_sinks_reach_the_kernels_within_the_bound_on_the_lengths(host, window, sinks, want):
    """Larger ones mean the same, and would pass 32 bits in the kernels' differences."""
    s = step(max_kv=1000, window=window, sinks=sinks)
    for path in (0, 1, 2):
        host.set_paths(path, path)
        assert forward(host, *s, size(host, *s)) == moe.MOE_OK
        assert (host.last_window(), host.last_sinks()) == want


@pytest.mark.parametrize("dim,heads,kv_heads,page", [(64, 8, 8, 16), (128, 16, 2, 64), (256, 16, 2, 64), (128, 5, 1, 16),
                                                    (64, 24, 4, 256), (256, 64, 8, 32)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 1), (512, 4), (5000, 100)])
def test_a_larger_steps_workspace_serves_a_smaller_one(dim, heads, kv_heads, page, window, sinks):
    """No bound of the step lowers the size: over the grid, each size against those one bound below it, with the lengths
    about those up to which items are not cut and those at which the many-row kernels need one pass more."""
    build.build()
    c = moe.moe_kv_cache(10, page, kv_heads, dim, P, P, P, P, P, P, P)
    seqs = [1, 2, 3, 8, 15, 16, 17, 31, 32, 33, 64, 65, 128, 300]
    tokens = [1, 2, 4, 7, 16, 33, 64, 65, 129, 257, 600, 3000, 40000]
    new = [1, 2, 3, 4, 8, 9, 17, 129, 257, 600, 3000]
    tile = 128 * dim * 4  # bytes of an expanded tile of 128 keys and their values
    passes = [128 * (2 ** 31 // tile // n) for n in (1, 2, 3, 4, 5, 8, 64, 600)]
    kv = sorted({1, 100, 400, 447, 448, 449, 600, 895, 896, 897, 1100, 1500, 2047, 2048, 2049, 2100, 32768, 1 << 24}
                | {p + d for p in passes for d in (-129, -1, 0, 1, 128) if 0 < p + d <= 1 << 24})
    got = {}
    for i, s in enumerate(seqs):
        for j, t in enumerate(tokens):
            for k, m in enumerate(new):
                for l, v in enumerate(kv):
                    n = moe.moe_attention_workspace_size(c, moe.moe_kv_batch(s, t, m, v, P, P, P, 64),
                                                         moe.moe_attention(heads, window, sinks, 0.1))
                    got[i, j, k, l] = n
                    for at in ((i - 1, j, k, l), (i, j - 1, k, l), (i, j, k - 1, l), (i, j, k, l - 1)):
                        assert got.get(at, 1) <= n, (s, t, m, v, at)
