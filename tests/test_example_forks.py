"""The decoder example with several continuations of each prompt: shared pages, copied before they are written, and attention
that shares what they have in common, against plain attention over what the cache holds."""
import os
import sys

import pytest

import bit_moe_expert_routing_gb300 as moe
from bit_moe_expert_routing_gb300 import build, synth

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("path", [0, 2])
def test_continuations_of_a_prompt(path):
    import decoder
    from test_example_decoder import plain_attend
    build.build()
    D, prompts, steps, n = 256, [70, 9, 33], 20, 3
    dec = decoder.build(2, prompts, steps, 8, 2, 64, 16, lambda i: synth.make_layer(i, D, 16, 4, 128), window=24, sinks=2,
                        continuations=n)
    x = torch.randn(sum(prompts), D, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    y = dec.prompt(x)
    assert y.shape == (3, D) and torch.isfinite(y).all()
    held = dec.pages.held.tolist()
    dec.fork()
    assert dec.pages.held.tolist() == [h for h in held[::n] for _ in range(n)]
    g = torch.Generator(device="cuda").manual_seed(2)
    y = y.repeat_interleave(n, 0) + torch.randn(n * len(prompts), D, generator=g, device="cuda").bfloat16()
    seen = []
    for layer in dec.layers:
        attend = layer.attend
        layer.attend = lambda x, batch, pos, ws, attend=attend: seen.append((x, batch, pos, attend(x, batch, pos, ws))) or seen[-1][3]
    lengths = [p for p in prompts for _ in range(n)]
    # as for the example's other test: bf16 roundings of the output, the product and the sum, values of order 4
    close = dict(atol=2.0 ** -5, rtol=2.0 ** -7)
    moe.moe_set_option(moe.MOE_OPT_FORCE_PATH, path)  # (2: the attention shares whatever its size; the experts' GEMM path)
    try:
        y = dec.step(y)
    finally:
        moe.moe_set_option(moe.MOE_OPT_FORCE_PATH, 0)
    for t in range(steps):
        if t:
            y = dec.step(y.clone())
        lengths = [p + 1 for p in lengths]
        assert dec.kv_len.tolist() == lengths and torch.isfinite(y).all()
        dec.check()
        if t in (0, 7, steps - 1):
            # the captured step's tensors, filled by the replay: the two calls before were the one outside the capture
            for layer, (xi, batch, pos, got) in zip(dec.layers, seen[2:]):
                torch.testing.assert_close(got.double(), plain_attend(layer, xi, batch, pos, lengths, list(range(len(lengths) + 1))),
                                           **close)
    # every prompt's whole pages are its continuations' all, and what they wrote is each one's own
    table, refs = dec.pages.table.cpu(), dec.pages.refs.cpu()
    assert dec.pages.held.tolist() == [-(-p // 16) for p in lengths]
    for i, p in enumerate(prompts):
        rows = table[i * n:(i + 1) * n]
        for j in range(-(-lengths[i * n] // 16)):
            pages = set(rows[:, j].tolist())
            assert len(pages) == (1 if j < p // 16 else n)
            assert all(refs[q] == (n if j < p // 16 else 1) for q in pages)
