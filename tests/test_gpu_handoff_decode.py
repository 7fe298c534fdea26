"""What the decode worker of lossless_bf16_kv_gb300.handoff computes, step by step
and layer by layer: its queries, the tokens it appends to the cache that arrived,
and its attention, each against the definition in 64 bits on the stored bits, so
that nothing but the operator's own roundings is allowed for."""
import pytest
import torch

from lossless_bf16_kv_gb300 import handoff
from lossless_bf16_kv_gb300 import splitzip as sz
from tests import serving_ref as ref
from tests.gpu_helpers import ensure_library
from tests.test_gpu_serving import close

pytestmark = pytest.mark.gpu


def check_decode(s: handoff.Shape, arrived: int):
    """arrived: tokens of the prompt that the decode worker has."""
    r = handoff.run(s)
    m, kv = r["layers"], r["decoded"]
    bits = torch.int16 if s.fmt == "bf16" else torch.uint8
    assert torch.equal(kv[:, :, :arrived].view(bits), r["there"][:, :, :arrived].view(bits))
    for step in range(s.steps):
        x = m.new[step:step + 1]
        pos = torch.tensor([s.tokens + step], device="cuda")
        n = arrived + step + 1
        for layer in range(s.layers):
            qr, kr, vr = m.project(layer, x)
            q, out = r["queries"][step, layer][None, None], r["outs"][step, layer][None, None]
            want, tol = ref.norm_rope(qr, m.norm[layer][0], pos, m.table, 1e-6, False)
            close(q[0], want, tol + want.abs() * 2.0 ** -8, f"queries {step} {layer}")
            want, tol = ref.norm_rope(kr, m.norm[layer][1], pos, m.table, 1e-6, False)
            tol = tol + (want.abs() * 2.0 ** -8 if s.fmt == "bf16" else want.abs() * 2.0 ** -3 + 2.0 ** -17)
            close(kv[layer, 0, n - 1][None].float(), want, tol, f"keys {step} {layer}")
            assert torch.equal(kv[layer, 1, n - 1].float(), vr[0].to(s.dtype).float())
            k, v = kv[layer:layer + 1, 0, :n], kv[layer:layer + 1, 1, :n]
            attend = lambda size: ref.attention(q, k, v, torch.tensor([size], device="cuda"), 0, 0, s.dim ** -0.5)  # noqa: E731
            o, _, tol, _ = attend(n)
            close(out, o, tol, f"outputs {step} {layer}")
            # The bound tells the new token's part from none.
            without = attend(n - 1)[0] if n > 1 else torch.zeros_like(o)
            assert bool(((without - o).abs() > 2 * tol).any())
            x = m.mix(layer, x, out[0])


@pytest.mark.parametrize("fmt,heads,dim", [("bf16", (8, 2), 128), ("e5m2", (6, 2), 64)])
def test_decode_over_a_thinned_cache(fmt, heads, dim):
    ensure_library()
    check_decode(handoff.Shape(layers=2, tokens=300, q_heads=heads[0], kv_heads=heads[1], dim=dim, window=120, sinks=4,
                               budget=70, observe=16, steps=3, fmt=fmt, seed=3), 70)


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("tokens,budget", [(50, 128), (5, 6), (40, 40)])
def test_decode_after_a_prompt_shorter_than_the_budget(tokens, budget, fmt):
    """Only the prompt's tokens are there to attend to, however many would be kept."""
    ensure_library()
    check_decode(handoff.Shape(layers=2, tokens=tokens, q_heads=8, kv_heads=2, dim=64, window=32, sinks=4, budget=budget,
                               observe=16, steps=2, fmt=fmt, seed=4), tokens)


def test_no_query_to_weigh_by_is_refused():
    """With none to observe, none decides; not all of the prompt's."""
    ensure_library()
    with pytest.raises(sz.SplitZipError):
        handoff.run(handoff.Shape(layers=1, tokens=30, q_heads=2, kv_heads=1, dim=64, budget=10, observe=0, steps=1))
