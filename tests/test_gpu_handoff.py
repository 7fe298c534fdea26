"""The operators together: a prompt's cache from prefill through eviction and
the codec to a decode worker (lossless_bf16_kv_gb300.handoff), each part
against its definition in 64 bits."""
import pytest
import torch

from lossless_bf16_kv_gb300 import handoff
from tests import serving_ref as ref
from tests.gpu_helpers import ensure_library
from tests.test_gpu_serving import close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,heads,dim", [("bf16", (8, 2), 128), ("e5m2", (6, 2), 64)])
def test_prefill_thin_send_decode(fmt, heads, dim):
    ensure_library()
    s = handoff.Shape(layers=2, tokens=300, q_heads=heads[0], kv_heads=heads[1], dim=dim, window=120, sinks=4, budget=70,
                      observe=16, steps=3, fmt=fmt, seed=3)
    r = handoff.run(s)
    m, kv = r["layers"], r["kv"]
    bits = torch.int16 if fmt == "bf16" else torch.uint8
    assert torch.equal(r["small"].view(bits), r["there"].view(bits))
    for layer in range(s.layers):
        for h in range(s.kv_heads):
            keep = ref.evict_slots(r["weights"][layer, h].tolist(), s.tokens, s.budget, s.sinks, s.observe)
            assert r["index"][layer, h].tolist() == keep
            assert torch.equal(r["small"][layer, :, :, h].view(bits), kv[layer, :, keep, h].view(bits))
        # Every one of the last queries gives away a weight of one per query head.
        total = r["weights"][layer].double().sum().item()
        assert abs(total - s.observe * s.q_heads) < 1e-3 * s.observe * s.q_heads
    # The first layer's first new token: its query over the thinned cache and its own key.
    qr, kr, vr = m.project(0, m.new[:1])
    pos = torch.tensor([s.tokens], device="cuda")
    q = ref.norm_rope(qr, m.norm[0][0], pos, m.table, 1e-6, False)[0].bfloat16()[None]
    k = ref.norm_rope(kr, m.norm[0][1], pos, m.table, 1e-6, False)[0].to(s.dtype)
    one = torch.stack([k.float(), vr.float()]).to(s.dtype)[None]                       # [1, 2, 1, heads, dim]
    cache = torch.cat([r["there"][:1].float(), one.float()], dim=2).to(s.dtype)
    lens = torch.tensor([s.budget + 1], dtype=torch.int32, device="cuda")
    o, _, tol, _ = ref.attention(q, cache[:, 0], cache[:, 1], lens, 0, 0, dim ** -0.5)
    # The query and key above may round the other way in their last bit: 2^-8 of a
    # BF16 (2^-3 of an E5M2) value in the one key, 2^-8 in the query, as a score error.
    score = ref.scores(q, cache[:, 0], dim ** -0.5)[1].max()
    slack = score * (2.0 ** -8 + (2.0 ** -8 if fmt == "bf16" else 2.0 ** -3))
    mass = torch.ones_like(o) * cache[:, 1].double().abs().max()
    close(r["outs"][0, 0][None, None], o, tol + 2 * slack * mass, "decode")


def test_command_line(capsys):
    ensure_library()
    assert handoff.main(["--layers", "1", "--tokens", "200", "--budget", "50", "--steps", "1", "--q-heads", "4",
                         "--kv-heads", "2"]) == 0
    assert "arrived bit for bit: True" in capsys.readouterr().out
