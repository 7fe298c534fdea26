"""The decode worker on pages: every operator of the paged cache in the run of the
whole chain, each step held to the definition over what the pages hold."""
import pytest
import torch

from lossless_bf16_kv_gb300 import handoff
from lossless_bf16_kv_gb300 import pages as pg
from lossless_bf16_kv_gb300 import splitzip as sz
from tests import pages_ref as ref
from tests.gpu_helpers import ensure_library
from tests.test_gpu_pages import close

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built():
    ensure_library()


@pytest.mark.parametrize("fmt,pages", [("bf16", "bf16"), ("bf16", "int8"), ("bf16", "e2m1"), ("e5m2", "e5m2"), ("e5m2", "int8")])
def test_decode_over_pages(fmt, pages):
    s = handoff.Shape(layers=2, tokens=333, q_heads=8, kv_heads=2, dim=64, window=128, budget=101, observe=16, steps=4, fmt=fmt,
                      pages=pages, seed=3)
    r = handoff.run(s)
    pool, table = r["decoded"], r["table"]
    assert torch.equal(r["there"].view(torch.uint8), r["small"].view(torch.uint8))
    one = torch.tensor([0, 1], dtype=torch.int32)
    for layer in range(s.layers):
        # What the pages hold of the cache that came is what the format makes of it.
        for i, x in enumerate("kv"):
            rows, exps = ref.codes(r["there"][layer, i].bfloat16(), pages)
            assert torch.equal(ref.sequence(pool, table[layer], s.kept, x), ref.values(rows, exps, pages))
        for step in range(s.steps):
            n = s.kept + step + 1
            found = ref.attention(r["queries"][step, layer:layer + 1], pool, table[layer:layer + 1], one, torch.tensor([n]), n, 0, 0,
                                  s.dim ** -0.5)
            (_, o, _, tol, _), = found
            close(r["outs"][step, layer:layer + 1], o, tol, f"layer {layer}, step {step}")


def test_pages_go_back_through_the_codec():
    """Quantised pages, read back, are BF16 values that the lossless codec packs and gives back bit for bit."""
    s = handoff.Shape(layers=2, tokens=200, q_heads=4, kv_heads=2, dim=128, window=64, budget=64, observe=8, steps=2, pages="int8")
    r = handoff.run(s)
    n = s.kept + s.steps
    kv = torch.zeros((s.layers, 2, n, s.kv_heads, s.dim), dtype=torch.bfloat16, device="cuda")
    pg.splitzip_pages_load(r["decoded"], r["table"], None, kv[:, 0], kv[:, 1])
    for layer in range(s.layers):
        for i, x in enumerate("kv"):
            assert torch.equal(kv[layer, i].double(), ref.sequence(r["decoded"], r["table"][layer], n, x))
    codec = sz.ChunkLocalSplitZipGPU(device="cuda", chunk_size=1024)
    codec.calibrate(kv)
    assert torch.equal(codec.decode(codec.encode(kv)).view(torch.int16), kv.view(torch.int16))


def test_the_command_runs_on_pages(capsys):
    assert handoff.main(["--layers", "2", "--tokens", "300", "--budget", "64", "--steps", "2", "--pages", "e2m1"]) == 0
    assert "outputs finite: True" in capsys.readouterr().out
