"""The operators around the KV cache at the far end of what they accept, and next
to it.  Long inputs are views whose rows overlap (a stride shorter than a row),
so that few bytes hold many tokens."""
import pytest
import torch

from lossless_bf16_kv_gb300 import serving
from tests import serving_ref as ref
from tests.gpu_helpers import ensure_library
from tests.test_gpu_serving import close, gen, rope_table

pytestmark = pytest.mark.gpu
DEV = "cuda"


def test_norm_rope_of_more_than_two_to_the_32_threads():
    """Three heads of 64 with rot_dim 8 take 24 threads a token: 2^32 are passed from
    178956971 tokens on (q_out alone holds 23 GB)."""
    ensure_library()
    d, rot, n, ends = 64, 8, 178_960_003, 40
    store = torch.randn(8 * n + d, generator=gen(1), device=DEV).bfloat16()
    x = store.as_strided((n, 1, d), (8, d, 1))
    pos = (torch.arange(n, device=DEV, dtype=torch.int32) % 50)
    table = rope_table(50, rot)
    slots = torch.full((n,), -1, dtype=torch.int64, device=DEV)
    at = torch.cat([torch.arange(ends, device=DEV), torch.arange(n - ends, n, device=DEV)])
    slots[at] = torch.arange(2 * ends, device=DEV)
    kv = torch.zeros((2, 2 * ends, 1, d), dtype=torch.bfloat16, device=DEV)
    out = torch.full((n, 1, d), float("nan"), dtype=torch.bfloat16, device=DEV)
    serving.splitzip_qk_norm_rope(x, x, x, None, None, pos, table, slots, out, kv[0], kv[1])
    want, tol = ref.norm_rope(x[at], None, pos[at], table, 1e-6, False)
    close(out[at], want, tol + want.abs() * 2.0 ** -8, "q")
    close(kv[0], want, tol + want.abs() * 2.0 ** -8, "k")
    assert torch.equal(kv[1], x[at])
    assert not any(bool(torch.isnan(part).any()) for part in out.split(1 << 24))


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("layout", ["planes", "heads first", "padded"])
def test_norm_rope_drops_slots_between_sequences(layout, fmt):
    """A row behind a sequence's last token is another plane's, another head's or
    padding: every slot of the whole range is offered, and only the cache changes."""
    ensure_library()
    b, t, h, d = 3, 40, 2, 64
    dtype = torch.bfloat16 if fmt == "bf16" else torch.float8_e5m2
    if layout == "planes":
        store = torch.full((b, 2, t, h, d), 7.0, device=DEV).to(dtype)
        k, v = store[:, 0], store[:, 1]
    elif layout == "heads first":
        store = torch.full((2, b, h, t, d), 7.0, device=DEV).to(dtype)
        k, v = store[0].transpose(1, 2), store[1].transpose(1, 2)
    else:
        store = torch.full((2, b, t + 9, h, d), 7.0, device=DEV).to(dtype)
        k, v = store[0, :, :t], store[1, :, :t]
    step = k.stride(0) // k.stride(1)
    n = b * step + 5
    x = torch.randn((n, h, d), generator=gen(4), device=DEV).bfloat16()
    out = torch.empty_like(x)
    serving.splitzip_qk_norm_rope(x, x, x, None, None, None, None, torch.arange(n, device=DEV), out, k, v)
    want, tol = ref.norm_rope(x, None, None, None, 1e-6, False)
    tol = tol + (want.abs() * 2.0 ** -8 if fmt == "bf16" else want.abs() * 2.0 ** -3 + 2.0 ** -17)
    for i in range(b):
        rows = slice(i * step, i * step + t)
        close(k[i].float(), want[rows], tol[rows], "k")
        assert torch.equal(v[i].float(), x[rows].to(dtype).float())
    if layout == "padded":
        assert bool((store[:, :, t:].float() == 7.0).all())
