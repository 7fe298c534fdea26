"""Attention over E5M2 caches where its 16-bit operands have the least room."""
import pytest
import torch

from tests import serving_ref as ref
from tests.gpu_helpers import ensure_library
from tests.test_gpu_serving import attend, close, lens_of

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("tq,tk", [(1, 200), (1, 70_001), (20, 70_001), (100, 70_001), (300, 20_000)])
@pytest.mark.parametrize("first", [True, False])
def test_many_small_weights_next_to_a_large_one(first, tq, tk, dim):
    """One slot takes nearly all of the weight, as a first token does, and has the value
    0: the output is what the others leave, 2^-25.6 of its weight each.  Their sum is
    held to the bound of any other, relative to itself."""
    ensure_library()
    q = torch.ones((1, tq, 1, dim), dtype=torch.bfloat16, device=DEV)
    kv = torch.zeros((1, 2, tk, 1, dim), device=DEV)
    at = 0 if first else tk - tq            # seen by every query
    kv[0, 0, at] = 0.25 * 64 / dim
    kv[0, 0, at, 0, :7] += 0.25             # 17.75 over all
    kv[0, 1] = 1.0
    kv[0, 1, at] = 0.0
    kv = kv.to(torch.float8_e5m2)
    assert kv[0, 0, at].double().sum().item() == 17.75
    out, lse = attend(q, kv, None, scale=1.0)
    o, l, tol, ltol = ref.attention(q, kv[:, 0], kv[:, 1], lens_of([tk]), 0, 0, 1.0)
    close(out, o, tol, "out")
    close(lse, l, ltol, "lse")
