"""Attention over E5M2 caches where its 16-bit operands have the least room."""
import pytest
import torch

from tests import serving_ref as ref
from tests.gpu_helpers import ensure_library
from tests.test_gpu_serving import attend, close, lens_of, make

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


@pytest.mark.parametrize("fmt", ["e5m2", "bf16"])
@pytest.mark.parametrize("tq,tk,hq,hk,dim,window,length", [
    (4, 5000, 40, 2, 128, 0, 7), (4, 5000, 40, 2, 64, 0, 7), (100, 1000, 2, 2, 128, 1, None), (100, 1000, 2, 2, 64, 1, None),
    (300, 6000, 4, 2, 128, 0, 400), (300, 6000, 4, 2, 64, 5, None)])
def test_splits_that_have_no_slots(tq, tk, hq, hk, dim, window, length, fmt):
    """Most of a row tile's splits are empty, as the plan goes by the cache's size: what
    they hand to the join is nothing, in every one of many calls.  (A warp of an empty
    split that was late with its queries wrote them over another's partial result.)"""
    ensure_library()
    q, kv = make(1, tq, tk, hq, hk, dim, fmt=fmt, seed=dim)
    lens = lens_of([length or tk])
    o, l, tol, ltol = ref.attention(q, kv[:, 0], kv[:, 1], lens, window, 0, dim ** -0.5)
    calls = [attend(q, kv, lens, window) for _ in range(600)]
    for out, lse in calls[:1]:
        close(out, o, tol, "out")
        close(lse, l, ltol, "lse")
    differ = [i for i, (out, lse) in enumerate(calls) if not (torch.equal(out, calls[0][0]) and torch.equal(lse, calls[0][1]))]
    assert not differ, f"{len(differ)} of {len(calls)} calls differ from the first"
