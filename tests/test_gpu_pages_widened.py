"""Attention of so many new tokens that quantised and E5M2 caches are widened ahead of the products."""
import pytest
import torch

from tests import pages_ref, serving_ref
from tests.gpu_helpers import ensure_library
from tests.test_gpu_pages import DEV, attend, batch_of, close, ints

pytestmark = pytest.mark.gpu
WIDENED = ["e5m2", "int8", "e2m1"]


@pytest.fixture(autouse=True)
def _built():
    ensure_library()


def ones_of_either_sign(p, fmt):
    """Values 1 in even slots of a page and -1 in odd ones."""
    neg = torch.arange(p.page_tokens, device=DEV)[None, :, None, None] % 2 == 1
    one = {"int8": (64, -64, 121), "e2m1": (0x22, 0xAA, 127), "e5m2": (1.0, -1.0, None)}[fmt]
    p.v.copy_(torch.where(neg, one[1], one[0]).expand(p.v.shape).to(p.v.dtype))
    if p.v_exp is not None:
        p.v_exp.fill_(one[2])


@pytest.mark.parametrize("fmt", WIDENED)
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("counts", [[200], [600], [600, 1, 220, 530]], ids=["tiles", "widened", "both"])
def test_weights_keep_eleven_bits(counts, dim, fmt):
    """Queries that see two slots, with values 1 and -1: the output is the difference of two weights, and where they are
    nearly alike it shows their rounding.  FP16 weights are off by at most 2^-11 of their sum, the output's own rounding
    is 2^-8 of it; 2^-13 and the scores' errors (which the bound of lse has) are serving_ref's."""
    lens = [n + 150 for n in counts]
    q, p, table, start, lens = batch_of(counts, lens, 8, 2, dim, 16, fmt, seed=dim)
    ones_of_either_sign(p, fmt)
    out, lse = attend(q, p, table, start, lens, window=2)
    near = 0
    for b, n in enumerate(lens.tolist()):
        i, j = start[b].item(), start[b + 1].item()
        k, v = (pages_ref.sequence(p, table[b], n, x)[None] for x in "kv")
        o, l, _, ltol = serving_ref.attention(q[None, i:j], k, v, ints([n]), 2, 0, dim ** -0.5)
        tol = o[0].abs() * 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -13 + 2 * ltol[0].T[..., None]
        near += int((o.abs() < 2.0 ** -4).sum())
        close(out[i:j], o[0], tol, "out")
        close(lse[:, i:j], l[0], ltol[0], "lse")
    assert near > 1000
