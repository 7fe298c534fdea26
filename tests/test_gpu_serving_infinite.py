"""Queries all of whose visible scores are -infinity, next to others: they take
nothing from the cache and give no weight, as those that see nothing."""
import math

import pytest
import torch

from lossless_bf16_kv_gb300 import serving
from tests import serving_ref as ref
from tests.gpu_helpers import ensure_library
from tests.test_gpu_serving import attend, close, lens_of, make

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("fmt", ["bf16", "e5m2"])
@pytest.mark.parametrize("b,tq,tk,hq,hk,dim", [(1, 12, 40, 2, 2, 128), (1, 12, 40, 8, 2, 64), (2, 60, 300, 4, 2, 128),
                                               (1, 200, 2000, 2, 2, 64), (1, 600, 600, 4, 2, 128), (2, 300, 300, 6, 2, 64)])
def test_rows_of_minus_infinity(b, tq, tk, hq, hk, dim, fmt):
    ensure_library()
    q, kv = make(b, tq, tk, hq, hk, dim, fmt=fmt, seed=tq)
    q[..., 3] = q[..., 3].abs() + 0.125
    first = tk - tq                        # position of the first query
    n = first + 9                          # slots whose scores are -infinity for every query
    kv[:, 0, :n, :, 3] = -math.inf
    out, lse = attend(q, kv, None)
    lost = n - first                       # queries at positions 0 .. n - 1 see no other
    assert bool((out[:, :lost] == 0).all()) and bool((lse[:, :, :lost] == -math.inf).all())
    o, l, tol, ltol = ref.attention(q[:, lost:], kv[:, 0, n:], kv[:, 1, n:], lens_of([tk - n] * b), 0, 0, dim ** -0.5)
    close(out[:, lost:], o, tol, "out")
    close(lse[:, :, lost:], l, ltol, "lse")
    w = torch.full((b, hk, tk), float("nan"), device=DEV)
    serving.splitzip_attention_weights(q, kv[:, 0], lse, w)
    assert bool((w[..., :n] == 0).all())
    want, wtol = ref.weights(q[:, lost:], kv[:, 0, n:], lse[:, :, lost:], lens_of([tk - n] * b), 0, 0, dim ** -0.5)
    close(w[..., n:], want, wtol, "weights")
