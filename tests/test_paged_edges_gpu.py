"""Paged 8-bit cache on the GPU at the edges of what the calls allow: references that
move in every page, against the oracle with the bounds of test_paged_gpu.py."""
import numpy as np
import pytest
import torch

import oracle.paged_oracle as po
from bit_kv_cache_25_b200 import vq
from test_paged_gpu import Paged, _q

pytestmark = pytest.mark.gpu


def _rising(D, fmt, pages, step, n, dtype, G=1):
    """A cache whose scores rise by `step` nats from page to page, and queries for it (softmax scale 1)."""
    p = Paged(1, 1, D, fmt, pages, seed=pages)
    p.fill([pages * 64 - 5])
    for j in range(pages):
        page = p.table[0, j]
        c = p.g.integers(-3, 4, (64, D)).astype(np.float64)
        c[:, 0] = 96.0
        p.o["k"][page, 0] = po.encode(c, fmt)
        p.o["k_scale"][page, 0] = step / 96.0 * (j + 1)
    p.push()
    q = _q(p, G, n, dtype, 0.02)
    q[..., 0] = 1.0
    return p, q


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G,pages", [(60, 1, 9), (130, 1, 6), (150, 2, 9)])
def test_a_reference_that_moves_in_every_page(n, G, pages, D, fmt, dtype):
    """Each page's best score passes the one before by more than 8 in log2, so both pages of every key tile move the
    row's reference, and what the first of them stored is rescaled by the second."""
    p, q = _rising(D, fmt, pages, 6.5, n, dtype, G)
    p.attend(q, 1.0)
