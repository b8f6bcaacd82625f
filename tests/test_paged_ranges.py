"""Borders of the arguments that the paged cache's entry points accept (no GPU): what
vq.h allows passes every check on the host."""

import pytest
import torch

from bit_kv_cache_25_b200 import vq
from test_paged_checks import BAD, INV, _attention, _query, _weights


@pytest.mark.parametrize("kw", [dict(softcap=1e-6), dict(softcap=1e6), dict(softcap=0.0), dict(softmax_scale=1e6),
                                dict(softmax_scale=1e-30), dict(first=BAD), dict(first=BAD, causal=1, prefix=BAD)])
def test_borders_of_queries_are_accepted(kw):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present: the pointers would be followed")
    assert _attention(q=_query(**kw)) == vq.VQ_ERR_CUDA and _weights(q=_query(**kw)) == vq.VQ_ERR_CUDA


@pytest.mark.parametrize("kw", [dict(softcap=9e-7), dict(softcap=1.1e6), dict(softmax_scale=1.1e6)])
def test_what_lies_beyond_is_refused(kw):
    assert _attention(q=_query(**kw)) == INV and _weights(q=_query(**kw)) == INV
