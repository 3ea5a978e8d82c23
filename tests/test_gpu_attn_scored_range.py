"""Scored attention at the ends of its inputs' range, against the oracle in 64
bits with the bounds of test_gpu_attn_scored."""

import numpy as np
import pytest
import torch

from test_gpu_attn_scored import _check, _run

pytestmark = pytest.mark.gpu

BIG = 255 * 2.0 ** 120      # the largest bf16

OPTIONS = [dict(), dict(slopes=1.0), dict(cap=30.0), dict(cap=30.0, slopes=1.0), dict(cap=200.0)]
NAMES = ["plain", "bias", "cap", "both", "large-cap"]


@pytest.mark.parametrize("opts", OPTIONS, ids=NAMES)
@pytest.mark.parametrize("mask,bad,fine", [
    (dict(causal=True), (200, 300), (0, 200)),                           # later tokens
    (dict(off=[0, 100, 290]), (100, 300), (0, 100)),                     # the next document, and none
    (dict(off=[0, 100, 290]), (0, 100), (100, 290)),                     # the document before
    (dict(off=[0, 140, 290], causal=False), (140, 300), (0, 140)),
    (dict(off=[0, 250], pre=[60]), (200, 300), (0, 200)),
], ids=["later", "next", "before", "full", "prefix"])
def test_unseen_finite_values_add_nothing(mask, bad, fine, opts):
    """Keys and values of the largest size, of either sign, where a row does not
    see them: a probability of 2^-126 instead of 0 would add 3 to its sum."""
    case = dict(p=1, T=300, h=2, hkv=1, **mask, **opts)

    def poison(Q, K, V, inside):
        K[:, bad[0]:bad[1]] = BIG
        K[:, bad[0] + 1:bad[1]:2] = -BIG
        V[:, bad[0]:bad[1], :64] = BIG
        V[:, bad[0]:bad[1], 64:] = -BIG

    host, slopes, seen, inside, O, LSE = _run(case, poison=poison)
    rows = np.zeros(300, bool)
    rows[fine[0]:fine[1]] = True
    _check(case, host, slopes, seen, inside, O, LSE, rows=rows)
