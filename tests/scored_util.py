"""Inputs and bounds shared by the scored-attention tests."""

import math

import numpy as np
import torch

import megatron_tensor_sharded_b200 as tp
from oracle import attn_oracle as A

U = 2.0 ** -8            # bf16: half a step, relative


def bf16(rng, *shape, std=1.0):
    t = torch.from_numpy((std * rng.standard_normal(shape)).astype(np.float32)).cuda().bfloat16()
    return t, t.double().cpu().numpy()


def head(x, i, j):
    """Head j of shard i of [p][T][heads * 128]."""
    return x[i][:, j * 128:(j + 1) * 128]


def score_error(q, k, scale, cap, slope, T):
    """Bound of one score's error: the tensor core's fp32 sum of 128 exact bf16
    products (128 * 2^-24 of the sum of magnitudes), the cap's polynomial and
    roundings (8e-7 < 2^-20 of the cap), the bias's roundings (2^-22 of it),
    and the exponent's own (its argument and approximation: 2^-18)."""
    mag = (np.abs(q) @ np.abs(k).T).max() if len(q) else 0.0
    return 2.0 ** -17 * scale * mag + 2.0 ** -20 * cap + 2.0 ** -22 * abs(slope) * T + 2.0 ** -18


def make_mask(offsets, prefix, causal, T):
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    pre = None if prefix is None else torch.tensor(prefix, dtype=torch.int32, device="cuda")
    n = tp.tp_attention_mask_size(T)
    mask = torch.full((n,), 0xAB, dtype=torch.uint8, device="cuda")
    tp.tp_attention_mask(off, len(offsets) - 1, pre, causal, mask, n, T)
    return mask


def make_score(case, slopes=None):
    """(ScoreParams, visible [T, T], inside [T]) of a case dict."""
    T = case["T"]
    off, pre, causal = case.get("off"), case.get("pre"), case.get("causal", True)
    mask = make_mask(off, pre, causal, T) if off is not None else None
    score = tp.score_params(scale=case.get("scale", 0.0), softcap=case.get("cap", 0.0), slopes=slopes,
                            mask=mask, causal=causal)
    return (score, *A.visible(T, causal, off, pre))


def slopes_of(case, h):
    if not case.get("slopes"):
        return None, np.zeros(h)
    s = np.array([2.0 ** (-8.0 * (i + 1) / h) * case["slopes"] for i in range(h)], np.float32)
    return torch.from_numpy(s).cuda(), s.astype(np.float64)


def case_scale(case):
    return case.get("scale", 0.0) or 1 / math.sqrt(128)


# The sizes and masks where it can go wrong: one token, one past a tile, short
# tails, several units a CTA, grouped heads; empty, one-token and tile-crossing
# documents, tokens in none; prefixes of nothing, of part, of more than all.
CASES = [
    dict(p=1, T=1, h=1, hkv=1),
    dict(p=1, T=1, h=2, hkv=1, cap=30.0),
    dict(p=2, T=129, h=4, hkv=4, cap=20.0),
    dict(p=2, T=300, h=4, hkv=2, cap=50.0, causal=False),
    dict(p=1, T=257, h=2, hkv=1, slopes=1.0),
    dict(p=1, T=385, h=2, hkv=2, slopes=1.0, causal=False),
    dict(p=1, T=300, h=2, hkv=1, slopes=-0.02, cap=10.0),
    dict(p=1, T=300, h=2, hkv=2, cap=200.0, std=4.0),          # a cap past the bound: with a maximum
    dict(p=1, T=200, h=2, hkv=1, cap=2.0, std=2.0),            # scores far beyond the cap
    dict(p=1, T=260, h=2, hkv=2, std=3.0, scale=0.25),         # peaked scores, a scale of its own
    dict(p=1, T=300, h=2, hkv=1, off=[0, 100, 100, 101, 290], cap=30.0),
    dict(p=2, T=700, h=4, hkv=2, off=[0, 1, 128, 129, 384, 650], slopes=1.0),
    dict(p=1, T=520, h=2, hkv=1, off=[0, 10, 200, 520], causal=False),
    dict(p=1, T=400, h=2, hkv=1, off=[7, 130, 131, 390], pre=[50, 3, 1000], cap=30.0),
    dict(p=1, T=300, h=2, hkv=1, off=[0, 300], pre=[200]),
    dict(p=1, T=300, h=2, hkv=1, off=[0, 300], pre=[-5], slopes=1.0),
    dict(p=1, T=140, h=1, hkv=1, off=[0, 0, 0]),               # every row in no document
    dict(p=1, T=900, h=3, hkv=1, off=[0, 600, 610], cap=15.0), # whole tiles in no document
    dict(p=1, T=64, h=1, hkv=1, off=list(range(65))),          # documents of one token
    dict(p=8, T=383, h=16, hkv=8, off=[0, 200, 380], slopes=1.0, cap=40.0),
    dict(p=4, T=1500, h=8, hkv=4, cap=50.0),
    dict(p=1, T=1300, h=64, hkv=8, off=[0, 300, 900, 1290], cap=50.0),
    dict(p=1, T=1300, h=40, hkv=8),
]
IDS = ["-".join("%s=%s" % (k, v if not isinstance(v, list) else len(v)) for k, v in c.items()) for c in CASES]
