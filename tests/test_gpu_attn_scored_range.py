"""Scored attention at the ends of its inputs' range, against the oracle in 64
bits with the bounds of test_gpu_attn_scored."""

import numpy as np
import pytest
import torch

import megatron_tensor_sharded_b200 as tp
import scored_util as S
from oracle import attn_oracle as A
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


@pytest.mark.parametrize("at", [1, 70, 128, 200, 299])
def test_later_tokens_add_nothing_to_plain_heads(at):
    """tp_attention_heads, causal, with the largest finite keys and values from
    token `at` on."""
    p, T, h, hkv = 1, 300, 2, 1
    rng = np.random.default_rng(at)
    (Q, Qh), (K, Kh), (V, Vh) = (S.bf16(rng, p, T, n * 128) for n in (h, hkv, hkv))
    K[:, at:], V[:, at:] = -BIG, BIG
    O = torch.zeros_like(Q)
    tp.tp_attention_heads(Q, K, V, O, T, p, h, hkv, 128, True)
    tp.tp_sync_status()
    for j in range(h):
        q, k, v = S.head(Qh, 0, j), S.head(Kh, 0, 0), S.head(Vh, 0, 0)
        want, _ = A.scored_head(q, k, v, np.tri(T, dtype=bool), 128 ** -0.5)
        E = S.score_error(q, k, 128 ** -0.5, 0.0, 0.0, T)
        tol = (S.U + 2 * E) * np.abs(v).max() + S.U * np.abs(want)
        assert np.all((np.abs(O[0, :, j * 128:j * 128 + 128].double().cpu().numpy() - want) <= tol)[:at])


@pytest.mark.parametrize("slope", [0.0, 0.01], ids=["plain", "bias"])
@pytest.mark.parametrize("key", [0, 2, 4, 15, 16, 19, 40, 131])
def test_infinite_scores(key, slope):
    """A key whose score is +inf: softmax is NaN and the log of the sum +inf in
    the rows that see it; one whose score is -inf has no weight, whatever its
    value."""
    T = 200
    rng = np.random.default_rng(key)
    (Q, Qh), (K, Kh), (V, Vh) = (S.bf16(rng, 1, T, 128) for _ in range(3))
    Q[0, :, 5], Qh[0, :, 5] = 1.0, 1.0
    sl = torch.tensor([slope], device="cuda") if slope else None
    score = tp.score_params(slopes=sl, causal=True)
    for value in (np.inf, -np.inf):
        K2, V2 = K.clone(), V.clone()
        K2[0, key, 5] = value
        V2[0, key] = 1.0 if value > 0 else BIG
        O, LSE = torch.zeros_like(Q), torch.zeros(1, 1, T, device="cuda")
        tp.tp_attention_scored(Q, K2, V2, O, LSE, T, 1, 1, 1, 128, score)
        tp.tp_sync_status()
        O, LSE = O[0].double().cpu().numpy(), LSE[0, 0].double().cpu().numpy()
        seen = np.tri(T, dtype=bool)
        rows = np.arange(T) < key if value > 0 else np.arange(T) != key
        if value > 0:
            assert np.isnan(O[key:]).all() and (LSE[key:] == np.inf).all()
        else:
            seen[:, key] = False
            if key == 0:
                assert LSE[0] == -np.inf
        want, lse = A.scored_head(Qh[0], Kh[0], Vh[0], seen, 128 ** -0.5, 0.0, slope)
        E = S.score_error(Qh[0], Kh[0], 128 ** -0.5, 0.0, slope, T)
        tol = (S.U + 2 * E) * np.abs(Vh).max() + S.U * np.abs(want)
        assert np.all((np.abs(O - want) <= tol)[rows])
        assert np.all(np.abs(LSE[rows] - lse[rows]) <= E + 2.0 ** -22 * np.abs(lse[rows]))


def _lse_bound(q, k, scale, z):
    """Of one row's log of the sum: the products' sums, then 2^-20 of the scores
    (the cap's arithmetic is relative to the score, not to the cap)."""
    return 2.0 ** -17 * scale * (np.abs(k) @ np.abs(q)).max() + 2.0 ** -20 * np.abs(z).max() + 2.0 ** -18


@pytest.mark.parametrize("cap", [1e3, 1e4, 1e6])
def test_scores_far_below_the_cap(cap):
    """Prompt and single token: what is lost of a small score does not grow
    with the cap; nor beside scores that are near it."""
    T = 150
    rng = np.random.default_rng(7)
    (Q, Qh), (K, Kh), (V, Vh) = (S.bf16(rng, 1, T, 128) for _ in range(3))
    peak = 77                       # one query and one key whose product is about the cap
    Q[0, peak], K[0, peak] = 0, 0
    Q[0, peak, 0], K[0, peak, 0] = 1.0, 11.3 * cap
    Q[0, :peak, 0] = 0
    Q[0, peak + 1:, 0] = 0
    Qh, Kh = Q.double().cpu().numpy(), K.double().cpu().numpy()
    O, LSE = torch.zeros_like(Q), torch.zeros(1, 1, T, device="cuda")
    tp.tp_attention_scored(Q, K, V, O, LSE, T, 1, 1, 1, 128, tp.score_params(softcap=cap, causal=True))
    n = tp.tp_attention_decode_workspace_size(T, T, 1, 1, 1, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    cache = [x[:, None].expand(1, T, T, 128).contiguous() for x in (K, V)]
    lengths = torch.arange(1, T + 1, dtype=torch.int32, device="cuda")
    O1, LSE1 = torch.zeros_like(Q), torch.zeros(1, 1, T, device="cuda")
    tp.tp_attention_decode(Q, None, None, *cache, lengths, O1, LSE1, ws, n, T, T, 1, 1, 1, 128,
                           tp.score_params(softcap=cap))
    tp.tp_sync_status()
    for name, o, lse in (("prompt", O, LSE), ("token", O1, LSE1)):
        o, lse = o[0].double().cpu().numpy(), lse[0, 0].double().cpu().numpy()
        for i in range(T):
            want, l = A.scored_row(Qh[0, i], Kh[0, :i + 1], Vh[0, :i + 1], 128 ** -0.5, cap)
            z = cap * np.tanh(128 ** -0.5 * (Kh[0, :i + 1] @ Qh[0, i]) / cap)
            E = _lse_bound(Qh[0, i], Kh[0, :i + 1], 128 ** -0.5, z)
            assert abs(lse[i] - l) <= E + 2.0 ** -22 * abs(l), (name, i)
            tol = (S.U + 2 * E) * np.abs(Vh).max() + S.U * np.abs(want)
            assert np.all(np.abs(o[i] - want) <= tol), (name, i)


@pytest.mark.parametrize("cap,ratio,size", [(50.0, 9.9e5, 0.0), (50.0, 9.9e5, 1e-4), (1.0, 9e5, 1e-3), (1e6, 9e5, 0.0),
                                            (1e6, 1.1e-9, 6000.0), (1e-3, 1.1e-9, 6000.0), (1e-3, 9e5, 1e-4),
                                            (30.0, 1e-8, 2000.0)])
@pytest.mark.parametrize("slope", [0.0, 0.01])
def test_scale_over_cap_at_the_ends_of_its_range(cap, ratio, size, slope):
    """Rows of zeros and rows whose scores lie around the cap."""
    T, scale = 140, cap * ratio
    rng = np.random.default_rng(2)
    (Q, Qh), (K, Kh) = (S.bf16(rng, 1, T, 128, std=size) for _ in range(2))
    V, Vh = S.bf16(rng, 1, T, 128)
    Q[0, 3], Qh[0, 3] = 0, 0
    sl = torch.tensor([slope], device="cuda") if slope else None
    O, LSE = torch.zeros_like(Q), torch.zeros(1, 1, T, device="cuda")
    score = tp.score_params(scale=scale, softcap=cap, slopes=sl, causal=True)
    scale = float(score.scale)          # as fp32
    tp.tp_attention_scored(Q, K, V, O, LSE, T, 1, 1, 1, 128, score)
    dO, _ = S.bf16(rng, 1, T, 128)
    g = [torch.zeros_like(x) for x in (Q, K, V)]
    n = tp.tp_attention_scored_backward_workspace_size(T, 1, 1, 1, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    tp.tp_attention_scored_backward(Q, K, V, O, LSE, dO, *g, ws, n, T, 1, 1, 1, 128, score)
    n = tp.tp_attention_decode_workspace_size(T, T, 1, 1, 1, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    cache = [x[:, None].expand(1, T, T, 128).contiguous() for x in (K, V)]
    O1, LSE1 = torch.zeros_like(Q), torch.zeros(1, 1, T, device="cuda")
    tp.tp_attention_decode(Q, None, None, *cache, torch.arange(1, T + 1, dtype=torch.int32, device="cuda"), O1, LSE1,
                           ws, n, T, T, 1, 1, 1, 128, score)
    tp.tp_sync_status()
    assert all(torch.isfinite(x).all() for x in g)
    want, lse = A.scored_head(Qh[0], Kh[0], Vh[0], np.tri(T, dtype=bool), scale, cap, slope)
    for name, o, l in (("prompt", O, LSE), ("token", O1, LSE1)):
        o, l = o[0].double().cpu().numpy(), l[0, 0].double().cpu().numpy()
        for i in range(T):
            x = scale * (Kh[0, :i + 1] @ Qh[0, i])
            z = cap * np.tanh(x / cap) - slope * np.arange(i, -1, -1)
            # the products' rounding as far as the cap's derivative lets it through
            mag = 2.0 ** -17 * scale * (np.abs(Kh[0, :i + 1]) @ np.abs(Qh[0, i]))
            near = np.maximum(np.abs(x) - mag, 0)
            E = (mag / np.cosh(np.minimum(near / cap, 300.0)) ** 2).max() + 2.0 ** -20 * np.abs(z).max() + 2.0 ** -18
            assert abs(l[i] - lse[i]) <= E + 2.0 ** -22 * abs(lse[i]), (name, i)
            tol = (S.U + 2 * E) * np.abs(Vh).max() + S.U * np.abs(want[i])
            assert np.all(np.abs(o[i] - want[i]) <= tol), (name, i)


@pytest.mark.parametrize("cap,slopes", [(50.0, 0.0), (55.0, 0.0), (50.0, 1e-3), (60.0, 0.0)])
@pytest.mark.parametrize("side", [1.0, -1.0])
def test_range_of_v(cap, slopes, side):
    """Every score next to +-cap: V as large as the sums allow (within a factor
    of four) and, at -cap, as small as keeps its digits."""
    p, T, h = 1, 300, 1
    rng = np.random.default_rng(3)
    (Q, Qh), (K, Kh) = (S.bf16(rng, p, T, 128, std=0.01) for _ in range(2))
    Q[..., 0], K[..., 0] = 64.0, side * 64.0        # scale q.k = +-362, tanh = 1 but for 2^-17
    Qh, Kh = Q.double().cpu().numpy(), K.double().cpu().numpy()
    log2w = cap / np.log(2) if cap <= 55 and not slopes else 8.0
    for log2v in (np.floor(128 - log2w - np.log2(4 * T) - 2), np.ceil(-126 + log2w + 4)):
        V, Vh = S.bf16(rng, p, T, 128)
        V, Vh = V * 2.0 ** log2v, Vh * 2.0 ** log2v
        sl = torch.tensor([slopes], device="cuda") if slopes else None
        O, LSE = torch.zeros_like(Q), torch.zeros(1, 1, T, device="cuda")
        tp.tp_attention_scored(Q, K, V, O, LSE, T, p, h, h, 128, tp.score_params(softcap=cap, slopes=sl, causal=True))
        tp.tp_sync_status()
        want, lse = A.scored_head(Qh[0], Kh[0], Vh[0], np.tri(T, dtype=bool), 128 ** -0.5, cap, slopes)
        # (the cap leaves nothing of the products' rounding)
        E = 2.0 ** -20 * cap + 2.0 ** -22 * slopes * T + 2.0 ** -18
        vmax = np.maximum.accumulate(np.abs(Vh[0]).max(1))[:, None]
        assert np.all(np.abs(O[0].double().cpu().numpy() - want) <= (S.U + 2 * E) * vmax + S.U * np.abs(want))
        assert np.all(np.abs(LSE[0, 0].double().cpu().numpy() - lse) <= E + 2.0 ** -22 * np.abs(lse))


@pytest.mark.parametrize("opts", OPTIONS, ids=NAMES)
@pytest.mark.parametrize("mask,broken", [
    (dict(off=[7, 75, 190, 470, 600], causal=True), None), (dict(off=[30, 331, 560], causal=False), None),
    (dict(off=[11, 590], pre=[140], causal=True), None), (dict(off=[0, 75, 190, 470, 640], causal=True), (75, 190)),
    (dict(off=[0, 231, 390], causal=False), (231, 390))], ids=["documents", "full", "prefix", "document", "second"])
def test_the_bits_do_not_depend_on_time_nor_garbage(mask, broken, opts):
    """Forward and backward with each kind of garbage in the rows of no document:
    the same bits each time, and without a cap those that zeros there give (with
    one the columns of a warp choose the cap's form together).  The same with
    garbage in a document, whose rows see it."""
    p, T, h, hkv = 2, 640, 8, 4
    case = dict(mask, **opts)
    rng = np.random.default_rng(5)
    Q, K, V, dO = (S.bf16(rng, p, T, n // p * 128)[0] for n in (h, hkv, hkv, h))
    slopes, _ = S.slopes_of(case, h)
    offsets = mask["off"]
    out = torch.ones(T, dtype=torch.bool, device="cuda")
    out[offsets[0]:offsets[-1]] = False
    if broken:
        out[broken[0]:broken[1]] = True
    plan = S.make_mask(offsets, mask.get("pre"), mask["causal"], T)
    score = tp.score_params(softcap=case.get("cap", 0.0), slopes=slopes, mask=plan)
    n = tp.tp_attention_scored_backward_workspace_size(T, p, h, hkv, 128)

    def run(value):
        x = [t.clone() for t in (Q, K, V, dO)]
        for t in x:
            t[:, out] = value
        O, LSE = torch.zeros_like(Q), torch.zeros(p, h // p, T, device="cuda")
        tp.tp_attention_scored(*x[:3], O, LSE, T, p, h, hkv, 128, score)
        g = [torch.zeros_like(t) for t in x[:3]]
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
        tp.tp_attention_scored_backward(*x[:3], O, LSE, x[3], *g, ws, n, T, p, h, hkv, 128, score)
        tp.tp_sync_status()
        return [t[:, ~out] for t in [O] + g] + [LSE[..., ~out]]

    want = run(0.0)
    assert all(torch.isfinite(t).all() for t in want)
    for value in (float("nan"), float("inf"), -float("inf"), BIG, -BIG):
        if broken or "cap" in case:
            want = run(value)
            assert all(torch.isfinite(t).all() for t in want)
        for _ in range(20):
            assert all(torch.equal(a, b) for a, b in zip(run(value), want)), value


@pytest.mark.parametrize("cap", [0.0, 30.0, 200.0])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_visible_key_that_is_not_finite_reaches_its_queries(value, cap):
    """dQ of the queries that see it, each time, where a mask cuts the block and
    where none does, with O and LSE that are finite."""
    T, key = 300, 40
    rng = np.random.default_rng(1)
    Q, K, V, dO = (S.bf16(rng, 1, T, 128)[0] for _ in range(4))
    score = tp.score_params(softcap=cap, causal=True)
    O, LSE = torch.zeros_like(Q), torch.zeros(1, 1, T, device="cuda")
    tp.tp_attention_scored(Q, K, V, O, LSE, T, 1, 1, 1, 128, score)
    K[0, key, 3] = value
    n = tp.tp_attention_scored_backward_workspace_size(T, 1, 1, 1, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    for _ in range(10):
        dQ, dK, dV = (torch.zeros_like(x) for x in (Q, K, V))
        tp.tp_attention_scored_backward(Q, K, V, O, LSE, dO, dQ, dK, dV, ws, n, T, 1, 1, 1, 128, score)
        tp.tp_sync_status()
        # (0 or a rounding of it times an infinity: NaN or infinite)
        assert not torch.isfinite(dQ[0, key:, 3]).any() and torch.isfinite(dQ[0, :key]).all()
