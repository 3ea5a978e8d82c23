"""GPU parity of tp_attention_scored against the oracle in 64 bits.

Bound of an output element: every probability is off by its score's error E
(scored_util.score_error) and by half a bf16 step u = 2^-8, the row sum by E
(it is taken before the rounding), and O is rounded once:
    |O - O_ref| <= (u + 2 E) max|v| + u |O_ref|,  max|v| over the keys in sight;
    |LSE - LSE_ref| <= E + 2^-22 |LSE_ref|."""

import numpy as np
import pytest
import torch

import megatron_tensor_sharded_b200 as tp
import scored_util as S
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu


def _run(case, seed=0, poison=None):
    p, T, h, hkv = case["p"], case["T"], case["h"], case["hkv"]
    rng = np.random.default_rng(seed + T)
    std = case.get("std", 1.0)
    (Q, Qh), (K, Kh), (V, Vh) = (S.bf16(rng, p, T, n // p * 128, std=s) for n, s in ((h, std), (hkv, std), (hkv, 1.0)))
    slopes, slopes_h = S.slopes_of(case, h)
    score, seen, inside = S.make_score(case, slopes)
    if poison is not None:
        poison(Q, K, V, inside)
    O, LSE = torch.full_like(Q, 7.0), torch.full((p, h // p, T), 5.0, device="cuda")
    tp.tp_attention_scored(Q, K, V, O, LSE, T, p, h, hkv, 128, score)
    tp.tp_sync_status()
    return (Qh, Kh, Vh), slopes_h, seen, inside, O.double().cpu().numpy(), LSE.double().cpu().numpy()


def _check(case, host, slopes, seen, inside, O, LSE, rows=None, heads=None):
    p, T, hq, hk = case["p"], case["T"], case["h"] // case["p"], case["hkv"] // case["p"]
    Q, K, V = host
    scale, cap = S.case_scale(case), case.get("cap", 0.0)
    rows = inside if rows is None else rows & inside
    for i in range(p):
        for j in range(hq):
            if heads is not None and (i, j) not in heads:
                continue
            q, k, v = S.head(Q, i, j), S.head(K, i, j * hk // hq), S.head(V, i, j * hk // hq)
            sl = slopes[i * hq + j]
            o, lse = A.scored_head(q, k, v, seen, scale, cap, sl)
            E = S.score_error(q, k, scale, cap, sl, T)
            vmax = np.where(seen, np.abs(v).max(1)[None, :], 0.0).max(1, keepdims=True)
            got = S.head(O, i, j)
            tol = (S.U + 2 * E) * vmax + S.U * np.abs(o)
            assert np.all((np.abs(got - o) <= tol)[rows]), (i, j)
            assert np.all((np.abs(LSE[i, j] - lse) <= E + 2.0 ** -22 * np.abs(lse))[rows]), (i, j)
            # the rows of no document are the caller's
            assert np.all(got[~inside] == 7.0) and np.all(LSE[i, j][~inside] == 5.0)


@pytest.mark.parametrize("case", S.CASES, ids=S.IDS)
def test_matches_oracle(case):
    heads = None if case["h"] < 32 else {(0, 0), (0, 9), (0, case["h"] - 1)}
    _check(case, *_run(case), heads=heads)


@pytest.mark.parametrize("case", [
    dict(p=2, T=700, h=96, hkv=48, off=[0, 1, 128, 129, 384, 650], slopes=1.0),
    dict(p=1, T=600, h=64, hkv=64, off=list(range(0, 601, 25)), cap=30.0),
    dict(p=2, T=500, h=128, hkv=64, cap=50.0), dict(p=1, T=130, h=200, hkv=200),
    dict(p=1, T=300, h=120, hkv=8, off=[0, 0, 3, 260], std=3.0)], ids=["docs", "short", "causal", "tiny", "peaked"])
def test_several_units_a_block_of_threads(case):
    """More (head, tile) units than the GPU has SMs, masks in most blocks."""
    last = (case["p"] - 1, case["h"] // case["p"] - 1)
    _check(case, *_run(case), heads={(0, 0), (0, 17), last})


def test_no_options_is_plain_attention():
    p, T, h = 2, 200, 4
    rng = np.random.default_rng(0)
    (Q, _), (K, _), (V, _) = (S.bf16(rng, p, T, h // p * 128) for _ in range(3))
    O = [torch.empty_like(Q) for _ in range(2)]
    tp.tp_attention_scored(Q, K, V, O[0], None, T, p, h, h, 128)
    tp.tp_attention_heads(Q, K, V, O[1], T, p, h, h, 128, False)
    tp.tp_sync_status()
    assert (O[0].float() - O[1].float()).abs().max() <= 2 * S.U * V.float().abs().max()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("case", [
    dict(p=1, T=300, h=2, hkv=1, off=[0, 100, 290], cap=30.0),
    dict(p=1, T=300, h=2, hkv=1, off=[0, 100, 290], slopes=1.0),
    dict(p=1, T=300, h=2, hkv=1, off=[0, 100, 290])], ids=["cap", "bias", "plain"])
def test_what_a_row_does_not_see_adds_nothing(case, value):
    """Garbage in the rows of no document, and one bad key in the middle of a
    document: the rows before it (causal) and the other document are as ever."""
    def poison(Q, K, V, inside):
        out = torch.from_numpy(~inside).cuda()
        for x in (Q, K, V):
            x[:, out] = value
        K[:, 60, 3] = value
        V[:, 60, 100] = value
        V[:, 250] = value

    host, slopes, seen, inside, O, LSE = _run(case, poison=poison)
    fine = inside.copy()
    fine[60:100] = False
    fine[250:290] = False
    _check(case, host, slopes, seen, inside, O, LSE, rows=fine)
    for j in range(2):
        assert not np.isfinite(S.head(O, 0, j)[60:100]).all(1).any()
        assert not np.isfinite(S.head(O, 0, j)[250:290]).all(1).any()


@pytest.mark.parametrize("cap,slopes", [(0.0, 0.0), (30.0, 0.0), (0.0, 1.0), (30.0, 1.0)])
def test_visible_nan_is_not_lost(cap, slopes):
    """A NaN key in every column position of a whole (unmasked) block reaches
    the rows that see it."""
    p, T, h = 1, 384, 1
    rng = np.random.default_rng(1)
    (Q, _), (K, _), (V, _) = (S.bf16(rng, p, T, 128) for _ in range(3))
    sl = torch.tensor([0.01 * slopes], device="cuda") if slopes else None
    for key in list(range(0, 16)) + [64, 127]:
        K2 = K.clone()
        K2[0, key, 5] = float("nan")
        O, LSE = torch.zeros_like(Q), torch.zeros(1, 1, T, device="cuda")
        tp.tp_attention_scored(Q, K2, V, O, LSE, T, p, h, h, 128, tp.score_params(softcap=cap, slopes=sl, causal=True))
        assert torch.isnan(O[0, key:]).all() and torch.isfinite(O[0, :key]).all(), key
        assert torch.isnan(LSE[0, 0, key:]).all()
    tp.tp_sync_status()


def test_offsets_that_lie_are_clamped():
    """Offsets outside [0, T], and decreasing ones: nothing out of range is touched."""
    T = 260
    rng = np.random.default_rng(4)
    (Q, _), (K, _), (V, _) = (S.bf16(rng, 1, T, 128) for _ in range(3))
    for off, pre in (([-50, 100, 10 ** 9], [10 ** 9, 5]), ([200, 100, 50, 260], None), ([300, 400], [0]),
                     ([-2 ** 31, 2 ** 31 - 1], [2 ** 31 - 1])):
        guard = torch.full((3, T, 128), 3.0, device="cuda", dtype=torch.bfloat16)
        mask = S.make_mask(off, pre, True, T)
        tp.tp_attention_scored(Q, K, V, guard[1:2], None, T, 1, 1, 1, 128, tp.score_params(mask=mask))
        tp.tp_sync_status()
        assert (guard[0] == 3).all() and (guard[2] == 3).all() and torch.isfinite(guard.float()).all()
    # clamped to the whole sequence
    ref = torch.empty(1, T, 128, device="cuda", dtype=torch.bfloat16)
    tp.tp_attention_scored(Q, K, V, ref, None, T, 1, 1, 1, 128, tp.score_params(mask=S.make_mask([-50, 10 ** 9], None, True, T)))
    want = torch.empty_like(ref)
    tp.tp_attention_scored(Q, K, V, want, None, T, 1, 1, 1, 128, tp.score_params(causal=True))
    assert torch.equal(ref, want)


def test_same_bits_again_and_on_a_captured_side_stream():
    case = dict(p=1, T=700, h=4, hkv=2, off=[0, 300, 690], cap=30.0)
    T = case["T"]
    rng = np.random.default_rng(9)
    (Q, _), (K, _), (V, _) = (S.bf16(rng, 1, T, n * 128) for n in (4, 2, 2))
    off = torch.tensor(case["off"], dtype=torch.int32, device="cuda")
    n = tp.tp_attention_mask_size(T)
    mask = torch.empty(n, dtype=torch.uint8, device="cuda")
    score = tp.score_params(softcap=30.0, mask=mask)
    outs = [torch.zeros_like(Q) for _ in range(3)]

    def call(out):
        tp.tp_attention_mask(off, 2, None, True, mask, n, T)
        tp.tp_attention_scored(Q, K, V, out, None, T, 1, 4, 2, 128, score)

    call(outs[0])
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        call(outs[1])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])
    off.copy_(torch.tensor([0, 500, 640], dtype=torch.int32))   # other documents under the same graph
    outs[1].zero_()
    g.replay()
    torch.cuda.synchronize()
    call(outs[2])
    assert torch.equal(outs[2], outs[1]) and not torch.equal(outs[0], outs[1])


def test_a_dropped_load_times_out():
    T = 300
    Q = torch.randn(1, T, 128, device="cuda").bfloat16()
    O = torch.empty_like(Q)
    tp.tp_set_wait_timeout_ns(50_000_000)
    try:
        tp.tp_debug_drop_load(1)
        tp.tp_attention_scored(Q, Q, Q, O, None, T, 1, 1, 1, 128, tp.score_params(causal=True))
        with pytest.raises(tp.TPError) as e:
            tp.tp_sync_status()
        assert e.value.name == "TP_ERR_DEVICE_TIMEOUT"
    finally:
        tp.tp_set_wait_timeout_ns(0)
        tp.tp_debug_drop_load(-1)
    tp.tp_attention_scored(Q, Q, Q, O, None, T, 1, 1, 1, 128, tp.score_params(causal=True))
    tp.tp_sync_status()


@pytest.mark.parametrize("case", [dict(p=1, T=300, h=2, hkv=1, off=[0, 100, 290], cap=30.0),
                                  dict(p=1, T=270, h=2, hkv=2, off=[5, 140, 261], slopes=1.0)], ids=["cap", "bias"])
def test_large_values_are_not_taken_for_infinities(case):
    # a factor of 2^90 in V is the same factor in O, bit for bit: products of
    # two such values are beyond bf16 and fp32
    def enlarge(Q, K, V, inside):
        V *= 2.0 ** 90

    inside, O = _run(case)[3:5]
    large = _run(case, poison=enlarge)[4]
    assert np.array_equal(large[:, inside], O[:, inside] * 2.0 ** 90)
