"""GPU parity of tp_attention_scored_backward against the oracle in 64 bits.

The call is given O (rounded to bf16) and LSE (fp32) of the oracle's own
forward, so only the backward is measured, against the formula with those D and
LSE.  u = 2^-8.  With E the bound of a score's error (scored_util), P is off by
P (2 E + 2^-22 |LSE|), then by u P when it is rounded; dP by 2^-17 sum|dO||v|
(fp32 sums of exact products), D by 2^-17 sum|dO||O|, 1 - t^2 by 2^-18; dS is
rounded by u.  The tile products add in fp32: 2^-13 of the sum of magnitudes is
above their rounding for these lengths.  Every gradient is rounded once:
    |dV - ref| <= (u + 2E + 2^-13) sum_i P |dO_i| + u |dV|
    |dQ - ref| <= scale sum_j err(dS_ij) |k_j| + u |dQ|      (dK likewise),
    err(dS) = P [(u + 2E + 2^-13) |dP - D| + 2^-17 (sum|dO||v| + sum|dO||O|)]
              + 2^-18 P |dP - D|.
Against the true gradient (D and P from exact O and LSE) the error stays within
four roundings (P, dS, O, the result) in the 2-norm: 4 u."""

import numpy as np
import pytest
import torch

import megatron_tensor_sharded_b200 as tp
import scored_util as S
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu


def _forward(case, Q, K, V, seen, slopes):
    p, T, hq, hk = case["p"], case["T"], case["h"] // case["p"], case["hkv"] // case["p"]
    O, LSE = np.zeros_like(Q), np.zeros((p, hq, T))
    for i in range(p):
        for j in range(hq):
            k, v = S.head(K, i, j * hk // hq), S.head(V, i, j * hk // hq)
            o, lse = A.scored_head(S.head(Q, i, j), k, v, seen, S.case_scale(case), case.get("cap", 0.0), slopes[i * hq + j])
            S.head(O, i, j)[:] = o
            LSE[i, j] = lse
    return O, LSE


def _setup(case, seed=0):
    p, T, h, hkv = case["p"], case["T"], case["h"], case["hkv"]
    rng = np.random.default_rng(seed + T)
    std = case.get("std", 1.0)
    dev, host = zip(*(S.bf16(rng, p, T, n // p * 128, std=s) for n, s in ((h, std), (hkv, std), (hkv, 1.0), (h, 1.0))))
    slopes, slopes_h = S.slopes_of(case, h)
    score, seen, inside = S.make_score(case, slopes)
    Q, K, V, dO = host
    O, LSE = _forward(case, Q, K, V, seen, slopes_h)
    O = torch.from_numpy(O).cuda().bfloat16()
    LSE = torch.from_numpy(np.where(inside, LSE, 123.0)).cuda().float()
    return dev, host, slopes_h, score, seen, inside, O, LSE


def _call(case, dev, score, O, LSE):
    p, T, h, hkv = case["p"], case["T"], case["h"], case["hkv"]
    Q, K, V, dO = dev
    g = [torch.full_like(x, 7.0) for x in (Q, K, V)]
    n = tp.tp_attention_scored_backward_workspace_size(T, p, h, hkv, 128)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    tp.tp_attention_scored_backward(Q, K, V, O, LSE, dO, *g, ws, n, T, p, h, hkv, 128, score)
    tp.tp_sync_status()
    return g


def _check(case, host, slopes, seen, inside, O, LSE, grads, rows=None, kv_heads=None):
    p, T, hq, hk = case["p"], case["T"], case["h"] // case["p"], case["hkv"] // case["p"]
    Q, K, V, dO = host
    O, LSE = O.double().cpu().numpy(), LSE.double().cpu().numpy()
    got = [x.double().cpu().numpy() for x in grads]
    scale, cap, group = S.case_scale(case), case.get("cap", 0.0), hq // hk
    rows = inside if rows is None else rows
    u = S.U
    for i in range(p):
        for n in range(hk):
            if kv_heads is not None and (i, n) not in kv_heads:
                continue
            k, v = S.head(K, i, n), S.head(V, i, n)
            sums = [np.zeros((T, 128)) for _ in range(4)]     # dk, dv and their bounds
            for j in range(n * group, n * group + group):
                q, do, o = S.head(Q, i, j), S.head(dO, i, j), S.head(O, i, j)
                sl, lse = slopes[i * hq + j], LSE[i, j][:, None]
                E = 2 * S.score_error(q, k, scale, cap, sl, T) + 2.0 ** -22 * np.abs(np.where(inside[:, None], lse, 0)).max()
                z, t = A.scores(q, k, scale, cap, sl)
                P = np.where(seen, np.exp(np.where(seen, z - lse, 0.0)), 0.0)
                d = do @ v.T - (do * o).sum(1, keepdims=True)
                mag = np.abs(do) @ np.abs(v).T + (np.abs(do) * np.abs(o)).sum(1, keepdims=True)
                f = 1.0 if t is None else 1 - t * t
                rel = u + E + 2.0 ** -13
                dS, err = P * d * f, P * f * (rel * np.abs(d) + 2.0 ** -17 * mag) + 2.0 ** -18 * P * np.abs(d)
                want, tol = scale * dS @ k, scale * err @ np.abs(k)
                a = S.head(got[0], i, j)
                assert np.all((np.abs(a - want) <= tol + u * np.abs(want))[rows & inside]), ("dQ", i, j)
                assert np.all(a[~inside] == 7.0)
                for x, y in zip(sums, (scale * dS.T @ q, P.T @ do, scale * err.T @ np.abs(q), rel * P.T @ np.abs(do))):
                    x += y
            for name, a, want, tol in (("dK", S.head(got[1], i, n), sums[0], sums[2]), ("dV", S.head(got[2], i, n), sums[1], sums[3])):
                assert np.all((np.abs(a - want) <= tol + u * np.abs(want))[rows & inside]), (name, i, n)
                assert np.all(a[~inside] == 7.0)


SMALL = [(c, i) for c, i in zip(S.CASES, S.IDS) if c["h"] < 32]


@pytest.mark.parametrize("case", [c for c, _ in SMALL], ids=[i for _, i in SMALL])
def test_matches_oracle(case):
    dev, host, slopes, score, seen, inside, O, LSE = _setup(case)
    grads = _call(case, dev, score, O, LSE)
    _check(case, host, slopes, seen, inside, O, LSE, grads)
    again = _call(case, dev, score, O, LSE)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


@pytest.mark.parametrize("case", [
    dict(p=1, T=1300, h=16, hkv=2, off=[0, 300, 900, 1290], cap=50.0),
    dict(p=2, T=1100, h=8, hkv=2, cap=30.0), dict(p=1, T=900, h=4, hkv=4, slopes=1.0),
    dict(p=1, T=1500, h=6, hkv=1, causal=False), dict(p=1, T=600, h=8, hkv=8, off=[0, 600], pre=[333], slopes=1.0, cap=20.0)])
def test_forward_then_backward_gives_the_true_gradient(case):
    p, T, h, hkv = case["p"], case["T"], case["h"], case["hkv"]
    dev, host, slopes, score, seen, inside, _, _ = _setup(case, seed=3)
    O, LSE = torch.zeros_like(dev[0]), torch.zeros(p, h // p, T, device="cuda")
    tp.tp_attention_scored(dev[0], dev[1], dev[2], O, LSE, T, p, h, hkv, 128, score)
    got = [x.double().cpu().numpy() for x in _call(case, dev, score, O, LSE)]
    hq, hk = h // p, hkv // p
    want = [np.zeros_like(x) for x in host[:3]]
    for i in range(p):
        for j in range(hq):
            n = j * hk // hq
            g = A.scored_head_backward(S.head(host[0], i, j), S.head(host[1], i, n), S.head(host[2], i, n),
                                       S.head(host[3], i, j), seen, S.case_scale(case), case.get("cap", 0.0), slopes[i * hq + j])
            S.head(want[0], i, j)[:] = g[0]
            S.head(want[1], i, n)[:] += g[1]
            S.head(want[2], i, n)[:] += g[2]
    for a, b in zip(got, want):
        a, b = a[:, inside], b[:, inside]
        assert np.linalg.norm(a - b) <= 4 * S.U * np.linalg.norm(b)


@pytest.mark.parametrize("case", [
    dict(p=2, T=700, h=48, hkv=48, off=[0, 1, 128, 129, 384, 650], slopes=1.0),
    dict(p=1, T=600, h=64, hkv=64, off=list(range(0, 601, 25)), cap=30.0),
    dict(p=2, T=500, h=64, hkv=64, cap=50.0)], ids=["docs", "short", "causal"])
def test_several_units_a_block_of_threads(case):
    """More (head, tile) units than the GPU has SMs, masks in most blocks."""
    dev, host, slopes, score, seen, inside, O, LSE = _setup(case, seed=2)
    grads = _call(case, dev, score, O, LSE)
    last = (case["p"] - 1, case["hkv"] // case["p"] - 1)
    _check(case, host, slopes, seen, inside, O, LSE, grads, kv_heads={(0, 0), (0, 7), last})


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_what_is_not_seen_adds_nothing(value):
    """Garbage in the rows of no document and in one whole document: the other
    document's gradients are as ever."""
    case = dict(p=1, T=400, h=4, hkv=2, off=[0, 150, 310, 390], cap=30.0)
    dev, host, slopes, score, seen, inside, O, LSE = _setup(case)
    broken = ~inside
    broken[150:310] = True
    at = torch.from_numpy(broken).cuda()
    for x in (*dev, O):
        x[:, at] = value
    LSE[..., at] = value
    grads = _call(case, dev, score, O, LSE)
    O, LSE = O.clone(), LSE.clone()
    O[:, at] = 0
    LSE[..., at] = 0
    _check(case, host, slopes, seen, inside, O, LSE, grads, rows=~broken)


def test_a_visible_nan_is_not_lost():
    """One query row's upstream gradient is NaN: dK and dV of every key that
    it sees, and its own dQ; one NaN query row: the same."""
    T = 300
    case = dict(p=1, T=T, h=2, hkv=1, off=[0, T])
    for what in ("dO", "Q"):
        for row in (5, 130, 131, 132, 133, 134, 135, 136, 137, 299):
            dev, host, slopes, score, seen, inside, O, LSE = _setup(case)
            (dev[3] if what == "dO" else dev[0])[0, row, 3] = float("nan")
            dQ, dK, dV = _call(case, dev, score, O, LSE)
            assert torch.isnan(dQ[0, row, :128]).all() and torch.isfinite(dQ[0, :row]).all()
            assert torch.isnan(dK[0, :row + 1]).all() and torch.isfinite(dK[0, row + 1:]).all()
            assert torch.isnan(dV[0, :row + 1, 3]).all() and torch.isfinite(dV[0, row + 1:]).all()


def test_captured_with_the_forward():
    case = dict(p=2, T=500, h=8, hkv=4, cap=50.0, off=[0, 211, 480])
    dev, host, slopes, score, seen, inside, O, LSE = _setup(case)
    T, p, h, hkv = case["T"], case["p"], case["h"], case["hkv"]
    g = [torch.zeros_like(x) for x in dev[:3]]
    n = tp.tp_attention_scored_backward_workspace_size(T, p, h, hkv, 128)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")

    def step():
        tp.tp_attention_scored(dev[0], dev[1], dev[2], O, LSE, T, p, h, hkv, 128, score)
        tp.tp_attention_scored_backward(dev[0], dev[1], dev[2], O, LSE, dev[3], *g, ws, n, T, p, h, hkv, 128, score)

    step()
    want = [x.clone() for x in g]
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=s):
        step()
        for x in g:       # a torch kernel right behind the call sees its results
            x.mul_(2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, 2 * b) for a, b in zip(g, want))


@pytest.mark.parametrize("launch", [0])
def test_a_dropped_load_times_out(launch):
    case = dict(p=1, T=300, h=1, hkv=1, cap=30.0)
    dev, host, slopes, score, seen, inside, O, LSE = _setup(case)
    tp.tp_set_wait_timeout_ns(50_000_000)
    try:
        tp.tp_debug_drop_load(1)
        with pytest.raises(tp.TPError) as e:
            _call(case, dev, score, O, LSE)
        assert e.value.name == "TP_ERR_DEVICE_TIMEOUT"
    finally:
        tp.tp_set_wait_timeout_ns(0)
        tp.tp_debug_drop_load(-1)
    _check(case, host, slopes, seen, inside, O, LSE, _call(case, dev, score, O, LSE))


@pytest.mark.parametrize("case,heads", [
    # 900 key tiles: each CTA takes several whole ones in turn
    (dict(p=1, T=129, h=450, hkv=450, cap=30.0), [(0, 0), (0, 222), (0, 449)]),
    # as many behind a mask, whose empty and short tiles lie on the CTAs' shares
    (dict(p=2, T=270, h=300, hkv=300, off=[3, 4, 130, 131, 260], slopes=1.0), [(0, 0), (0, 77), (1, 149)]),
    # shares of a few steps, each tile's sums on many CTAs
    (dict(p=1, T=600, h=24, hkv=1, slopes=1.0), [(0, 0)]),
], ids=["whole", "mask", "split"])
def test_key_tiles_dealt_to_the_ctas(case, heads):
    dev, host, slopes, score, seen, inside, O, LSE = _setup(case)
    grads = _call(case, dev, score, O, LSE)
    _check(case, host, slopes, seen, inside, O, LSE, grads, kv_heads=heads)
    assert all(torch.equal(a, b) for a, b in zip(grads, _call(case, dev, score, O, LSE)))


@pytest.mark.parametrize("case", [
    dict(p=2, T=1, h=4, hkv=2, slopes=1.0),
    dict(p=1, T=200, h=2, hkv=1, off=list(range(3, 198)), cap=30.0),
    dict(p=1, T=140, h=2, hkv=2, off=[0, 1, 2, 3, 140], causal=False),
], ids=["token", "documents", "some"])
def test_a_query_with_one_key_has_no_gradient(case):
    # softmax of one score is 1 whatever the score: exact zeros, not the rounding of dP - D
    dev, host, slopes, score, seen, inside, O, LSE = _setup(case)
    dQ, dK, dV = _call(case, dev, score, O, LSE)
    one = torch.from_numpy(seen.sum(1) == 1).cuda() & torch.from_numpy(inside).cuda()
    assert one.any() and torch.all(dQ[:, one] == 0)
    alone = one & torch.from_numpy(seen.sum(0) == 1).cuda()
    assert torch.all(dK[:, alone] == 0)
    # an infinite key is still seen
    dev[1][:, one.nonzero()[0, 0]] = float("nan")
    dQ, dK, dV = _call(case, dev, score, O, LSE)
    assert torch.all(torch.isnan(dQ[:, one.nonzero()[0, 0]]))


def test_many_tiles_of_documents():
    """More query tiles than are sorted: a document among many gives what it
    gives alone, O within both calls' roundings (2 u of sum P|v| each), the
    gradients within 8 u in the 2-norm (4 u each, see above)."""
    T, h = 66000, 2
    off = list(range(0, T - 700, 517)) + [T - 30]
    n = len(off) // 2
    rng = np.random.default_rng(3)
    (Q, _), (K, _), (V, _), (dO, _) = (S.bf16(rng, 1, T, w * 128) for w in (h, 1, 1, h))
    slopes = torch.tensor([0.5, 0.03], device="cuda")

    def run(lo, hi, offsets):
        t = hi - lo
        x = [y[:, lo:hi].contiguous() for y in (Q, K, V, dO)]
        size = tp.tp_attention_mask_size(t)
        mask = torch.empty(size, dtype=torch.uint8, device="cuda")
        tp.tp_attention_mask(torch.tensor(offsets, dtype=torch.int32, device="cuda"), len(offsets) - 1, None, True, mask, size, t)
        score = tp.score_params(slopes=slopes, mask=mask, causal=True)
        O, LSE = torch.zeros_like(x[0]), torch.zeros(1, h, t, device="cuda")
        tp.tp_attention_scored(*x[:3], O, LSE, t, 1, h, 1, 128, score)
        g = [torch.zeros_like(y) for y in x[:3]]
        w = tp.tp_attention_scored_backward_workspace_size(t, 1, h, 1, 128)
        tp.tp_attention_scored_backward(*x[:3], O, LSE, x[3], *g, torch.empty(w, dtype=torch.uint8, device="cuda"), w, t, 1, h, 1, 128, score)
        tp.tp_sync_status()
        return O, g

    O, g = run(0, T, off)
    for d in (0, n, len(off) - 2):
        lo, hi = off[d], off[d + 1]
        O1, g1 = run(lo, hi, [0, hi - lo])
        assert (O[:, lo:hi].float() - O1.float()).abs().max() <= 4 * S.U * V.float().abs().max()
        for a, b in zip(g, g1):
            a, b = a[:, lo:hi].double(), b.double()
            assert (a - b).norm() <= 8 * S.U * b.norm()
    assert all(torch.all(x[:, T - 30:] == 0) for x in [O] + g)


def test_two_calls_at_once():
    """On two streams, each with its own workspace and outputs: the bits of the
    calls one after the other."""
    cases = [dict(p=1, T=700, h=8, hkv=2, cap=50.0), dict(p=2, T=520, h=8, hkv=4, off=[0, 130, 470], slopes=1.0)]
    sets = [_setup(c) for c in cases]
    alone = [_call(c, s[0], s[3], s[6], s[7]) for c, s in zip(cases, sets)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for c, s, st in zip(cases, sets, streams):
        p, T, h, hkv = c["p"], c["T"], c["h"], c["hkv"]
        with torch.cuda.stream(st):
            g = [torch.full_like(x, 7.0) for x in s[0][:3]]
            n = tp.tp_attention_scored_backward_workspace_size(T, p, h, hkv, 128)
            ws = torch.empty(n, dtype=torch.uint8, device="cuda")
            for _ in range(4):
                tp.tp_attention_scored_backward(*s[0][:3], s[6], s[7], s[0][3], *g, ws, n, T, p, h, hkv, 128, s[3])
        got.append((g, ws))
    torch.cuda.synchronize()
    tp.tp_sync_status()
    for a, (g, _) in zip(alone, got):
        assert all(torch.equal(x, y) for x, y in zip(a, g))


@pytest.mark.parametrize("case", [
    dict(p=1, T=2300, h=20, hkv=20, causal=False, cap=30.0),
    dict(p=2, T=2300, h=20, hkv=4, off=[0, 2200]),
], ids=["full", "causal"])
def test_long_runs_of_blocks_that_no_mask_cuts(case):
    """Many key blocks of one query tile in a row that are seen whole, several
    such tiles a CTA: every wait ends, and the same bits again and again."""
    dev, host, slopes, score, seen, inside, O, LSE = _setup(case)
    grads = _call(case, dev, score, O, LSE)
    _check(case, host, slopes, seen, inside, O, LSE, grads, kv_heads={(0, 0)})
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(grads, _call(case, dev, score, O, LSE)))


@pytest.mark.parametrize("case", [
    dict(p=1, T=300, h=4, hkv=2, off=list(range(0, 301, 2))), dict(p=1, T=300, h=4, hkv=2, off=list(range(0, 301, 3)), cap=30.0),
    dict(p=1, T=290, h=2, hkv=2, off=list(range(0, 280, 7)) + [285], slopes=1.0),
    dict(p=1, T=200, h=2, hkv=1, off=list(range(0, 201, 20)), causal=False, std=2.0)], ids=["twos", "threes", "sevens", "peaked"])
def test_short_documents_against_the_true_gradient(case):
    """Forward, then backward, element by element against the gradient from exact
    O and LSE.  Beside the bound at the top, D is off by what O is:
    sum_d |dO_d| ((u + 2E) max_j|v_jd| + u |O_d|) in every dS of the row, times P f."""
    p, T, h, hkv = case["p"], case["T"], case["h"], case["hkv"]
    dev, host, slopes, score, seen, inside, _, _ = _setup(case, seed=4)
    O, LSE = torch.zeros_like(dev[0]), torch.zeros(p, h // p, T, device="cuda")
    tp.tp_attention_scored(dev[0], dev[1], dev[2], O, LSE, T, p, h, hkv, 128, score)
    got = [x[0].double().cpu().numpy() for x in _call(case, dev, score, O, LSE)]
    Q, K, V, dO = host
    scale, cap, u, group = S.case_scale(case), case.get("cap", 0.0), S.U, h // hkv
    for n in range(hkv):
        k, v = S.head(K, 0, n), S.head(V, 0, n)
        vmax = np.where(seen[:, :, None], np.abs(v)[None], 0.0).max(1)
        want, tol = [np.zeros((T, 128)) for _ in range(2)], [np.zeros((T, 128)) for _ in range(2)]
        for j in range(n * group, n * group + group):
            q, do, sl = S.head(Q, 0, j), S.head(dO, 0, j), slopes[j]
            E = 2 * S.score_error(q, k, scale, cap, sl, T)
            z, t = A.scores(q, k, scale, cap, sl)
            o, lse = A.scored_head(q, k, v, seen, scale, cap, sl)
            E += 2.0 ** -22 * np.abs(np.where(inside, lse, 0)).max()
            P = np.where(seen, np.exp(np.where(seen, z - np.where(inside, lse, 0.0)[:, None], 0.0)), 0.0)
            d = do @ v.T - (do * o).sum(1, keepdims=True)
            mag = np.abs(do) @ np.abs(v).T + (np.abs(do) * np.abs(o)).sum(1, keepdims=True)
            off = (np.abs(do) * ((u + E) * vmax + u * np.abs(o))).sum(1, keepdims=True)
            f = 1.0 if t is None else 1 - t * t
            rel = u + E + 2.0 ** -13
            dS = P * d * f
            err = P * f * (rel * np.abs(d) + 2.0 ** -17 * mag + (1 + rel) * off) + 2.0 ** -18 * P * np.abs(d)
            dq, bound = scale * dS @ k, scale * err @ np.abs(k)
            assert np.all((np.abs(got[0][:, j * 128:j * 128 + 128] - dq) <= bound + u * np.abs(dq))[inside]), ("dQ", j)
            for x, y in zip(want + tol, (scale * dS.T @ q, P.T @ do, scale * err.T @ np.abs(q), rel * P.T @ np.abs(do))):
                x += y
        for name, a, w, b in (("dK", got[1], want[0], tol[0]), ("dV", got[2], want[1], tol[1])):
            a = a[:, n * 128:n * 128 + 128]
            assert np.all((np.abs(a - w) <= b + u * np.abs(w))[inside]), (name, n)
