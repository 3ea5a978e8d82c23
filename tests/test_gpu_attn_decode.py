"""GPU parity of tp_attention_decode against the oracle in 64 bits: bounds as
in test_gpu_attn_scored (P rounded to bf16 before P V, O once):
    |O - O_ref| <= (u + 2E) max|v| + u |O_ref|,  |LSE - ref| <= E + 2^-22 |ref|."""

import math

import numpy as np
import pytest
import torch

import megatron_tensor_sharded_b200 as tp
import scored_util as S
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu


def _case(p, h, hkv, lens, capacity, cap=0.0, slopes=0.0, append=True, seed=0, std=1.0, garbage=float("nan")):
    """Runs the call on caches whose rows behind each length hold garbage."""
    B = len(lens)
    rng = np.random.default_rng(seed + B + capacity)
    (Q, Qh), (Kn, Knh), (Vn, Vnh) = (S.bf16(rng, p, B, n // p * 128, std=std) for n in (h, hkv, hkv))
    (Kc, Kch), (Vc, Vch) = (S.bf16(rng, p, B, capacity, hkv // p * 128, std=std) for _ in range(2))
    for b, n in enumerate(lens):
        Kc[:, b, max(n, 0):], Vc[:, b, max(n, 0):] = garbage, garbage
    K0, V0 = Kc.clone(), Vc.clone()
    sl, slh = S.slopes_of(dict(slopes=slopes), h)
    O, LSE = torch.full_like(Q, 7.0), torch.full((p, h // p, B), 5.0, device="cuda")
    n = tp.tp_attention_decode_workspace_size(B, capacity, p, h, hkv, 128)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    length = torch.tensor(lens, dtype=torch.int32, device="cuda")
    new = (Kn, Vn) if append else (None, None)
    tp.tp_attention_decode(Q, *new, Kc, Vc, length, O, LSE, ws, n, B, capacity, p, h, hkv, 128,
                           tp.score_params(softcap=cap, slopes=sl))
    status = tp.tp_sync_status(check=False)
    Oh, Lh = O.double().cpu().numpy(), LSE.double().cpu().numpy()
    hq, hk, scale = h // p, hkv // p, 1 / math.sqrt(128)
    for b, n in enumerate(lens):
        fits = 0 <= n and n + append <= capacity
        if append and fits:
            assert torch.equal(Kc[:, b, n], Kn[:, b]) and torch.equal(Vc[:, b, n], Vn[:, b])
            K0[:, b, n], V0[:, b, n] = Kn[:, b], Vn[:, b]
        if not fits:
            assert (O[:, b] == 7).all() and (LSE[..., b] == 5).all()
            continue
        for i in range(p):
            for j in range(hq):
                c = slice(j * hk // hq * 128, j * hk // hq * 128 + 128)
                k, v = Kch[i, b, :n, c], Vch[i, b, :n, c]
                if append:
                    k, v = np.vstack([k, Knh[i, b, c]]), np.vstack([v, Vnh[i, b, c]])
                q = Qh[i, b, j * 128:j * 128 + 128]
                o, lse = A.scored_row(q, k, v, scale, cap, slh[i * hq + j])
                got = Oh[i, b, j * 128:j * 128 + 128]
                if len(k) == 0:
                    assert not got.any() and Lh[i, j, b] == -np.inf
                    continue
                E = S.score_error(q[None], k, scale, cap, slh[i * hq + j], len(k))
                tol = (S.U + 2 * E) * np.abs(v).max() + S.U * np.abs(o)
                assert np.all(np.abs(got - o) <= tol), (b, i, j, n)
                assert abs(Lh[i, j, b] - lse) <= E + 2.0 ** -22 * abs(lse), (b, i, j, n)
    assert torch.equal(Kc.view(torch.int16), K0.view(torch.int16))     # nothing else was written
    assert torch.equal(Vc.view(torch.int16), V0.view(torch.int16))
    return status


@pytest.mark.parametrize("kw", [
    dict(p=1, h=1, hkv=1, lens=[0], capacity=1),
    dict(p=1, h=1, hkv=1, lens=[1], capacity=1, append=False),
    dict(p=1, h=8, hkv=1, lens=[0], capacity=64, append=False),
    dict(p=2, h=4, hkv=2, lens=[0, 1, 15, 16, 17, 63, 64, 65], capacity=80, cap=30.0),
    dict(p=2, h=16, hkv=4, lens=[127, 128, 129, 500, 3, 511], capacity=512, slopes=1.0),
    dict(p=8, h=64, hkv=8, lens=[1000, 4, 700, 1023], capacity=1024, cap=50.0),
    dict(p=1, h=24, hkv=1, lens=[300, 5], capacity=320, cap=20.0, slopes=1.0),     # 24 heads on one key head
    dict(p=1, h=40, hkv=2, lens=[333], capacity=400),
    dict(p=1, h=2, hkv=1, lens=[9000], capacity=9001, std=2.0),                    # one item over many CTAs
    dict(p=1, h=12, hkv=12, lens=[77] * 40, capacity=100, append=False, cap=15.0, std=2.0),
    dict(p=1, h=2, hkv=2, lens=[30] * 300, capacity=33),                           # more sequences than threads
    dict(p=2, h=4, hkv=2, lens=[-1, 40, -5, 0, 20], capacity=64, slopes=1.0),      # unused slots
    dict(p=1, h=4, hkv=4, lens=[0, 0, 0], capacity=16, append=False),
    dict(p=4, h=32, hkv=32, lens=[2000, 1, 1500], capacity=2048, cap=50.0, garbage=float("inf")),
])
def test_matches_oracle(kw):
    assert _case(**kw) == 0


def test_a_length_that_does_not_fit_is_reported():
    assert _case(1, 4, 2, [64, 10, 1000, 63], 64, cap=30.0) == 1
    assert _case(1, 4, 2, [65, 64], 64, append=False) == 1
    assert _case(1, 4, 2, [63, 64], 64, append=False) == 0


def test_a_nan_key_in_sight_is_not_lost():
    for key in (0, 5, 18, 63, 64, 99):
        Q = torch.randn(1, 1, 256, device="cuda").bfloat16()
        Kc, Vc = torch.randn(1, 1, 100, 128, device="cuda").bfloat16(), torch.randn(1, 1, 100, 128, device="cuda").bfloat16()
        Kc[0, 0, key, 7] = float("nan")
        O, n = torch.zeros_like(Q), tp.tp_attention_decode_workspace_size(1, 100, 1, 2, 1, 128)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        for cap in (0.0, 30.0):
            tp.tp_attention_decode(Q, None, None, Kc, Vc, torch.tensor([100], dtype=torch.int32, device="cuda"), O, None,
                                   ws, n, 1, 100, 1, 2, 1, 128, tp.score_params(softcap=cap))
            assert torch.isnan(O).all()
            tp.tp_attention_decode(Q, None, None, Kc, Vc, torch.tensor([key], dtype=torch.int32, device="cuda"), O, None,
                                   ws, n, 1, 100, 1, 2, 1, 128, tp.score_params(softcap=cap))
            assert torch.isfinite(O).all()
    tp.tp_sync_status()


def test_a_step_after_a_prompt_in_one_graph():
    """The operators as a serving step uses them: the prompt's pass fills the
    cache; then norm, rotation and decode of the next tokens, captured once and
    replayed as lengths and positions move on, against the prompt's pass over
    all the tokens."""
    p, h, hkv, T, steps, D = 2, 8, 4, 200, 5, 128
    rng = np.random.default_rng(0)
    total = T + steps
    (Q, _), (K, _), (V, _) = (S.bf16(rng, p, total, n // p * D) for n in (h, hkv, hkv))
    wq, wk = torch.rand(D, device="cuda") + 0.5, torch.rand(D, device="cuda") + 0.5
    plan, pos = tp.rope_plan(rotary_dim=64, base=10000.0), torch.arange(total, dtype=torch.int32, device="cuda")
    sl, _ = S.slopes_of(dict(slopes=0.1), h)
    Qr, Kr, want = torch.empty_like(Q), torch.empty_like(K), torch.empty_like(Q)
    tp.tp_qk_norm_rope(Q, K, wq, wk, pos, Qr, Kr, total, p, h, hkv, D, plan, 1e-6, tp.TP_BF16)
    tp.tp_attention_scored(Qr, Kr, V, want, None, total, p, h, hkv, D, tp.score_params(softcap=30.0, slopes=sl, causal=True))

    capacity = 256
    Kc, Vc = (torch.full((p, 1, capacity, hkv // p * D), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    Kc[:, 0, :T], Vc[:, 0, :T] = Kr[:, :T], V[:, :T]
    q1, k1, v1 = (torch.empty(p, 1, x.shape[2], device="cuda", dtype=torch.bfloat16) for x in (Q, K, V))
    at, out = torch.full((1,), T, dtype=torch.int32, device="cuda"), torch.empty_like(q1)
    n = tp.tp_attention_decode_workspace_size(1, capacity, p, h, hkv, D)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    score = tp.score_params(softcap=30.0, slopes=sl)

    def step():
        tp.tp_qk_norm_rope(q1, k1, wq, wk, at, q1, k1, 1, p, h, hkv, D, plan, 1e-6, tp.TP_BF16)
        tp.tp_attention_decode(q1, k1, v1, Kc, Vc, at, out, None, ws, n, 1, capacity, p, h, hkv, D, score)
        at.add_(1)

    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        step()
    at.fill_(T)
    vmax = V.float().abs().max()
    for i in range(steps):
        for x, y in ((q1, Q), (k1, K), (v1, V)):
            x.copy_(y[:, T + i:T + i + 1])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Kc[:, 0, T + i], Kr[:, T + i])      # the same bits as in the prompt's pass
        assert (out[:, 0].float() - want[:, T + i].float()).abs().max() <= 2 * (2 * S.U) * vmax
    tp.tp_sync_status()
