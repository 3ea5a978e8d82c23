"""GPU parity of rotary positions, head norms with the rotation and their
backward against the oracle in 64 bits.

Tolerances (u = 2^-8 for bf16 outputs, 2^-24 for fp32).  Rotation: the angle
enters sincospi as an fp32 fraction of a half turn (off by at most pi 2^-25
rad), sine and cosine are off by at most 2 ulp (2^-23), each product and the
sum by 2^-24 of the terms; together below 2^-21 a (|x1| + |x2|), then one
rounding u |y|.  Norm: the sum of squares adds 16 terms a lane and log2(lanes)
more, all positive, so rstd is off by less than 16 * 2^-24 + the
approximation's 2^-22: below 2^-19 relative; with the weight and the rotation
below 2^-18 of the terms.  Backward: dx = rstd (g w - xhat m): g is off by
2^-21 (|g1| + |g2|), m by (dh) terms of either sign, at most
2^-18 mean|g w xhat|; together below 2^-17 rstd (|g1 w| + |g2 w| + |xhat| mean|g w xhat|).
dw: sums of products that are off by 2^-18 of themselves, added in chains of
at most 2^10 (2^-14 of the sum of magnitudes is far above that)."""

import numpy as np
import pytest
import torch

import megatron_tensor_sharded_b200 as tp
from oracle import attn_oracle as A

pytestmark = pytest.mark.gpu

EPS = 1e-5
U = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}

# p, T, h, h_kv, head_dim, rotary_dim, layout, scaling, dtype, offset
CASES = [
    (1, 1, 1, 1, 2, 2, "half", "none", "f32", 0),
    (1, 3, 2, 1, 6, 4, "interleaved", "none", "bf16", 0),
    (2, 5, 4, 2, 64, 64, "half", "bands", "bf16", 0),
    (2, 130, 12, 12, 64, 32, "interleaved", "linear", "bf16", 0),
    (4, 300, 8, 4, 128, 128, "half", "ramp", "bf16", 0),
    (8, 1030, 64, 8, 128, 128, "half", "bands", "bf16", 0),
    (8, 700, 64, 8, 128, 128, "interleaved", "base", "bf16", 0),
    (1, 33, 3, 1, 256, 96, "half", "none", "f32", 0),
    (1, 70, 5, 5, 250, 250, "half", "none", "bf16", 0),
    (1, 70, 2, 1, 256, 130, "interleaved", "none", "f32", 0),
    (2, 513, 4, 2, 96, 48, "half", "ramp", "f32", 0),
    (2, 65, 4, 2, 80, 80, "half", "none", "bf16", 1),        # buffers off their 16 bytes
    (3, 41, 9, 3, 128, 54, "half", "none", "bf16", 0),
    (1, 4100, 8, 2, 128, 64, "interleaved", "none", "bf16", 0),
]


def _plan_args(r, scaling):
    return dict(base=10000.0, scaling=scaling, factor=4.0, original_len=2048.0, low=1.0,
                high=32.0 if scaling == "ramp" else 4.0)


def _tensor(rng, shape, dtype, offset):
    """Values on the device at `offset` elements from a 256-byte boundary, and in 64 bits."""
    n = int(np.prod(shape))
    buf = torch.empty(n + offset, dtype=TORCH[dtype], device="cuda")
    t = buf[offset:].view(shape)
    t.copy_(torch.from_numpy(rng.standard_normal(shape).astype(np.float32)))
    return t, t.double().cpu().numpy()


def _setup(case, seed=0):
    p, T, h, hkv, D, r, layout, scaling, dtype, off = case
    rng = np.random.default_rng(seed + T)
    Q, Qh = _tensor(rng, (p, T, h // p * D), dtype, off)
    K, Kh = _tensor(rng, (p, T, hkv // p * D), dtype, off)
    pos = rng.integers(-50, 3_000_000, T).astype(np.int32)
    pos[0] = 2 ** 31 - 1 if T > 1 else 7
    pos[-1] = -2 ** 31 if T > 2 else pos[-1]
    plan = tp.rope_plan(rotary_dim=r, layout=layout, **_plan_args(r, scaling))
    a = _plan_args(r, scaling)
    w = A.rope_frequencies(r, **a)
    return Q, K, Qh, Kh, pos, torch.from_numpy(pos).cuda(), plan, w


def _heads(x, D):
    return x.reshape(x.shape[0], x.shape[1], -1, D)


def _others(x, r, layout):
    """|x1| + |x2| at both elements of each pair, |x| at the others."""
    y = np.abs(x)
    n = r // 2
    a, b = (slice(0, n), slice(n, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    s = y[..., a] + y[..., b]
    y[..., a] = s
    y[..., b] = s
    return y


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_rope(case, inverse):
    p, T, h, hkv, D, r, layout, scaling, dtype, off = case
    Q, K, Qh, Kh, pos, dpos, plan, w = _setup(case)
    Qo, Ko = (torch.full_like(x, float("nan")) for x in (Q, K))
    if off:
        Qo, Ko = (torch.empty(x.numel() + off, dtype=x.dtype, device="cuda")[off:].view(x.shape) for x in (Q, K))
    tp.tp_rope(Q, K, dpos, Qo, Ko, T, p, h, hkv, D, plan, tp.DTYPE[dtype], inverse)
    tp.tp_sync_status()
    for got, x in ((Qo, Qh), (Ko, Kh)):
        got = _heads(got.double().cpu().numpy(), D)
        for i in range(p):
            xi = _heads(x, D)[i]
            want = A.rope_rotate(xi, pos, w, layout, plan.amplitude, inverse)
            tol = U[dtype] * np.abs(want) + 2.0 ** -21 * plan.amplitude * _others(xi, r, layout)
            assert np.all(np.abs(got[i] - want) <= tol)
    # in place, and one tensor alone: the same bits
    Q2 = Q.clone() if not off else Q
    tp.tp_rope(Q2, None, dpos, Q2, None, T, p, h, 0, D, plan, tp.DTYPE[dtype], inverse)
    tp.tp_sync_status()
    assert torch.equal(Q2, Qo)


def test_positions_default_to_the_token_index():
    p, T, h, D = 2, 37, 4, 128
    Q = torch.randn(p, T, h // p * D, device="cuda").bfloat16()
    plan = tp.rope_plan(rotary_dim=D)
    a, b = torch.empty_like(Q), torch.empty_like(Q)
    tp.tp_rope(Q, None, None, a, None, T, p, h, 0, D, plan, tp.TP_BF16)
    tp.tp_rope(Q, None, torch.arange(T, device="cuda", dtype=torch.int32), b, None, T, p, h, 0, D, plan, tp.TP_BF16)
    assert torch.equal(a, b)
    assert torch.equal(a[:, 0], Q[:, 0])


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_norm_rope_and_backward(case, weights):
    p, T, h, hkv, D, r, layout, scaling, dtype, off = case
    Q, K, Qh, Kh, pos, dpos, plan, w = _setup(case, seed=1)
    rng = np.random.default_rng(5)
    wts = [1 + 0.3 * rng.standard_normal(D).astype(np.float32) for _ in range(2)]
    dw = [torch.from_numpy(x).cuda() if weights else None for x in wts]
    hw = [x.astype(np.float64) if weights else None for x in wts]
    if T > 2:
        Q[0, 1] = 0          # a head of zeros: eps alone
        Qh[0, 1] = 0
    Qo, Ko = torch.full_like(Q, float("nan")), torch.full_like(K, float("nan"))
    tp.tp_qk_norm_rope(Q, K, dw[0], dw[1], dpos, Qo, Ko, T, p, h, hkv, D, plan, EPS, tp.DTYPE[dtype])
    dQo, dQoh = _tensor(rng, tuple(Q.shape), dtype, off)
    dKo, dKoh = _tensor(rng, tuple(K.shape), dtype, off)
    dQ, dK = torch.full_like(Q, float("nan")), torch.full_like(K, float("nan"))
    gw = [torch.full((D,), float("nan"), device="cuda") for _ in range(2)]
    n = tp.tp_qk_norm_rope_backward_workspace_size(T, p, h, hkv, D)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    args = (Q, K, dw[0], dw[1], dpos, dQo, dKo)
    tail = (ws, n, T, p, h, hkv, D, plan, EPS, tp.DTYPE[dtype])
    tp.tp_qk_norm_rope_backward(*args, dQ, dK, gw[0], gw[1], *tail)
    tp.tp_sync_status()
    for y, x, dy, dx, g, wt in ((Qo, Qh, dQoh, dQ, gw[0], hw[0]), (Ko, Kh, dKoh, dK, gw[1], hw[1])):
        y, dx = (_heads(t.double().cpu().numpy(), D) for t in (y, dx))
        sum_w, mag_w = np.zeros(D), np.zeros(D)
        for i in range(p):
            xi, gi = _heads(x, D)[i], _heads(dy, D)[i]
            normed = A.head_norm(xi, wt, EPS)
            want = A.rope_rotate(normed, pos, w, layout, plan.amplitude)
            tol = U[dtype] * np.abs(want) + 2.0 ** -18 * plan.amplitude * _others(normed, r, layout)
            assert np.all(np.abs(y[i] - want) <= tol)
            back = A.rope_rotate(gi, pos, w, layout, plan.amplitude, inverse=True)
            want, dwi = A.head_norm_backward(xi, wt, back, EPS)
            rms = np.sqrt((xi * xi).mean(-1, keepdims=True) + EPS)
            xhat, gmag = np.abs(xi / rms), plan.amplitude * _others(gi, r, layout)
            gmag_w = gmag * (1.0 if wt is None else np.abs(wt))
            tol = U[dtype] * np.abs(want) + 2.0 ** -17 / rms * (
                gmag_w + xhat * (gmag_w * xhat).mean(-1, keepdims=True))
            assert np.all(np.abs(dx[i] - want) <= tol)
            sum_w += dwi
            mag_w += (gmag * xhat).sum((0, 1))
        assert np.all(np.abs(g.double().cpu().numpy() - sum_w) <= 2.0 ** -14 * mag_w)
    # the gradient in its upstream's place, weights' gradients again: the same bits
    if not off:
        q2, k2, g2 = dQo.clone(), dKo.clone(), [torch.empty_like(x) for x in gw]
        tp.tp_qk_norm_rope_backward(Q, K, dw[0], dw[1], dpos, q2, k2, q2, k2, g2[0], g2[1], *tail)
        tp.tp_sync_status()
        assert torch.equal(q2, dQ) and torch.equal(k2, dK)
        assert torch.equal(g2[0], gw[0]) and torch.equal(g2[1], gw[1])


def test_norm_alone_one_tensor_and_no_tokens():
    T, h, D = 50, 4, 128
    K = torch.randn(1, T, h * D, device="cuda").bfloat16()
    wk, out = torch.rand(D, device="cuda") + 0.5, torch.empty_like(K)
    tp.tp_qk_norm_rope(None, K, None, wk, None, None, out, T, 1, 0, h, D, None, EPS, tp.TP_BF16)
    want = A.head_norm(_heads(K.double().cpu().numpy(), D)[0], wk.double().cpu().numpy(), EPS)
    got = _heads(out.double().cpu().numpy(), D)[0]
    assert np.all(np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -18) * np.abs(want))
    g = torch.full((D,), 3.0, device="cuda")
    tp.tp_qk_norm_rope_backward(None, None, None, None, None, None, None, None, None, g, None, None,
                                0, 0, 1, h, h, D, None, EPS, tp.TP_BF16)
    tp.tp_sync_status()
    assert torch.count_nonzero(g).item() == 0


def test_captured_and_replayed_on_a_side_stream():
    p, T, h, hkv, D = 2, 64, 4, 2, 128
    Q, K = torch.randn(p, T, h // p * D, device="cuda"), torch.randn(p, T, hkv // p * D, device="cuda")
    plan, pos = tp.rope_plan(rotary_dim=D), torch.arange(T, device="cuda", dtype=torch.int32)
    Qo, Ko = torch.empty_like(Q), torch.empty_like(K)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(g, stream=s):
        tp.tp_qk_norm_rope(Q, K, None, None, pos, Qo, Ko, T, p, h, hkv, D, plan, EPS, tp.TP_F32)
        tp.tp_rope(Qo, Ko, pos, Qo, Ko, T, p, h, hkv, D, plan, tp.TP_F32, inverse=True)
    for _ in range(2):
        Q.normal_()
        pos.add_(100000)
        g.replay()
        torch.cuda.synchronize()
        want = A.head_norm(_heads(Q.double().cpu().numpy(), D)[1], None, EPS)
        assert np.allclose(_heads(Qo.double().cpu().numpy(), D)[1], want, atol=2e-5)


def test_as_many_tokens_as_int32_counts():
    """2^31 - 1 tokens of one head of two elements: forward and backward at the
    first and the last tokens."""
    T, D = 2 ** 31 - 1, 2
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 27 GB")
    w = torch.tensor([1.5, -0.5], device="cuda")
    x, dy = (torch.empty(T * D, dtype=torch.bfloat16, device="cuda").normal_() for _ in range(2))
    y = torch.zeros_like(x)
    plan, freq = tp.rope_plan(rotary_dim=D, base=10000.0), A.rope_frequencies(D, 10000.0)
    tp.tp_qk_norm_rope(x, None, w, None, None, y, None, T, 1, 1, 0, D, plan, EPS, tp.TP_BF16)
    n = tp.tp_qk_norm_rope_backward_workspace_size(T, 1, 1, 0, D)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    dx = torch.zeros_like(x)
    tp.tp_qk_norm_rope_backward(x, None, w, None, None, dy, None, dx, None, None, None, ws, n, T, 1, 1, 0, D, plan,
                                EPS, tp.TP_BF16)
    tp.tp_sync_status()
    for lo in (0, 2 ** 30 - 7, T - 5000):
        at = slice(lo * D, (lo + 5000) * D)
        xh, dyh = (t[at].double().cpu().numpy().reshape(-1, 1, D) for t in (x, dy))
        pos, wh = np.arange(lo, lo + 5000), w.double().cpu().numpy()
        normed = A.head_norm(xh, wh, EPS)
        want = A.rope_rotate(normed, pos, freq)
        tol = U["bf16"] * np.abs(want) + 2.0 ** -18 * _others(normed, D, "half")
        assert np.all(np.abs(y[at].double().cpu().numpy().reshape(want.shape) - want) <= tol)
        want, _ = A.head_norm_backward(xh, wh, A.rope_rotate(dyh, pos, freq, inverse=True), EPS)
        rms = np.sqrt((xh * xh).mean(-1, keepdims=True) + EPS)
        g, xhat = _others(dyh, D, "half") * np.abs(wh), np.abs(xh / rms)
        tol = U["bf16"] * np.abs(want) + 2.0 ** -17 / rms * (g + xhat * (g * xhat).mean(-1, keepdims=True))
        assert np.all(np.abs(dx[at].double().cpu().numpy().reshape(want.shape) - want) <= tol)
