"""Rotation plans and the refusals of tp_rope and tp_qk_norm_rope*, without a GPU."""

import ctypes

import numpy as np
import pytest

import megatron_tensor_sharded_b200 as tp
from oracle import attn_oracle as A

A1, A2, A3, A4, A5 = (0x10000000 * i for i in range(1, 6))   # never dereferenced


@pytest.mark.parametrize("scaling", list(tp.ROPE_SCALING))
@pytest.mark.parametrize("r,base,factor,length,low,high", [
    (128, 500000.0, 8.0, 8192.0, 1.0, 4.0), (64, 10000.0, 4.0, 4096.0, 1.0, 32.0),
    (2, 10000.0, 3.0, 512.0, 1.0, 4.0), (18, 77.0, 1.0, 10.0, 0.5, 40.0), (256, 1e6, 16.0, 32768.0, 1.0, 32.0)])
def test_plan_matches_the_formulas(scaling, r, base, factor, length, low, high):
    plan = tp.rope_plan(rotary_dim=r, layout="interleaved", base=base, scaling=scaling,
                        factor=factor, original_len=length, low=low, high=high)
    w = A.rope_frequencies(r, base, scaling, factor, length, low, high)
    got = np.array(list(plan.turn[:r // 2]), dtype=np.longdouble) / np.longdouble(2) ** 64
    want = w / (2 * np.longdouble("3.14159265358979323846264338327950288"))
    assert np.all(np.abs(got - want) <= want * 2.0 ** -50 + np.longdouble(2) ** -63)
    assert list(plan.turn[r // 2:]) == [0] * (128 - r // 2)
    assert (plan.rotary_dim, plan.layout) == (r, 1)
    amp = 0.1 * np.log(factor) + 1 if scaling == "ramp" else 1.0
    assert abs(plan.amplitude - amp) < 1e-6
    assert tp.rope_plan(rotary_dim=r, amplitude=1.25).amplitude == 1.25


def test_plan_refusals():
    def init(**kw):
        a = dict(rotary_dim=64, layout=0, scaling=0, base=1e4, factor=2.0, original_len=100.0, low=1.0,
                 high=4.0, amplitude=0.0)
        a.update(kw)
        return tp.tp_rope_plan_init(tp.RopeConfig(**a), tp.RopePlan(), check=False)

    assert init() == 0
    for bad in (dict(rotary_dim=0), dict(rotary_dim=7), dict(rotary_dim=258), dict(layout=2),
                dict(scaling=5), dict(scaling=-1), dict(base=1.0), dict(base=float("nan")),
                dict(base=float("inf")), dict(scaling=1, factor=0.5), dict(scaling=3, original_len=0.0),
                dict(scaling=3, low=0.0), dict(scaling=4, high=1.0), dict(amplitude=-1.0),
                dict(amplitude=float("nan")), dict(scaling=2, factor=float("inf"))):
        assert init(**bad) == 1, bad
    lib = ctypes.CDLL(tp.LIB_PATH)
    assert lib.tp_rope_plan_init(None, None) == 1


def _rope(**kw):
    a = dict(Q=A1, K=A2, positions=None, Q_out=A3, K_out=A4, T=4, p=2, n_heads=4, n_kv_heads=2,
             head_dim=64, plan=tp.rope_plan(rotary_dim=64), dtype=tp.TP_BF16, stream=0, check=False)
    a.update(kw)
    return tp.tp_rope(**a)


BAD_CALLS = [
    (dict(p=0), 1), (dict(T=-1), 1), (dict(n_heads=0), 1), (dict(n_heads=3), 2),
    (dict(n_kv_heads=5), 2), (dict(head_dim=0), 1), (dict(head_dim=258), 4), (dict(head_dim=62), 1),
    (dict(dtype=7), 1), (dict(Q_out=None), 1), (dict(K=None), 1),
    (dict(Q=None, K=None, Q_out=None, K_out=None), 1), (dict(Q=A1 + 1), 3),
    (dict(dtype=tp.TP_F32, K=A2 + 2), 3), (dict(positions=A5 + 2), 3),
    (dict(Q_out=A1 + 128), 1),         # partly the input
    (dict(Q_out=A2), 1),               # another input's buffer
    (dict(K_out=A3), 1),               # both outputs in one place
    (dict(positions=A3), 1), (dict(T=2 ** 31), 4),
]


@pytest.mark.parametrize("kw,status", BAD_CALLS)
def test_rope_refusals(kw, status):
    assert _rope(**kw) == status


def test_rope_plan_of_the_caller_is_checked():
    assert _rope(plan=None) == 1
    for field, value in (("rotary_dim", 3), ("rotary_dim", 66), ("rotary_dim", 0), ("layout", 9)):
        plan = tp.rope_plan(rotary_dim=64)
        setattr(plan, field, value)
        assert _rope(plan=plan) == 1


def test_nothing_to_do():
    n0 = tp.tp_kernel_launch_count()
    assert _rope(T=0) == 0
    assert tp.tp_qk_norm_rope(None, None, None, None, None, None, None, 0, 1, 1, 1, 64, None, 1e-6,
                              tp.TP_BF16, stream=0, check=False) == 0
    assert tp.tp_kernel_launch_count() == n0


def _norm(**kw):
    a = dict(Q=A1, K=A2, wq=None, wk=None, positions=None, Q_out=A3, K_out=A4, T=4, p=2, n_heads=4,
             n_kv_heads=2, head_dim=64, plan=tp.rope_plan(rotary_dim=64), eps=1e-6,
             dtype=tp.TP_BF16, stream=0, check=False)
    a.update(kw)
    return tp.tp_qk_norm_rope(**a)


@pytest.mark.parametrize("kw,status", BAD_CALLS + [
    (dict(eps=0.0), 1), (dict(eps=float("nan")), 1), (dict(wq=A5 + 1), 3), (dict(wk=A3 + 8), 1)])
def test_norm_refusals(kw, status):
    assert _norm(**kw) == status


def _bwd(**kw):
    a = dict(Q=A1, K=A2, wq=None, wk=None, positions=None, dQ_out=A3, dK_out=A4, dQ=A5, dK=6 * A1,
             dwq=7 * A1, dwk=8 * A1, workspace=9 * A1, workspace_bytes=1 << 22, T=4, p=2, n_heads=4,
             n_kv_heads=2, head_dim=64, plan=tp.rope_plan(rotary_dim=64), eps=1e-6,
             dtype=tp.TP_BF16, stream=0, check=False)
    a.update(kw)
    return tp.tp_qk_norm_rope_backward(**a)


def test_backward_refusals():
    n = tp.tp_qk_norm_rope_backward_workspace_size(4, 2, 4, 2, 64)
    assert n > 0
    assert tp.tp_qk_norm_rope_backward_workspace_size(4, 2, 3, 2, 64) == 0
    assert tp.tp_qk_norm_rope_backward_workspace_size(4, 2, 4, 2, 300) == 0
    for kw, status in ((dict(workspace=None), 7), (dict(workspace_bytes=n - 1), 7),
                       (dict(workspace=9 * A1 + 16), 3), (dict(dQ_out=None), 1), (dict(dK=None), 1),
                       (dict(dwq=7 * A1 + 2), 3), (dict(dwk=7 * A1), 1), (dict(dQ=A1), 1),
                       (dict(dwq=9 * A1), 1), (dict(eps=-1.0), 1), (dict(n_heads=5), 2)):
        assert _bwd(**kw) == status, kw


def test_an_output_in_place_of_two_inputs():
    """In place is one input's buffer; where another input is read there too its
    rows would be overwritten before they are read."""
    for call in (_rope, _norm):
        assert call(K=A1, Q_out=A1) == 1           # Q turned in place, K read from Q
        assert call(K=A1, K_out=A1) == 1
    assert _bwd(dK_out=A3, dQ=A3) == 1
    assert _bwd(Q=A3, dQ=A3) == 1
    assert _bwd(dK_out=A3, dK=A3) == 1


@pytest.mark.parametrize("r,base", [(128, 500000.0), (64, 10000.0), (256, 1e6), (18, 77.0)])
def test_plan_is_rounded_to_the_nearest(r, base):
    """Against 60 decimal digits: half a unit, and 2^-62 of the frequency for the
    power in long double."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    two_pi = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494")
    turn = tp.rope_plan(rotary_dim=r, base=base).turn
    for i in range(r // 2):
        want = Decimal(base) ** (Decimal(-2 * i) / Decimal(r)) / two_pi * 2 ** 64
        assert abs(Decimal(turn[i]) - want) <= Decimal("0.5") + want / 2 ** 62, i
