"""The bound that holds fp32 attention to fp32 (cache_bounds.py), on the CPU: fp32 arithmetic in
another order meets it, and inputs with a third of their bits cut off do not."""
import numpy as np
import pytest

import cache_bounds as cb
from oracle import cache_oracle as co


def visible_of(case, causal=True):
    B, H, Hk, Nq, P, S, D, window, sinks, lens = case
    return lambda n: co.visible(n, Nq, S, window, sinks, causal)


def over(case, x, causal=True):
    """How far the call on other inputs x is from the call on the case's own, in bounds."""
    B, H, Hk, Nq, P, S, D, window, sinks, lens = case
    own = cb.inputs(5, B, H, Hk, Nq, P, S, D)
    pre = lambda y: dict(kp=y[3], vp=y[4]) if P else {}  # noqa: E731
    see = visible_of(case, causal)
    o, tol, got, wtol = cb.call(*own[:3], lens, cb.SCALE, see, causal=causal, **pre(own))
    x = x(own)
    o2, _, got2, _ = cb.call(*x[:3], lens, cb.SCALE, see, causal=causal, **pre(x))
    some = wtol > 0
    return (np.abs(o2 - o) / tol).max(), (np.abs(got2 - got)[some] / wtol[some]).max()


@pytest.mark.parametrize("case", cb.SINK[:2] + cb.PREFIX[:1] + cb.CACHE)
def test_inputs_cut_to_16_bits_leave_the_bound(case):
    assert over(case, lambda x: x) == (0.0, 0.0)
    for which in (0, 1, 2):                       # queries, keys, values
        def one_cut(x):
            y = [z.copy() for z in x]
            for i in ((0,), (1, 3), (2, 4))[which]:
                y[i] = cb.cut(y[i], 16)
            return y
        out, weights = over(case, one_cut)
        assert out > 2
        assert which == 2 or weights > 2


def test_the_oracle_gives_the_same():
    for case in cb.SINK[:2] + cb.PREFIX[:1] + cb.CACHE[:2]:
        B, H, Hk, Nq, P, S, D, window, sinks, lens = case
        x = cb.inputs(6, B, H, Hk, Nq, P, S, D)
        pre = dict(kp=x[3], vp=x[4]) if P else {}
        o, _, got, _ = cb.call(*x[:3], lens, cb.SCALE, visible_of(case), **pre)
        want, weights, _ = co.cache_attention(*x[:3], lens, cb.SCALE, window=window, sinks=sinks, **pre)
        assert np.abs(o - want).max() < 1e-12 and np.abs(got - weights).max() < 1e-12


@pytest.mark.parametrize("case", cb.CACHE)
def test_fp32_arithmetic_meets_the_bound(case):
    B, H, Hk, Nq, P, S, D, window, sinks, lens = case
    q, k, v, _, _ = x = cb.inputs(7, B, H, Hk, Nq, P, S, D)
    o, tol, _, _ = cb.call(*x[:3], lens, cb.SCALE, visible_of(case))
    f = np.float32
    for b in range(B):
        see = visible_of(case)(lens[b])
        for h in range(H):
            s = (q[b, h] @ k[b, h * Hk // H].T * f(cb.SCALE)).astype(f)
            s = np.where(see, s, f(-np.inf))
            top = s.max(1, keepdims=True)
            e = np.exp((s - np.where(np.isfinite(top), top, f(0))).astype(f)).astype(f)
            w = (e / np.maximum(e.sum(1, keepdims=True, dtype=f), f(1e-30))).astype(f)
            assert (np.abs((w @ v[b, h * Hk // H]).astype(f) - o[b, h]) <= tol[b, h]).all()
