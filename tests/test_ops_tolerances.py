"""The bounds of the GPU tests catch what they are there for: mistakes planted in float64
statements of the operators, on the CPU."""
import numpy as np
import pytest

from oracle import bf16_round, ops

U32 = 2.0 ** -24


def _parts(x, count):
    """x as the sum of its first `count` bf16 parts."""
    x = x.astype(np.float32).astype(np.float64)
    total = np.zeros_like(x)
    for _ in range(count):
        total += bf16_round(x - total)
    return total


def _off(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def _inputs(seed):
    r = np.random.default_rng(seed)
    n, B, H, d = 400, 1, 2, 32
    q, k, v = (_parts(r.standard_normal((n, B, H, d)), 3) for _ in range(3))
    return q, k, v, np.log([0.9, 0.99])


def test_three_parts_hold_an_fp32_value():
    x = np.random.default_rng(0).standard_normal(10000).astype(np.float32)
    assert np.array_equal(_parts(x, 3), x.astype(np.float64))


@pytest.mark.parametrize("lost", ["q", "k", "v"])
def test_a_lost_part_of_a_prompt_is_above_the_bound(lost):
    q, k, v, ld = _inputs(1)
    o, S = ops.linattn(q, k, v, ld)
    cut = {name: _parts(t, 2) if name == lost else t for name, t in (("q", q), ("k", k), ("v", v))}
    o2, S2 = ops.linattn(cut["q"], cut["k"], cut["v"], ld)
    assert _off(o2, o) > 9.7 * U32
    if lost != "q":
        assert _off(S2, S) > 14.6 * U32


def test_a_lost_part_of_a_linear_layer_is_above_the_bound():
    r = np.random.default_rng(2)
    for nin in (512, 8192):
        x, w = _parts(r.standard_normal((20, nin)), 3), _parts(r.standard_normal((30, nin)), 3)
        assert _off(_parts(x, 2) @ w.T, x @ w.T) > (5 + np.sqrt(nin / 128 / 3)) * U32


def test_scores_or_states_of_one_part_are_above_the_bound():
    # results rounded to bf16 once, with and without scores and states rounded to it before
    q, k, v, ld = _inputs(3)
    q, k, v = (bf16_round(t) for t in (q, k, v))
    o, _ = ops.linattn(q, k, v, ld)
    n = q.shape[0]
    lag = np.arange(n)[:, None] - np.arange(n)[None, :]
    rough = np.empty_like(o)
    for h in range(2):
        P = np.where(lag >= 0, np.exp(np.maximum(lag, 0) * ld[h]), 0.0) * (q[:, 0, h] @ k[:, 0, h].T)
        rough[:, 0, h] = bf16_round(P) @ v[:, 0, h]
    bound = 2.0 ** -8 / np.sqrt(3.0) + 2.0 ** -16
    assert _off(bf16_round(o), o) <= bound < _off(bf16_round(rough), o)
