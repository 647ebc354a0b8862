"""Pins of the prompt and rotation oracle: closed forms, and equality with the decode oracle (CPU)."""

import numpy as np
import pytest

import oracle.attention as OA
import oracle.prompt as OP


def _case(lens, starts, heads=2, kv=1, D=8, seed=0):
    rng = np.random.default_rng(seed)
    pool = rng.normal(size=(9, kv, 16, D)).astype(np.float16)
    vals = rng.normal(size=(9, kv, 16, D)).astype(np.float16)
    tables = np.array([[3, 0, 7], [5, 8, 1]])[:len(lens)]
    q = rng.normal(size=(starts[-1], heads, D)).astype(np.float16)
    return q, pool, vals, tables, np.array(lens), np.array(starts)


def test_each_causal_query_is_a_decode_of_its_own_length():
    q, k, v, tables, lens, starts = _case([20, 37], [0, 20, 25])
    got, bound = OP.attention(q, k, v, tables, lens, starts, 0.4, "f16")
    for s, n in ((0, 20), (1, 5)):
        for i in range(n):
            t = starts[s] + i
            want = OA.paged_attention_decode(q[t:t + 1], k, v, tables[s:s + 1], np.array([lens[s] - n + i + 1]), 0.4, 1, "f16")
            assert np.allclose(got[t], want[0], rtol=1e-12, atol=1e-14)
    assert (bound > 0).all()


@pytest.mark.parametrize("window", [1, 5, 16, 100])
def test_window_is_the_sliding_decode(window):
    q, k, v, tables, lens, starts = _case([40], [0, 7])
    got, _ = OP.attention(q, k, v, tables, lens, starts, 0.4, "f16", window=window)
    for i in range(7):
        want = OA.paged_attention_decode_window(q[i:i + 1], k, v, tables, np.array([34 + i]), 0.4, 1, "f16", window)
        assert np.allclose(got[i], want[0], rtol=1e-12, atol=1e-14)


def test_cross_attention_ignores_order_and_empty_rows_are_zero():
    q, k, v, tables, lens, starts = _case([33, 0], [0, 3, 4])
    got, _ = OP.attention(q, k, v, tables, lens, starts, 0.4, "f16", causal=False)
    assert not got[3].any()
    back, _ = OP.attention(q[[2, 1, 0, 3]], k, v, tables, lens, starts, 0.4, "f16", causal=False)
    assert np.allclose(got[:3], back[[2, 1, 0]])
    # more queries than tokens: those before the first position see nothing
    got, _ = OP.attention(q, k, v, tables, np.array([1, 1]), starts, 0.4, "f16")
    assert not got[:2].any()
    assert np.array_equal(got[2, 0], v[3, 0, 0].astype(float))


def test_prefix_tables_take_the_first_members_blocks():
    tables = np.array([[4, 5, 6], [-1, -1, 7], [1, 2, 3], [9, 9, 8]])
    got = OP.prefix_tables(tables, [0, 2, 4], [2, 1])
    assert got.tolist() == [[4, 5, 6], [4, 5, 7], [1, 2, 3], [1, 9, 8]]


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_turns_pairs_by_the_angle(interleaved):
    rng = np.random.default_rng(1)
    x = rng.normal(size=(5, 3, 32))
    R = 16
    freq = 100.0 ** (-np.arange(R // 2) / (R // 2))
    angle = np.outer(np.arange(50), freq)
    table = np.concatenate((np.cos(angle), np.sin(angle)), 1)
    pos = [0, 7, 7, 49, 3]
    y = OP.rotate(x, pos, table, interleaved)
    assert np.allclose(y[0], x[0]) and np.array_equal(y[..., R:], x[..., R:])
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    # a quarter turn of the pair takes (a, b) to (-b, a)
    quarter = np.concatenate((np.zeros((1, R // 2)), np.ones((1, R // 2))), 1)
    y = OP.rotate(x[:1], [0], quarter, interleaved)
    a, b = (x[0, :, 0], x[0, :, 1]) if interleaved else (x[0, :, 0], x[0, :, R // 2])
    assert np.allclose(y[0, :, 0], -b) and np.allclose(y[0, :, 1 if interleaved else R // 2], a)
    # scores of rotated queries and keys depend on the distance alone
    qk = [(OP.rotate(x[:1], [p], table, interleaved)[0, 0] @ OP.rotate(x[1:2], [p + 4], table, interleaved)[0, 0]) for p in (2, 31)]
    assert np.isclose(*qk)
