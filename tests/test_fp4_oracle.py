"""The plain 4-bit forms against what the format fixes."""
import numpy as np
import pytest

import oracle
from oracle import fp4 as F
from paged_kv_attention_fwd_gb300 import workloads as W


def test_grid_values_and_ties():
    # a block whose largest magnitude is 6 with head scale 1 has scale 1: the
    # elements are rounded to the grid themselves
    x = np.zeros((1, 16), np.float32)
    x[0, :10] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.75, -5.0]
    codes, byte = F.encode(x, 1.0)
    assert oracle.e4m3_to_f64(byte)[0, 0] == 1.0
    assert codes[0, :10].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8 + 2, 8 + 6]  # ties to the even code
    assert not codes[0, 10:].any()


@pytest.mark.parametrize("head", [1.0, 0.37, 3e-3])
def test_error_is_at_most_half_a_step(head):
    x = W.normal_f32(3, 1, 64 * 128).reshape(64, 128)
    codes, byte = F.encode(x, head)
    s = np.repeat(oracle.e4m3_to_f64(byte), 16, -1) * np.float32(head)
    n = codes.astype(int)
    v = np.where(n >= 8, -1, 1) * F.GRID[n & 7] * s
    # the widest gap of the grid is 2; a scale rounded down by up to 2^-4 lets 6 stand for up to 6 (1 + 2^-4)
    assert (np.abs(v - x) <= s * 1.0 + 1e-12).all()
    small = np.abs(x) <= 2 * s
    assert (np.abs(v - x)[small] <= 0.25 * s[small] * (1 + 1e-6)).all()


def test_zero_nan_and_infinite_blocks():
    x = np.ones((4, 16), np.float32)
    x[0] = 0
    x[1, 3] = np.nan
    x[2, 5] = -np.inf
    x[3] = 1e-30
    codes, byte = F.encode(x, 1.0)
    assert byte[0, 0] == 0 and not codes[0].any()
    assert byte[1, 0] == 0x7F and not codes[1].any()
    assert byte[2, 0] == 0x7E and codes[2, 5] == 15  # -6 * 448
    assert byte[3, 0] == 0 and not codes[3].any()


def test_pool_round_trip_and_append():
    d, hk = 64, 3
    head = np.array([0.01, 1.0, 5.0], np.float32)
    x = W.normal_f32(5, 2, 4 * hk * 64 * d).reshape(4, hk, 64, d)
    pool = F.make_pool(x, head)
    assert pool.shape == (4, hk, 64 * (d // 2 + d // 16))
    v = F.decode_pool(pool, head, d)
    assert np.abs(v - x).max() < 0.6 and np.corrcoef(v.ravel(), x.ravel())[0, 1] > 0.98
    again = F.make_pool(v.astype(np.float32), head)  # stored values read back and stored again do not move
    assert np.allclose(F.decode_pool(again, head, d), v, rtol=1e-6, atol=0)
    # writing the same rows token by token gives the same pool
    bits = W.f32_to_bf16_bits(x)
    table = np.array([[2, 0], [3, 1]], np.int32)
    rows = np.concatenate([bits[2].transpose(1, 0, 2), bits[0].transpose(1, 0, 2), bits[3].transpose(1, 0, 2),
                           bits[1].transpose(1, 0, 2)])
    got = F.append(rows, np.array([0, 128, 256]), [0, 0], table, np.zeros_like(pool), head, d)
    assert np.array_equal(got, F.make_pool(oracle.bf16_to_f64(bits), head))


def test_attend_is_the_mean_of_equal_scores():
    d = 64
    k = np.zeros((2, 1, 64, d))
    v = np.random.default_rng(0).standard_normal((2, 1, 64, d))
    q = W.f32_to_bf16_bits(np.ones((1, 2, d), np.float32))
    out, lse, *_ = F.attend(q, k, v, np.array([[1, 0]]), [100], 0.1)
    want = np.concatenate([v[1, 0], v[0, 0]])[:100].mean(0)
    assert np.allclose(out[0], want) and np.allclose(lse, np.log(100))


def test_norm_rope_turns_and_keeps_length():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 2, 64))
    angle = np.arange(9)[:, None] * 0.3 ** np.arange(16)
    cs = np.concatenate([np.cos(angle), np.sin(angle)], -1)
    pos = np.array([[0, 1, 2, 3, 8]])
    for inter in (False, True):
        y, _ = F.norm_rope(x, None, pos, cs, 32, inter, [16], 0.0)
        assert np.allclose((y ** 2).mean(-1), 1)  # unit mean square, and the rotation keeps it
        assert np.allclose(y[0], x[0] / np.sqrt((x[0] ** 2).mean(-1, keepdims=True)))  # position 0 does not turn
    # the product of a query and a key depends on the distance alone
    a, b = rng.standard_normal((1, 1, 64)), rng.standard_normal((1, 1, 64))
    dot = lambda i, j: float((F.norm_rope(a, None, np.array([[i]]), cs, 32, False, [16], 0.0, norm=False)[0]
                              * F.norm_rope(b, None, np.array([[j]]), cs, 32, False, [16], 0.0, norm=False)[0]).sum())
    assert np.isclose(dot(7, 5), dot(4, 2))
