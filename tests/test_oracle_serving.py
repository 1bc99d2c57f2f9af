"""Pins of the plain forms of the serving operators: closed cases worked by
hand, and cases where they must reduce to the pinned base operators."""
import numpy as np
import pytest

import oracle
from oracle import serving


def rng_i8(r, *shape):
    return r.integers(-128, 128, shape, dtype=np.int8)


@pytest.fixture(scope="module", autouse=True)
def built():
    oracle.build()


@pytest.mark.parametrize("rounding", [0, 1])
def test_no_adapter_is_the_base_layer(rounding):
    r = np.random.default_rng(1)
    X, W = rng_i8(r, 6, 32), rng_i8(r, 48, 32)
    bias = r.integers(-5000, 5000, 48, dtype=np.int32)
    b, c = r.integers(0, 1 << 20, 48, dtype=np.int32), r.integers(20, 31, 48).astype(np.int8)
    ad = (rng_i8(r, 2, 16, 32), np.full((2, 16), 1 << 20, np.int32), np.full((2, 16), 28, np.int8), rng_i8(r, 2, 48, 16))
    skip = rng_i8(r, 6, 48)
    for idx in ([-1, 2, 7], [-5, 100, 2]):
        got = serving.linear_lora(X, W, bias, b, c, ad, idx, 2, 7, skip, (3, 2, 2), rounding)
        np.testing.assert_array_equal(got, oracle.linear_requant(X, W, bias, b, c, 7, skip, (3, 2, 2), rounding))


def test_exact_adapter_is_the_merged_weight():
    """With t = X A^T exact (b_t = 1, c_t = 0, small values), X W^T + t B^T = X (W + B A)^T."""
    r = np.random.default_rng(2)
    X, W = r.integers(-2, 3, (8, 32), dtype=np.int8), r.integers(-20, 21, (16, 32), dtype=np.int8)
    A, B = r.integers(-1, 2, (3, 16, 32), dtype=np.int8), r.integers(-2, 3, (3, 16, 16), dtype=np.int8)
    ad = (A, np.ones((3, 16), np.int32), np.zeros((3, 16), np.int8), B)
    b, c = np.full(16, 3, np.int32), np.full(16, 4, np.int8)
    got = serving.linear_lora(X, W, None, b, c, ad, [2, 0, 1, 2], 2)
    for q, a in enumerate([2, 0, 1, 2]):
        merged = W.astype(np.int64) + B[a].astype(np.int64) @ A[a].astype(np.int64)
        assert np.abs(merged).max() <= 127
        want = oracle.linear_requant(X[2 * q:2 * q + 2], merged.astype(np.int8), None, b, c)
        np.testing.assert_array_equal(got[2 * q:2 * q + 2], want)


def test_adapter_requant_saturates_and_floors():
    """One rank entry by hand: t = sat_8((3 * 100 * 100) >> 4) = 127, and (3 * -7) >> 2 = -6 (floor)."""
    X = np.zeros((2, 16), np.int8)
    X[0, 0], X[1, 0] = 100, -7
    A = np.zeros((1, 16, 16), np.int8)
    B = np.zeros((1, 16, 16), np.int8)
    W = np.zeros((16, 16), np.int8)
    one, zero = np.ones(16, np.int32), np.zeros(16, np.int8)
    B[0, 5, 0] = 1
    A[0, 0, 0] = 100
    ad = (A, np.full((1, 16), 3, np.int32), np.full((1, 16), 4, np.int8), B)
    assert serving.linear_lora(X, W, None, one, zero, ad, [0], 2)[0, 5] == 127
    A[0, 0, 0] = 1
    ad = (A, np.full((1, 16), 3, np.int32), np.full((1, 16), 2, np.int8), B)
    assert serving.linear_lora(X, W, None, one, zero, ad, [0], 2)[1, 5] == -6
    # round half up: (-21 + 2) >> 2 = -5
    assert serving.linear_lora(X, W, None, one, zero, ad, [0], 2, rounding=1)[1, 5] == -5


def test_branch_end_by_hand():
    skip = np.full((2, 16), 10, np.int8)
    branch = np.full((2, 16), -3, np.int8)
    gate = np.full((1, 16), 4, np.int8)
    scale = np.full(16, -5, np.int32)
    y, z = serving.residual_norm(skip, branch, scale, 7, 3, gate=gate, gate_rows=2)
    assert z is None and (y == ((7 * 10 + (-5) * (-3) * 4) >> 3)).all()       # 130 >> 3 = 16
    y, _ = serving.residual_norm(skip, branch, -scale, 7, 3, gate=gate, gate_rows=2)
    assert (y == ((70 - 60) >> 3)).all()
    y, _ = serving.residual_norm(skip, branch, scale * 1000, 7, 0)
    assert (y == 127).all()


def test_branch_end_with_unit_scales_is_two_norms():
    r = np.random.default_rng(3)
    x = rng_i8(r, 5, 48)
    g, be = rng_i8(r, 48), r.integers(-9000, 9000, 48, dtype=np.int32)
    post, pre = (g, be, 7, 23, (3, 9)), (g[::-1].copy(), be, 5, 20, (1, 6))
    zero = np.zeros_like(x)
    y, z = serving.residual_norm(zero, x, np.ones(48, np.int32), 0, 0, post=post, pre=pre)
    n = oracle.layernorm(x, *post)
    np.testing.assert_array_equal(y, n)
    np.testing.assert_array_equal(z, oracle.layernorm(n, *pre))


def test_zero_weight_is_plain_attention():
    """lam = 0: each half of V attends with the first map alone, as ivit_attention's heads do."""
    r = np.random.default_rng(4)
    B, N, H = 2, 21, 2
    qkv = rng_i8(r, B * N, 3 * 128 * H)
    args = ((1 << 20, 31), 8, 9, 30, 8)
    got = serving.attention_diff(qkv, B, N, H, *args, np.zeros(H, np.int32), (1, 4))
    t = qkv.reshape(B * N, 3, H, 2, 64)
    for half in range(2):
        one = np.stack((t[:, 0, :, 0], t[:, 1, :, 0], t[:, 2, :, half]), 1).reshape(B * N, 3 * H * 64)
        want = oracle.attention(one, B, N, H, *args, (1, 4)).reshape(B * N, H, 64)
        np.testing.assert_array_equal(got.reshape(B * N, H, 2, 64)[:, :, half], want)


def test_equal_maps_with_full_weight_cancel():
    r = np.random.default_rng(5)
    qkv = rng_i8(r, 9, 3, 1, 2, 64)
    qkv[:, :2, :, 1] = qkv[:, :2, :, 0]
    args = ((1 << 20, 31), 8, 9, 30, 8)
    ctx = serving.attention_diff(qkv.reshape(9, -1), 1, 9, 1, *args, np.array([1 << 30]), (1, 0))
    assert not ctx.any()


def test_maps_by_hand():
    """I0 = 4: ShiftExp(0) = 4, ShiftExp(-4): Ip = -4 - 2 + 1 = -5 = -(1 * 4 + 1), (4 - 1) >> 1 = 1."""
    p1, p2 = serving.diff_maps([[0, -4]], [[3, 3]], 4, 10, 8, 512)
    assert p1.tolist() == [[(1024 // 5 * 4) >> 3, (1024 // 5) >> 3]]
    assert p2.tolist() == [[(512 // 8 * 4) >> 3] * 2]
    assert serving.diff_maps([[0]], [[0]], 4, 10, 8, 5000)[1].tolist() == [[128]]   # lam clamped to 2^M
    assert serving.diff_maps([[0]], [[0]], 4, 10, 8, -3)[1].tolist() == [[0]]
