"""Pins of the decoder-layer oracle: hand-worked values and slow restatements in plain Python."""

import math

import numpy as np

from oracle import decode_oracle as D


def test_unpack_order():
    assert D.unpack4(np.array([[0x21, 0xf0]], np.uint8)).tolist() == [[1, 2, 0, 15]]


def test_group_weights_by_hand():
    s = np.array([[0.5, 2.0]], np.float16)
    z = np.array([[1.0, 7.5]], np.float16)
    codes = np.array([[0, 3, 8, 15]])
    assert D.group_weights(codes, s, z, 2).tolist() == [[-0.5, 1.0, 1.0, 15.0]]
    assert D.group_weights(codes - 8, s, None, 2).tolist() == [[-4.0, -2.5, 0.0, 14.0]]


def test_gemm_group_is_a_triple_loop():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 64)).astype(np.float16)
    codes = rng.integers(-8, 8, (3, 64))
    s = rng.uniform(0.01, 0.1, (3, 2)).astype(np.float16)
    y, bound = D.gemm_group(x, codes, s, None, 32)
    for i in range(2):
        for j in range(3):
            want = math.fsum(float(x[i, k]) * float(s[j, k // 32]) * int(codes[j, k]) for k in range(64))
            assert abs(y[i, j] - want) < 1e-12 and bound[i, j] > 0


def test_code_groups_by_hand():
    x = np.array([[-1.0, 0.0, 0.5, 2.0, 3.0, 3.0, 3.0, 3.0]], np.float16)
    u, step, low, val = D.code_groups(x, 4)
    # step 3 / 15 = 0.2 in fp16 (0.199951...), low -1: codes 0, 5, 7.5 -> 8 (0.5 + 1 = 1.5; 1.5 / 0.19995 = 7.502), 15
    assert u.tolist() == [[0, 5, 8, 15, 0, 0, 0, 0]]
    assert float(step[0, 0]) == float(np.float16(0.2)) and step[0, 1] == 0 and low.tolist() == [[-1.0, 3.0]]
    assert val[0, 4:].tolist() == [3.0] * 4 and abs(float(val[0, 3]) - 2.0) < 2e-3


def test_values_are_within_half_a_step():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((50, 128)) * np.exp(rng.standard_normal((50, 1)) * 3)).astype(np.float16)
    u, step, low, val = D.code_groups(x, 32)
    st = np.repeat(step.astype(np.float64), 32, -1)
    # half a step, the rounding of 15 steps to fp16 at the top, and the rounding of the value
    assert (np.abs(val.astype(np.float64) - x) <= st * (0.5 + 15 * 2.0 ** -11) + np.abs(x) * 2.0 ** -10 + 1e-7).all()


def test_norm_and_rotation():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((3, 2, 64)).astype(np.float16)
    w = rng.uniform(0.5, 2, 64).astype(np.float16)
    y = D.head_norm(x, w, 1e-6)
    exact = x.astype(np.float64) / np.sqrt((x.astype(np.float64) ** 2).mean(-1, keepdims=True) + 1e-6) * w
    assert np.allclose(y, exact, rtol=1e-6)
    angle = np.array([0.3, 2.0])[None] * np.arange(5)[:, None]
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    pos = np.array([0, 4, 2])
    for pairs in (False, True):
        z = D.rotate(y, cos, sin, pos, pairs).astype(np.float64)
        assert np.allclose(z[0], y[0], atol=2e-3) and np.allclose(z[..., 4:], y[..., 4:], atol=4e-3)
        a, b = (y[..., 0], y[..., 1]) if pairs else (y[..., 0], y[..., 2])
        turned = (a + 1j * b) * np.exp(1j * 0.3 * pos)[:, None]
        i, j = (0, 1) if pairs else (0, 2)
        assert np.allclose(z[..., i], turned.real, atol=4e-3) and np.allclose(z[..., j], turned.imag, atol=4e-3)


def test_attention_against_loops():
    rng = np.random.default_rng(3)
    codes = rng.integers(0, 256, (4, 2, 1, 16, 32)).astype(np.uint8)
    params = rng.uniform(-0.3, 0.3, (4, 2, 1, 16, 2, 2)).astype(np.float16)
    table = np.array([[2, 0], [3, 1]])
    lens, cu = np.array([19, 1]), np.array([0, 2, 5])
    q = rng.standard_normal((5, 2, 64)).astype(np.float16)
    out, lse, tol, tol_lse = D.attention(q, codes, params, table, lens, cu, 0.2, window=18)

    def value(page, kv, tok, d):
        byte = int(codes[page, kv, 0, tok, d // 2])
        s, lo = params[page, kv, 0, tok, d // 32]
        return float(lo) + float(s) * (byte >> 4 if d % 2 else byte & 15)
    for t, (b, p) in enumerate([(0, 17), (0, 18), (1, -2), (1, -1), (1, 0)]):
        keys = [j for j in range(p + 1) if j > p - 18]
        for h in range(2):
            s = [0.2 * math.fsum(float(q[t, h, d]) * value(table[b, j // 16], 0, j % 16, d) for d in range(64))
                 for j in keys]
            if not keys:
                assert not out[t, h].any() and lse[t, h] == -math.inf
                continue
            total = math.fsum(math.exp(x) for x in s)
            assert abs(lse[t, h] - math.log(total)) < 1e-10
            for d in (0, 31, 63):
                want = math.fsum(math.exp(x) / total * value(table[b, j // 16], 1, j % 16, d) for x, j in zip(s, keys))
                assert abs(out[t, h, d] - want) < 1e-10 and tol[t, h, d] > 0
