"""The oracle of the operators on drafted tokens against what must hold of them."""

import numpy as np
import pytest

from oracle import decode_oracle as D
from oracle import draft_oracle as O


def pool(rng, pages, heads, page, d, group):
    u, step, low, _ = D.code_groups(rng.standard_normal((pages, 2, heads, page, d)).astype(np.float16), group)
    return u[..., 0::2] | (u[..., 1::2] << 4), np.stack([step, low], -1)


@pytest.mark.parametrize("window", [0, 9])
def test_a_chain_is_plain_attention(window):
    """Nodes that each follow the one before are new tokens in a row."""
    rng = np.random.default_rng(0)
    codes, params = pool(rng, 5, 2, 16, 64, 32)
    q = rng.standard_normal((7, 4, 64)).astype(np.float16)
    table, lens, cu = np.array([[1, 0, 0], [2, 4, 3]]), [11, 40], [0, 3, 7]
    masks = [np.tril(np.ones((3, 3), bool)), np.tril(np.ones((4, 4), bool))]
    a = D.attention(q, codes, params, table, lens, cu, 0.2, window)
    b = O.tree_attention(q, codes, params, table, lens, cu, masks, 0.2, window)
    for x, y in zip(a, b):
        assert np.allclose(x, y, rtol=1e-12, atol=0)


def test_masks():
    m = O.bits_of([-1, 0, 0, 1, -2, 3])
    assert m.astype(int).tolist() == [[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 0, 1, 0, 0, 0], [1, 1, 0, 1, 0, 0],
                                      [0, 0, 0, 0, 0, 0], [1, 1, 0, 1, 0, 1]]
    assert O.words_of([m], 2)[:, 0].tolist() == [1, 3, 5, 11, 0, 43]
    wide = O.words_of([np.ones((64, 64), bool)], 1)
    assert wide[0, 0] == -1


def test_sample_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.1, 0.3, 0.1]))
    assert [O.sample(x, u)[0] for u in (0.0, 0.05, 0.11, 0.55, 0.75, 0.95)] == [0, 0, 1, 2, 3, 4]
    assert O.sample(x, 0.99, k=2)[0] == 3 and O.sample(x, 0.5, k=2)[0] == 1
    assert O.sample(x, 0.99, k=3)[0] == 3 and O.sample(x, 0.0, k=3)[0] == 0          # of equal ones the lower index
    assert O.sample(x, 0.99, p=0.39)[2] == 1 and O.sample(x, 0.99, p=0.41)[2] == 2
    assert O.sample(x, 0.5, m=0.7)[2] == 2 and O.sample(x, 0.5, m=1.0)[2] == 1
    assert O.sample(x, 0.9, temperature=0.0)[0] == 1
    assert O.sample([-np.inf] * 3, 0.5)[0] == -1
    assert abs(O.sample(x, 0.99, k=2)[1] - np.log(3 / 7)) < 1e-12


def test_accept_by_hand():
    #      0
    #    1   2
    #   3 4   5
    masks = [O.bits_of([-1, 0, 0, 1, 1, 2])]
    tokens = [9, 5, 6, 7, 8, 7]
    codes = np.arange(2 * 2 * 1 * 16 * 32, dtype=np.int64).reshape(1, 2, 2, 1, 16, 32)
    params = np.zeros((1, 2, 2, 1, 16, 1, 2))

    def run(targets):
        c = codes.copy()
        r = O.accept(tokens, targets, masks, [0, 6], [20], [[0, 1]], c, params.copy())
        return r, c
    (path, n, last, lens), c = run([6, 0, 7, 0, 0, 3])
    assert path == [[0, 2, 5]] and n == [3] and last == [3] and lens == [17]
    # places 14, 15, 16: the second and third come from 16 and 19
    assert (c[0, 0, :, :, 15] == codes[0, 1, :, :, 0]).all() and (c[0, 1, :, :, 0] == codes[0, 1, :, :, 3]).all()
    (path, n, last, lens), c = run([1, 2, 3, 4, 5, 6])
    assert path == [[0]] and last == [1] and lens == [15] and (c == codes).all()
