"""The acceptance of a branch on the GPU against the oracle: paths, tokens, lengths and every byte of the caches."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import quantized_mixed_precision_gb300 as bq  # noqa: E402
from oracle import draft_oracle as O  # noqa: E402
from tests.test_gpu_attn_tree import random_tree, tree_tensor  # noqa: E402
from tests.test_gpu_parity import dev, host  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bq.lib()
    yield
    torch.cuda.synchronize()
    assert bq.bq_device_status(reset=True) == bq.BQ_OK


def make(seed, ns, befores, layers=2, heads=2, page=16, d=64, group=32, padding=0.0, likely=0.8):
    rng = np.random.default_rng(seed)
    parents = [random_tree(rng, n, padding) for n in ns]
    masks = [O.bits_of(p) for p in parents]
    tokens = rng.integers(0, 4, sum(ns)).astype(np.int32)         # few of them, so that siblings meet
    targets = rng.integers(0, 4, sum(ns)).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
    for b, p in enumerate(parents):
        for i, up in enumerate(p):
            if up >= 0 and rng.random() < likely:
                targets[cu[b] + up] = tokens[cu[b] + i]
    lens = np.array([n + m for n, m in zip(ns, befores)], np.int32)
    need = [-(-int(n) // page) for n in lens]
    pages = sum(need) + 2
    order = rng.permutation(pages)
    table = np.full((len(ns), max(need + [1])), 10 ** 9, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    codes = rng.integers(0, 256, (layers, pages, 2, heads, page, d // 2)).astype(np.uint8)
    params = rng.standard_normal((layers, pages, 2, heads, page, d // group, 2)).astype(np.float16)
    return dict(tokens=tokens, targets=targets, masks=masks, cu=cu, lens=lens, table=table, codes=codes, params=params)


def check(c, uniform=False, words=None, flat=False):
    codes, params = dev(c["codes"]), dev(c["params"])
    most = int(np.diff(c["cu"]).max())
    got = bq.bq_kv4_accept(dev(c["tokens"]), dev(c["targets"]), tree_tensor(c["masks"], words),
                           codes[0] if flat else codes, params[0] if flat else params, dev(c["table"]), dev(c["lens"]),
                           cu_q=None if uniform else dev(c["cu"]), max_q=most)
    path, accepted, last, lens = (host(t) for t in got)
    wc, wp = c["codes"].copy(), c["params"].copy()
    wpath, wn, wlast, wlens = O.accept(c["tokens"], c["targets"], c["masks"], c["cu"], c["lens"], c["table"],
                                       wc[:1] if flat else wc, wp[:1] if flat else wp)
    for b, p in enumerate(wpath):
        assert path[b].tolist() == p + [-1] * (most - len(p))
    assert accepted.tolist() == wn and last.tolist() == wlast and lens.tolist() == wlens
    assert (host(codes) == wc).all() and (host(params).view(np.uint16) == wp.view(np.uint16)).all()
    return wn


@pytest.mark.parametrize("d,group,page", [(64, 32, 16), (64, 64, 32), (128, 32, 64), (128, 64, 16), (128, 128, 128),
                                          (256, 64, 16), (256, 128, 256)])
@pytest.mark.parametrize("layers,heads", [(1, 1), (3, 5)])
def test_shapes(d, group, page, layers, heads):
    n = check(make(d + page, [1, 8, 31, 64], [0, 5, 37, 100], layers, heads, page, d, group))
    assert max(n) > 2


@pytest.mark.parametrize("n", [1, 2, 3, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 500, 1024])
def test_nodes(n):
    check(make(n, [n, max(1, n // 3)], [3, 50]), words=max(1, -(-n // 64)))
    check(make(n + 1, [n], [17], padding=0.2, likely=0.95))


def test_chains_longer_than_a_step():
    """Every line of a long branch moves by one place, through pages."""
    n = 150
    c = make(1, [n], [13], page=16)
    m = np.zeros((n, n), bool)
    m[0, 0] = m[1, 1] = True
    m[1, 0] = True
    for i in range(2, n):
        m[i] = m[i - 1] if i > 2 else m[0]
        m[i, i] = True
    c["masks"] = [m]
    c["tokens"][:] = np.arange(n)
    c["targets"][:] = np.arange(n) + 1
    c["targets"][0] = 2
    assert check(c) == [n - 1]


def test_many_sequences_and_layers():
    check(make(2, [13] * 70, [int(x) for x in np.random.default_rng(2).integers(0, 40, 70)], layers=5, heads=3),
          uniform=True)


def test_one_pool_without_layers():
    check(make(3, [9, 9], [4, 20], layers=1), flat=True, uniform=True)


def test_no_nodes_padding_and_no_root():
    c = make(4, [0, 5, 6, 0], [0, 7, 30, 9])
    c["masks"][1][:] = False                      # padding alone
    check(c)
    c["masks"][2][0] = False                      # the root is padding: its children's bits name it still
    check(c)


def test_bits_behind_a_node_do_not_count():
    c = make(5, [20, 20], [3, 8])
    want = check(c)
    wide = [np.concatenate([m, np.zeros((20, 44), bool)], 1) for m in c["masks"]]
    for m in wide:
        for i in range(20):
            m[i, i + 1:] = m[i].any()
    codes, params = dev(c["codes"]), dev(c["params"])
    _, n, _, _ = bq.bq_kv4_accept(dev(c["tokens"]), dev(c["targets"]), tree_tensor(wide, 1), codes, params,
                                  dev(c["table"]), dev(c["lens"]))
    assert host(n).tolist() == want


def test_reported_and_left_out():
    c = make(6, [6, 6], [4, 9], likely=1.0)
    for change in (dict(lens=np.array([5, 15], np.int32)), dict(lens=np.array([10 ** 6, 15], np.int32)),
                   dict(cu=np.array([-3, 6, 12], np.int32))):
        bad = dict(c, **change)
        codes, params = dev(c["codes"]), dev(c["params"])
        path, n, last, lens = bq.bq_kv4_accept(dev(c["tokens"]), dev(c["targets"]), tree_tensor(c["masks"]), codes, params,
                                               dev(c["table"]), dev(bad["lens"]), cu_q=dev(bad["cu"]), max_q=6)
        assert bq.bq_device_status(reset=True) == bq.BQ_ERR_INVALID_ARG
        assert host(n)[0] == 0 and host(last)[0] == -1 and host(lens)[0] == bad["lens"][0] and (host(path)[0] == -1).all()
        assert host(n)[1] > 0
    # a page outside the pool: its lines stay, the others move
    bad = c["table"].copy()
    bad[0, :] = 10 ** 8
    codes, params = dev(c["codes"]), dev(c["params"])
    got = bq.bq_kv4_accept(dev(c["tokens"]), dev(c["targets"]), tree_tensor(c["masks"]), codes, params, dev(bad),
                           dev(c["lens"]))
    want = O.accept(c["tokens"], c["targets"], c["masks"], c["cu"], c["lens"], c["table"], c["codes"].copy(), c["params"])
    assert host(got[1]).tolist() == want[1]
    bq.bq_device_status(reset=True)


def test_captured():
    c = make(7, [12, 12], [5, 40])
    args = [dev(c["tokens"]), dev(c["targets"]), tree_tensor(c["masks"]), dev(c["codes"]), dev(c["params"]),
            dev(c["table"]), dev(c["lens"])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        path, n, last, lens = bq.bq_kv4_accept(*args)
    graph.replay()
    wc, wp = c["codes"].copy(), c["params"].copy()
    want = O.accept(c["tokens"], c["targets"], c["masks"], c["cu"], c["lens"], c["table"], wc, wp)
    assert host(n).tolist() == want[1] and (host(args[3]) == wc).all()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    args[3] = dev(c["codes"])
    torch.cuda.synchronize()
    got = bq.bq_kv4_accept(*args, stream=side)
    side.synchronize()
    assert host(got[3]).tolist() == want[3]


def test_refusals():
    c = make(8, [4, 4], [3, 3])
    args = [dev(c["tokens"]), dev(c["targets"]), tree_tensor(c["masks"]), dev(c["codes"]), dev(c["params"]),
            dev(c["table"]), dev(c["lens"])]

    def call(i, v, **kw):
        a = list(args)
        a[i] = v
        return bq.bq_kv4_accept(*a, **kw)
    with pytest.raises(TypeError):
        call(0, args[0].long())
    with pytest.raises(TypeError):
        call(2, args[2].int())
    with pytest.raises(ValueError):
        call(1, args[1][:3])
    with pytest.raises(ValueError):
        call(2, args[2][:3])
    with pytest.raises(ValueError):
        call(3, args[3][:1])
    with pytest.raises(ValueError):
        call(3, args[3].transpose(0, 1))
    with pytest.raises(ValueError):
        call(6, args[6][:1])
    with pytest.raises(ValueError):
        call(0, args[0], max_q=3)
