"""The choice of tokens on the GPU against the float64 oracle: the same tokens, logarithms to fp32."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import quantized_mixed_precision_gb300 as bq  # noqa: E402
from oracle import draft_oracle as O  # noqa: E402

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bq.lib()
    yield
    torch.cuda.synchronize()
    assert bq.bq_device_status(reset=True) == bq.BQ_OK


def cuda(x, dtype):
    return None if x is None else torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


def check(x, u, t=None, k=None, p=None, m=None, **kw):
    """x: a CUDA tensor (R, V); the rest numpy or None."""
    tokens, logs = bq.bq_sample(x, cuda(u, torch.float32), cuda(t, torch.float32), cuda(k, torch.int32),
                                cuda(p, torch.float32), cuda(m, torch.float32), logprob=True, **kw)
    rows = x.double().cpu().numpy()
    got, glog = tokens.cpu().numpy(), logs.double().cpu().numpy()
    f32 = [None if v is None else np.asarray(v, np.float32) for v in (u, t, p, m)]
    for i in range(len(rows)):
        want, wlog, _ = O.sample(rows[i], f32[0][i], 1.0 if t is None else f32[1][i], 0 if k is None else int(k[i]),
                                 1.0 if p is None else f32[2][i], 0.0 if m is None else f32[3][i])
        assert got[i] == want, (i, got[i], want)
        # one rounding to fp32, and sums that are good to 2**-28 (a weight) of the whole
        assert glog[i] == wlog or abs(glog[i] - wlog) <= 2.0 ** -24 * abs(wlog) + 2.0 ** -27, (i, glog[i], wlog)
    return tokens


def logits(seed, r, v, dtype, std=2.0, top=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((r, v), generator=g, device="cuda") * std
    if top and v > top:
        x.scatter_add_(1, torch.randint(0, v, (r, top), generator=g, device="cuda"),
                       torch.full((r, top), 6.0, device="cuda"))
    return x.to(TYPES[dtype])


def settings(seed, r, v):
    rng = np.random.default_rng(seed)
    return dict(u=rng.random(r), t=np.where(rng.random(r) < 0.1, 0.0, rng.uniform(0.3, 2.0, r)),
                k=np.where(rng.random(r) < 0.4, 0, rng.integers(1, max(2, v), r)),
                p=np.where(rng.random(r) < 0.3, 1.0, rng.uniform(0.05, 0.999, r)),
                m=np.where(rng.random(r) < 0.5, 0.0, rng.uniform(0.001, 0.3, r)))


@pytest.mark.parametrize("v", [1, 2, 7, 31, 32, 33, 63, 255, 1000, 1023, 1025, 4099, 32000, 50021])
@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_sizes_with_all_filters(v, dtype):
    check(logits(v, 12, v, dtype), **settings(v, 12, v))


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("std", [0.01, 1.0, 3.0, 12.0])
@pytest.mark.parametrize("which", ["none", "t", "k", "p", "m"])
def test_large_vocabularies(dtype, std, which):
    r, v = 6, 131072
    s = settings(int(std * 100), r, v)
    s["t"] = np.maximum(s["t"], 0.3)
    one = dict(u=s["u"])
    if which == "k":
        s["k"] = np.array([1, 2, 50, 1000, 60000, 131071])
    if which != "none":
        one[which] = s[which]
    check(logits(3, r, v, dtype, std, top=0), **one)


def test_the_largest_vocabulary():
    check(logits(4, 2, 1 << 19, "f16", 0.5, top=0), **settings(4, 2, 1 << 19))


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_many_draws_of_one_flat_row(dtype):
    """The borders between 30000 about equal tokens, each hit to the last bits: every u gives the oracle's token."""
    v, r = 30011, 256
    x = logits(5, 1, v, dtype, 0.3, top=0).expand(r, v).contiguous()
    u = np.random.default_rng(5).random(r)
    check(x, u)
    check(x, u, p=np.full(r, 0.9))
    check(x, u, t=np.full(r, 0.7), k=np.full(r, 20000), p=np.full(r, 0.8))


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_equal_logits(dtype):
    """Ties go to the lower index, in every filter."""
    v = 5000
    x = torch.zeros((8, v), device="cuda")
    x[:, 1::3] = 1.0
    x[:, 7] = -0.0
    u = [0.0, 0.3, 0.5, 0.999, 0.1, 0.7, 0.9, 0.99]
    check(x.to(TYPES[dtype]), u, k=[1, 2, 1000, 1700, 3000, 4999, 5000, 0])
    check(x.to(TYPES[dtype]), u, p=[0.01, 0.2, 0.5, 0.57, 0.6, 0.8, 0.9, 0.999])
    check(x.to(TYPES[dtype]), u, k=[4000] * 8, p=[0.01, 0.2, 0.5, 0.57, 0.6, 0.8, 0.9, 0.999], m=[1.0, .3, .4, 0, 0, 0, 0, 0])
    check(x.to(TYPES[dtype]), u, t=[0.0] * 8)
    check(torch.full((8, v), 3.0, device="cuda").to(TYPES[dtype]), u, p=[0.01, 0.2, 0.5, 0.57, 0.6, 0.8, 0.9, 0.999])


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_infinities_and_nan(dtype):
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[-inf, 1, -inf, 2], [nan, 1, nan, 2], [-inf] * 4, [nan] * 4, [1, inf, inf, 2],
                      [-inf, -inf, -inf, -5], [-60000, 60000, -60000, 59000]], device="cuda").to(TYPES[dtype])
    for u in (0.0, 0.5, 0.999):
        us = [u] * 7
        check(x, us)
        check(x, us, t=[0.5] * 7, k=[3] * 7, p=[0.99] * 7, m=[0.01] * 7)
        check(x, us, k=[1] * 7)


@pytest.mark.parametrize("dtype", sorted(TYPES))
def test_min_p_alone(dtype):
    """From a few kept tokens to all of them, rows of infinities among them, with and without top-k."""
    for v in (5, 4000, 70001):
        for std in (0.01, 0.5, 3.0):
            x = logits(v, 24, v, dtype, std)
            x[1] = float("-inf")
            x[2, v // 2] = float("inf")
            x[3, v - 1] = float("inf")
            x[4, : v // 2] = float("nan")
            x[5] = x[5].sort().values                 # the largest last: all before it were the largest once
            x[6] = x[6].sort(descending=True).values
            x[7] = 1.0
            u = np.random.default_rng(v).random(24)
            m = np.resize([0.001, 0.05, 0.3, 0.9, 1.0], 24)
            check(x, u, m=m)
            check(x, u, t=np.resize([0.3, 1.0, 2.0], 24), m=m, k=np.resize([0, 1, 5, 40, 3000], 24))


def test_settings_at_the_edges():
    inf, nan = float("inf"), float("nan")
    x = logits(6, 12, 777, "f16")
    u = np.linspace(0, 0.99, 12)
    check(x, u, t=[0, -1, nan, 1e-6, 1e-3, 1e3, 1e6, 1, 1, 1, 1, 1])
    check(x, u, k=[0, -1, 1, 777, 778, 10 ** 9, -2 ** 31, 2, 3, 4, 5, 6])
    check(x, u, p=[0, -1, 1, 2, 1e-30, 1e-6, 0.9999999, inf, 0.5, 0.5, 0.5, 0.5])
    check(x, u, m=[0, -1, 1, 2, 1e-30, 0.999999, inf, 0.1, 0.2, 0.3, 0.4, 0.5])
    check(x, [0.0, -1.0, 1.0, 2.0, nan, 1 - 2.0 ** -24, 2.0 ** -149, 0.5, 0.5, 0.5, 0.5, 0.5])
    same, _ = bq.bq_sample(x, cuda(u, torch.float32))
    for name in ("top_p", "min_p"):
        got, _ = bq.bq_sample(x, cuda(u, torch.float32), **{name: cuda([nan] * 12, torch.float32)})
        assert torch.equal(got, same)
    flat, lp = bq.bq_sample(x, cuda(u, torch.float32), temperature=cuda([inf] * 12, torch.float32), logprob=True)
    assert flat.tolist() == [int(v * 777) for v in np.float32(u)] and (lp + np.log(777)).abs().max() < 1e-6


@pytest.mark.parametrize("v", [777, 20000])
def test_infinite_temperature_with_limits(v):
    x = logits(7, 8, v, "f16")
    u = np.linspace(0.01, 0.99, 8)
    t = [float("inf")] * 8
    check(x, u, t=t, m=[1.0, 0.5, 1e-30, 2.0, 1.0, 1.0, 0.9, 0.0])
    check(x, u, t=t, m=[1.0, 0.5, 1e-30, 2.0, 1.0, 1.0, 0.9, 0.0], k=[0, 3, 100, 5, 1, 50, v, 2 * v])
    check(x, u, t=t, m=[1.0, 0.5, 1e-30, 2.0, 1.0, 1.0, 0.9, 0.0], p=[0.3, 0.001, 0.77, 0.5, 0.9, 1.0, 0.0, 0.6])


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("shift", [0, 1, 3, 5])
def test_strides_and_alignment(dtype, shift):
    v = 1000
    wide = torch.full((5, v + 37), float("inf"), device="cuda").to(TYPES[dtype])
    x = wide[:, shift:shift + v]
    x.copy_(logits(7, 5, v, dtype))
    assert not x.is_contiguous()
    check(x, **settings(7, 5, v))


def test_rows_do_not_depend_on_one_another():
    x = logits(8, 300, 9001, "bf16")
    s = settings(8, 300, 9001)
    every = check(x[:40], **{k: v[:40] for k, v in s.items()})
    args = {k: cuda(v, torch.int32 if k == "k" else torch.float32) for k, v in s.items()}

    def call(rows):
        return bq.bq_sample(x[rows], *(args[k][rows] for k in "utkpm"))[0]
    whole = call(slice(None))
    assert torch.equal(whole[:40], every)
    for a, b in ((0, 1), (5, 7), (100, 260)):
        assert torch.equal(call(slice(a, b)), whole[a:b])


@pytest.mark.parametrize("dtype", sorted(TYPES))
@pytest.mark.parametrize("v", [300, 5000, 70001])
def test_small_k_with_other_filters(dtype, v):
    """First k of a few to more than a list holds, each with top-p and min-p at every strictness."""
    r = 48
    rng = np.random.default_rng(v)
    k = np.resize([1, 2, 3, 17, 50, 255, 999, 1024, 1025, 2047, 2048, 4000], r)
    p = np.resize([1.0, 0.0, 0.3, 0.9, 0.999], r)
    m = np.resize([0.0, 0.0, 0.05, 1.0, 0.5, 2.0, 0.0], r)
    for std in (0.05, 2.0):
        x = logits(v, r, v, dtype, std)
        check(x, rng.random(r), t=rng.uniform(0.5, 1.5, r), k=k, p=p, m=m)
        check(x, rng.random(r), k=k)
        check(x, rng.random(r), k=k, m=m)


def test_no_rows_and_no_tokens():
    x = torch.zeros((0, 10), device="cuda")
    assert bq.bq_sample(x, torch.zeros(0, device="cuda"))[0].shape == (0,)
    t, lp = bq.bq_sample(torch.zeros((2, 0), device="cuda"), torch.zeros(2, device="cuda"), logprob=True)
    assert t.tolist() == [-1, -1] and torch.isneginf(lp).all()


def test_captured_out_and_stream():
    x = logits(9, 20, 40000, "f16")
    s = settings(9, 20, 40000)
    args = [cuda(s[k], torch.int32 if k == "k" else torch.float32) for k in "utkpm"]
    want, _ = bq.bq_sample(x, *args)
    out = torch.empty(20, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _ = bq.bq_sample(x, *args, out=out)
    assert got is out
    for _ in range(2):
        out.fill_(-7)
        graph.replay()
        assert torch.equal(out, want)
    args[0].copy_(torch.rand(20, device="cuda"))
    graph.replay()
    assert torch.equal(out, bq.bq_sample(x, *args)[0])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    third, lp = bq.bq_sample(x, *args, stream=side, logprob=True)
    side.synchronize()
    assert torch.equal(third, out) and torch.isfinite(lp).all()


def test_refusals():
    x, u = torch.zeros((3, 8), device="cuda"), torch.zeros(3, device="cuda")
    with pytest.raises(TypeError):
        bq.bq_sample(x.double(), u)
    with pytest.raises(TypeError):
        bq.bq_sample(x, u.double())
    with pytest.raises(TypeError):
        bq.bq_sample(x, u, top_k=u)
    with pytest.raises(ValueError):
        bq.bq_sample(x, u[:2])
    with pytest.raises(ValueError):
        bq.bq_sample(x[0].expand(3, 8), u)
    with pytest.raises(ValueError):
        bq.bq_sample(x.t(), torch.zeros(8, device="cuda"))
    with pytest.raises(ValueError):
        bq.bq_sample(x[0], u)
    with pytest.raises(bq.BqError):
        bq.bq_sample(torch.zeros((1, (1 << 19) + 1), device="cuda"), u[:1])
