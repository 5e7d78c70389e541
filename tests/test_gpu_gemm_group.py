"""fp16 x 4-bit weights with group scales on the GPU against the float64 oracle, within the oracle's derived bound."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import quantized_mixed_precision_gb300 as bq  # noqa: E402
from oracle import bq_oracle as O  # noqa: E402
from oracle import decode_oracle as D  # noqa: E402
from tests.test_gpu_parity import dev, host  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    bq.lib()
    yield
    torch.cuda.synchronize()
    assert bq.bq_device_status(reset=True) == bq.BQ_OK


def make(seed, m, n, k, group, zp):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((m, k)).astype(np.float16)
    s = rng.uniform(1e-3, 1e-2, (n, k // group)).astype(np.float16)
    if zp:
        codes = rng.integers(0, 16, (n, k))
        z = rng.integers(0, 16, (n, k // group)).astype(np.float16)
        z[::3] += np.float16(0.25)
        return x, codes, s, z
    return x, rng.integers(-8, 8, (n, k)), s, None


def pack(codes, layout):
    return dev(O.pack(((codes + 8) % 16 - 8).astype(np.int8), 4, layout))


def check(x, codes, s, z, group, layout, act="none", **kw):
    y = bq.bq_gemm_f16xi4_group(dev(x) if isinstance(x, np.ndarray) else x, pack(codes, layout), dev(s), group,
                                zero_point=None if z is None else dev(z), layout=layout, activation=act, **kw)
    x = x if isinstance(x, np.ndarray) else host(x)
    want, bound = D.gemm_group(x, codes, s, z, group, act)
    got = host(y).astype(np.float64)
    assert got.shape == want.shape and (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())
    return y


@pytest.mark.parametrize("layout", ["plain", "interleaved"])
@pytest.mark.parametrize("zp", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (1, 17, 384), (2, 100, 1152), (5, 33, 4096), (8, 257, 640), (9, 64, 896)])
def test_small(m, n, k, group, zp, layout):
    x, codes, s, z = make(m * n + k, m, n, k, group, zp)
    check(x, codes, s, z, group, layout)


@pytest.mark.parametrize("m,n,k,group,zp", [(1, 11008, 4096, 128, False), (16, 4096, 4096, 64, True),
                                            (17, 1001, 2048, 32, True), (33, 520, 1024, 128, False),
                                            (64, 300, 1088, 64, False), (65, 70, 512, 32, True),
                                            (200, 130, 256, 128, True), (1, 5, 65536, 128, True),
                                            (3, 4099, 32, 32, False)])
def test_large(m, n, k, group, zp):
    x, codes, s, z = make(m + n + k, m, n, k, group, zp)
    check(x, codes, s, z, group, "interleaved")


@pytest.mark.parametrize("act", ["relu", "gelu"])
def test_activation(act):
    x, codes, s, z = make(4, 3, 200, 512, 64, True)
    check(x, codes, s, z, 64, "interleaved", act)


def test_strided_rows_and_out():
    x, codes, s, z = make(5, 6, 90, 256, 32, False)
    wide = torch.full((6, 512), float("nan"), dtype=torch.float16, device="cuda")
    wide[:, 128:384] = dev(x)
    out = torch.empty((6, 90), dtype=torch.float16, device="cuda")
    assert check(wide[:, 128:384], codes, s, z, 32, "plain", out=out) is out


@pytest.mark.parametrize("zp", [False, True])
@pytest.mark.parametrize("m,k,group", [(9, 64, 32), (12, 32, 32), (20, 192, 64), (40, 1088, 32), (40, 1088, 64),
                                       (70, 1216, 64), (33, 1248, 32), (17, 4224, 128)])
def test_strided_rows_with_a_ragged_end(m, k, group, zp):
    """Rows apart by more than K, K that ends inside a slab of 128, and NaN beside every row; the last row ends the storage."""
    x, codes, s, z = make(m + k, m, 150, k, group, zp)
    flat = torch.full(((m - 1) * (k + 24) + k,), float("nan"), dtype=torch.float16, device="cuda")
    view = flat.as_strided((m, k), (k + 24, 1))
    view.copy_(dev(x))
    for layout in ("plain", "interleaved"):
        check(view, codes, s, z, group, layout)


def test_wait_limit_is_reported():
    """With no time to wait, waits for the copies of a slab give up: reported once, and the next call is right."""
    x, codes, s, z = make(12, 64, 256, 4096, 128, False)
    xd, w, sd = dev(x), pack(codes, "interleaved"), dev(s)
    torch.cuda.synchronize()
    assert bq.bq_device_status(reset=True) == bq.BQ_OK
    old = bq.bq_set_wait_timeout_ns(0)
    try:
        bq.bq_gemm_f16xi4_group(xd, w, sd, 128)
        torch.cuda.synchronize()
        assert bq.bq_device_status(reset=True) == bq.BQ_ERR_TIMEOUT
    finally:
        bq.bq_set_wait_timeout_ns(old)
    check(x, codes, s, z, 128, "interleaved")


def test_large_and_tiny_activations():
    """Activations up to the fp16 limits: nothing overflows or vanishes on the way."""
    x, codes, s, z = make(6, 4, 64, 512, 64, False)
    x[0] = 0
    x[0, 5] = 60000.0
    x[1] *= np.float16(2.0 ** -14)
    x[2] *= np.float16(2000.0)
    check(x, codes, s / np.float16(16), z, 64, "interleaved")


def test_same_bits_on_every_run_and_batch():
    """A row's result does not depend on the launch, and repeats bit for bit."""
    x, codes, s, z = make(7, 8, 600, 2048, 128, True)
    w, sd, zd = pack(codes, "interleaved"), dev(s), dev(z)
    a = bq.bq_gemm_f16xi4_group(dev(x), w, sd, 128, zero_point=zd)
    b = bq.bq_gemm_f16xi4_group(dev(x), w, sd, 128, zero_point=zd)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_quantiser_gives_the_layout():
    """bq_quantize_sym over the groups, then the packer, then this call."""
    rng = np.random.default_rng(8)
    w = (rng.standard_normal((96, 512)) * 0.02).astype(np.float16)
    q, sw = bq.bq_quantize_sym(dev(w).view(-1, 64), 4)
    wp = bq.bq_pack_weights(q.view(96, 512), 4, "interleaved")
    x = rng.standard_normal((2, 512)).astype(np.float16)
    y = bq.bq_gemm_f16xi4_group(dev(x), wp, sw.view(96, 8), 64)
    want, bound = D.gemm_group(x, host(q).reshape(96, 512).astype(np.int64), host(sw).reshape(96, 8), None, 64)
    assert (np.abs(host(y) - want) <= bound).all()


def test_empty_and_zero_k():
    e = torch.empty((0, 64), dtype=torch.float16, device="cuda")
    w = torch.zeros((5, 32), dtype=torch.uint8, device="cuda")
    s = torch.ones((5, 1), dtype=torch.float16, device="cuda")
    assert bq.bq_gemm_f16xi4_group(e, w, s, 64).shape == (0, 5)
    y = bq.bq_gemm_f16xi4_group(torch.empty((3, 0), dtype=torch.float16, device="cuda"), w[:, :0].contiguous(),
                                s[:, :0].contiguous(), 64)
    assert y.shape == (3, 5) and not y.any()


def test_side_stream():
    x, codes, s, z = make(9, 1, 500, 1024, 64, True)
    xd, w, sd, zd = dev(x), pack(codes, "plain"), dev(s), dev(z)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    y = bq.bq_gemm_f16xi4_group(xd, w, sd, 64, zero_point=zd, layout="plain", stream=st)
    st.synchronize()
    want, bound = D.gemm_group(x, codes, s, z, 64)
    assert (np.abs(host(y) - want) <= bound).all()


def test_refusals():
    x, codes, s, z = make(10, 2, 40, 256, 64, True)
    xd, w, sd, zd = dev(x), pack(codes, "plain"), dev(s), dev(z)
    for bad in (dict(group=48), dict(group=256)):
        with pytest.raises(ValueError):
            bq.bq_gemm_f16xi4_group(xd, w, sd, **bad)
    for args in ((xd.float(), w, sd), (xd, w.to(torch.int8), sd), (xd, w, sd.float())):
        with pytest.raises(TypeError):
            bq.bq_gemm_f16xi4_group(*args, 64)
    for args in ((xd[:, :128], w, sd), (xd, w, sd[:, :2]), (xd, w[::2], sd), (xd.t(), w, sd), (xd[0], w, sd)):
        with pytest.raises(ValueError):
            bq.bq_gemm_f16xi4_group(*args, 64)
    with pytest.raises(ValueError):
        bq.bq_gemm_f16xi4_group(xd, w, sd, 64, zero_point=zd[:1])
    with pytest.raises(bq.BqError):      # row starts that are not 16-byte aligned
        wide = torch.zeros((2, 260), dtype=torch.float16, device="cuda")
        bq.bq_gemm_f16xi4_group(wide[:, :256], w, sd, 64)
