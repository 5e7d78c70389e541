"""The three decoder-layer operators together, as examples/decode_layer.py runs them: a prompt and some decode steps
against the float64 oracle fed with the same 4-bit cache, and the example itself."""

import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import quantized_mixed_precision_gb300 as bq  # noqa: E402
from oracle import bq_oracle as O  # noqa: E402
from oracle import decode_oracle as D  # noqa: E402
from tests.test_gpu_parity import host  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


def test_prompt_and_steps():
    from decode_layer import Cache, Layer
    batch, prompt, steps = 3, 37, 4
    layer = Layer(hidden=256, q_heads=4, kv_heads=2, head_dim=64, group=64)
    cache = Cache(layer, batch, prompt + steps, page=16, group=32)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)

    def weights(w):
        packed, scale = (host(t) for t in w)
        return O.unpack(packed, 2 * packed.shape[1], 4, "interleaved").astype(np.int64), scale

    (wq, sq), (wo, so) = weights(layer.qkv), weights(layer.out)
    codes, params = np.zeros_like(host(cache.codes)), np.zeros_like(host(cache.params))
    lens = torch.zeros((batch,), dtype=torch.int32, device="cuda")
    for n in [prompt] + [1] * steps:
        x = torch.randn((batch * n, 256), generator=g, device="cuda").half()
        seq = torch.arange(batch, device="cuda").repeat_interleave(n)
        pos = (lens.repeat_interleave(n) + torch.arange(n, device="cuda").repeat(batch)).to(torch.int32)
        lens += n
        slots = cache.slots(seq, pos)
        cu = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * n
        y = layer(x, cache, slots, pos, lens, cu_q=cu if n > 1 else None, max_q=n)

        # the oracle's layer, from the projection's fp16 result on: q, k and v as the GPU has them
        qkv = host(bq.bq_gemm_f16xi4_group(x, *layer.qkv, 64))
        want, bound = D.gemm_group(host(x), wq, sq, None, 64)
        assert (np.abs(qkv - want) <= bound).all()
        h = qkv.reshape(-1, 8, 64)
        q, _, _ = D.write(h[:, :4], h[:, 4:6], h[:, 6:], codes, params, host(slots), host(pos), host(cache.cos),
                          host(cache.sin), host(layer.q_norm), host(layer.k_norm), 1e-6, False)
        assert (host(cache.codes) == codes).all() and (host(cache.params) == params).all()
        o, _, tol, _ = D.attention(q, codes, params, host(cache.table), host(lens), host(cu), 64 ** -0.5)
        got, _ = bq.bq_attn_kv4(torch.from_numpy(q).cuda(), cache.codes, cache.params, cache.table, lens,
                                cu_q=cu, max_q=n)
        assert (np.abs(host(got) - o) <= tol).all()
        want, bound = D.gemm_group(host(got).reshape(-1, 256), wo, so, None, 64)
        assert (np.abs(host(y) - want) <= bound).all()
    assert bq.bq_device_status(reset=True) == bq.BQ_OK


@pytest.mark.parametrize("args", [[], ["--batch", "1", "--prompt", "1", "--steps", "3"]])
def test_example_runs(args):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "decode_layer.py"), *args], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "us a decode step" in r.stdout
