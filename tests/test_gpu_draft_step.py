"""The operators on drafted tokens together, as examples/draft_step.py runs them: steps of a small model, every part
against its oracle on what the GPU had, the caches against those of token-by-token decoding, and the example itself."""

import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

import quantized_mixed_precision_gb300 as bq  # noqa: E402
from oracle import draft_oracle as O  # noqa: E402
from tests.test_gpu_parity import host  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))


@pytest.mark.parametrize("heads,kv", [(4, 2), (8, 1)])       # few query rows a kv head, and many
def test_steps(heads, kv):
    from draft_step import PARENTS, Caches, Checker, Model
    batch, n, most, steps = 3, len(PARENTS), 200, 5
    model = Model(vocab=500, hidden=256, layers=2, q_heads=heads, kv_heads=kv, head_dim=64, group=64)
    caches = Caches(model, batch, most, page=16, group=32)
    g = torch.Generator(device="cuda").manual_seed(3)
    lens = torch.zeros((batch,), dtype=torch.int32, device="cuda")
    last = torch.randint(0, 500, (batch,), generator=g, device="cuda", dtype=torch.int32)
    check = Checker(model, caches, lens, last, most, temperature=0.5)
    masks, cu = [O.bits_of(PARENTS)] * batch, np.arange(batch + 1) * n
    emitted = [[] for _ in range(batch)]
    kept = 0
    for _ in range(steps):
        u = torch.rand(batch * n, generator=g, device="cuda")
        seen = {}
        real = model.logits
        model.logits = lambda x: seen.setdefault("logits", real(x))
        before = host(check.lens) + n
        old = caches.codes.clone(), caches.params.clone()
        accept = bq.bq_kv4_accept

        def recorded(*args, **kw):
            seen["codes"], seen["params"] = host(args[3]).copy(), host(args[4]).copy()
            return accept(*args, **kw)
        try:
            bq.bq_kv4_accept = recorded
            tokens, targets, path, accepted = check.step(u)
        finally:
            bq.bq_kv4_accept, model.logits = accept, real
        assert not torch.equal(old[0], caches.codes)
        logits = host(seen["logits"]).astype(np.float64)
        for i in range(batch * n):
            assert int(targets[i]) == O.sample(logits[i], np.float32(host(u)[i]), np.float32(0.5), p=np.float32(0.9))[0]
        wpath, wn, wlast, wlens = O.accept(host(tokens), host(targets), masks, cu, before, host(caches.table),
                                           seen["codes"], seen["params"])
        assert host(accepted).tolist() == wn and host(check.last).tolist() == wlast and host(check.lens).tolist() == wlens
        assert (host(caches.codes) == seen["codes"]).all() and (host(caches.params) == seen["params"]).all()
        for b in range(batch):
            emitted[b] += [int(host(tokens)[b * n + j]) for j in wpath[b]]
        kept += sum(wn)
    assert kept > batch * steps                      # more than a token a step: branches were taken

    # the first layer's keys and values depend on a token and its place alone: token by token they are the same bytes
    # (the projection's as well, with as many rows: a row's bits can differ between calls with other numbers of them)
    plain = Caches(model, batch, most, page=16, group=32)
    for b in range(batch):
        for i, t in enumerate(emitted[b]):
            pos = torch.tensor([i], dtype=torch.int32, device="cuda")
            x = model.embed[t:t + 1].repeat(batch * n, 1)
            layer = model.layers[0]
            qkv = bq.bq_gemm_f16xi4_group(x, *layer.qkv, layer.group)[:1].unflatten(1, (heads + 2 * kv, 64))
            bq.bq_qk_norm_rope_kv4(qkv[:, :heads], qkv[:, heads:heads + kv], qkv[:, heads + kv:], plain.codes[0],
                                   plain.params[0], plain.slots(torch.tensor([b], device="cuda"), pos), pos, plain.cos,
                                   plain.sin, q_weight=layer.q_norm, k_weight=layer.k_norm)
        at = np.arange(len(emitted[b]))
        pages = host(caches.table)[b][at // 16]
        assert len(at) == int(check.lens[b])
        for x, y in ((caches.codes, plain.codes), (caches.params, plain.params)):
            assert (host(x[0])[pages, :, :, at % 16] == host(y[0])[pages, :, :, at % 16]).all()
    assert bq.bq_device_status(reset=True) == bq.BQ_OK


@pytest.mark.parametrize("args", [[], ["--batch", "1", "--prompt", "1", "--steps", "3", "--temperature", "0"]])
def test_example_runs(args):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "draft_step.py"), *args], capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
    assert "tokens a step" in r.stdout
