"""The attention half of a decoder layer on 4-bit weights and a 4-bit cache: a prompt, then tokens one by one.

    python examples/decode_layer.py [--batch 4] [--prompt 300] [--steps 16]

One layer with random weights: QKV projection (bq_gemm_f16xi4_group), norm, rotation and the write into the cache
(bq_qk_norm_rope_kv4), attention over the cache (bq_attn_kv4), output projection.  A decode step is captured once in a
CUDA graph and replayed: lengths, slots and positions are tensors that the step itself moves on.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import quantized_mixed_precision_gb300 as bq  # noqa: E402


class Layer:
    """Weights of one layer's attention, quantised to 4 bits by groups along k."""

    def __init__(self, hidden=4096, q_heads=32, kv_heads=8, head_dim=128, group=128, seed=0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)
        self.q_heads, self.kv_heads, self.d, self.group = q_heads, kv_heads, head_dim, group

        def weight(n, k):
            w = (torch.randn((n, k), generator=g, device=device) * k ** -0.5).half()
            codes, scale = bq.bq_quantize_sym(w.view(-1, group), 4)
            return bq.bq_pack_weights(codes.view(n, k), 4), scale.view(n, k // group)

        self.qkv = weight((q_heads + 2 * kv_heads) * head_dim, hidden)
        self.out = weight(hidden, q_heads * head_dim)
        self.q_norm = (1 + 0.1 * torch.randn(head_dim, generator=g, device=device)).half()
        self.k_norm = (1 + 0.1 * torch.randn(head_dim, generator=g, device=device)).half()

    def __call__(self, x, cache, slots, positions, lens, cu_q=None, max_q=1, max_len=None):
        """x (tokens, hidden) fp16 -> (tokens, hidden); the tokens' keys and values go into the cache first."""
        hq, hkv, d = self.q_heads, self.kv_heads, self.d
        qkv = bq.bq_gemm_f16xi4_group(x, *self.qkv, self.group)
        q, _, _ = bq.bq_qk_norm_rope_kv4(qkv[:, :hq * d].unflatten(1, (hq, d)),
                                         qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d)),
                                         qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d)), cache.codes, cache.params,
                                         slots, positions, cache.cos, cache.sin, q_weight=self.q_norm,
                                         k_weight=self.k_norm)
        o, _ = bq.bq_attn_kv4(q, cache.codes, cache.params, cache.table, lens, cu_q=cu_q, max_q=max_q, max_len=max_len)
        return bq.bq_gemm_f16xi4_group(o.flatten(1), *self.out, self.group)


class Cache:
    """The layer's 4-bit cache: a pool of pages, dealt out to the sequences in turn."""

    def __init__(self, layer, batch, most, page=64, group=64, base=10000.0, device="cuda"):
        per = -(-most // page)
        self.codes, self.params = bq.bq_kv4_pool(batch * per, layer.kv_heads, layer.d, page, group, device)
        self.table = torch.arange(batch * per, dtype=torch.int32, device=device).view(per, batch).t().contiguous()
        self.page = page
        angle = torch.arange(most, device=device, dtype=torch.float64)[:, None] * \
            base ** (-torch.arange(layer.d // 2, device=device, dtype=torch.float64) * 2 / layer.d)
        self.cos, self.sin = angle.cos().float(), angle.sin().float()

    def slots(self, seq, position):
        """Places in the pool of the tokens at `position` of the sequences `seq`."""
        at = position.long()
        return (self.table[seq.long(), at // self.page] * self.page + position % self.page).to(torch.int32)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--steps", type=int, default=16)
    a = ap.parse_args()
    layer = Layer()
    hidden = layer.out[0].shape[0]
    cache = Cache(layer, a.batch, a.prompt + a.steps + 2)

    # the prompt: all tokens of all sequences at once
    seq = torch.arange(a.batch, device="cuda").repeat_interleave(a.prompt)
    pos = torch.arange(a.prompt, dtype=torch.int32, device="cuda").repeat(a.batch)
    lens = torch.full((a.batch,), a.prompt, dtype=torch.int32, device="cuda")
    cu = torch.arange(a.batch + 1, dtype=torch.int32, device="cuda") * a.prompt
    x = torch.randn((a.batch * a.prompt, hidden), device="cuda").half()
    y = layer(x, cache, cache.slots(seq, pos), pos, lens, cu_q=cu, max_q=a.prompt, max_len=a.prompt)
    token = y.view(a.batch, a.prompt, hidden)[:, -1].contiguous()

    # one step as a graph: the new token stands at position lens, then lens grows
    rows = torch.arange(a.batch, device="cuda")

    def step():
        pos = lens.clone()
        lens.add_(1)
        token.copy_(layer(token, cache, cache.slots(rows, pos), pos, lens, max_len=a.prompt + a.steps + 2))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                                     # warm-up, and the first step
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    assert int(lens[0]) == a.prompt + a.steps + 1 and torch.isfinite(token).all()
    print(f"{a.batch} sequences, prompt {a.prompt}: {begin.elapsed_time(end) * 1e3 / a.steps:.1f} us a decode step, "
          f"norm of the last token's output {token.float().norm(dim=1).mean().item():.3f}")


if __name__ == "__main__":
    main()
