"""A small attention layer that decodes with an 8-bit cache: prompts of several lengths are projected, rotated,
written into the cache and attended in one chunk each; then tokens are drawn one at a time. It runs the fused
projection (gemm), kv_append with rotary positions, attention_kv and the output projection on one GPU, the decode
step as a CUDA graph, and compares every step with the same layer computed by torch in 32 bits over an
unquantised cache.

    python examples/decode_layer.py [--steps 16] [--cache e4m3|int8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_tensor_core_tcgen05_gb300 as tg  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, PAGE = 1024, 16, 4, 64, 32
PROMPTS = [300, 17, 1, 129]


class Layer:
    """x -> x + attention(x) W_out, with the cache's state of a batch of sequences."""

    def __init__(self, batch, longest, cache_dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        width = (HEADS + 2 * KV_HEADS) * DIM
        self.w_in = (torch.randn(HIDDEN, width, generator=g, device="cuda") * HIDDEN ** -0.5).half()
        self.w_out = (torch.randn(HEADS * DIM, HIDDEN, generator=g, device="cuda") * (HEADS * DIM) ** -0.5).half()
        pages_a_sequence = -(-longest // PAGE)
        self.cache = tg.KvCache.empty(batch * pages_a_sequence, KV_HEADS, PAGE, DIM, dtype=cache_dtype)
        order = torch.randperm(batch * pages_a_sequence, generator=torch.Generator().manual_seed(seed))
        self.table = order.to(torch.int32).view(batch, pages_a_sequence).cuda()
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.freq, self.amplitude = tg.rope_frequencies(DIM, scaling="yarn", factor=4.0, trained=256)
        self.longest = longest

    def step(self, x, cu, new, max_new):
        """x (tokens, HIDDEN) of the sequences' new tokens, packed at cu; new: how many each has."""
        qkv = tg.gemm(x, self.w_in).view(x.shape[0], HEADS + 2 * KV_HEADS, DIM)
        q, k, v = qkv[:, :HEADS], qkv[:, HEADS:HEADS + KV_HEADS], qkv[:, HEADS + KV_HEADS:]
        # the queries are rotated where the projection left them
        tg.kv_append(self.cache, k, v, self.table, self.lens, cu, max_new=max_new, Q=q, out=q, inv_freq=self.freq, amplitude=self.amplitude)
        self.lens += new
        o = tg.attention_kv(q, self.cache, self.table, self.lens, cu, max_new=max_new, max_len=self.longest)
        return x + tg.gemm(o.view(x.shape[0], HEADS * DIM), self.w_out)


class Plain:
    """The same layer in 32 bits, each sequence's keys and values kept as they are."""

    def __init__(self, layer, batch):
        self.w_in, self.w_out, self.freq, self.amplitude = layer.w_in.float(), layer.w_out.float(), layer.freq, layer.amplitude
        self.k, self.v = [torch.zeros(0, KV_HEADS, DIM, device="cuda")] * batch, [torch.zeros(0, KV_HEADS, DIM, device="cuda")] * batch

    def rotate(self, x, first):
        angle = torch.arange(first, first + x.shape[0], device="cuda", dtype=torch.float64)[:, None] * self.freq
        c, s = (angle.cos() * self.amplitude).float()[:, None], (angle.sin() * self.amplitude).float()[:, None]
        a, b = x[..., :DIM // 2], x[..., DIM // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1)

    def step(self, parts):
        out = []
        for i, x in enumerate(parts):
            qkv = (x.float() @ self.w_in).view(-1, HEADS + 2 * KV_HEADS, DIM)
            held = self.k[i].shape[0]
            q = self.rotate(qkv[:, :HEADS], held)
            self.k[i] = torch.cat([self.k[i], self.rotate(qkv[:, HEADS:HEADS + KV_HEADS], held)])
            self.v[i] = torch.cat([self.v[i], qkv[:, HEADS + KV_HEADS:]])
            k, v = (t.repeat_interleave(HEADS // KV_HEADS, 1) for t in (self.k[i], self.v[i]))
            score = torch.einsum("qhd,khd->hqk", q, k) * DIM ** -0.5
            hidden = torch.arange(k.shape[0], device="cuda")[None] > held + torch.arange(x.shape[0], device="cuda")[:, None]
            o = torch.einsum("hqk,khd->qhd", score.masked_fill(hidden, -torch.inf).softmax(-1), v)
            out.append(x.float() + o.reshape(x.shape[0], -1) @ self.w_out)
        return torch.cat(out)


def main(steps=16, cache="e4m3"):
    batch = len(PROMPTS)
    layer = Layer(batch, max(PROMPTS) + steps, torch.float8_e4m3fn if cache == "e4m3" else torch.int8)
    plain = Plain(layer, batch)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(sum(PROMPTS), HIDDEN, generator=g, device="cuda").half()
    cu = torch.tensor([0] + PROMPTS, device="cuda").cumsum(0).to(torch.int32)
    new = torch.tensor(PROMPTS, device="cuda", dtype=torch.int32)
    worst = []

    def compare(y, parts):
        want = plain.step(parts)
        base = torch.cat(parts).float()
        worst.append(((y.float() - want).norm() / (want - base).norm()).item())

    compare(layer.step(x, cu, new, max(PROMPTS)), list(x.split(PROMPTS)))

    # the decode step, captured once: one token a sequence, no offsets needed
    token = torch.randn(batch, HIDDEN, generator=g, device="cuda").half()
    one = torch.ones(batch, dtype=torch.int32, device="cuda")
    kept = [t.clone() for t in (layer.cache.k.view(torch.uint8), layer.cache.v.view(torch.uint8), layer.cache.k_scale, layer.cache.v_scale, layer.lens)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(token, None, one, 1)  # before the capture, as every kernel's first launch should be
    torch.cuda.current_stream().wait_stream(side)
    for t, was in zip((layer.cache.k.view(torch.uint8), layer.cache.v.view(torch.uint8), layer.cache.k_scale, layer.cache.v_scale, layer.lens), kept):
        t.copy_(was)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.step(token, None, one, 1)
    for _ in range(steps):
        token.copy_(torch.randn(batch, HIDDEN, generator=g, device="cuda"))
        graph.replay()
        compare(out, list(token.split(1)))
    status, where = tg.tg_device_status(None)
    assert status == tg.OK, (status, where)
    print(f"{cache} cache: prompts of {PROMPTS}, {steps} tokens each; attention branch off by {worst[0]:.4f} (prompts), "
          f"{max(worst[1:], default=0.0):.4f} (decode, largest) of its size")
    return worst


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--steps", type=int, default=16)
    p.add_argument("--cache", choices=["e4m3", "int8"], default="e4m3")
    main(**vars(p.parse_args()))
