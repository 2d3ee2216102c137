"""The attention half of a decoder layer on quantized projections: prompts are
prefilled in chunks, then every sequence grows token by token from one captured
CUDA graph.

    x -> linear (fused q, k, v) -> kv_append (rotary positions, paged cache)
      -> paged_attention -> linear (output)

Weights are random int4; the script checks itself: what the growing cache gives
for the last token of each sequence must be what one chunk over the whole
sequence gives. With an 8-bit cache the heads of queries and keys are divided by
their norms too, in the same launch that rotates and stores them.

    python examples/decoder_attention.py [--steps 8] [--hidden 1024] [--cache 16 | int8 | e4m3]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import w4a16_group_quantized_linear_gb300 as w4  # noqa: E402


CACHES = {"16": torch.float16, "int8": torch.int8, "e4m3": torch.float8_e4m3fn}


class AttentionLayer:
    """Quantized projections, a paged cache and the pages of each sequence."""

    def __init__(self, hidden, heads, kv_heads, head_dim, sequences, places, page=16, seed=0, cache="16"):
        dev = "cuda"
        gen = torch.Generator(device=dev).manual_seed(seed)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        rows = (heads + 2 * kv_heads) * head_dim
        self.w_qkv = w4.pack(torch.randn(rows, hidden, generator=gen, device=dev) * hidden ** -0.5)
        self.w_out = w4.pack(torch.randn(hidden, heads * head_dim, generator=gen, device=dev) * hidden ** -0.5)
        self.table = w4.rope_table(places, head_dim, device=dev)
        per = -(-places // page)
        shape = (sequences * per, page, kv_heads, head_dim)
        self.k, self.v = (torch.empty(shape, dtype=CACHES[cache], device=dev) for _ in range(2))
        self.scales, self.norms = {}, {}
        if cache != "16":
            shape = (sequences * per, kv_heads, page)
            self.scales = {name: torch.empty(shape, device=dev) for name in ("k_scale", "v_scale")}
            self.norms = {name: 1 + 0.1 * torch.randn(head_dim, generator=gen, device=dev)
                          for name in ("q_norm", "k_norm")}
        # any assignment of pages will do
        self.pages = torch.randperm(sequences * per, generator=gen, device=dev).to(torch.int32).view(sequences, per)

    def __call__(self, x, q_offsets, kv_lens, max_q_len):
        """x fp16 [T, hidden], the new tokens of all sequences one after another."""
        H, G, D = self.heads, self.kv_heads, self.head_dim
        qkv = w4.linear(x, *self.w_qkv).unflatten(1, (H + 2 * G, D))
        batch = (self.k, self.v, self.pages[:kv_lens.shape[0]], q_offsets, kv_lens)
        q = w4.kv_append(qkv[:, H:H + G], qkv[:, H + G:], *batch, q=qkv[:, :H], table=self.table, **self.scales,
                         **self.norms)
        y = w4.paged_attention(q, *batch, max_q_len, **self.scales)
        return w4.linear(y.flatten(1), *self.w_out)


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(lens):
    return _ints([sum(lens[:i]) for i in range(len(lens) + 1)])


def run(prompts=(37, 300, 5), steps=8, hidden=1024, heads=16, kv_heads=4, head_dim=64, chunk=128, seed=0,
        cache="16"):
    """Returns (last tokens' outputs from the growing cache, the same from one
    chunk over each whole sequence): fp16 [sequences, hidden] twice."""
    B = len(prompts)
    total = [n + steps for n in prompts]
    layer, check = (AttentionLayer(hidden, heads, kv_heads, head_dim, B, max(total), seed=seed, cache=cache)
                    for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(seed + 1)
    tokens = [torch.randn(n, hidden, generator=gen, device="cuda").half() for n in total]

    # prompts in chunks: every call takes what is left of each sequence, up to `chunk`
    done = [0] * B
    while any(d < n for d, n in zip(done, prompts)):
        new = [min(chunk, n - d) for d, n in zip(done, prompts)]
        x = torch.cat([t[d:d + n] for t, d, n in zip(tokens, done, new)])
        done = [d + n for d, n in zip(done, new)]
        layer(x, _offsets(new), _ints(done), max(new))

    # then a token of each sequence per step, one graph for them all: the lengths are on the device
    offsets, lens = _offsets([1] * B), _ints(done)
    x = torch.empty(B, hidden, dtype=torch.float16, device="cuda")
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        x.copy_(torch.cat([t[d:d + 1] for t, d in zip(tokens, done)]))
        lens += 1
        y = layer(x, offsets, lens, 1)  # the first step, which also allocates
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y = layer(x, offsets, lens, 1)
        for step in range(1, steps):
            x.copy_(torch.cat([t[d + step:d + step + 1] for t, d in zip(tokens, done)]))
            lens += 1
            graph.replay()
        if steps == 1:
            graph.replay()  # the same token again, the same place
    torch.cuda.current_stream().wait_stream(stream)

    whole = check(torch.cat(tokens), _offsets(total), _ints(total), max(total))
    ends = [sum(total[:i + 1]) - 1 for i in range(B)]
    w4.device_status()
    return y, whole[ends]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--cache", choices=sorted(CACHES), default="16")
    a = ap.parse_args()
    grown, whole = run(steps=a.steps, hidden=a.hidden, cache=a.cache)
    worst = (grown.float() - whole.float()).abs().max().item()
    scale = whole.float().abs().max().item()
    print(f"{grown.shape[0]} sequences, {a.steps} tokens each from one graph: "
          f"largest difference {worst:.2e} of values up to {scale:.2e}")
    if worst > 0.01 * scale:
        raise SystemExit("the growing cache and the whole chunk disagree")


if __name__ == "__main__":
    main()
