"""One attention block of a transformer on quantised operators, as a serving loop would run it.

  query/key/value projection: 8-bit weights and 8-bit activations per token, under the scales of
                              the activation-aware search on calibration tokens;
  key/value cache:            4 bits, paged;
  attention:                  over the cache, prompts and single tokens through the same calls;
  output projection:          4-bit weights packed under its own search's scales, 16-bit activations.

Random weights and inputs: the point is the order of the calls.  A batch of prompts of different
lengths is taken in, then decoded a token at a time, the decoding step once as plain calls and
once captured into a HIP graph and replayed while lengths and inputs change.

    python examples/quantized_attention.py [--tokens 16]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import weight_only_quantization_act_amd as awq  # noqa: E402


class Block:
    """Weights, cache and page tables of one attention block (fp16)."""

    def __init__(self, hidden=4096, heads=32, kv_heads=8, head_dim=128, max_seqs=4, max_len=1024,
                 seed=0, device="cuda"):
        g = torch.Generator(device=device).manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.max_len = heads, kv_heads, head_dim, max_len
        rows = (heads + 2 * kv_heads) * head_dim
        w_qkv = torch.randn(rows, hidden, generator=g, device=device).half() * hidden ** -0.5
        w_out = torch.randn(hidden, heads * head_dim, generator=g, device=device).half() * hidden ** -0.5
        calib = torch.randn(512, hidden, generator=g, device=device).half()
        calib[:, ::97] *= 8  # a few channels stand out, as in real activations

        # the activation-aware search of both layers on the calibration tokens: the projection's scales
        # go into its 8-bit weights, the output layer is packed with its own to 4 bits
        self.w_qkv, self.w_out, self.calib = w_qkv, w_out, calib
        self.cfg4 = awq.qconfig(w_bit=4, group_size=128, zero_point=1)
        self.alphas = [i / 20 for i in range(20)]
        search = awq.awq_search_scales(w_qkv, calib, awq.awq_act_stats(calib), self.alphas, self.cfg4)
        self.s = search["s"]
        self.wq, self.wstep = awq.awq_int8_quantize(w_qkv, self.s, fold="multiply")
        layer = awq.quantize_layer(w_out, self.attend_plain(calib).half(), self.alphas, self.cfg4)
        self.s_out = layer["s"]
        self.codes, self.scales, self.zeros = layer["codes"], layer["scales"], layer["zeros"]

        self.kv = awq.awq_kv4_config(head_dim, kv_heads, page_size=64, group_size=64, zero_point=1)
        pages = -(-max_len // 64)
        self.cache = awq.awq_kv4_cache(max_seqs * pages, self.kv, device=device)
        self.table = torch.randperm(max_seqs * pages, generator=g, device=device).to(torch.int32)
        self.table = self.table.reshape(max_seqs, pages).contiguous()

    def forward(self, x, lens, starts, max_q, max_len=None):
        """x [tokens, hidden]: the last tokens of each sequence; lens, starts: as the cache takes
        them.  Returns [tokens, hidden]."""
        T, H, Hk, D = x.shape[0], self.heads, self.kv_heads, self.dim
        qkv = awq.awq_int8_linear(x, self.wq, self.wstep, s=self.s)
        # views into the projection's output: the cache and the attention take strides
        q, k, v = qkv.view(T, H + 2 * Hk, D).split([H, Hk, Hk], dim=1)
        awq.awq_kv4_append(k, v, self.cache, self.table, lens, starts, self.kv)
        o, _ = awq.awq_kv4_attention(q, self.cache, self.table, lens, starts, self.kv, max_q=max_q,
                                     max_len=max_len or self.max_len)
        return awq.awq_w4a16_matmul(o.view(T, H * D), self.codes, self.scales, self.zeros, self.cfg4,
                                    s=self.s_out)

    def attend_plain(self, x):
        """Projection and attention on 16-bit weights and keys, one whole sequence, in fp32."""
        T, H, Hk, D = x.shape[0], self.heads, self.kv_heads, self.dim
        qkv = (x.float() @ self.w_qkv.float().t()).view(T, H + 2 * Hk, D)
        q, k, v = qkv.split([H, Hk, Hk], dim=1)
        k, v = (t.repeat_interleave(H // Hk, dim=1).transpose(0, 1).contiguous() for t in (k, v))
        s = torch.matmul(q.transpose(0, 1).contiguous(), k.transpose(1, 2).contiguous()) * D ** -0.5
        s = s.masked_fill(torch.ones(T, T, dtype=torch.bool, device=x.device).triu(1), float("-inf"))
        return torch.matmul(s.softmax(-1), v).transpose(0, 1).reshape(T, H * D)

    def plain(self, x):
        """The whole block so."""
        return self.attend_plain(x) @ self.w_out.float().t()


def run(tokens=16, hidden=4096, heads=32, kv_heads=8, prompts=(200, 1, 77), max_len=1024):
    """Prompts, then `tokens` decoding steps; returns the block's outputs by sequence (prompt rows
    and decoded rows in order), those of the plain block, and the graph's last step against the
    plain calls'."""
    block = Block(hidden, heads, kv_heads, max_seqs=len(prompts), max_len=max_len)
    n = len(prompts)
    g = torch.Generator(device="cuda").manual_seed(1)
    x = [torch.randn(p + tokens, hidden, generator=g, device="cuda").half() for p in prompts]

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    # the prompts, all in one call
    starts = [0]
    for p in prompts:
        starts.append(starts[-1] + p)
    y = block.forward(torch.cat([x[b][:p] for b, p in enumerate(prompts)]), ints(list(prompts)), ints(starts),
                      max_q=max(prompts), max_len=max(prompts))
    out = [[y[starts[b]:starts[b + 1]]] for b in range(n)]

    # one token of every sequence a step
    one_each = ints(list(range(n + 1)))
    for i in range(tokens):
        row = torch.stack([x[b][p + i] for b, p in enumerate(prompts)])
        y = block.forward(row, ints([p + i + 1 for p in prompts]), one_each, max_q=1)
        for b in range(n):
            out[b].append(y[b:b + 1])
    last = y

    # the same steps as a graph: captured once, replayed with new lengths and inputs
    row, lens = torch.zeros(n, hidden, device="cuda").half(), ints([1] * n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.forward(row, lens, one_each, max_q=1)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        replayed = block.forward(row, lens, one_each, max_q=1)
    # (the first tokens were overwritten by the zeros above: take the prompts in once more)
    block.forward(torch.cat([x[b][:p] for b, p in enumerate(prompts)]), ints(list(prompts)), ints(starts),
                  max_q=max(prompts), max_len=max(prompts))
    for i in range(tokens):
        row.copy_(torch.stack([x[b][p + i] for b, p in enumerate(prompts)]))
        lens.copy_(ints([p + i + 1 for p in prompts]))
        graph.replay()
    return [torch.cat(o) for o in out], [block.plain(t) for t in x], replayed, last


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--tokens", type=int, default=16)
    got, want, replayed, last = run(ap.parse_args().tokens)
    for b, (o, w) in enumerate(zip(got, want)):
        print(f"sequence {b}: {len(o)} rows, difference to the 16-bit block "
              f"{float((o.float() - w).norm() / w.norm()):.4f} of its norm")
    print("graph replays equal the plain calls:", bool(torch.equal(replayed, last)))


if __name__ == "__main__":
    main()
