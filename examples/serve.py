"""An attention layer served from the 8-bit paged key/value cache.

One layer of a decoder with E4M3 weights (gemm_dequant), its keys and values
in the paged cache, over the life of a few requests: whole prompts, then
steps in which each request adds a token and drafts, some of which the next
step drops again; requests that end give their pages back and new ones take
them.  Everything a step decides on the GPU stays there: lengths, block tables,
slots and the stack of free pages are never read by the host.

    python examples/serve.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_quantized_mx_gb300 as mx  # noqa: E402


class Layer:
    """hidden -> heads x d attention -> hidden, weights in E4M3."""

    def __init__(self, hidden, q_heads, heads, d, seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(k, n):
            w = torch.randn(k, n, generator=g) * k ** -0.5
            return mx.mx_quantize(w.cuda(), mx.E4M3, k_strided=True)

        self.q_heads, self.heads, self.d = q_heads, heads, d
        self.w_qkv = weight(hidden, (q_heads + 2 * heads) * d)
        self.w_out = weight(q_heads * d, hidden)

    def qkv(self, x):
        """Queries, keys and values of x's tokens, as views of one product."""
        y = mx.gemm_dequant(x, self.w_qkv, out_dtype=torch.bfloat16)
        y = y.view(x.shape[0], self.q_heads + 2 * self.heads, self.d)
        return y.split([self.q_heads, self.heads, self.heads], 1)

    def out(self, o):
        return mx.gemm_dequant(o.reshape(o.shape[0], -1), self.w_out, out_dtype=torch.bfloat16)


class Server:
    """The cache of a layer and the requests that live in it."""

    def __init__(self, layer, requests, pages, page, longest, most_new, fmt=mx.E4M3):
        i32 = dict(dtype=torch.int32, device="cuda")
        self.layer, self.page = layer, page
        self.cache = mx.empty_kv_cache(fmt, pages, layer.heads, page, layer.d)
        self.table = torch.full((requests, -(-longest // page)), -1, **i32)
        self.stack = torch.arange(pages - 1, -1, -1, **i32)
        self.counts = torch.tensor([pages, 0], **i32)
        self.lens = torch.zeros(requests, **i32)
        self.workspace = torch.empty(
            mx.kv_attention_workspace_bytes(layer.q_heads, layer.heads, layer.d, most_new),
            dtype=torch.uint8, device="cuda")

    def step(self, keep, new, x, most_new):
        """keep, new: what each request keeps of its tokens and how many it adds
        (int32, on the GPU); x: the new tokens' hidden states, request by
        request; most_new: the most any request adds.  Returns the layer's
        output for them, and what the attention saw."""
        cut = mx.mx_kv_truncate(self.lens, keep, self.table, self.stack, self.counts, self.page)
        plan = mx.mx_kv_extend(cut.lens, new, self.table, self.stack, cut.counts, self.page,
                               x.shape[0])
        self.lens, self.counts = plan.lens, plan.counts
        q, k, v = self.layer.qkv(x)
        mx.mx_kv_append(self.cache, k, v, plan.slots)
        o = mx.mx_kv_attention(q, self.cache, self.table, plan.lens, plan.cu, most_new,
                               workspace=self.workspace)
        return self.layer.out(o), q, o, plan


def main():
    mx.build()
    hidden, longest = 2048, 1024
    layer = Layer(hidden, 16, 4, 128)
    server = Server(layer, requests=8, pages=160, page=64, longest=longest, most_new=512)
    g = torch.Generator(device="cuda").manual_seed(1)
    lens = [0] * 8                               # what the host knows too
    drafts = 3
    for step in range(12):
        keep, new = list(lens), []
        for b in range(8):
            if step and lens[b] > 300:           # this one ends; a new one takes its place
                keep[b] = 0
            elif step and lens[b]:               # a request drops some of its drafts
                keep[b] = lens[b] - (step + b) % (drafts + 1)
            new.append(1 + drafts if keep[b] else 37 * (b + 1) + 11 * step)
        x = torch.randn(sum(new), hidden, generator=g, device="cuda").bfloat16()
        i32 = dict(dtype=torch.int32, device="cuda")
        y, _, _, plan = server.step(torch.tensor(keep, **i32), torch.tensor(new, **i32), x, max(new))
        lens = [k + n for k, n in zip(keep, new)]
        free, refused = plan.counts.tolist()     # for the print below; a server need not look
        print("step %2d: %4d new tokens, lengths %s, %3d pages free, |y| %.3f" %
              (step, sum(new), plan.lens.tolist(), free, y.float().abs().mean().item()))
        assert refused == 0 and plan.lens.tolist() == lens
    assert mx.mx_last_error() == 0


if __name__ == "__main__":
    main()
