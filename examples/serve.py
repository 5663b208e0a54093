"""A decoder layer's attention half served from the 8-bit paged key/value cache.

h + attention(norm(h)), with E4M3 weights: the norm's output goes to MX codes in one
pass (mx_rmsnorm_quantize) and into the projection (mx_gemm), queries and keys are
turned to their positions (mx_rope), and the keys and values stand in the paged
cache, over the life of a few requests: whole prompts, then steps in which each
request adds a token and drafts, some of which the next step drops again; requests
that end give their pages back and new ones take them.  Requests may be forked: samples of
one prompt hold its pages together, get a copy of the last one when they write
it, and attend to what they share once for all.  Everything a step decides on the GPU
stays there: lengths, block tables, holders, slots and the stack of free pages are
never read by the host.

    python examples/serve.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_quantized_mx_gb300 as mx  # noqa: E402


class Layer:
    """hidden -> norm -> heads x d attention -> hidden, weights in E4M3."""

    def __init__(self, hidden, q_heads, heads, d, seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(k, n):
            w = torch.randn(k, n, generator=g) * k ** -0.5
            return mx.mx_quantize(w.cuda(), mx.E4M3, k_strided=True)

        self.q_heads, self.heads, self.d = q_heads, heads, d
        self.norm = 1.0 + 0.1 * torch.randn(hidden, generator=g).cuda()
        self.w_qkv = weight(hidden, (q_heads + 2 * heads) * d)
        self.w_out = weight(q_heads * d, hidden)
        self.rope = mx.rope_frequencies(d)

    def qkv(self, x, plan):
        """Queries, keys and values of x's tokens, as views of one product; queries
        and keys at their positions."""
        a, _ = mx.mx_rmsnorm_quantize(x, self.norm, mx.E4M3)
        y = mx.mx_gemm(a, self.w_qkv, out_dtype=torch.bfloat16)
        y = y.view(x.shape[0], self.q_heads + 2 * self.heads, self.d)
        q, k, v = y.split([self.q_heads, self.heads, self.heads], 1)
        mx.mx_rope(q, k, self.rope, lens=plan.lens, cu=plan.cu, out=(q, k))
        return q, k, v

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
        self.refs = torch.zeros(pages, **i32)
        self.lens = torch.zeros(requests, **i32)
        self.shared = torch.full((requests,), longest, **i32)     # as much as there is
        # for up to most_new rows of each request, each request a group of its own
        self.workspace = torch.empty(
            mx.kv_attention_shared_workspace_bytes(requests * most_new, layer.q_heads, layer.heads,
                                                   layer.d, most_new, requests, requests),
            dtype=torch.uint8, device="cuda")

    def step(self, keep, new, x, most_new, fork=None, groups=None):
        """keep, new: what each request keeps of its tokens and how many it adds
        (int32, on the GPU); x: the new tokens' hidden states, request by
        request; most_new: the most any request adds.  fork: (src, dst, tokens),
        requests that begin as copies of others' first tokens; groups: offsets of requests
        that may have a prefix in common, which stand side by side.  Returns the layer's output for the new tokens, and
        what the attention saw."""
        cut = mx.mx_kv_release(self.lens, keep, self.table, self.stack, self.counts, self.refs,
                               self.page)
        lens = cut.lens
        if fork is not None:
            lens = mx.mx_kv_fork(lens, *fork, self.table, self.refs, self.page).lens
        own = mx.mx_kv_own(self.cache, lens, new, self.table, self.stack, cut.counts, self.refs)
        plan = mx.mx_kv_extend(lens, own.new_tokens, self.table, self.stack, own.counts, self.page,
                               x.shape[0])
        self.lens, self.counts = plan.lens, plan.counts
        q, k, v = self.layer.qkv(x, plan)
        mx.mx_kv_append(self.cache, k, v, plan.slots)
        if groups is None:
            o = mx.mx_kv_attention(q, self.cache, self.table, plan.lens, plan.cu, most_new,
                                   workspace=self.workspace)
        else:
            o = mx.mx_kv_attention_shared(q, self.cache, self.table, plan.lens, plan.cu, most_new,
                                          groups, self.shared, workspace=self.workspace)
        return self.layer.out(o) + x, q, o, plan


def main():
    mx.build()
    hidden, longest = 2048, 1024
    layer = Layer(hidden, 16, 4, 128)
    server = Server(layer, requests=8, pages=160, page=64, longest=longest, most_new=512)
    g = torch.Generator(device="cuda").manual_seed(1)
    i32 = dict(dtype=torch.int32, device="cuda")
    lens = [0] * 8                               # what the host knows too
    drafts = 3

    def step(name, keep, new, **kw):
        x = torch.randn(sum(new), hidden, generator=g, device="cuda").bfloat16()
        y, _, _, plan = server.step(torch.tensor(keep, **i32), torch.tensor(new, **i32), x, max(new),
                                    **kw)
        free, refused = plan.counts.tolist()     # for the print below; a server need not look
        print("%s: %4d new tokens, lengths %s, %3d pages free, |y| %.3f" %
              (name, sum(new), plan.lens.tolist(), free, y.float().abs().mean().item()))
        assert refused == 0

    for i in range(12):
        keep, new = list(lens), []
        for b in range(8):
            if i and lens[b] > 300:              # this one ends; a new one takes its place
                keep[b] = 0
            elif i and lens[b]:                  # a request drops some of its drafts
                keep[b] = lens[b] - (i + b) % (drafts + 1)
            new.append(1 + drafts if keep[b] else 37 * (b + 1) + 11 * i)
        step("step %2d" % i, keep, new)
        lens = [k + n for k, n in zip(keep, new)]
        assert server.lens.tolist() == lens
    # one long prompt, and seven samples of it
    step("prompt ", [0] * 8, [500] + [0] * 7)
    fork = [torch.tensor(v, **i32) for v in ([0] * 7, list(range(1, 8)), [500] * 7)]
    groups = torch.tensor([0, 8], **i32)
    keep, lens = [500] + [0] * 7, [500] * 8
    for i in range(3):
        step("sample %d" % i, keep, [1] * 8, groups=groups, fork=None if i else fork)
        keep = lens = [n + 1 for n in lens]
    step("release ", [0] * 8, [1] + [0] * 7)
    assert server.counts.tolist()[0] == 159 and server.refs.sum().item() == 0
    assert mx.mx_last_error() == 0


if __name__ == "__main__":
    main()
