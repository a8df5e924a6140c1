"""One decoder attention block served with the library, end to end.

The q/k/v and output projections are SERQ W4A4 linears; between them the
queries and keys are normed, rotated and stored (rope_append), prompts attend
in one packed call (attn_prefill), and every further token of all users in one
call over a prefix that they share (attn_decode), captured once in a HIP graph
and replayed.

    python examples/serve_attention.py

Weights and inputs are random; the block's own arithmetic is real.
"""

from __future__ import annotations

import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4a4_linear_layers_amd as S  # noqa: E402

HIDDEN, HQ, HKV, D, PAGE, MAX_POS = 1024, 8, 2, 128, 16, 4096


def rms(x):
    return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class AttentionBlock:
    """x -> x + o(attention(qkv(norm x))), its keys and values in a paged cache."""

    def __init__(self, n_pages: int, seed: int = 0):
        rng = np.random.default_rng(seed)
        width = (HQ + 2 * HKV) * D
        amax = np.full(HIDDEN, 4.0, np.float32)
        amax[rng.choice(HIDDEN, 10, replace=False)] = 60.0
        qkv = S.calibrate(rng.standard_normal((HIDDEN, width), dtype=np.float32) * 0.04, amax, r=64)
        out = S.calibrate(rng.standard_normal((HQ * D, HIDDEN), dtype=np.float32) * 0.04,
                          np.full(HQ * D, 3.0, np.float32), r=64)
        self.qkv, self.out = qkv.to("cuda"), out.to("cuda")
        # the linears take their inputs in saliency order
        self.order_in, self.order_out = self.qkv.perm.long(), self.out.perm.long()
        self.q_norm = torch.from_numpy(1 + 0.1 * rng.standard_normal(D).astype(np.float32)).cuda()
        self.k_norm = torch.from_numpy(1 + 0.1 * rng.standard_normal(D).astype(np.float32)).cuda()
        # trained to 1024 positions, served to 4096
        self.table = torch.from_numpy(S.rope_table(D, MAX_POS, theta=500000.0, scaling="bands", factor=4.0,
                                                   orig_len=1024)).cuda()
        self.cache = S.KvCache.empty(n_pages, HKV, PAGE, D)

    def queries(self, x, pos, slot):
        """The rows' queries; their keys and values are stored."""
        qkv = S.linear(*S.quant_act(rms(x)[:, self.order_in].contiguous(), self.qkv), self.qkv)
        return S.rope_append(qkv, HQ, self.cache, pos, slot, self.table, q_norm=self.q_norm, k_norm=self.k_norm)

    def finish(self, x, o):
        o = o.view(o.shape[0], HQ * D)[:, self.order_out].contiguous()
        return x + S.linear(*S.quant_act(o, self.out), self.out)

    def prefill(self, x, pos, slot, cu, pages, kv_len, max_len):
        return self.finish(x, S.attn_prefill(self.queries(x, pos, slot), cu, self.cache, pages, kv_len, max_len=max_len))


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def slots(pages, seq, at):
    """Slots of tokens `at` of the sequences `seq` (rows of page ids)."""
    return (pages[seq, at // PAGE] * PAGE + at % PAGE).to(torch.int32)


def serve(steps: int = 24, prefix_len: int = 5 * PAGE, prompts=(7, 33, 1, 20), seed: int = 0, graph: bool = True):
    """Prefills a shared prefix and one prompt per user, then decodes `steps`
    tokens for all of them. Returns every step's outputs (users x hidden) and
    what checks them: the block and its state."""
    users, room = len(prompts), -(-(max(prompts) + steps) // PAGE)
    lead = prefix_len // PAGE                        # whole pages, so that a prompt can continue the prefix's row
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    block = AttentionBlock(lead + users * room + 1, seed)
    order = torch.randperm(lead + users * room, generator=g, device="cuda").to(torch.int32)
    prefix, own = order[:lead].contiguous(), order[lead:].view(users, room).contiguous()

    def embed(n):
        return torch.randn(n, HIDDEN, generator=g, device="cuda").to(torch.bfloat16)

    # the prefix, once
    at = torch.arange(prefix_len, device="cuda")
    block.prefill(embed(prefix_len), at.int(), slots(prefix[None], 0, at), ints([0, prefix_len]), prefix[None].contiguous(),
                  ints([prefix_len]), prefix_len)
    # every user's prompt, packed; each sees the prefix's pages and its own
    cu = [0] + list(np.cumsum(prompts))
    seq = torch.repeat_interleave(torch.arange(users, device="cuda"), torch.tensor(prompts, device="cuda"))
    at = torch.arange(cu[-1], device="cuda") - torch.tensor(cu[:-1], device="cuda")[seq]
    pages = torch.cat([prefix.expand(users, -1), own], 1).contiguous()
    kv_len = ints([prefix_len + n for n in prompts])
    y = block.prefill(embed(cu[-1]), (at + prefix_len).int(), slots(own, seq, at), ints(cu), pages, kv_len,
                      prefix_len + max(prompts))
    x = y[torch.tensor(cu[1:], device="cuda") - 1].clone()         # each user's last row
    have = ints(list(prompts))                                     # tokens in the users' own pages
    everyone = torch.arange(users, device="cuda")
    max_own = max(prompts) + steps

    def step():
        pos, slot = have + prefix_len, slots(own, everyone, have.long())
        q = block.queries(x, pos, slot)
        have.add_(1)
        o = S.attn_decode(q, block.cache, own, have, max_len=max_own, prefix=prefix, prefix_len=prefix_len)
        x.copy_(block.finish(x, o))
        return q, o

    outs = []
    if graph:
        keep = x.clone(), have.clone(), block.cache.k.clone(), block.cache.v.clone()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):                              # once outside, as captures want it
            step()
        torch.cuda.current_stream().wait_stream(side)
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            q, o = step()
        for dst, src in zip((x, have, block.cache.k, block.cache.v), keep):
            dst.copy_(src)
        for _ in range(steps):
            captured.replay()
            outs.append(x.clone())
    else:
        for _ in range(steps):
            q, o = step()
            outs.append(x.clone())
    torch.cuda.synchronize()
    return outs, dict(block=block, q=q, o=o, pages=pages, kv_len=have + prefix_len, prefix_len=prefix_len,
                      max_len=prefix_len + max_own)


def check(state) -> float:
    """The last decode step against the prompt attention over the same keys
    (one new token a sequence, the prefix's pages in its own row): the largest
    difference."""
    users = state["q"].shape[0]
    cu = torch.arange(users + 1, dtype=torch.int32, device="cuda")
    again = S.attn_prefill(state["q"], cu, state["block"].cache, state["pages"], state["kv_len"],
                           max_len=state["max_len"])
    return float((again.float() - state["o"].float()).abs().max())


if __name__ == "__main__":
    outs, state = serve()
    eager, _ = serve(graph=False)
    same = all(torch.equal(a, b) for a, b in zip(outs, eager))
    print(f"{len(outs)} steps of {outs[0].shape[0]} users over {state['prefix_len']} shared tokens; "
          f"graph and eager {'agree bit for bit' if same else 'DIFFER'}; "
          f"decode against prompt attention: {check(state):.4f} at most")
