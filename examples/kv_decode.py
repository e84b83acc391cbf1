"""One attention block of a decoder served with 4-bit weights and a 4-bit key/value cache.

A batch of prompts of different lengths is prefilled and then decoded token by token:

    plan       block tables, slots and positions of the step, on the GPU (kv_plan)
    project    q, k, v from the hidden states with NVFP4 weights (qmm for many rows, qmv_batch for few)
    append     the new keys and values, quantized into their pages (kv_append)
    attend     softmax attention over the cache (kv_attention)
    project    back to the hidden size, added to the hidden states

The decode step runs from a HIP graph: lengths, tables and pages live on the GPU, so the captured step serves
every token.  `--check` runs the block again in fp32 on the values the weights and the cache stand for.

    python examples/kv_decode.py [--steps N] [--check]
"""
import argparse
import math
import os
import sys
import time

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import block_scaled_bit_fp_amd as bs  # noqa: E402


class Block:
    """Weights, cache and tables of one attention block."""

    def __init__(self, hidden=5120, heads=64, kv_heads=8, head_dim=128, page_size=64, pages=256,
                 requests=8, max_pages=32, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=gen, device="cuda") * 0.02
            return bs.quantize(w.to(torch.bfloat16), bs.NVFP4)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim
        self.wq = weight(heads * head_dim, hidden)
        self.wk = weight(kv_heads * head_dim, hidden)
        self.wv = weight(kv_heads * head_dim, hidden)
        self.wo = weight(hidden, heads * head_dim)
        # global scales of the cache: the largest magnitude expected over 448 * 6
        amax = 6.0 * 0.02 * math.sqrt(hidden)
        self.cache = bs.empty_kv_cache(
            bs.NVFP4, pages, kv_heads, head_dim, page_size=page_size,
            k_scale=torch.full((1,), amax / 2688, device="cuda"),
            v_scale=torch.full((1,), amax / 2688, device="cuda"))
        self.table = torch.full((requests, max_pages), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        self.begin = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(self, x, q_lens, max_q, workspace):
        """The new tokens' hidden states x [tokens, hidden] through the block; returns (y, batch, the
        attention's output).  q_lens: new tokens of each request (device int32), at most max_q."""
        T, h = x.shape[0], self.normed(x)
        batch = bs.kv_plan(self.lens, q_lens, self.table, self.free, self.begin, tokens=T,
                           page_size=self.cache.page_size)
        if T <= 8:
            q, k, v = bs.qmv_batch(h, [self.wq, self.wk, self.wv])
        else:
            q, k, v = (bs.qmm(h, w) for w in (self.wq, self.wk, self.wv))
        D = self.head_dim
        bs.kv_append(self.cache, k.view(T, self.kv_heads, D), v.view(T, self.kv_heads, D), batch.slots)
        o = bs.kv_attention(q.view(T, self.heads, D), self.cache, batch, max_q=max_q, workspace=workspace)
        o = o.view(T, self.heads * D)
        y = x + (bs.qmv(o, self.wo) if T <= 8 else bs.qmm(o, self.wo))
        # the step's lengths and free pages are the next one's
        self.lens.copy_(batch.next_lens)
        self.begin.copy_(batch.state[:1])
        return y, batch, o

    @staticmethod
    def normed(x):
        f = x.float()
        return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def workspace(self, tokens, max_q):
        return bs.kv_attention_workspace(tokens, self.heads, self.cache, self.lens.numel(), max_q)

    def reference(self, x, batch):
        """The attention output of the step in fp32, on the values that weights and cache stand for."""
        D, H, Hk, P = self.head_dim, self.heads, self.kv_heads, self.cache.page_size
        q = (self.normed(x).float() @ bs.dequantize(self.wq).float().T).to(torch.bfloat16).float().view(-1, H, D)
        k, v = (bs.dequantize(t).float().view(-1, Hk, P, D) for t in (self.cache.k, self.cache.v))
        out = torch.zeros_like(q)
        starts, lens = batch.q_starts.tolist(), batch.kv_lens.tolist()
        for r, L in enumerate(lens):
            a, b = starts[r], starts[r + 1]
            if a == b or L == 0:
                continue
            pages = self.table[r, :-(-L // P)].long()
            kr, vr = (t[pages].transpose(0, 1).reshape(Hk, -1, D)[:, :L] for t in (k, v))
            s = torch.matmul(q[a:b].view(b - a, Hk, H // Hk, D).permute(1, 2, 0, 3).reshape(Hk, -1, D),
                             kr.transpose(1, 2).contiguous()).view(Hk, H // Hk, b - a, L) / math.sqrt(D)
            at = torch.arange(L, device="cuda")
            s.masked_fill_(at > torch.arange(L - (b - a), L, device="cuda")[:, None], -math.inf)
            o = torch.matmul(torch.softmax(s, -1).view(Hk, -1, L), vr.contiguous())
            out[a:b] = o.view(Hk, H // Hk, b - a, D).permute(2, 0, 1, 3).reshape(b - a, H, D)
        return out.view(-1, H * D)


def serve(block, prompt_lens, steps, check=False, seed=1):
    """Prefills the prompts, then decodes `steps` tokens of each from a HIP graph.  Returns the largest
    error against the fp32 reference, relative to its root mean square (0 without check), and the
    milliseconds per decode step."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    hidden, R = block.wq.cols, len(prompt_lens)
    worst = 0.0

    def compare(x, batch, o):
        want = block.reference(x, batch)
        return float((o.float() - want).abs().max() / want.square().mean().sqrt())

    T = sum(prompt_lens)
    x = torch.randn((T, hidden), generator=gen, device="cuda").to(torch.bfloat16)
    y, batch, o = block.step(x, torch.tensor(prompt_lens, dtype=torch.int32, device="cuda"),
                             max(prompt_lens), block.workspace(T, max(prompt_lens)))
    if check:
        worst = max(worst, compare(x, batch, o))
    x = y[batch.q_starts[1:].long() - 1].contiguous()

    one, workspace = torch.ones(R, dtype=torch.int32, device="cuda"), block.workspace(R, 1)
    state = block.lens.clone(), block.begin.clone()
    side = torch.cuda.Stream()  # a step outside the graph first, undone after
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x, one, 1, workspace)
    torch.cuda.current_stream().wait_stream(side)
    block.lens.copy_(state[0])
    block.begin.copy_(state[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, batch, o = block.step(x, one, 1, workspace)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    for _ in range(steps):
        graph.replay()
        if check:
            worst = max(worst, compare(x, batch, o))
        x.copy_(y)
    torch.cuda.synchronize()
    ms = (time.perf_counter() - t0) / max(steps, 1) * 1e3
    if int(batch.state[1]):
        raise RuntimeError("the page pool is too small: requests were refused")
    return worst, ms


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=64)
    ap.add_argument("--check", action="store_true")
    args = ap.parse_args()
    prompts = [700, 33, 1, 512, 129, 64, 257, 900]
    worst, ms = serve(Block(), prompts, args.steps, check=args.check)
    print(f"{len(prompts)} requests, prompts of {min(prompts)} to {max(prompts)} tokens, {args.steps} steps: "
          f"{ms:.3f} ms per step" + (f" (checked), largest error {worst:.4f} of the rms" if args.check else ""))


if __name__ == "__main__":
    main()
