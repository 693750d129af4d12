"""The attention block of a layer over quantized weights and a paged cache, as a server runs it.

    python -m gguf_block_quantized_gb300.attn_block [--type f16|q8_0] [--prompt 512] [--steps 16] [--seqs 4]

One grouped product makes q, k and v, syn_kv_append rotates q and k and writes the cache, the
attention reads it, and one product brings the result back to the model's width.  The command runs a
prompt of every sequence through the prefill form, then tokens one at a time through the decode form
captured as one CUDA graph, and compares each token's output with the prefill form's for the same
token.  The shapes are the attn_* matrices of a Llama-1B-shaped layer (Q4_K, 32 / 8 heads of 64).
"""
from __future__ import annotations

import argparse

from .workloads import F16, LLAMA1B_LAYER, Q8_0


class AttnBlock:
    """q, k, v and output weights (type, blocks, n_out, n_in each) with a cache and a rotation."""

    def __init__(self, weights: dict, cache, rope, n_heads: int, **options):
        self.w, self.cache, self.rope, self.n_heads, self.options = weights, cache, rope, n_heads, options
        self.dim = cache.head_dim

    def _steps(self, x, out, pos, slots, attend, stream):
        """The block's calls for n tokens, prepared over buffers of their own."""
        import torch

        from . import syn
        n, kv, dim = x.shape[0], self.cache.n_kv_heads, self.dim
        q = torch.empty((n, self.n_heads, dim), device=x.device)
        k, v = (torch.empty((n, kv, dim), device=x.device) for _ in range(2))
        mixed = torch.empty((n, self.n_heads, dim), device=x.device)
        q_rot = torch.empty(q.shape, dtype=torch.float16, device=x.device)
        products = syn.prepare_batch([(*self.w[name], x, y) for name, y in (("q", q), ("k", k), ("v", v))], n, stream=stream)
        append = syn.prepare_kv_append(self.cache, self.rope, k, v, pos, slots, q=q, q_out=q_rot, stream=stream)
        last = syn.prepare_batch([(*self.w["output"], mixed.view(n, -1), out)], n, stream=stream)
        return products, append, attend(q_rot, mixed, stream), last

    def prepare_prompt(self, x, out, pos, slots, starts, pages, lens, stream=None):
        """New tokens of several sequences (syn_attn_prefill); x and out: (n_tok, model width) fp32."""
        from . import syn
        steps = self._steps(x, out, pos, slots, lambda q, y, s: syn.prepare_attn_prefill(
            self.cache, q, starts, pages, lens, y, stream=s, **self.options), stream)
        return lambda: [step() for step in steps][-1]

    def prepare_token(self, x, out, pos, slots, pages, lens, stream=None):
        """One new token of each sequence (syn_attn_decode)."""
        from . import syn
        steps = self._steps(x, out, pos, slots, lambda q, y, s: syn.prepare_attn_decode(
            self.cache, q, pages, lens, y, stream=s, **self.options), stream)
        return lambda: [step() for step in steps][-1]


def llama1b_block(cache_type: int, seqs: int, rows: int, page: int = 64, seed: int = 7, **options):
    """A block with random Q4_K weights, its page table (seqs, pages) and the slot of row j of
    sequence s: slots[s, j]."""
    import torch

    from . import syn, synth
    heads, kv, dim = 32, 8, 64
    shapes = {m.name.removeprefix("attn_"): m for m in LLAMA1B_LAYER if m.name.startswith("attn_")}
    weights = {}
    for i, (name, m) in enumerate(shapes.items()):
        w = torch.from_numpy(synth.normal(seed + i, (m.n_out, m.n_in), 0.02)).cuda()
        weights[name] = (m.wtype, syn.quantize(m.wtype, w), m.n_out, m.n_in)
    per = -(-rows // page)
    cache = syn.KVCache.empty(cache_type, kv, dim, page, seqs * per)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    pages = torch.randperm(seqs * per, device="cuda", generator=gen).to(torch.int32).view(seqs, per)
    row = torch.arange(rows, device="cuda")
    slots = pages[:, row // page].long() * page + row % page
    rope = syn.Rope(dim, 500000.0, layout=syn.ROPE_ADJACENT)
    return AttnBlock(weights, cache, rope, heads, **options), pages, slots


def run(cache_type: int, prompt: int, steps: int, seqs: int) -> dict:
    """The prompt, then `steps` tokens from a graph: the largest difference of a token's output from the
    prefill form's, relative to the largest output, and both times (us)."""
    import torch

    from . import syn
    rows = prompt + steps
    block, pages, slots = llama1b_block(cache_type, seqs, rows)
    width = block.w["q"][3]
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn((seqs, rows, width), device="cuda", generator=gen)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        def prefill(n):  # rows 0 .. n - 1 of every sequence
            out = torch.empty((seqs * n, width), device="cuda")
            call = block.prepare_prompt(
                x[:, :n].reshape(-1, width), out, torch.arange(n, dtype=torch.int32, device="cuda").repeat(seqs),
                slots[:, :n].reshape(-1), torch.arange(0, seqs * n + 1, n, dtype=torch.int32, device="cuda"), pages,
                torch.full((seqs,), n, dtype=torch.int32, device="cuda"))
            return call, out.view(seqs, n, width)

        def timed(call):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            call()
            b.record()
            b.synchronize()
            return a.elapsed_time(b) * 1e3

        whole, want = prefill(rows)
        whole()
        want = want.clone()
        block.cache.k.zero_()
        block.cache.v.zero_()
        first, got = prefill(prompt)
        first()
        us_prompt = timed(first)
        diff = (got - want[:, :prompt]).abs().max()
        token = torch.empty((seqs, width), device="cuda")
        out = torch.empty((seqs, width), device="cuda")
        pos = torch.empty(seqs, dtype=torch.int32, device="cuda")
        at = torch.empty(seqs, dtype=torch.int64, device="cuda")
        lens = torch.empty(seqs, dtype=torch.int32, device="cuda")
        step = block.prepare_token(token, out, pos, at, pages, lens)

        def load(j):
            token.copy_(x[:, j])
            pos.fill_(j)
            at.copy_(slots[:, j])
            lens.fill_(j + 1)

        load(prompt)
        step()  # allocates the workspaces
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        us_token = []
        for j in range(prompt, rows):
            load(j)
            us_token.append(timed(graph.replay))
            diff = torch.maximum(diff, (out - want[:, j]).abs().max())
    torch.cuda.synchronize()
    syn.check(syn.device_status(), "device status")
    return {"difference": float(diff / want.abs().max()), "us_prompt": us_prompt, "us_token": sorted(us_token)[len(us_token) // 2]}


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--type", choices=("f16", "q8_0"), default="f16")
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--seqs", type=int, default=4)
    a = ap.parse_args()
    r = run(Q8_0 if a.type == "q8_0" else F16, a.prompt, a.steps, a.seqs)
    print(f"{a.seqs} sequences, {a.type} cache: prompt of {a.prompt} tokens {r['us_prompt']:.1f} us, one token of each "
          f"{r['us_token']:.1f} us; largest difference between the two forms {r['difference']:.2e} of the largest output")


if __name__ == "__main__":
    main()
