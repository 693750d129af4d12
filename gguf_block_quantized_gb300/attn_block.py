"""The attention block of a layer over quantized weights and a paged cache, as a server runs it.

    python -m gguf_block_quantized_gb300.attn_block [--type f16|q8_0] [--prompt 512] [--steps 16] [--seqs 4] [--draft NODES]

One grouped product makes q, k and v, syn_kv_append rotates q and k and writes the cache, the
attention reads it, and one product brings the result back to the model's width.  The command runs a
prompt of every sequence through the prefill form, then tokens one at a time through the decode form
captured as one CUDA graph, and compares each token's output with the prefill form's for the same
token.  With --draft it decodes speculatively instead: the prompt's pages are forked to every sequence,
and each step verifies a tree of drafted tokens in one call (syn_kv_extend, the block with syn_attn_tree, a
vocabulary product, syn_logprobs) and keeps the accepted path (syn_kv_compact, syn_kv_trim); the
tokens' log probabilities are compared with those of decoding one token at a time.  The shapes are the attn_* matrices of a Llama-1B-shaped layer (Q4_K, 32 / 8 heads of 64).
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


    def prepare_draft(self, x, out, pos, slots, starts, parents, pages, lens, stream=None):
        """Drafted tokens, nodes of a tree for each sequence (syn_attn_tree); pos: the context's length plus
        each node's depth."""
        from . import syn
        steps = self._steps(x, out, pos, slots, lambda q, y, s: syn.prepare_attn_tree(
            self.cache, q, starts, parents, pages, lens, y, stream=s, **self.options), stream)
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


def _draft(gen, sure, vocab: int, nodes: int):
    """A drafter's tree for one sequence: sure[0] is the token to come, sure[1:] what will follow it; a node has the right
    token to follow among up to three children seven times of ten.  -> tokens, parents, depths."""
    tokens, parents, depths, right = [sure[0]], [-1], [0], [0]
    while len(tokens) < nodes:
        at = right[-1] if gen.random() < 0.8 else gen.randrange(len(tokens))
        d = depths[at] + 1
        on_path = at == right[-1] and at == right[depths[at]] and d < len(sure)
        children = [gen.randrange(vocab) for _ in range(min(gen.randint(1, 3), nodes - len(tokens)))]
        if on_path and gen.random() < 0.7:
            children[gen.randrange(len(children))] = sure[d]
        for c in children:
            if on_path and c == sure[d] and len(right) == d:
                right.append(len(tokens))
            tokens.append(c)
            parents.append(at)
            depths.append(d)
    return tokens, parents, depths


def run_drafts(cache_type: int, prompt: int, tokens: int, seqs: int, nodes: int, vocab: int = 32000, page: int = 64) -> dict:
    """`tokens` tokens of each sequence, one at a time and by trees of up to `nodes` drafts: whether both give the same
    tokens (a near tie may go either way), the largest difference of their log probabilities, and tokens a step."""
    import random

    import torch

    from . import syn
    rows = prompt + tokens + nodes
    block, _, _ = llama1b_block(cache_type, 2 * seqs, rows, page)
    n_pages, width = block.cache.n_pages, block.w["q"][3]
    gen, rand = torch.Generator(device="cuda").manual_seed(3), random.Random(3)
    table = torch.randn((vocab, width), device="cuda", generator=gen)
    head = syn.quantize(syn.Q6_K, torch.randn((vocab, width), device="cuda", generator=gen) * 0.05)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")

    def score(out, ids=None, n_top=0):
        return syn.logprobs(syn.mul_mat(syn.Q6_K, head, vocab, width, out), ids, n_top)

    def forked(pages, lens, n):
        return syn.kv_fork(block.cache, refs, i32([0] * n), pages, lens)

    # the prompt, once; every sequence starts as a fork of it, with an alternative of its own as its first token
    pages, lens = torch.full((1, -(-rows // page)), -1, dtype=torch.int32, device="cuda"), i32([0])
    _, slots = syn.kv_extend(block.cache, refs, pages, lens, starts=i32([0, prompt]), n_tok=prompt)
    x = table[torch.randint(0, vocab, (prompt,), device="cuda", generator=gen)]
    out = torch.empty((prompt, width), device="cuda")
    block.prepare_prompt(x, out, torch.arange(prompt, dtype=torch.int32, device="cuda"), slots, i32([0, prompt]), pages, lens)()
    best = score(out[-1:].contiguous(), n_top=min(seqs, 64, vocab)).top[0].tolist()  # (64: the most that logprobs gives)
    first = [best[s % len(best)] for s in range(seqs)]

    def plain():  # one token at a time: tokens and log probabilities
        mine, ln = forked(pages, lens, seqs)
        now, said, sure = list(first), [[t] for t in first], [[] for _ in first]
        for _ in range(tokens + nodes):
            _, slots = syn.kv_extend(block.cache, refs, mine, ln)
            out = torch.empty((seqs, width), device="cuda")
            block.prepare_token(table[i32(now)], out, ln - 1, slots, mine, ln)()
            got = score(out, n_top=1)
            now = got.top[:, 0].tolist()
            for s, (t, p) in enumerate(zip(now, got.top_logprob[:, 0].tolist())):
                said[s].append(t)
                sure[s].append(p)
            if int(ln.max()) >= rows:
                break
        syn.kv_trim(block.cache, refs, mine, torch.zeros_like(ln))
        return said, sure

    want, sure = plain()
    mine, ln = forked(pages, lens, seqs)
    said, worst, steps = [[t] for t in first], 0.0, 0
    while min(len(x) for x in said) <= tokens:
        # (a sequence that is done drafts nothing more)
        trees = [_draft(rand, want[s][len(said[s]) - 1:], vocab, nodes) if len(said[s]) <= tokens else ([], [], []) for s in range(seqs)]
        n = [len(t[0]) for t in trees]
        starts = i32([sum(n[:s]) for s in range(seqs + 1)])
        depth = i32([d for t in trees for d in t[2]])
        of = torch.repeat_interleave(torch.arange(seqs, device="cuda"), i32(n))
        long, slots = syn.kv_extend(block.cache, refs, mine, ln, torch.empty_like(ln), starts=starts, n_tok=sum(n))
        out = torch.empty((sum(n), width), device="cuda")
        block.prepare_draft(table[i32([t for x in trees for t in x[0]])], out, ln[of] + depth, slots, starts,
                            i32([a for t in trees for a in t[1]]), mine, long)()
        got = score(out, n_top=1)
        top, logp, at, paths = got.top[:, 0].tolist(), got.top_logprob[:, 0].tolist(), 0, []
        for s, (tok, parents, _) in enumerate(trees):
            path = [0] if tok else []
            while path:  # the target's token after the path's last node, and the child that has it
                i = path[-1]
                worst = max(worst, abs(logp[at + i] - sure[s][len(said[s]) - 1]))
                said[s].append(top[at + i])
                child = [j for j in range(i + 1, len(tok)) if parents[j] == i and tok[j] == top[at + i]]
                if not child:
                    break
                path.append(child[0])
            paths.append(path)
            at += len(tok)
        keep = i32([sum(len(x) for x in paths[:s]) for s in range(seqs + 1)])
        ln = syn.kv_compact(block.cache, refs, mine, ln, keep, i32([i for x in paths for i in x]))
        syn.kv_trim(block.cache, refs, mine, ln)
        steps += 1
    syn.kv_trim(block.cache, refs, mine, torch.zeros_like(ln))
    syn.kv_trim(block.cache, refs, pages, torch.zeros_like(lens))
    held = int((refs != 0).sum())
    syn.check(syn.device_status(), "device status")
    same = all(a[:tokens + 1] == b[:tokens + 1] for a, b in zip(said, want))
    return {"same": same, "difference": worst, "per_step": sum(len(x) - 1 for x in said) / steps / seqs, "held": held}


def main() -> None:
    ap = argparse.ArgumentParser()
    ap.add_argument("--type", choices=("f16", "q8_0"), default="f16")
    ap.add_argument("--prompt", type=int, default=512)
    ap.add_argument("--steps", type=int, default=16)
    ap.add_argument("--seqs", type=int, default=4)
    ap.add_argument("--draft", type=int, default=0, metavar="NODES")
    a = ap.parse_args()
    if min(a.prompt, a.steps, a.seqs) < 1 or a.draft < 0:
        ap.error("--prompt, --steps and --seqs: at least 1; --draft: 0 or more")
    if a.draft:
        r = run_drafts(Q8_0 if a.type == "q8_0" else F16, a.prompt, a.steps, a.seqs, a.draft)
        print(f"{a.seqs} sequences, {a.type} cache, trees of {a.draft} drafts: {r['per_step']:.2f} tokens a step and sequence, "
              f"the same tokens: {r['same']}; largest difference of a log probability from decoding "
              f"one token at a time {r['difference']:.2e}")
        return
    r = run(Q8_0 if a.type == "q8_0" else F16, a.prompt, a.steps, a.seqs)
    print(f"{a.seqs} sequences, {a.type} cache: prompt of {a.prompt} tokens {r['us_prompt']:.1f} us, one token of each "
          f"{r['us_token']:.1f} us; largest difference between the two forms {r['difference']:.2e} of the largest output")


if __name__ == "__main__":
    main()
