"""One product, repeated a few times, for profiler captures of a single kernel.

    python -m gguf_block_quantized_gb300.profile_case --case gemv_q6k_lm_head --reps 3

Cases (synthetic weights ~N(0, 0.02), activations ~N(0, 1)):
  gemv_q6k_lm_head   Q6_K 128256 x 2048, 1 token    (216 MB of weights: larger than L2)
  gemv_q6k_lm_head_4tok  the same, 4 tokens
  gemv_q4k_wide      Q4_K 32768 x 8192, 1 token     (151 MB)
  gemv_q8_0_wide     Q8_0 16384 x 8192, 1 token     (143 MB)
  gemm_q4k_ffn_up    Q4_K 14336 x 4096, 512 tokens  (prefill, tensor cores)
  gemm_q4k_ffn_down  Q4_K 4096 x 14336, 512 tokens
  gemv_llama1b_layer the seven decode products of a Llama-1B-shaped layer, one grouped call
  gemv_llama8b_layers  the grouped decode calls of two Llama-8B Q4_K_M layers, alternating:
                     layer 0 (Q6_K attn_v / ffn_down) and layer 4 (all Q4_K), the weights and
                     inputs of the benchmark's sweep
  prefill_llama8b_layer  one Llama-8B layer at 2048 tokens as a model calls it: q/k/v grouped
                     on one input, o, gate/up grouped on one input, down (Q4_K, Q6_K v/down)
  kv_append_f16, kv_append_q8  4096 tokens of 32 / 8 heads of 128 into a paged cache (150 MB moved)
  attn_decode_f16, attn_decode_q8  one token of each of 48 sequences of 2000 cached tokens, 32 / 8
                     heads of 128, pages of 64 (F16: 393 MB of rows)
  attn_decode_long_f16, attn_decode_long_q8  one token of one sequence of 96000 rows
  attn_prefill_f16, attn_prefill_q8  a prompt of 4096 tokens, 32 / 8 heads of 128 (Q8_0: expanded ahead)
  attn_prefill_batch_f16, attn_prefill_batch_q8  8 prompts of 512 tokens (Q8_0: expanded in the kernel)
  kv_read_f16, kv_read_q8  the rows of 4096 tokens back as fp16
  attn_tree_f16, attn_tree_q8  trees of 24 drafts over each of 48 sequences of 2000 rows (F16: 393 MB)
  attn_tree_long_f16, attn_tree_long_q8  a tree of 64 drafts over one sequence of 96000 rows
  kv_compact_f16, kv_compact_q8  one sequence of 40000 rows packed to every second one
  logprobs_f32, logprobs_f16  512 and 1024 rows of 128256 logits (263 MB), one token and the 8 most likely of each
"""
from __future__ import annotations

import argparse

CASES = {
    "gemv_q6k_lm_head": (3, 128256, 2048, 1),
    "gemv_q6k_lm_head_4tok": (3, 128256, 2048, 4),
    "gemv_q4k_wide": (2, 32768, 8192, 1),
    "gemv_q8_0_wide": (1, 16384, 8192, 1),
    "gemm_q4k_ffn_up": (2, 14336, 4096, 512),
    "gemm_q4k_ffn_down": (2, 4096, 14336, 512),
}


ATTN = ["kv_append_f16", "kv_append_q8", "attn_decode_f16", "attn_decode_q8", "attn_decode_long_f16",
        "attn_decode_long_q8", "attn_prefill_f16", "attn_prefill_q8", "attn_prefill_batch_f16", "attn_prefill_batch_q8",
        "kv_read_f16", "kv_read_q8"]
DRAFTS = ["attn_tree_f16", "attn_tree_q8", "attn_tree_long_f16", "attn_tree_long_q8", "kv_compact_f16", "kv_compact_q8",
          "logprobs_f32", "logprobs_f16"]


def attn_case(case: str, reps: int):
    """The paged-cache operators on random rows (the cache's content does not change their time)."""
    import torch

    from gguf_block_quantized_gb300 import syn

    heads, kv, dim, page = 32, 8, 128, 64
    t = syn.Q8_0 if case.endswith("q8") else syn.F16
    seqs, rows = (1, 96000) if "long" in case else (48, 2000) if "decode" in case else (8, 512) if "batch" in case else (1, 4096)
    per = -(-rows // page)
    cache = syn.KVCache.empty(t, kv, dim, page, seqs * per)
    pages = torch.randperm(seqs * per, device="cuda").to(torch.int32).view(seqs, per)
    n = min(rows, 8192)  # rows appended at once
    row = torch.arange(n, device="cuda")
    fused = torch.randn((n, heads + 2 * kv, dim), device="cuda")
    parts = {"q": fused[:, :heads], "k": fused[:, heads:heads + kv], "v": fused[:, heads + kv:]}
    rope = syn.Rope(dim, 500000.0, layout=syn.ROPE_ADJACENT)
    pos = row.to(torch.int32)
    for s, base in [(s, b) for s in range(seqs) for b in range(0, rows - n + 1, n)]:
        at = base + row
        slots = pages[s].long()[at // page] * page + at % page
        append = syn.prepare_kv_append(cache, rope, parts["k"], parts["v"], pos, slots, parts["q"])
        q = append()
    lens = torch.full((seqs,), rows, dtype=torch.int32, device="cuda")
    if case.startswith("kv_append"):
        step = append
    elif case.startswith("kv_read"):
        step = syn.prepare_kv_read(cache, slots)
    elif "decode" in case:
        step = syn.prepare_attn_decode(cache, q[:seqs].contiguous(), pages, lens)
    else:
        step = syn.prepare_attn_prefill(cache, torch.cat([q] * seqs), torch.arange(0, seqs * rows + 1, rows, dtype=torch.int32, device="cuda"),
                                        pages, lens)
    for _ in range(reps):
        step()
    torch.cuda.synchronize()
    assert syn.device_status() == syn.OK
    print(f"{case}: {reps} calls done")


def draft_case(case: str, reps: int):
    """The operators of drafted tokens: 32 / 8 heads of 128, pages of 64, zeroed caches."""
    import torch

    from gguf_block_quantized_gb300 import syn

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    if case.startswith("logprobs"):
        rows, dtype = (512, torch.float32) if case.endswith("f32") else (1024, torch.float16)
        logits = (4.0 * torch.randn((rows, 128256), device="cuda")).to(dtype)
        step = syn.prepare_logprobs(logits, ids=torch.randint(128256, (rows, 1), device="cuda").to(torch.int32), n_top=8)
    else:
        seqs, rows, n = (1, 40000, 20000) if "compact" in case else (1, 96000, 64) if "long" in case else (48, 2000, 24)
        per = -(-rows // 64)
        cache = syn.KVCache.empty(syn.Q8_0 if case.endswith("q8") else syn.F16, 8, 128, 64, seqs * per)
        pages = torch.randperm(seqs * per, device="cuda").to(torch.int32).view(seqs, per)
        if "compact" in case:
            step = syn.prepare_kv_compact(cache, None, pages, ints([0]), ints([0, n]), ints(range(1, rows, 2)))
        else:
            q = torch.randn((seqs * n, 32, 128), device="cuda").half()
            parents = ints([(i + 1) // 2 - 1 for i in range(n)] * seqs)
            step = syn.prepare_attn_tree(cache, q, ints(range(0, seqs * n + 1, n)), parents, pages, ints([rows] * seqs))
    for _ in range(reps):
        step()
    torch.cuda.synchronize()
    assert syn.device_status() == syn.OK
    print(f"{case}: {reps} calls done")


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--case", required=True, choices=sorted(CASES) + ["gemv_llama1b_layer", "gemv_llama8b_layers",
                                                                     "prefill_llama8b_layer"] + ATTN + DRAFTS)
    ap.add_argument("--reps", type=int, default=3)
    args = ap.parse_args()
    import torch

    from gguf_block_quantized_gb300 import syn, synth

    if args.case in ATTN:
        attn_case(args.case, args.reps)
        return
    if args.case in DRAFTS:
        draft_case(args.case, args.reps)
        return
    if args.case == "gemv_llama1b_layer":
        from gguf_block_quantized_gb300 import workloads
        mats = workloads.LLAMA1B_LAYER
        Ws = [syn.quantize(m.wtype, torch.from_numpy(synth.weight(2, i, m.n_out, m.n_in)).cuda()) for i, m in enumerate(mats)]
        Xs = [torch.from_numpy(synth.activations(2, i, 1, m.n_in)).cuda() for i, m in enumerate(mats)]
        Ys = [torch.empty((1, m.n_out), device="cuda") for m in mats]
        for _ in range(args.reps):
            syn.mul_mat_batch([(m.wtype, Ws[i], m.n_out, m.n_in, Xs[i], Ys[i]) for i, m in enumerate(mats)], 1)
        torch.cuda.synchronize()
        assert syn.device_status() == syn.OK
        print(f"{args.case}: {args.reps} grouped calls done")
        return
    if args.case == "gemv_llama8b_layers":
        from gguf_block_quantized_gb300 import workloads
        mats = workloads.llama8b_q4_k_m()
        d, f = mats[0].n_in, mats[6].n_in
        xs = [torch.from_numpy(synth.activations(5, j, 1, n)).cuda() for j, n in enumerate([d, d, d, f])]
        src = [xs[0], xs[0], xs[0], xs[1], xs[2], xs[2], xs[3]]
        calls = []
        for k in (0, 4):
            lay = mats[7 * k:7 * k + 7]
            Ws = [syn.quantize(m.wtype, torch.from_numpy(synth.weight(5, 7 * k + i, m.n_out, m.n_in)).cuda())
                  for i, m in enumerate(lay)]
            Ys = [torch.empty((1, m.n_out), device="cuda") for m in lay]
            calls.append([(m.wtype, Ws[i], m.n_out, m.n_in, src[i], Ys[i]) for i, m in enumerate(lay)])
        for _ in range(args.reps):
            for c in calls:
                syn.mul_mat_batch(c, 1)
        torch.cuda.synchronize()
        assert syn.device_status() == syn.OK
        print(f"{args.case}: {args.reps} x 2 grouped calls done")
        return
    if args.case == "prefill_llama8b_layer":
        from gguf_block_quantized_gb300 import workloads
        lay = workloads.llama8b_q4_k_m(n_layers=1, lm_head=False)  # a Q6_K attn_v / ffn_down layer
        n_tok = 2048
        Ws = [syn.quantize(m.wtype, torch.from_numpy(synth.normal(20 + i, (m.n_out, m.n_in), 0.02)).cuda())
              for i, m in enumerate(lay)]
        XA, XO, XF = (torch.from_numpy(synth.normal(30 + i, (n_tok, lay[0].n_in))).cuda() for i in range(3))
        XD = torch.from_numpy(synth.normal(33, (n_tok, lay[6].n_in))).cuda()
        Ys = [torch.empty((n_tok, m.n_out), device="cuda") for m in lay]
        syn.syn_reserve(lay[6].n_in, n_tok, torch.cuda.current_stream().cuda_stream)
        for _ in range(args.reps):
            syn.mul_mat_batch([(lay[i].wtype, Ws[i], lay[i].n_out, lay[i].n_in, XA, Ys[i]) for i in range(3)], n_tok)
            syn.mul_mat(lay[3].wtype, Ws[3], lay[3].n_out, lay[3].n_in, XO, Y=Ys[3])
            syn.mul_mat_batch([(lay[i].wtype, Ws[i], lay[i].n_out, lay[i].n_in, XF, Ys[i]) for i in (4, 5)], n_tok)
            syn.mul_mat(lay[6].wtype, Ws[6], lay[6].n_out, lay[6].n_in, XD, Y=Ys[6])
        torch.cuda.synchronize()
        assert syn.device_status() == syn.OK
        print(f"{args.case}: {args.reps} layer passes done")
        return
    wt, n_out, n_in, n_tok = CASES[args.case]
    W = syn.quantize(wt, torch.from_numpy(synth.normal(5, (n_out, n_in), 0.02)).cuda())
    X = torch.from_numpy(synth.normal(6, (n_tok, n_in))).cuda()
    Y = torch.empty((n_tok, n_out), device="cuda")
    syn.syn_reserve(n_in, n_tok, torch.cuda.current_stream().cuda_stream)
    for _ in range(args.reps):
        syn.mul_mat(wt, W, n_out, n_in, X, Y=Y)
    torch.cuda.synchronize()
    assert syn.device_status() == syn.OK
    print(f"{args.case}: {args.reps} products done")


if __name__ == "__main__":
    main()
