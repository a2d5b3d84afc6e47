"""Run a few verify calls on one preset workload (a target for profilers).

    python -m speculative_decoding_verification_36_gb300.run_case c4 [--batch B] [--calls N]

Builds the library if needed, generates the preset's synthetic inputs on
cuda:0 and makes N calls of the entry point the preset exercises
(spec_verify for c1-c4, or spec_verify_early_exit with --early-exit;
spec_tree_verify_greedy for c5, its early exit with --early-exit;
spec_tree_verify_sampling at tau = 1 on the
c5 tree for c5s; spec_ngram_draft (n 1..4, K = 8) on 256 repetitive
histories of up to 131072 tokens for ngram; spec_count_tokens and
spec_process_logits on the c3 target rows (process) or the c5 tree's
(process-tree), then the greedy verify of what comes out; spec_kv_append, the
greedy tree verify and spec_kv_commit on the c5 tree with 4 layers of 8 heads
of 128 (cache)), then synchronises.
"""
from __future__ import annotations

import argparse
import sys


def main(argv=None) -> int:
    ap = argparse.ArgumentParser()
    ap.add_argument("preset", choices=["c1", "c2", "c3", "c4", "c5", "c5s", "ngram", "process", "process-tree", "cache"])
    ap.add_argument("--early-exit", action="store_true", help="c1-c5: the early-exit verify")
    ap.add_argument("--batch", type=int, default=0, help="sequences (default: the preset's B)")
    ap.add_argument("--calls", type=int, default=3)
    args = ap.parse_args(argv)

    import torch

    from . import build, spec_get_status, spec_ngram_draft, spec_tree_verify_greedy, spec_tree_verify_sampling
    from . import spec_verify, spec_verify_early_exit
    from . import spec_count_tokens, spec_kv_append, spec_kv_commit, spec_process_logits, spec_rope_turns, spec_token_state
    from . import workloads as wl

    build.build()
    dev = torch.device("cuda", 0)
    if args.preset == "ngram":
        B, L = args.batch or 256, 131072
        h = wl.make_ngram_histories(16, L, seed=1)
        reps = (B + 15) // 16
        tok = h["tokens"].repeat(reps, 1)[:B].contiguous().to(dev)
        ln = h["lengths"].repeat(reps)[:B].contiguous().to(dev)
        for _ in range(args.calls):
            spec_ngram_draft(tok, ln, 1, 4, 8)
        torch.cuda.synchronize()
        flags = spec_get_status()
        print(f"ngram B={B} L<={L}: {args.calls} calls, status flags {flags}")
        return 0 if flags == 0 else 1
    if args.preset in ("process", "process-tree"):
        tree = args.preset == "process-tree"
        p = wl.preset("c5" if tree else "c3", **({"B": args.batch} if args.batch else {}))
        x = wl.make_tree(p, device=dev, seed=0) if tree else wl.make_chain(p, device=dev, seed=0)
        B, rows, V = x["target"].shape
        o = wl.make_settings(B, rows, V, seed=0, device=dev)
        state, out = spec_token_state(B, V, dev), torch.empty_like(x["target"])
        for _ in range(args.calls):
            spec_count_tokens(state, o["tokens"], V, o["lengths"], o["prompt_lengths"], reset=True)
            spec_process_logits(x["target"], x["tokens"], x["parents"] if tree else None, state, o["repetition"],
                                o["frequency"], o["presence"], o["bias_tokens"], o["bias_values"], o["allowed_mask"],
                                out=out)
            if tree:
                spec_tree_verify_greedy(out, x["tokens"], x["parents"])
            else:
                spec_verify(out, None, x["tokens"], 0.0, 0)
        torch.cuda.synchronize()
        flags = spec_get_status()
        print(f"{args.preset} B={B}: {args.calls} calls, status flags {flags}")
        return 0 if flags == 0 else 1
    if args.preset == "cache":
        x = wl.make_tree(wl.preset("c5", **({"B": args.batch} if args.batch else {})), device=dev, seed=0)
        B, N = x["tokens"].shape
        c = wl.make_cache_step(B, N + 1, 32, 8, 128, layers=4, device=dev)
        turns, lengths = spec_rope_turns(c["inv_freq"], dev), c["lengths"]
        for _ in range(args.calls):
            for i in range(4):
                spec_kv_append(c["k"][i], c["v"][i], c["key_cache"][i], c["value_cache"][i], c["page_table"], lengths,
                               turns=turns, q=c["q"][i], parent_idx=x["parents"])
            path, n, _ = spec_tree_verify_greedy(x["target"], x["tokens"], x["parents"])
            spec_kv_commit(c["key_cache"], c["value_cache"], c["page_table"], lengths, x["tokens"], x["parents"], path, n)
        torch.cuda.synchronize()
        flags = spec_get_status()
        print(f"cache B={B}: {args.calls} calls, status flags {flags}")
        return 0 if flags == 0 else 1
    name = "c5" if args.preset == "c5s" else args.preset
    p = wl.preset(name, B=args.batch) if args.batch else wl.preset(name)
    if args.preset == "c5s":
        x = wl.make_tree_sampling(p, 1.0, device=dev, seed=0)
        for i in range(args.calls):
            spec_tree_verify_sampling(x["target"], x["draft"], x["tokens"], x["parents"], 1.0, i)
    elif args.preset == "c5":
        x = wl.make_tree(p, device=dev, seed=0)
        for _ in range(args.calls):
            spec_tree_verify_greedy(x["target"], x["tokens"], x["parents"], early_exit=args.early_exit)
    else:
        x = wl.make_chain(p, device=dev, seed=0)
        verify = spec_verify_early_exit if args.early_exit else spec_verify
        for i in range(args.calls):
            verify(x["target"], x["draft"], x["tokens"], x["temperature"], i)
    torch.cuda.synchronize()
    flags = spec_get_status()
    print(f"{args.preset} B={p.B}: {args.calls} calls, status flags {flags}")
    return 0 if flags == 0 else 1


if __name__ == "__main__":
    sys.exit(main())
