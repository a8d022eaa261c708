"""Speculative decoding on a quantised paged cache: what one layer runs per step, on random weights.

A prompt's keys are normed, rotated and written to pages; then every step projects a tree of drafted tokens,
writes their keys and values behind the prefix, lets the nodes attend the prefix and their ancestors, keeps
the longest path that a (here: random) verdict accepts, and moves its keys and values to the places after
the prefix by reading the cache and writing it back.

    python examples/draft_step.py [--format int8|e4m3|e2m1] [--steps 8] [--sequences 4]
"""
import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import random_access_kv_gb300 as rk  # noqa: E402

HEADS_Q, HEADS_KV, D, PAGE, EPS = 32, 8, 128, 64, 1e-6


def rope_table(positions: int, device) -> torch.Tensor:
    angle = torch.arange(positions, device=device).double()[:, None] * 10000.0 ** (-torch.arange(D // 2, device=device).double() / (D // 2))
    return torch.cat([angle.cos(), angle.sin()], 1).float().contiguous()


def tree_of(parents):
    """Depth of each node and the bits of the nodes that it sees: its ancestors and itself."""
    depth, seen = [], []
    for i, p in enumerate(parents):
        depth.append(0 if p < 0 else depth[p] + 1)
        seen.append((0 if p < 0 else seen[p]) | 1 << i)
    return depth, seen


def run(fmt: str = "int8", steps: int = 8, sequences: int = 4, prompt: int = 300, hidden: int = 512, seed: int = 0):
    """Returns the lengths of the sequences and the last step's outputs."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = torch.bfloat16
    parents = [-1, 0, 0, 1, 1, 2, 3, 3]                       # a tree of 8 drafted tokens
    depth, seen = tree_of(parents)
    nodes, most = len(parents), prompt + 8 * steps
    each = -(-(most + nodes) // PAGE)

    ctx = rk.qc_create(fmt, D, HEADS_KV, PAGE)
    pages = rk.alloc_pages(ctx, sequences * each)
    table = torch.randperm(sequences * each, generator=gen, device="cuda").reshape(sequences, each).int()
    workspace = rk.alloc_attend_workspace(ctx, sequences, nodes, HEADS_Q, most)
    rope = rope_table(most + nodes, "cuda")
    w_qkv = torch.randn((hidden, (HEADS_Q + 2 * HEADS_KV) * D), generator=gen, device="cuda").to(dtype) / math.sqrt(hidden)
    w_q, w_k = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
    tree = torch.tensor(seen, dtype=torch.int32, device="cuda").reshape(1, nodes, 1).repeat(sequences, 1, 1)
    at_depth = torch.tensor(depth, device="cuda")
    lens = torch.zeros(sequences, dtype=torch.int32, device="cuda")

    def slots_of(places):                                     # places [sequences, n] of each sequence
        page = torch.gather(table.long(), 1, places // PAGE)
        return (page * PAGE + places % PAGE).reshape(-1)

    def project(n):                                           # a layer's queries, keys and values of n tokens
        x = torch.randn((n, hidden), generator=gen, device="cuda").to(dtype)
        return (x @ w_qkv).view(n, HEADS_Q + 2 * HEADS_KV, D).split([HEADS_Q, HEADS_KV, HEADS_KV], 1)

    # the prompt: norm and rotate in place, then into the pages
    q, k, v = project(sequences * prompt)
    places = torch.arange(prompt, device="cuda").repeat(sequences, 1)
    rk.qc_norm_rope(ctx, q, k, w_q, w_k, EPS, places.reshape(-1), rope, D, False, q, k)
    rk.qc_write(ctx, k, v, slots_of(places), pages)
    lens += prompt

    out = torch.empty((sequences, nodes, HEADS_Q, D), dtype=dtype, device="cuda")
    lse = torch.empty((sequences, nodes, HEADS_Q), device="cuda")
    for _ in range(steps):
        q, k, v = project(sequences * nodes)
        behind = lens.long()[:, None] + torch.arange(nodes, device="cuda")
        rk.qc_norm_rope(ctx, q, k, w_q, w_k, EPS, (lens.long()[:, None] + at_depth).reshape(-1), rope, D, False, q, k)
        rk.qc_write(ctx, k, v, slots_of(behind), pages)
        rk.qc_attend(ctx, pages, q.view(sequences, nodes, HEADS_Q, D), table, lens, None, tree, 1 / math.sqrt(D), most, out, lse, workspace)
        # the verdict: a path through the tree for each sequence, root first
        tip = torch.randint(0, nodes, (sequences,), generator=gen, device="cuda").tolist()
        paths = []
        for node in tip:
            path = [node]
            while parents[path[0]] >= 0:
                path.insert(0, parents[path[0]])
            paths.append(path)
        longest = max(map(len, paths))
        came = torch.tensor([p + [p[-1]] * (longest - len(p)) for p in paths], device="cuda")
        kept = torch.tensor([[1] * len(p) + [0] * (longest - len(p)) for p in paths], device="cuda").bool()
        held = [torch.empty((sequences * longest, HEADS_KV, D), dtype=torch.float32, device="cuda") for _ in range(2)]
        rk.qc_read(ctx, pages, slots_of(lens.long()[:, None] + came), *held)
        to = slots_of(lens.long()[:, None] + torch.arange(longest, device="cuda"))
        rk.qc_write(ctx, *held, torch.where(kept.reshape(-1), to, -1), pages)
        lens += kept.sum(1).int()
    flags = rk.qc_status(ctx)
    if flags:
        raise RuntimeError(f"the cache reports flags {flags}")
    rk.qc_destroy(ctx)
    return lens, out, lse


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--format", default="int8", choices=("int8", "e4m3", "e2m1"))
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--sequences", type=int, default=4)
    a = ap.parse_args()
    lengths, out, lse = run(a.format, a.steps, a.sequences)
    print(f"{a.format}: {a.steps} steps, lengths now {lengths.tolist()}, last outputs of magnitude {out.float().abs().mean():.4f}, "
          f"log-sums {lse.mean():.3f}")
