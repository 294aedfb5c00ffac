"""The attention of one layer whose heads keep their own keys and values (a drafter's layer),
as a serving loop runs it: prompts of different lengths packed into one call, then one new
token a request at a time, over a paged cache.

    python examples/grouped_head_layer.py [--fp8 | --blocks]

With --blocks the cache has a scale for each block of positions and head, the page tables are
built on the GPU, later prompts run behind their cached prefix, and several new tokens of a
request (drafts) are attended at once.  Each step of the loop is checked against the same layer
run over the whole sequences at once.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import paged_mla_latent_gb300 as pm  # noqa: E402


def indptr(lens, device):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device=device)


class GroupedHeadLayer:
    """q, k and v of `q_heads` / `kv_heads` heads from one projection, rotated, cached in pages
    of `page` tokens (bf16, or e4m3 with one scale for keys and one for values) and attended."""

    def __init__(self, width=1024, q_heads=16, kv_heads=4, dim=128, page=64, pages=256, max_pos=8192,
                 fp8=False, device="cuda", seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        self.q_heads, self.kv_heads, self.dim, self.page = q_heads, kv_heads, dim, page
        self.device = torch.device(device)
        self.w = torch.randn(width, (q_heads + 2 * kv_heads) * dim, generator=g, device=device)
        self.w = (self.w * width ** -0.5).bfloat16()
        inv = 10000.0 ** (-torch.arange(dim // 2, device=device, dtype=torch.float64) * 2 / dim)
        ang = torch.arange(max_pos, device=device, dtype=torch.float64)[:, None] * inv
        self.cos_sin = torch.cat([ang.cos(), ang.sin()], dim=1).float()
        kind = torch.float8_e4m3fn if fp8 else torch.bfloat16
        shape = (pages, page, kv_heads, dim)
        self.k_cache = torch.empty(shape, dtype=kind, device=device)
        self.v_cache = torch.empty(shape, dtype=kind, device=device)
        self.k_scale = torch.tensor(0.02, device=device) if fp8 else None
        self.v_scale = torch.tensor(0.02, device=device) if fp8 else None
        self.error_word = torch.zeros(1, dtype=torch.int32, device=device)
        self.workspace = pm.make_gqa_decode_workspace(1, q_heads, kv_heads, dim, device)
        self.free = list(torch.randperm(pages, generator=torch.Generator().manual_seed(seed)))
        self.tables, self.lens = [], []

    def _append(self, x, positions, slots, keep_k):
        """Project x, rotate, write keys and values at the slots: rotated q, rotated k (where
        the caller attends to it directly), v."""
        t, d = x.shape[0], self.dim
        qkv = x @ self.w
        q = qkv[:, :self.q_heads * d].view(t, self.q_heads, d)
        k = qkv[:, self.q_heads * d:(self.q_heads + self.kv_heads) * d].view(t, self.kv_heads, d)
        v = qkv[:, (self.q_heads + self.kv_heads) * d:].view(t, self.kv_heads, d)
        # in place: q and k are views of the projection
        pm.mla_gqa_rope_and_cache(q, k, v, positions, self.cos_sin, 1, slots, q, self.k_cache,
                                  self.v_cache, self.error_word, self.k_scale, self.v_scale,
                                  k_out=k if keep_k else None)
        return q, k, v

    def _slots(self, b, start, stop):
        while len(self.tables[b]) * self.page < stop:
            self.tables[b].append(int(self.free.pop()))
        return [self.tables[b][j // self.page] * self.page + j % self.page for j in range(start, stop)]

    def prompt(self, xs):
        """New requests: xs[b] (T_b, width).  Returns o of all their tokens (sum T, heads, dim)."""
        first, slots, pos = len(self.lens), [], []
        for x in xs:
            self.tables.append([])
            self.lens.append(x.shape[0])
            slots += self._slots(len(self.lens) - 1, 0, x.shape[0])
            pos += range(x.shape[0])
        ints = lambda a: torch.tensor(a, dtype=torch.int32, device=self.device)
        q, k, v = self._append(torch.cat(xs), ints(pos), ints(slots), keep_k=True)
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
        ptr = indptr(self.lens[first:], self.device)
        pm.mla_prompt_attention(q, k, v, o, ptr, ptr, self.dim ** -0.5, self.error_word)
        return o

    def step(self, x):
        """One new token a request: x (B, width).  Returns o (B, heads, dim)."""
        slots = [self._slots(b, n, n + 1)[0] for b, n in enumerate(self.lens)]
        ints = lambda a: torch.tensor(a, dtype=torch.int32, device=self.device)
        q, _, _ = self._append(x, ints(self.lens), ints(slots), keep_k=False)
        self.lens = [n + 1 for n in self.lens]
        o = torch.empty_like(q, memory_format=torch.contiguous_format)
        pm.mla_gqa_decode(q, self.k_cache, self.v_cache, o, indptr([len(t) for t in self.tables], self.device),
                          ints(sum(self.tables, [])), ints([(n - 1) % self.page + 1 for n in self.lens]),
                          self.dim ** -0.5, self.k_scale, self.v_scale, workspace=self.workspace)
        return o

    def check(self):
        """Device-side errors since the last check."""
        status = pm.mla_check_error(self.workspace)
        bits = int(self.error_word.item())
        if status or bits:
            raise RuntimeError(f"{pm.mla_status_string(status)}, error bits {bits}")


def run(fp8=False, lens=(37, 400, 1, 129), steps=70, device="cuda"):
    """Largest difference between the steps' outputs and the same tokens' rows of one prompt
    over the whole sequences."""
    width = 1024
    g = torch.Generator(device=device).manual_seed(1)
    xs = [torch.randn(n + steps, width, generator=g, device=device).bfloat16() for n in lens]
    layer = GroupedHeadLayer(width, fp8=fp8, device=device)
    first = layer.prompt([x[:n] for x, n in zip(xs, lens)])
    outs = [layer.step(torch.stack([x[n + i] for x, n in zip(xs, lens)])) for i in range(steps)]
    layer.check()
    whole = GroupedHeadLayer(width, device=device).prompt(xs).float()
    worst, at, start = 0.0, 0, 0
    for b, n in enumerate(lens):
        worst = max(worst, (first[start:start + n].float() - whole[at:at + n]).abs().max().item())
        for i in range(steps):
            worst = max(worst, (outs[i][b].float() - whole[at + n + i]).abs().max().item())
        start, at = start + n, at + n + steps
    return worst


class BlockScaledLayer(GroupedHeadLayer):
    """The layer over an e4m3 cache with a scale for each `block` positions and head.  Requests'
    lengths, page tables and the stack of free pages live on the GPU."""

    def __init__(self, requests, width=1024, q_heads=16, kv_heads=4, dim=128, page=64, pages=256, block=16,
                 max_new=8, **kw):
        super().__init__(width, q_heads, kv_heads, dim, page, pages, fp8=True, **kw)
        ints = lambda *shape, fill=0: torch.full(shape, fill, dtype=torch.int32, device=self.device)
        scales = (pages, page // block, kv_heads)
        self.k_scale, self.v_scale = (torch.zeros(scales, device=self.device) for _ in range(2))
        self.max_new, self.seq_lens = max_new, ints(requests)
        self.block_table, self.kv_indices = ints(requests, pages, fill=-1), ints(pages)
        self.free_pages = torch.tensor(self.free, dtype=torch.int32, device=self.device)
        self.free_count = ints(1, fill=pages)
        self.qo_indptr, self.key_indptr, self.kv_indptr = (ints(requests + 1) for _ in range(3))
        self.last = ints(requests)
        self.error_word = ints(2)
        self.workspace = pm.make_gqa_block_decode_workspace(q_heads, kv_heads, dim, max_new, self.device)

    def forward(self, xs):
        """The next tokens of every request: xs[b] (T_b, width), T_b >= 0.  Returns o of all of
        them (sum T, heads, dim)."""
        new = torch.tensor([x.shape[0] for x in xs], dtype=torch.int32, device=self.device)
        t, d = sum(x.shape[0] for x in xs), self.dim
        self.seq_lens += new
        positions, slots = (torch.empty(t, dtype=torch.int32, device=self.device) for _ in range(2))
        pm.mla_build_page_table(self.seq_lens, new, self.block_table, self.page, self.qo_indptr, self.key_indptr,
                                self.kv_indptr, self.kv_indices, self.last, self.error_word, positions=positions,
                                slot_mapping=slots, free_pages=self.free_pages, free_count=self.free_count,
                                free_count_out=self.free_count)
        qkv = torch.cat(xs) @ self.w
        q, k, v = (y.unflatten(1, (-1, d)) for y in qkv.split([self.q_heads * d, self.kv_heads * d, self.kv_heads * d], 1))
        lists = self.kv_indptr, self.kv_indices, self.last
        pm.mla_gqa_block_append(q, k, v, positions, self.cos_sin, 1, self.qo_indptr, *lists, q, self.k_cache,
                                self.v_cache, self.k_scale, self.v_scale, self.error_word, k_out=k)
        o = torch.empty(q.shape, dtype=q.dtype, device=self.device)
        if max(x.shape[0] for x in xs) <= self.max_new:
            pm.mla_gqa_block_decode(q, self.k_cache, self.v_cache, self.k_scale, self.v_scale, o, self.qo_indptr,
                                    *lists, self.max_new, d ** -0.5, workspace=self.workspace)
            return o
        rows = int(self.key_indptr[-1])            # prompts: the cached positions as rows, the new ones behind
        k_rows, v_rows = (torch.empty(rows, self.kv_heads, d, dtype=q.dtype, device=self.device) for _ in range(2))
        pm.mla_gqa_block_gather(self.k_cache, self.v_cache, self.k_scale, self.v_scale, *lists, self.key_indptr,
                                k_rows, v_rows, self.error_word, qo_indptr=self.qo_indptr, k_new=k, v_new=v)
        pm.mla_prompt_attention(q, k_rows, v_rows, o, self.qo_indptr, self.key_indptr, d ** -0.5, self.error_word)
        return o

    def check(self):
        status = pm.mla_check_error(self.workspace)
        bits = int(self.error_word[0])
        if status or bits:
            raise RuntimeError(f"{pm.mla_status_string(status)}, error bits {bits}")


def block_errors(lens=(37, 400, 1, 129), steps=20, device="cuda"):
    """The same for the block-scaled cache: a prompt in two parts, then steps of one to five
    tokens a request (none, now and then).  Returns {(part, request): (largest difference, root mean
    square of the differences over that of the outputs)}, parts "prompt", "prefix" and "decode"."""
    width = 1024
    counts = [[(i * 7 + 3 * b) % 6 for b in range(len(lens))] for i in range(steps)]
    more = [n // 2 + 20 for n in lens]
    total = [n + m + sum(c[b] for c in counts) for b, (n, m) in enumerate(zip(lens, more))]
    g = torch.Generator(device=device).manual_seed(1)
    xs = [torch.randn(n, width, generator=g, device=device).bfloat16() for n in total]
    layer = BlockScaledLayer(len(lens), width, device=device)
    whole = GroupedHeadLayer(width, device=device).prompt(xs).float().split(total)
    at, rows = [0] * len(lens), {}
    for part, new in [("prompt", lens), ("prefix", more)] + [("decode", c) for c in counts]:
        o = layer.forward([x[a:a + n] for x, a, n in zip(xs, at, new)]).float()
        for b, (got, w, a, n) in enumerate(zip(o.split(list(new)), whole, at, new)):
            if n:
                rows.setdefault((part, b), []).append((got, w[a:a + n]))
        at = [a + n for a, n in zip(at, new)]
    layer.check()
    out = {}
    for key, pairs in rows.items():
        got, want = (torch.cat(x) for x in zip(*pairs))
        out[key] = (got - want).abs().max().item(), ((got - want).norm() / want.norm()).item()
    return out


def run_blocks(lens=(37, 400, 1, 129), steps=20, device="cuda"):
    return max(largest for largest, _ in block_errors(lens, steps, device).values())


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--fp8", action="store_true", help="an e4m3 cache")
    ap.add_argument("--blocks", action="store_true", help="an e4m3 cache with a scale for each block and head")
    args = ap.parse_args()
    print(f"largest difference to the whole prompt: {run_blocks() if args.blocks else run(args.fp8):.4f}")
