"""Generating with a key-value cache that is kept within a budget.

    python examples/bounded_cache.py [--sequences 4] [--prompt 900] [--steps 200] [--budget 512] [--observe 32]

One attention layer with random projections stands for a model. The prompts'
tokens attend with a sliding window and the first tokens always visible
(``window_attn``), their keys and values go into pages (``cache_append``), and each further token
attends its sequence's pages (``paged_attn``), which also adds the weight that
every cell received to a running mass. When a cache has grown past its budget
by a few pages, ``cache_evict`` keeps the first cells, the most recent ones and
those of largest mass, in new pages, and the old pages are free again.

``window_attn`` gives no masses. What the prompt's cells are worth is learnt from
its last tokens (``--observe``), which attend the pages once more, each as a row of
``paged_attn`` with a length of its own, and from the steps: a cache is cut only
after a step has attended it.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_kv_qsa_gb300 as qsa  # noqa: E402

D = 128


class PagedCache:
    """Keys and values of a batch of sequences in pages of one pool, with a running mass per cell."""

    def __init__(self, sequences: int, pages: int, page: int, nkv: int, cells: int, device, dtype=torch.bfloat16):
        self.page, self.device = page, device
        self.k = torch.zeros((pages, page, nkv, D), dtype=dtype, device=device)
        self.v = torch.zeros_like(self.k)
        self.free = list(range(pages))
        self.pages = [[] for _ in range(sequences)]          # each sequence's pages, in order
        self.length = [0] * sequences                        # the host's copy of lens
        self.columns = -(-cells // page)
        self.table = torch.zeros((sequences, self.columns), dtype=torch.int32, device=device)
        self.lens = torch.zeros(sequences, dtype=torch.int32, device=device)
        self.mass = torch.zeros((sequences, self.columns * page), device=device)

    def _reserve(self, s: int, cells: int) -> None:
        while len(self.pages[s]) * self.page < cells:
            self.table[s, len(self.pages[s])] = self.free[-1]
            self.pages[s].append(self.free.pop())

    def append(self, s: int, k: torch.Tensor, v: torch.Tensor) -> None:
        """New cells ``[n, nkv, 128]`` at the end of sequence ``s``."""
        n, at = k.shape[0], self.length[s]
        self._reserve(s, at + n)
        self.length[s] = at + n
        self.lens[s] = at + n
        cu = None if n == 1 else torch.tensor([0, n], dtype=torch.int32, device=self.device)
        qsa.cache_append(k, v, self.k, self.v, self.table[s:s + 1], self.lens[s:s + 1], cu=cu)

    def attend(self, q: torch.Tensor, window: int = -1, sinks: int = 0) -> torch.Tensor:
        """Each sequence's newest token ``q [sequences, heads, 128]`` over its cells; the mass grows."""
        out, _ = qsa.paged_attn(q, self.k, self.v, self.table, self.lens, window=window, sinks=sinks, mass=self.mass)
        return out

    def observe(self, s: int, q: torch.Tensor, window: int = -1, sinks: int = 0) -> None:
        """Adds the weights that the last tokens ``q [n, heads, 128]`` of sequence ``s`` give its cells to its mass."""
        n = q.shape[0]
        lens = torch.arange(self.length[s] - n + 1, self.length[s] + 1, dtype=torch.int32, device=self.device)
        mass = torch.zeros((n, self.mass.shape[1]), device=self.device)
        qsa.paged_attn(q, self.k, self.v, self.table[s].repeat(n, 1), lens, window=window, sinks=sinks, mass=mass)
        self.mass[s] += mass.sum(0)

    def evict(self, budget: int, sinks: int, recent: int) -> torch.Tensor:
        """Every sequence down to ``budget`` cells, in new pages; returns the kept cells' old places."""
        each = -(-budget // self.page)
        new = [[self.free.pop() for _ in range(each)] for _ in self.pages]
        new_table = torch.tensor(new, dtype=torch.int32, device=self.device)
        kept, self.lens, mass = qsa.cache_evict(self.k, self.v, self.table, self.lens, self.mass, new_table, budget,
                                                sinks=sinks, recent=recent, new_mass=torch.empty_like(self.mass))
        for s, old in enumerate(self.pages):
            self.length[s] = min(self.length[s], budget)
            used = -(-self.length[s] // self.page)
            self.free += old + new[s][used:]
            self.pages[s] = new[s][:used]
        self.table = torch.zeros_like(self.table)
        self.table[:, :each] = new_table
        self.mass = mass
        return kept


def generate(sequences: int = 4, prompt: int = 900, steps: int = 200, budget: int = 512, sinks: int = 4, recent: int = 64,
             window: int = 256, heads: int = 8, nkv: int = 2, page: int = 16, seed: int = 0, report=None, observe: int = 0):
    """Runs prompts and steps; returns ``(outputs of the prompts, outputs of every step, cache)``. ``report`` is
    called with a text now and then. ``observe``: how many of a prompt's last tokens tell what its cells are worth."""
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    width = heads * D
    project = torch.randn((width, (heads + 2 * nkv) * D), generator=g, device=dev, dtype=torch.bfloat16) * width ** -0.5

    def qkv(x):                                              # [n, width] -> q, k, v as slices of one projection
        y = (x @ project).view(x.shape[0], heads + 2 * nkv, D)
        return y[:, :heads], y[:, heads:heads + nkv], y[:, heads + nkv:]

    slack = 4 * page                                         # evicting every few pages, not every token
    lengths = [prompt - (prompt // (2 * sequences)) * s for s in range(sequences)]
    most = max(max(lengths), budget) + slack
    pages = sequences * (-(-most // page) + -(-budget // page) + 1)
    cache = PagedCache(sequences, pages, page, nkv, most, dev)

    # The prompts, packed one after the other.
    starts = torch.tensor([sum(lengths[:s]) for s in range(sequences + 1)], dtype=torch.int32, device=dev)
    x = torch.randn((sum(lengths), width), generator=g, device=dev, dtype=torch.bfloat16)
    q, k, v = qkv(x)
    prompts, _ = qsa.window_attn(q, k, v, starts, starts, max(lengths), window=window, sinks=sinks)
    for s in range(sequences):
        a, b = sum(lengths[:s]), sum(lengths[:s + 1])
        cache.append(s, k[a:b], v[a:b])
        if observe > 0:
            cache.observe(s, q[max(a, b - observe):b])
    if report:
        report(f"prompts of {lengths} tokens, {len(cache.free)} of {pages} pages free")

    # One token at a time; a step's output is the next step's input.
    ends = starts[1:].long() - 1
    x = prompts[ends].reshape(sequences, width)
    made = []
    for step in range(steps):
        q, k, v = qkv(torch.nn.functional.normalize(x.float(), dim=1).to(torch.bfloat16) * width ** 0.5)
        for s in range(sequences):
            cache.append(s, k[s:s + 1], v[s:s + 1])
        out = cache.attend(q)
        made.append(out)
        if max(cache.length) >= budget + slack:   # with this step's weights in the masses
            before = list(cache.length)
            cache.evict(budget, sinks, recent)
            if report:
                report(f"step {step}: {before} -> {cache.length} cells, {len(cache.free)} pages free")
        x = out.reshape(sequences, width)
    return prompts, made, cache


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("sequences", 4), ("prompt", 900), ("steps", 200), ("budget", 512), ("observe", 32)):
        ap.add_argument("--" + name, type=int, default=default)
    a = ap.parse_args()
    _, made, cache = generate(a.sequences, a.prompt, a.steps, a.budget, report=print, observe=a.observe)
    torch.cuda.synchronize()
    print(f"{len(made)} steps of {a.sequences} sequences; caches of {cache.length} cells")


if __name__ == "__main__":
    main()
