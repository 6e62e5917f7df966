"""Answering many sequences that continue the same few texts.

    python examples/shared_prefix.py [--texts 2] [--readers 24] [--text 900] [--question 40] [--steps 60] [--int8]

One attention layer with random projections stands for a model. Each text is read
in once: its tokens' keys are rotated by position on their way into pages, and
kept for the prompt's own attention beside that (``cache_append``, then
``window_attn``). Each reader's question follows it: ``cache_append`` puts its tokens
behind the text (positions go on from there, cells are the reader's own) and every
further step appends one token per reader and answers it over the shared text and
the reader's own cells in one call (``prefix_attn``). The steps run from one
captured graph: lengths, positions and tables are updated in place.
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_attention_kv_qsa_gb300 as qsa  # noqa: E402

D = 128


def generate(texts: int = 2, readers: int = 24, text: int = 900, question: int = 40, steps: int = 60, heads: int = 8,
             nkv: int = 2, page: int = 16, int8: bool = False, seed: int = 0, each_step=None):
    """Returns the last step's outputs ``[texts * readers, heads, 128]``. ``each_step(state)`` is called after every step
    with what it read and wrote. The first text has ``text`` tokens, each further one 100 fewer, but one at least."""
    if min(texts, readers, text, question, steps) < 1:
        raise ValueError("texts, readers, text, question and steps are 1 at least")
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    width, nseq = heads * D, texts * readers
    project = torch.randn((width, (heads + 2 * nkv) * D), generator=g, device=dev, dtype=torch.bfloat16) * width ** -0.5
    freqs = torch.pow(torch.tensor(10000.0, dtype=torch.float64), -torch.arange(D // 2) / (D // 2)).float().to(dev)

    def qkv(x):                                              # [n, width] -> q, k, v as slices of one projection
        y = (x @ project).view(x.shape[0], heads + 2 * nkv, D)
        return y[:, :heads], y[:, heads:heads + nkv], y[:, heads + nkv:]

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device=dev)

    # One pool: pages of the texts, then of the readers.
    text_lens = [max(1, text - 100 * t) for t in range(texts)]
    columns, own_columns = -(-text // page), -(-(question + steps) // page)
    npages = texts * columns + nseq * own_columns
    kind = torch.int8 if int8 else torch.bfloat16
    k_pages, v_pages = (torch.zeros((npages, page, nkv, D), dtype=kind, device=dev) for _ in range(2))
    scales = {}
    if int8:
        scales = {n: torch.zeros((npages, page, nkv), dtype=torch.float16, device=dev) for n in ("k_scale_f16", "v_scale_f16")}
    order = torch.randperm(npages, generator=g, device=dev).to(torch.int32)
    text_table, own_table = order[:texts * columns].view(texts, columns), order[texts * columns:].view(nseq, own_columns)
    groups = ints([readers * t for t in range(texts + 1)])

    # The texts, packed one after the other: positions are the cells' numbers.
    cu = ints([sum(text_lens[:t]) for t in range(texts + 1)])
    x = torch.randn((sum(text_lens), width), generator=g, device=dev, dtype=torch.bfloat16)
    q, k, v = qkv(x)
    turned = torch.empty((x.shape[0], nkv, D), dtype=torch.bfloat16, device=dev)
    q, turned = qsa.cache_append(k, v, k_pages, v_pages, text_table, ints(text_lens), cu=cu, q=q, freqs=freqs, k_out=turned, **scales)
    read, _ = qsa.window_attn(q, turned, v, cu, cu, max(text_lens))

    # The readers' questions: cells from 0 on, positions behind their text. Their last tokens are answered below.
    lens = torch.full((nseq,), question, dtype=torch.int32, device=dev)
    behind = ints(text_lens).repeat_interleave(readers)
    x = torch.randn((nseq * question, width), generator=g, device=dev, dtype=torch.bfloat16)
    x[::question] += read[cu[1:].long() - 1].reshape(texts, width).repeat_interleave(readers, 0)
    _, k, v = qkv(x)
    positions = (behind[:, None] + torch.arange(question, device=dev, dtype=torch.int32)).reshape(-1)
    qsa.cache_append(k, v, k_pages, v_pages, own_table, lens, cu=ints([question * s for s in range(nseq + 1)]), freqs=freqs,
                     positions=positions, **scales)

    # One token of every reader at a time, captured once.
    x = torch.randn((nseq, width), generator=g, device=dev, dtype=torch.bfloat16)
    out = torch.zeros((nseq, heads, D), dtype=torch.bfloat16, device=dev)
    at = torch.empty_like(lens)
    state = {"text_table": text_table, "text_lens": text_lens, "own_table": own_table, "lens": lens, "k": k_pages, "v": v_pages,
             "out": out, "at": at, "freqs": freqs, **scales}

    def step():
        lens.add_(1)
        torch.add(behind, lens, alpha=1, out=at).sub_(1)
        q, k, v = qkv(x)
        turned_q, _ = qsa.cache_append(k, v, k_pages, v_pages, own_table, lens, q=q, positions=at, freqs=freqs, **scales)
        state["q"], state["turned_q"], state["new_k"], state["new_v"] = q, turned_q, k, v
        qsa.prefix_attn(turned_q, k_pages, v_pages, text_table, ints_text_lens, groups, own_table, lens, out=out, **scales)
        x.copy_(torch.nn.functional.normalize(out.reshape(nseq, width).float(), dim=1) * width ** 0.5)

    ints_text_lens = ints(text_lens)
    graph = None
    for n in range(steps):
        if n == 1:                                           # the first step warms the allocator up
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is None:
            step()
        else:
            graph.replay()
        if each_step is not None:
            each_step(state)
    return out


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("texts", 2), ("readers", 24), ("text", 900), ("question", 40), ("steps", 60)):
        ap.add_argument("--" + name, type=int, default=default)
    ap.add_argument("--int8", action="store_true")
    a = ap.parse_args()
    out = generate(a.texts, a.readers, a.text, a.question, a.steps, int8=a.int8)
    torch.cuda.synchronize()
    print(f"{a.steps} steps of {out.shape[0]} readers of {a.texts} texts; all finite: {bool(torch.isfinite(out).all())}")


if __name__ == "__main__":
    main()
