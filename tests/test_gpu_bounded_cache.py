"""The example that runs the bounded-cache operators together: every step's
output equals plain attention over the cells that a plain copy of the cache
holds, and the caches stay within budget and slack."""
import os
import sys

import pytest
import torch

import cache_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_example_agrees_with_a_plain_cache(monkeypatch):
    import bounded_cache as ex
    cells = {}                                   # per sequence: the keys and values it should hold, and their masses
    checked = []

    append, attend, evict = ex.PagedCache.append, ex.PagedCache.attend, ex.PagedCache.evict

    def plain_append(self, s, k, v):
        ks, vs, mass = cells.get(s, (k[:0], v[:0], []))
        cells[s] = (torch.cat([ks, k]), torch.cat([vs, v]), mass + [0.0] * k.shape[0])
        append(self, s, k, v)

    def plain_attend(self, q, **kw):
        out = attend(self, q, **kw)
        for s, (k, v, mass) in cells.items():
            n, group = k.shape[0], q.shape[1] // k.shape[1]
            seen = torch.ones((1, n), dtype=torch.bool, device=q.device)
            gained = torch.zeros(n, dtype=torch.float64, device=q.device)
            for h in range(k.shape[1]):
                hs = slice(h * group, (h + 1) * group)
                o, l, p, size, S = ref.attend(q[s, hs][:, None], k[:, h], v[:, h], seen, 128 ** -0.5)
                tol, _ = ref.bounds(o, l, size, S, n, q.dtype, 2.0 ** -17)
                ref.check(out[s, hs], o[:, 0], tol[:, 0], (s, h))
                gained += p.sum((0, 1))
            assert n == self.length[s]
            # the masses that eviction goes by, as the kernel summed them (near the plain sum)
            got = self.mass[s, :n]
            want = torch.tensor(mass, dtype=torch.float64, device=q.device) + gained
            assert torch.allclose(got.double(), want, rtol=1e-4, atol=1e-5)
            cells[s] = (k, v, got.tolist())
        checked.append(1)
        return out

    def plain_evict(self, budget, sinks, recent):
        want = {s: ref.evict(m, len(m), budget, sinks, recent) for s, (_, _, m) in cells.items()}
        kept = evict(self, budget, sinks, recent)
        for s, keep in want.items():
            assert kept[s].tolist() == keep + [-1] * (budget - len(keep))
            k, v, m = cells[s]
            cells[s] = (k[keep], v[keep], [m[j] for j in keep])
        return kept

    monkeypatch.setattr(ex.PagedCache, "append", plain_append)
    monkeypatch.setattr(ex.PagedCache, "attend", plain_attend)
    monkeypatch.setattr(ex.PagedCache, "evict", plain_evict)
    said = []
    prompts, made, cache = ex.generate(sequences=3, prompt=300, steps=90, budget=160, sinks=4, recent=24, report=said.append)
    assert len(made) == len(checked) == 90 and sum("->" in s for s in said) >= 2
    assert max(cache.length) <= 160 + 64 and torch.isfinite(made[-1]).all() and torch.isfinite(prompts).all()
    held = {p for pages in cache.pages for p in pages}
    assert len(held) == sum(len(p) for p in cache.pages) and not held & set(cache.free)
    assert len(held) + len(cache.free) == cache.k.shape[0]
