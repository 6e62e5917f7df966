"""The example's first eviction: the masses it goes by are weights that the
prompt's cells received, from the steps so far and, where asked for, from the
prompt's last tokens."""
import os
import sys

import pytest
import torch

import cache_ref as ref

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("observe", [0, 24])
def test_no_eviction_goes_by_masses_that_nothing_gave(monkeypatch, observe):
    import bounded_cache as ex
    at_eviction = []
    evict = ex.PagedCache.evict

    def looked_at(self, *a, **kw):
        at_eviction.append([self.mass[s, :n].clone() for s, n in enumerate(self.length)])
        return evict(self, *a, **kw)

    monkeypatch.setattr(ex.PagedCache, "evict", looked_at)
    _, made, cache = ex.generate(sequences=3, prompt=300, steps=80, budget=160, sinks=4, recent=24, observe=observe)
    assert len(made) == 80 and max(cache.length) <= 160 + 64 and len(at_eviction) >= 2
    heads = 8
    for s, mass in enumerate(at_eviction[0]):
        assert bool((mass > 0).all())                # no cell without a weight: ties decide nothing
        rows = 1 + min(observe, mass.numel() - 1)    # each row's weights sum to 1 per head, within 2^-10 of it
        assert abs(float(mass.double().sum()) - heads * rows) < heads * rows * 2.0 ** -10


def test_masses_from_the_last_tokens(monkeypatch):
    """`observe` equals the weights of plain attention of the last tokens, each over the cells up to its own."""
    import bounded_cache as ex
    observe, seen = ex.PagedCache.observe, []

    def checked(self, s, q):
        observe(self, s, q)
        n, m, group = self.length[s], q.shape[0], q.shape[1] // self.k.shape[2]
        j = torch.arange(n, device=q.device)
        see = j <= (n - m + torch.arange(m, device=q.device))[:, None]
        page, slot = self.table[s].long()[j // self.page], j % self.page
        gained = torch.zeros(n, dtype=torch.float64, device=q.device)
        for h in range(self.k.shape[2]):
            k, v = self.k[page, slot, h], self.v[page, slot, h]
            _, _, p, _, _ = ref.attend(q[:, h * group:(h + 1) * group].transpose(0, 1), k, v, see, 128 ** -0.5)
            gained += p.sum((0, 1))
        assert torch.allclose(self.mass[s, :n].double(), gained, rtol=1e-4, atol=1e-5)
        assert torch.count_nonzero(self.mass[s, n:]) == 0
        seen.append((n, m))

    monkeypatch.setattr(ex.PagedCache, "observe", checked)
    ex.generate(sequences=3, prompt=90, steps=1, budget=160, sinks=4, recent=24, observe=50)
    assert [m for _, m in seen] == [50, 50, 50] and len({n for n, _ in seen}) == 3
