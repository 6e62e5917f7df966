"""qsa_cache_evict against a plain sort: the kept cells, their order, the
copied keys, values and scales, and the carried masses are equal bit for bit."""
import math

import pytest
import torch

import cache_ref as ref
import sparse_attention_kv_qsa_gb300 as qsa
from test_gpu_paged_attn import BF16, F16, I8, Cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def run(dev, lens, budget, sinks, recent, nkv=2, page=16, kv=BF16, layout="nhd", mass=None, mass_cols=None, cols=None):
    per = -(-budget // page)
    c = Cache(dev, lens, nkv, page, kv, layout, spare=per * len(lens) + 2, cols=cols)
    new_table = c.free[:per * len(lens)].view(len(lens), per)
    if mass is None:
        g = torch.Generator(device=dev).manual_seed(7)
        mass = torch.rand((len(lens), c.cols * page), generator=g, device=dev)
    elif isinstance(mass, list):
        full = torch.full((len(lens), c.cols * page), math.nan, device=dev)
        for s, m in enumerate(mass):
            full[s, :len(m)] = torch.tensor(m, device=dev)
        mass = full
    tensors = [t for t in (c.k, c.v, c.ks, c.vs) if t is not None]
    before = [t.clone() for t in tensors]
    nm = None if mass_cols is None else torch.full((len(lens), mass_cols), -3.0, device=dev)
    kept, new_lens, new_mass = qsa.cache_evict(c.k, c.v, c.table, c.lens, mass, new_table, budget, sinks=sinks,
                                               recent=recent, k_scale_f16=c.ks, v_scale_f16=c.vs, new_mass=nm)
    for s, n in enumerate(lens):
        n = max(0, min(n, c.cols * page))
        want = ref.evict(mass[s, :n].tolist(), n, budget, sinks, recent)
        assert kept[s].tolist() == want + [-1] * (budget - len(want)), s
        assert int(new_lens[s]) == len(want)
        j = torch.tensor(want, dtype=torch.long, device=dev)
        i = torch.arange(len(want), device=dev)
        assert torch.equal(new_mass[s, :len(want)].view(torch.int32), mass[s, j].view(torch.int32))
        assert torch.count_nonzero(new_mass[s, len(want):]) == 0
        for t, b in zip(tensors, before):
            b[new_table[s, i // page].long(), i % page] = b[c.table[s, j // page].long(), j % page]
    for t, b in zip(tensors, before):                      # the copies, and nothing else changed
        kind = torch.int8 if t.dtype == I8 else torch.int16
        assert torch.equal(t.contiguous().view(kind), b.contiguous().view(kind))
    return c, kept


@pytest.mark.parametrize("kv", [BF16, F16, I8])
@pytest.mark.parametrize("layout,nkv,page", [("nhd", 2, 16), ("hnd", 3, 7), ("joint", 8, 64), ("nhd", 1, 1)])
def test_every_length(dev, kv, layout, nkv, page):
    run(dev, [0, 1, 63, 64, 65, 66, 100, 128, 1000, 1025, 2500], 64, 4, 16, nkv, page, kv, layout)


@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (5, 2, 3), (40, 0, 0), (40, 40, 0),
                                                 (40, 0, 40), (999, 3, 5), (1000, 1, 1), (1300, 7, 100)])
def test_budgets(dev, budget, sinks, recent):
    run(dev, [1000, 999, 40, 2100], budget, sinks, recent)


@pytest.mark.parametrize("lens,budget", [([70000], 9000), ([40000, 3, 20000], 16384), ([131072], 130000),
                                         ([300000], 1000)])
def test_long_caches(dev, lens, budget):
    run(dev, lens, budget, 4, 100, 1, 64, I8)


def test_ties_keep_the_lower_cells(dev):
    n = 3000
    for values in ([1.0] * n, [float(j % 2) for j in range(n)], [float(j % 7 == 3) for j in range(n)],
                   [0.0, -0.0] * (n // 2), [math.inf] * n, [-math.inf] * n):
        run(dev, [n, n - 1], 500, 3, 30, mass=[values, values[:n - 1]])


@pytest.mark.parametrize("n,budget", [(700, 200), (30000, 5000)])
@pytest.mark.parametrize("high,low", [(2.0, 0.5), (1.0625, 1.0), (1.0000001192092896, 1.0), (-0.5, -math.inf), (1e-45, 0.0)])
def test_exactly_the_larger_masses_fit(dev, n, budget, high, low):
    """The cells to keep are all those of one mass, told apart by the first, second or last bits; and one more, one less."""
    for more in (-1, 0, 1):
        mass = [low] * n
        for i in range(budget - 4 - 20 + more):
            mass[4 + (i * 7919) % (n - 24)] = high             # 7919 is prime: other cells every time
        run(dev, [n], budget, 4, 20, 1, 16, I8, mass=[mass])


@pytest.mark.parametrize("lens", [[9000, 16000, 0, 4097, 15999], [20000, 33333, 6], [20000 - 700 * i for i in range(21)]])
def test_several_middle_sized_caches(dev, lens):
    run(dev, lens, 3000, 4, 100, 1, 16, I8)


def test_more_cells_than_shared_memory_holds(dev):
    run(dev, [700001], 9001, 4, 100, 1, 64, I8)


def test_masses_of_every_kind(dev):
    """NaN counts as the lowest, infinities and tiny differences are told apart."""
    n = 2000
    g = torch.Generator().manual_seed(4)
    wild = torch.randint(-2 ** 31, 2 ** 31, (n,), generator=g).to(torch.int32).view(torch.float32)
    close = (torch.randint(0, 40, (n,), generator=g) + 0x3F800000).to(torch.int32).view(torch.float32)
    run(dev, [n, n, n], 700, 4, 64, mass=[wild.tolist(), close.tolist(), [math.nan] * n])


def test_mass_buffer_wider_than_the_budget(dev):
    run(dev, [500, 20, 64], 64, 4, 8, mass_cols=211)


def test_bad_pages_are_skipped(dev):
    """A copy from or to a page outside the pool does not happen; the list of kept cells does not depend on it."""
    c = Cache(dev, [64], 1, 16, BF16, spare=4)
    mass = torch.arange(64, device=dev, dtype=torch.float32).repeat(1, c.cols * 16 // 64 + 1)[:, :c.cols * 16].contiguous()
    new = c.free[:2].view(1, 2).clone()
    good, new[0, 1] = int(new[0, 0]), c.k.shape[0]
    c.table[0, 2] = -4
    k0, free = c.k.clone(), int(c.free[2])
    kept, n, _ = qsa.cache_evict(c.k, c.v, c.table, c.lens, mass, new, 32, sinks=0, recent=0)
    assert kept[0].tolist() == list(range(32, 64)) and int(n[0]) == 32
    # cells 32..47 come from the bad page, 48..63 would go to the bad page
    assert torch.equal(c.k[good], k0[good]) and torch.equal(c.k[free], k0[free])


def test_evicted_cache_is_attended(dev):
    """Attention over the new pages equals attention over the kept cells."""
    lens = [500, 64, 300]
    c, kept = run(dev, lens, 128, 4, 32, nkv=2)
    new = c.free[:8 * 3].view(3, 8)
    q = torch.randn((3, 8, 128), device=dev).to(BF16)
    new_lens = torch.tensor([min(n, 128) for n in lens], dtype=torch.int32, device=dev)
    out, _ = qsa.paged_attn(q, c.k, c.v, new, new_lens)
    for s in range(3):
        j = kept[s][kept[s] >= 0].long()
        k, v = (t[c.table[s, j // 16].long(), j % 16].float() for t in (c.k, c.v))
        for h in range(8):
            p = torch.softmax(k[:, h // 4] @ q[s, h].float() / 128 ** 0.5, 0)
            assert torch.allclose(out[s, h].float(), p @ v[:, h // 4], rtol=2 ** -7, atol=1e-3)


def test_graph(dev):
    c = Cache(dev, [900, 160], 2, 16, BF16, spare=2 * 8)
    mass = torch.rand((2, c.cols * 16), device=dev)
    new = c.free[:16].view(2, 8)
    bufs = [torch.empty((2, 128), dtype=torch.int32, device=dev), torch.empty(2, dtype=torch.int32, device=dev),
            torch.empty((2, 128), device=dev)]
    call = lambda: qsa.cache_evict(c.k, c.v, c.table, c.lens, mass, new, 128, sinks=4, recent=16, kept=bufs[0],  # noqa: E731
                                   new_lens=bufs[1], new_mass=bufs[2])
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    for step in range(10):
        lens = [900 - 80 * step, 70 + 10 * step]
        c.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        mass.uniform_()
        graph.replay()
        torch.cuda.synchronize()
        for s, n in enumerate(lens):
            want = ref.evict(mass[s, :n].tolist(), n, 128, 4, 16)
            assert bufs[0][s].tolist() == want + [-1] * (128 - len(want))
            j, i = torch.tensor(want, device=dev), torch.arange(len(want), device=dev)
            assert torch.equal(c.k[new[s, i // 16].long(), i % 16], c.k[c.table[s, j // 16].long(), j % 16])


def test_refusals_of_the_binding(dev):
    c = Cache(dev, [20, 30], 2, 16, BF16, spare=4)
    mass = torch.zeros((2, c.cols * 16), device=dev)
    new = c.free[:4].view(2, 2)
    for args in ((mass[:, :10], new, 32), (mass, new, 33), (mass, new, 0), (mass, new[:1], 32), (mass.double(), new, 32),
                 (mass, new.long(), 32)):
        with pytest.raises(ValueError):
            qsa.cache_evict(c.k, c.v, c.table, c.lens, *args)
    with pytest.raises(ValueError):
        qsa.cache_evict(c.k, c.v, c.table, c.lens, mass, new, 20, sinks=11, recent=10)
    with pytest.raises(ValueError):
        qsa.cache_evict(c.k, c.v, c.table, c.lens, mass, new, 20, kept=torch.empty((2, 21), dtype=torch.int32, device=dev))
