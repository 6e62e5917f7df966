"""qsa_paged_attn (one new token per sequence over a paged cache) against the
plain 64-bit form. Tolerances: cache_ref.bounds; the weights enter the product
with the values with at least 17 significant bits (16-bit cells) or 22 (int8),
so p_half = 2^-17 (bfloat16 cells) or 2^-22."""
import math

import pytest
import torch

import cache_ref as ref
import sparse_attention_kv_qsa_gb300 as qsa

pytestmark = pytest.mark.gpu
BF16, F16, F32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8
KINDS = [(BF16, BF16), (F16, F16), (I8, F32), (I8, BF16), (I8, F16)]


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


class Cache:
    """A paged cache whose pages are a random order of a pool; everything that no sequence can see is poisoned."""

    def __init__(self, dev, lens, nkv, page, kv, layout="nhd", seed=0, spare=3, cols=None):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.lens_list, self.page, self.nkv, self.kv, self.dev = list(lens), page, nkv, kv, dev
        need = [-(-max(n, 0) // page) for n in lens]
        self.cols = cols if cols is not None else max(need + [1]) + 1
        npages = sum(need) + spare
        shape = {"nhd": (npages, page, nkv, 128), "hnd": (npages, nkv, page, 128),
                 "joint": (npages, 2, page, nkv, 128)}[layout]

        def values(shape):
            if kv == I8:
                return torch.randint(-128, 128, shape, generator=g, device=dev, dtype=I8)
            return torch.randn(shape, generator=g, device=dev, dtype=kv)

        if layout == "joint":
            self.k, self.v = values(shape).unbind(1)
        else:
            self.k, self.v = values(shape), values(shape)
            if layout == "hnd":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.ks = self.vs = None
        if kv == I8:
            sc = lambda: torch.exp2(torch.rand((npages, nkv, page), generator=g, device=dev) * 4 - 9).to(F16)  # noqa: E731
            self.ks, self.vs = sc().transpose(1, 2), sc().transpose(1, 2)
        order = torch.randperm(npages, generator=g, device=dev).to(torch.int32)
        # what lies past a sequence's pages is never looked up: ids far out of range
        self.table = torch.full((len(lens), self.cols), 2 ** 31 - 1, dtype=torch.int32, device=dev)
        at = 0
        for s, c in enumerate(need):
            self.table[s, :c] = order[at:at + c]
            at += c
        self.free = order[at:]
        self.lens = torch.tensor(lens, dtype=torch.int32, device=dev)

    def poison(self, window, sinks):
        """NaN in every cell that no sequence sees (codes of int8 cells get NaN scales)."""
        used = torch.zeros(self.k.shape[:2], dtype=torch.bool, device=self.dev)
        for s, n in enumerate(self.lens_list):
            j = torch.arange(max(n, 0), device=self.dev)
            j = j[(j >= n - window) | (j < sinks)] if window >= 0 else j
            used[self.table[s, j // self.page].long(), j % self.page] = True
        hidden = ~used
        for t in (self.k, self.v) if self.kv != I8 else (self.ks, self.vs):
            t[hidden] = math.nan
        return self

    def call(self, q, **kw):
        return qsa.paged_attn(q, self.k, self.v, self.table, self.lens, k_scale_f16=self.ks, v_scale_f16=self.vs, **kw)

    def check(self, q, out, lse, window=-1, sinks=0, scale=128 ** -0.5, mass=None, mass_out=None):
        heads = q.shape[1]
        g = heads // self.nkv
        p_half = 2.0 ** -17 if self.kv == BF16 else 2.0 ** -22
        for s, n in enumerate(self.lens_list):
            n = max(0, min(n, self.cols * self.page))
            gained, loose = torch.zeros(n, dtype=torch.float64, device=self.dev), 0.0
            j = torch.arange(n, device=self.dev)
            seen = torch.ones_like(j, dtype=torch.bool)
            if window >= 0:
                seen = (j >= n - window) | (j < sinks)
            for h in range(self.nkv):
                k, ok = ref.paged_cells(self.k, self.ks, self.table[s], n, h, self.page)
                v, _ = ref.paged_cells(self.v, self.vs, self.table[s], n, h, self.page)
                o, l, p, size, S = ref.attend(q[s, h * g:(h + 1) * g][:, None], k, v, (seen & ok)[None], scale)
                tol, ltol = ref.bounds(o, l, size, S, n, q.dtype, p_half)
                ref.check(out[s, h * g:(h + 1) * g], o[:, 0], tol[:, 0], ("out", s, h))
                ref.check(lse[s, h * g:(h + 1) * g], l[:, 0], ltol[:, 0], ("lse", s, h))
                gained += p.sum((0, 1))
                loose = max(loose, float((2 * 256 * ref.U * S + 2 * ltol).max()) if n else 0.0)
            if mass is not None:
                want = mass[s, :n].double() + gained
                tol = gained * (loose + 64 * ref.U) + want.abs() * 4 * ref.U
                ref.check(mass_out[s, :n], want, tol, ("mass", s))


def queries(dev, nseq, heads, dtype, seed=1):
    g = torch.Generator(device=dev).manual_seed(seed)
    return torch.randn((nseq, heads, 128), generator=g, device=dev).to(dtype)


LENS = [1, 0, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 200, 511, 513, 1000, 2049]


@pytest.mark.parametrize("kv,qt", KINDS)
@pytest.mark.parametrize("nkv,group,page,layout", [(1, 1, 16, "nhd"), (2, 4, 16, "hnd"), (8, 4, 64, "joint"),
                                                   (2, 3, 1, "nhd"), (1, 8, 48, "joint"), (3, 5, 7, "hnd"),
                                                   (1, 9, 128, "nhd"), (2, 16, 32, "nhd"), (1, 17, 16, "hnd"),
                                                   (1, 40, 16, "nhd")])
def test_every_length(dev, kv, qt, nkv, group, page, layout):
    c = Cache(dev, LENS, nkv, page, kv, layout).poison(-1, 0)
    q = queries(dev, len(LENS), nkv * group, qt)
    out, lse = c.call(q)
    c.check(q, out, lse)
    assert torch.count_nonzero(out[1]) == 0 and bool((lse[1] == -math.inf).all())
    again, lse2 = c.call(q)
    assert torch.equal(out, again) and torch.equal(lse, lse2)      # a fixed order of sums


@pytest.mark.parametrize("kv,qt", [(BF16, BF16), (F16, F16), (I8, F32)])
@pytest.mark.parametrize("nkv,group,page", [(1, 9, 16), (2, 16, 48), (1, 12, 64), (1, 40, 16)])
def test_many_heads_on_wide_tables(dev, kv, qt, nkv, group, page):
    """Tables for more cells than stay in L2: 9 to 16 heads of 16-bit cells share one reading."""
    lens = LENS + [9000, 20000]
    cols = max(20000 // page + 2, 1 + (128 << 20) // (512 * nkv * page * len(lens)))
    c = Cache(dev, lens, nkv, page, kv, cols=cols)
    q = queries(dev, len(lens), nkv * group, qt)
    out, lse = c.call(q)
    c.check(q, out, lse)
    again, lse2 = c.call(q)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    mass = torch.zeros((len(lens), c.cols * page), device=dev)
    out, lse = c.poison(700, 9).call(q, window=700, sinks=9, mass=mass)
    c.check(q, out, lse, 700, 9, mass=torch.zeros_like(mass), mass_out=mass)


@pytest.mark.parametrize("kv,qt", [(BF16, BF16), (I8, F32)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 3), (1, 0), (1, 1), (16, 4), (100, 70), (511, 0), (512, 1),
                                          (4096, 5), (64, 5000), (0, 2 ** 31 - 1), (2 ** 31 - 1, 4)])
def test_windows_and_sinks(dev, kv, qt, window, sinks):
    c = Cache(dev, LENS, 2, 16, kv).poison(window, sinks)
    q = queries(dev, len(LENS), 8, qt)
    out, lse = c.call(q, window=window, sinks=sinks)
    c.check(q, out, lse, window, sinks)
    if window == 0 and sinks == 0:
        assert torch.count_nonzero(out) == 0 and bool((lse == -math.inf).all())


@pytest.mark.parametrize("kv,qt", KINDS)
@pytest.mark.parametrize("lens", [[30000], [20000, 1, 9000], [4096] * 5 + [70001]])
def test_long_caches(dev, kv, qt, lens):
    """Few rows: the cells of a row are split over the GPU and joined."""
    c = Cache(dev, lens, 2, 64, kv)
    q = queries(dev, len(lens), 8, qt)
    out, lse = c.call(q)
    c.check(q, out, lse)


def test_many_sequences(dev):
    lens = [(37 * i) % 90 for i in range(700)]
    c = Cache(dev, lens, 1, 16, BF16).poison(-1, 0)
    q = queries(dev, 700, 4, BF16)
    out, lse = c.call(q)
    c.check(q, out, lse)


@pytest.mark.parametrize("kv,qt", KINDS)
@pytest.mark.parametrize("window,sinks", [(-1, 0), (100, 4), (0, 0)])
def test_mass(dev, kv, qt, window, sinks):
    lens = LENS + [5000]
    c = Cache(dev, lens, 2, 16, kv).poison(window, sinks)
    q = queries(dev, len(lens), 12, qt)
    g = torch.Generator(device=dev).manual_seed(3)
    wide = torch.rand((len(lens), c.cols * 16 + 5), generator=g, device=dev)
    mass, out_mass = wide[:, :c.cols * 16], torch.full_like(wide, -5.0)[:, :c.cols * 16]
    before = mass.clone()
    out, lse = c.call(q, window=window, sinks=sinks, mass=mass, mass_out=out_mass)
    c.check(q, out, lse, window, sinks, mass=mass, mass_out=out_mass)
    assert torch.equal(mass, before)
    for s, n in enumerate(lens):
        assert bool((out_mass[s, n:] == -5.0).all())               # columns past the length are not written
    out2, _ = c.call(q, window=window, sinks=sinks, mass=mass)     # in place, same bits
    assert torch.equal(out, out2)
    for s, n in enumerate(lens):
        assert torch.equal(mass[s, :n], out_mass[s, :n]) and torch.equal(mass[s, n:], before[s, n:])


def test_bad_pages_are_skipped(dev):
    """Page ids below 0 or past the pool are as if their cells were hidden; a sequence of such pages alone is empty."""
    c = Cache(dev, [100, 64, 40], 2, 16, F16)
    c.table[0, 2] = -1
    c.table[0, 4] = c.k.shape[0]
    c.table[1, :4] = torch.tensor([-7, 2 ** 31 - 1, -2 ** 31, c.k.shape[0]], dtype=torch.int32)
    q = queries(dev, 3, 4, F16)
    mass = torch.zeros((3, c.cols * 16), device=dev)
    out, lse = c.call(q, mass=mass)
    c.check(q, out, lse, mass=torch.zeros_like(mass), mass_out=mass)
    assert torch.count_nonzero(out[1]) == 0 and torch.count_nonzero(mass[1]) == 0


def test_lengths_are_clamped(dev):
    c = Cache(dev, [-5, 64, 33], 1, 16, BF16, cols=4)
    c.lens[1] = 10 ** 9
    q = queries(dev, 3, 4, BF16)
    out, lse = c.call(q)
    c.check(q, out, lse)
    assert torch.count_nonzero(out[0]) == 0


def test_strided_arguments(dev):
    """Queries as a slice of a fused projection, a table as a view, one output buffer given."""
    c = Cache(dev, [300, 5, 77], 2, 16, BF16)
    fused = queries(dev, 3, 8 + 2 * 2, BF16)
    q = fused[:, :8]
    out, lse = c.call(q)
    c.check(q, out, lse)
    qt = queries(dev, 8, 3, BF16).transpose(0, 1)                  # heads outside sequences
    wide = torch.full((3, c.cols + 3), -1, dtype=torch.int32, device=dev)
    wide[:, :c.cols] = c.table
    c.table = wide[:, :c.cols]
    buf = torch.empty((3, 8, 128), dtype=BF16, device=dev)
    out, lse = c.call(qt, out=buf)
    assert out is buf
    c.check(qt, out, lse)


@pytest.mark.parametrize("qmul,scale", [(60.0, 128 ** -0.5), (1e-12, 128 ** -0.5), (1.0, 3.0), (1.0, 1e-30)])
@pytest.mark.parametrize("kv,qt", [(BF16, BF16), (F16, F16), (I8, F32)])
def test_input_ranges(dev, qmul, scale, kv, qt):
    """One-hot and uniform softmax: no overflow, no loss of the small."""
    c = Cache(dev, [700, 64, 1], 2, 16, kv)
    q = (queries(dev, 3, 8, F32) * qmul).to(qt)
    out, lse = c.call(q, scale=scale)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    c.check(q, out, lse, scale=scale)


@pytest.mark.parametrize("lo,hi", [(-24, -20), (10, 15), (-24, 15)])
def test_int8_scale_ranges(dev, lo, hi):
    """Value scales over the whole binary16 range, subnormal ones and zero among them."""
    c = Cache(dev, [900, 130], 2, 16, I8)
    g = torch.Generator(device=dev).manual_seed(9)
    c.vs.copy_(torch.exp2(torch.rand(c.vs.shape, generator=g, device=dev) * (hi - lo) + lo).to(F16))
    c.vs[:, ::5] = 0.0
    q = queries(dev, 2, 8, F32)
    out, lse = c.call(q)
    c.check(q, out, lse)


def test_a_visible_nan_reaches_its_own_row_only(dev):
    c = Cache(dev, [100, 100], 2, 16, BF16)
    c.v[c.table[0, 3].long(), 5, 1] = math.nan
    q = queries(dev, 2, 8, BF16)
    out, _ = c.call(q)
    assert torch.isnan(out[0, 4:]).all()
    assert torch.isfinite(out[0, :4]).all() and torch.isfinite(out[1]).all()


def test_other_stream_and_graph(dev):
    """Captured once, replayed for other lengths, queries and pages."""
    c = Cache(dev, [600, 100, 1000], 2, 16, I8)
    q = queries(dev, 3, 8, F32)
    out, lse = torch.empty((3, 8, 128), device=dev), torch.empty((3, 8), device=dev)
    mass = torch.zeros((3, c.cols * 16), device=dev)
    scratch = torch.empty(qsa.paged_attn_scratch_bytes(3, 8, 2, c.cols, 16, True), dtype=torch.uint8, device=dev)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        c.call(q, out=out, lse=lse, mass=mass, scratch=scratch)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            c.call(q, out=out, lse=lse, mass=mass, scratch=scratch)
    for step in range(20):
        c.lens_list = [600 - 29 * step, 80 + step, max(0, 1000 - 60 * step)]
        c.lens.copy_(torch.tensor(c.lens_list, dtype=torch.int32))
        q.copy_(queries(dev, 3, 8, F32, seed=step))
        mass.zero_()
        out.fill_(math.nan)
        scratch.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        c.check(q, out, lse, mass=torch.zeros_like(mass), mass_out=mass)
    assert qsa.device_error(dev) == 0


def test_offsets_past_32_bits(dev):
    """A pool of more than 2^32 bytes: the last page's cells are read right."""
    page, nkv = 128, 8
    npages = (1 << 32) // (page * nkv * 128 * 2) + 40
    k = torch.zeros((npages, page, nkv, 128), dtype=BF16, device=dev)
    v = torch.zeros_like(k)
    g = torch.Generator(device=dev).manual_seed(2)
    k[-3:] = torch.randn((3, page, nkv, 128), generator=g, device=dev, dtype=BF16)
    v[-3:] = torch.randn((3, page, nkv, 128), generator=g, device=dev, dtype=BF16)
    small = Cache(dev, [300], nkv, page, BF16, cols=3)
    small.k, small.v = k, v
    small.table = torch.tensor([[npages - 1, npages - 3, npages - 2]], dtype=torch.int32, device=dev)
    q = queries(dev, 1, 32, BF16)
    out, lse = small.call(q)
    small.check(q, out, lse)


def test_refusals_of_the_binding(dev):
    c = Cache(dev, [20, 30], 2, 16, BF16)
    q = queries(dev, 2, 8, BF16)
    bad = [lambda: c.call(q.float()), lambda: c.call(q[:1]), lambda: c.call(q[:, :7]), lambda: c.call(q[..., :64]),
           lambda: c.call(q.cpu()), lambda: c.call(q, mass_out=torch.zeros((2, 99), device=dev)),
           lambda: c.call(q, mass=torch.zeros((2, 3), device=dev)), lambda: c.call(q, scratch=q),
           lambda: c.call(q, out=torch.empty((2, 8, 128), device=dev)), lambda: c.call(q[..., ::2]),
           lambda: qsa.paged_attn(q, c.k, c.v[:1], c.table, c.lens),
           lambda: qsa.paged_attn(q, c.k, c.v, c.table.long(), c.lens),
           lambda: qsa.paged_attn(q, c.k, c.v, c.table, c.lens[:1]),
           lambda: qsa.paged_attn(q, c.k, c.v, c.table, c.lens, k_scale_f16=c.k[..., 0], v_scale_f16=c.k[..., 0]),
           lambda: qsa.paged_attn(q, c.k.to(I8), c.v.to(I8), c.table, c.lens)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for kw in (dict(scale=0.0), dict(scale=math.nan), dict(sinks=-1)):
        with pytest.raises(qsa.QSAError):
            c.call(q, **kw)
