"""qsa_prefix_attn (one new token per sequence, groups of which share a prefix) against the plain 64-bit form over the
prefix's cells and the sequence's own. Tolerances: cache_ref.bounds; weights of prefix cells are rounded once to the
operand type (bfloat16 or binary16), or keep 22 bits for fp32 queries.

Binary16 weights below its normal numbers are off by up to 2^-25, half its smallest step. Prefix weights (value scale
included) are held so that a row's largest is at least 2^7, so that is 2^-32 of the largest (the remainders that fp32
queries keep too); weights of own cells keep a remainder times 2^11 and reach at least 1: 2^-36. For n cells a column is off by
n times that, times the largest weight, scale and |code|; with codes of up to 128 whose largest in a cell is at least 64 that
is at most twice the largest p_j |v_jd| of any column, which the largest column's sum of |p v| bounds. It counts in a column
where the cell that has nearly all the weight has a value of 0: relative to that column's own sum it is not small."""
import math

import pytest
import torch

import cache_ref as ref
import sparse_attention_kv_qsa_gb300 as qsa

pytestmark = pytest.mark.gpu
BF16, F16, F32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8
KINDS = [(BF16, BF16), (F16, F16), (I8, F32), (I8, BF16), (I8, F16)]   # pages, queries


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


class Shared:
    """Groups of sequences (members, prefix length) over a pool whose pages stand in a random order; everything that no
    sequence sees holds NaN (int8 cells: their scales), and table entries past a length are no page's."""

    def __init__(self, dev, groups, lens, nkv, group, page, kv, qt, layout="nhd", seed=0, before=0):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.groups, self.lens_list, self.page, self.nkv, self.group, self.kv, self.dev = groups, list(lens), page, nkv, group, kv, dev
        nseq = len(lens)
        need = [-(-max(n, 0) // page) for _, n in groups] + [-(-max(n, 0) // page) for n in lens]
        npages = sum(need) + 3
        shape = {"nhd": (npages, page, nkv, 128), "hnd": (npages, nkv, page, 128), "joint": (npages, 2, page, nkv, 128)}[layout]

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
        ng = len(groups)
        self.ptable = torch.full((ng, max(need[:ng] + [0]) + 1), 2 ** 31 - 1, dtype=torch.int32, device=dev)
        self.table = torch.full((nseq, max(need[ng:] + [0]) + 1), -7, dtype=torch.int32, device=dev)
        at = 0
        for i, c in enumerate(need):
            (self.ptable[i] if i < ng else self.table[i - ng])[:c] = order[at:at + c]
            at += c
        self.plens = torch.tensor([n for _, n in groups], dtype=torch.int32, device=dev)
        self.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        starts = [before]
        for m, _ in groups:
            starts.append(starts[-1] + m)
        self.starts = starts
        self.cu = torch.tensor(starts, dtype=torch.int32, device=dev)
        self.q = torch.randn((nseq, nkv * group, 128), generator=g, device=dev).to(qt)
        used = torch.zeros(self.k.shape[:2], dtype=torch.bool, device=dev)
        for row, n in [(self.ptable[i], n) for i, (_, n) in enumerate(groups)] + [(self.table[i], n) for i, n in enumerate(lens)]:
            j = torch.arange(max(n, 0), device=dev)
            used[row[j // page].long(), j % page] = True
        for t in (self.k, self.v) if kv != I8 else (self.ks, self.vs):
            t[~used] = math.nan

    def call(self, **kw):
        return qsa.prefix_attn(self.q, self.k, self.v, self.ptable, self.plens, self.cu, self.table, self.lens,
                               k_scale_f16=self.ks, v_scale_f16=self.vs, **kw)

    def check(self, out, lse, scale=128 ** -0.5, only=None):
        qt, grp = self.q.dtype, self.group
        p_half = 2.0 ** -22 if qt == F32 else ref.half_step(BF16 if self.kv == BF16 else F16)
        assert out.dtype == qt and out.shape == self.q.shape
        cells = lambda pages, sc, row, n, h: ref.paged_cells(pages, sc, row, n, h, self.page)  # noqa: E731
        group_of = {s: g for g in range(len(self.groups)) for s in range(self.starts[g], self.starts[g + 1])}
        for h in range(self.nkv):
            prefix = {}
            for s in range(len(self.lens_list)) if only is None else only:
                g = group_of.get(s)
                if g is not None and g not in prefix:
                    n = max(0, min(self.groups[g][1], self.ptable.shape[1] * self.page))
                    prefix = {g: (cells(self.k, self.ks, self.ptable[g], n, h), cells(self.v, self.vs, self.ptable[g], n, h))}
                n = max(0, min(self.lens_list[s], self.table.shape[1] * self.page))
                (k, ok), (v, _) = cells(self.k, self.ks, self.table[s], n, h), cells(self.v, self.vs, self.table[s], n, h)
                if g is not None:
                    (pk, pok), (pv, _) = prefix[g]
                    k, v, ok = torch.cat((pk, k)), torch.cat((pv, v)), torch.cat((pok, ok))
                o, l, _, size, S = ref.attend(self.q[s, h * grp:(h + 1) * grp][:, None], k, v, ok[None], scale)
                tol, ltol = ref.bounds(o, l, size, S, k.shape[0], qt, p_half)
                if self.kv != BF16 and k.shape[0] > 0:
                    tol = tol + 2 * k.shape[0] * 2.0 ** -32 * size.amax(-1, keepdim=True)
                for name, got, want, t in (("out", out, o, tol), ("lse", lse, l, ltol)):
                    got = got[s, h * grp:(h + 1) * grp]
                    if bool(torch.isnan(want).all()):        # the formula's own NaN
                        assert torch.isnan(got).all(), (name, s, h)
                    else:
                        ref.check(got, want[:, 0], t[:, 0], (name, s, h))


def lens_of(n, most=70, seed=0):
    return [(7919 * (i + 1 + seed)) % (most + 1) for i in range(n)]


@pytest.mark.parametrize("kv,qt", KINDS)
@pytest.mark.parametrize("groups,nkv,group,page",
                         [([(1, 1)], 1, 1, 16), ([(3, 129)], 2, 4, 16), ([(5, 128), (1, 127), (2, 300)], 1, 8, 48),
                          ([(31, 500), (33, 40), (64, 257), (65, 1000)], 2, 4, 16), ([(20, 385)], 3, 7, 7),
                          ([(9, 2000)], 1, 16, 128), ([(130, 777)], 1, 2, 1), ([(4, 0), (2, 50), (3, 0), (7, 640)], 2, 5, 32)])
def test_against_the_formula(dev, groups, nkv, group, page, kv, qt):
    b = Shared(dev, groups, lens_of(sum(m for m, _ in groups)), nkv, group, page, kv, qt)
    b.check(*b.call())


@pytest.mark.parametrize("layout", ["hnd", "joint"])
@pytest.mark.parametrize("kv,qt", KINDS)
def test_layouts(dev, kv, qt, layout):
    b = Shared(dev, [(6, 450), (40, 200)], lens_of(46), 2, 4, 16, kv, qt, layout)
    b.check(*b.call())


@pytest.mark.parametrize("kv,qt", KINDS)
def test_long_prefix_split_over_all_ctas(dev, kv, qt):
    b = Shared(dev, [(7, 40000)], lens_of(7, 300), 2, 4, 16, kv, qt)
    b.check(*b.call())


@pytest.mark.parametrize("kv,qt", KINDS)
def test_many_rows(dev, kv, qt):
    """More rows than two tiles: several blocks of a group."""
    b = Shared(dev, [(150, 3000)], lens_of(150, 40), 1, 8, 32, kv, qt)
    b.check(*b.call(), only=list(range(0, 150, 7)) + [149])


@pytest.mark.parametrize("kv,qt", KINDS)
def test_many_small_groups(dev, kv, qt):
    groups = [(1 + i % 3, (i * 37) % 300) for i in range(250)]
    b = Shared(dev, groups, lens_of(sum(m for m, _ in groups), 20), 4, 2, 16, kv, qt)
    b.check(*b.call())


@pytest.mark.parametrize("kv,qt", KINDS)
def test_rows_without_a_cell_and_without_a_group(dev, kv, qt):
    """Sequences before the first group and behind the last have no prefix; some have nothing at all."""
    lens = [0, 5, 0, 0, 9, 0, 3, 0]
    b = Shared(dev, [(2, 0), (2, 140)], lens, 2, 3, 16, kv, qt, before=2)
    out, lse = b.call(out=torch.full_like(b.q, math.nan))
    b.check(out, lse)
    for s in (0, 2, 3, 7):
        assert torch.count_nonzero(out[s]) == 0 and bool((lse[s] == -math.inf).all())


@pytest.mark.parametrize("kv,qt", KINDS)
def test_no_groups_and_no_columns(dev, kv, qt):
    b = Shared(dev, [(3, 60)], [10, 0, 70], 2, 4, 16, kv, qt)
    b.groups, b.starts = [], [0]
    b.ptable, b.plens, b.cu = b.ptable[:0], b.plens[:0], b.cu[:1]
    b.check(*b.call())
    b = Shared(dev, [(3, 60)], [10, 0, 70], 2, 4, 16, kv, qt)
    b.table, b.lens_list = b.table[:, :0], [0, 0, 0]
    b.check(*b.call())
    b.ptable, b.groups = b.ptable[:, :0], [(3, 0)]
    out, lse = b.call()
    assert torch.count_nonzero(out) == 0 and bool((lse == -math.inf).all())


@pytest.mark.parametrize("prefix,own", [(100, 20), (96, 16)])   # the first: cells of NaN between the length and the page's end
@pytest.mark.parametrize("kv,qt", KINDS)
def test_lengths_and_pages_out_of_range(dev, kv, qt, prefix, own):
    b = Shared(dev, [(2, prefix), (2, 90), (1, 33)], [own, 3, 40, 8, 5], 2, 4, 16, kv, qt)
    b.plens[0], b.lens[0] = 2 ** 31 - 1, 2 ** 31 - 1          # the tables' capacity; what lies past the pages is none
    b.groups[0], b.lens_list[0] = (2, 2 ** 31 - 1), 2 ** 31 - 1
    b.plens[2], b.lens[4] = -5, -1
    b.groups[2], b.lens_list[4] = (1, 0), 0
    b.ptable[1, 2], b.table[2, 1] = -1, b.k.shape[0]          # holes
    b.check(*b.call())


@pytest.mark.parametrize("cu", [[5, 2, 3], [-9, 4, 99], [0, 5, 1], [2 ** 31 - 1, -2 ** 31, 0]])
def test_whatever_cu_holds(dev, cu):
    """Garbage in device memory: the call ends, and writes its own results alone."""
    b = Shared(dev, [(2, 500), (3, 700)], lens_of(5), 2, 4, 16, BF16, BF16)
    b.cu.copy_(torch.tensor(cu))
    need = qsa.prefix_attn_scratch_bytes(5, 2, 8, 2, b.ptable.shape[1], b.table.shape[1], 16)
    room = torch.full((need + 4096,), 77, dtype=torch.uint8, device=dev)
    b.call(scratch=room[:need])
    torch.cuda.synchronize()
    assert bool((room[need:] == 77).all()) and qsa.device_error(dev) == 0


@pytest.mark.parametrize("kv,qt", KINDS)
def test_same_every_time_and_whatever_scratch_holds(dev, kv, qt):
    b = Shared(dev, [(40, 3000), (3, 10)], lens_of(43, 200), 2, 4, 16, kv, qt)
    need = qsa.prefix_attn_scratch_bytes(43, 2, 8, 2, b.ptable.shape[1], b.table.shape[1], 16)
    want = b.call()
    for fill in (0x00, 0xFF, 0x7F):
        got = b.call(scratch=torch.full((need,), fill, dtype=torch.uint8, device=dev))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kv,qt", KINDS)
def test_strided_queries_given_outputs_and_scale(dev, kv, qt):
    b = Shared(dev, [(9, 300)], lens_of(9), 2, 4, 16, kv, qt)
    wide = torch.zeros((9, 12, 128), device=dev, dtype=qt)
    wide[:, 2:10] = b.q
    b.q = wide[:, 2:10]
    out, lse = torch.empty((9, 8, 128), device=dev, dtype=qt), torch.empty((9, 8), device=dev)
    got = b.call(out=out, lse=lse, scale=0.31)
    assert got[0].data_ptr() == out.data_ptr() and got[1].data_ptr() == lse.data_ptr()
    b.check(out, lse, scale=0.31)


@pytest.mark.parametrize("kv,qt", KINDS)
def test_peaked_and_growing_logits(dev, kv, qt):
    """Maxima that grow along the prefix move the reference again and again; large queries make it one cell's."""
    b = Shared(dev, [(40, 2500)], lens_of(40, 50), 1, 4, 16, kv, qt)
    grow = torch.linspace(0.01, 6.0, 2500, device=dev)
    j = torch.arange(2500, device=dev)
    at = (b.ptable[0, j // 16].long(), j % 16)
    if kv == I8:
        b.ks[at] = (b.ks[at].float() * grow[:, None]).to(F16)
    else:
        b.k[at] = (b.k[at].float() * grow[:, None, None]).to(kv)
    b.check(*b.call())
    b.q = b.q * 8
    b.check(*b.call())


@pytest.mark.parametrize("qt", [F32, BF16, F16])
def test_scales_of_the_whole_range(dev, qt):
    """int8 value scales from binary16's smallest to its largest, and key scales of 0."""
    b = Shared(dev, [(5, 600)], lens_of(5), 2, 4, 16, I8, qt)
    g = torch.Generator(device=dev).manual_seed(5)
    fine = ~torch.isnan(b.vs.float())
    b.vs.copy_(torch.where(fine, torch.exp2(torch.rand(b.vs.shape, generator=g, device=dev) * 39 - 24).to(F16), b.vs))
    b.ks[b.ptable[0, 3].long()] = 0
    b.check(*b.call(scale=0.02), scale=0.02)


@pytest.mark.parametrize("qmul,scale", [(1e36, 1e-37), (1e-36, 1e35)])
def test_queries_of_the_whole_range_over_int8_cells(dev, qmul, scale):
    b = Shared(dev, [(5, 600), (30, 300)], lens_of(35), 2, 4, 16, I8, F32)
    b.q = b.q.clamp(-4, 4) * qmul
    b.check(*b.call(scale=scale), scale=scale)


@pytest.mark.parametrize("qt,qmul,scale", [(F32, 1e-13, 1e-30), (F32, 1.0, 1e-42), (BF16, 1.0, 1e-42), (F16, 1e-3, 1e-42), (F32, 0.0, 1e-42)])
def test_small_queries_and_scales_over_int8_cells(dev, qt, qmul, scale):
    """Logits that vanish: the mean of the cells that are there, beside absent ones (a tile's end, a hole)."""
    b = Shared(dev, [(5, 600), (3, 128), (30, 300), (2, 1)], lens_of(40), 2, 4, 16, I8, qt)
    b.ptable[0, 4] = -1
    b.q = b.q * qmul
    b.check(*b.call(scale=scale), scale=scale)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("kv,qt", [(BF16, BF16), (F16, F16)])
def test_odd_values_reach_who_sees_them_alone(dev, kv, qt, bad):
    """One group's prefix has an infinity or NaN in column 5 of its values; another group, the other KV head and the other
    columns stay as they were, and so does lse."""
    b = Shared(dev, [(6, 300), (4, 200)], lens_of(10), 2, 4, 16, kv, qt)
    out, lse = b.call()
    b.v[b.ptable[0, 4].long(), 3, 0, 5] = bad
    odd, odd_lse = b.call()
    assert torch.equal(odd_lse, lse) and not torch.isfinite(odd[:6, :4, 5]).any()
    keep = [c for c in range(128) if c != 5]
    assert torch.equal(odd[6:], out[6:]) and torch.equal(odd[:, 4:], out[:, 4:]) and torch.equal(odd[..., keep], out[..., keep])


@pytest.mark.parametrize("kv,qt", KINDS)
def test_odd_queries_spoil_their_own_row(dev, kv, qt):
    b = Shared(dev, [(40, 300)], lens_of(40), 2, 4, 16, kv, qt)
    out, lse = b.call()
    b.q[7, 2, 9] = math.nan
    odd, odd_lse = b.call()
    assert torch.isnan(odd[7, 2]).all() and torch.isnan(odd_lse[7, 2])
    same = torch.ones((40, 8), dtype=torch.bool, device=dev)
    same[7, 2] = False
    assert torch.equal(odd[same], out[same]) and torch.equal(odd_lse[same], lse[same])


def test_streams_and_graphs(dev):
    """A captured call follows lengths, groups and tables in place; two graphs on one scratch, one after the other."""
    b = Shared(dev, [(20, 900), (14, 300)], [30] * 34, 2, 4, 16, BF16, BF16)
    want = b.call()
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        got = b.call()
    torch.cuda.current_stream(dev).wait_stream(side)
    assert torch.equal(got[0], want[0])
    need = qsa.prefix_attn_scratch_bytes(34, 2, 8, 2, b.ptable.shape[1], b.table.shape[1], 16)
    scratch = torch.empty((need,), dtype=torch.uint8, device=dev)
    outs = [(torch.zeros_like(b.q), torch.zeros((34, 8), device=dev)) for _ in range(2)]
    graphs = []
    for o, l in outs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.call(out=o, lse=l, scratch=scratch)
            b.call(out=o, lse=l, scratch=scratch)
        graphs.append(g)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for o, l in outs:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    b.plens.copy_(torch.tensor([200, 299]))
    b.lens.fill_(17)
    b.cu[1] = 9
    b.groups, b.starts, b.lens_list = [(9, 200), (25, 299)], [0, 9, 34], [17] * 34
    graphs[0].replay()
    graphs[1].replay()
    torch.cuda.synchronize()
    for o, l in outs:
        b.check(o, l)


def test_as_paged_attention_over_both(dev):
    """The same cells in one table: paged_attn's results."""
    b = Shared(dev, [(8, 512)], [16] * 8, 2, 4, 16, BF16, BF16)
    out, lse = b.call()
    table = torch.cat((b.ptable[:, :32].expand(8, 32), b.table[:, :1]), 1).contiguous()
    want, want_lse = qsa.paged_attn(b.q, b.k, b.v, table, b.lens + 512)
    # two forms: weights rounded (2^-8) in one, results in both
    assert float((out.float() - want.float()).abs().max()) <= 3 * 2.0 ** -8 * float(b.v.nan_to_num().abs().max())
    assert float((lse - want_lse).abs().max()) <= 2 * (512 * ref.U * 128 ** 0.5 * 4 + 800 * ref.U)


def test_past_32_bit_offsets(dev):
    npages = 2 ** 31 // (16 * 128) + 40
    b = Shared(dev, [(3, 200)], [20, 1, 0], 1, 4, 16, BF16, BF16)
    k, v = (torch.zeros((npages, 16, 1, 128), device=dev, dtype=BF16) for _ in range(2))
    n = b.k.shape[0]
    k[-n:], v[-n:] = b.k, b.v
    want = b.call()
    b.k, b.v = k, v
    b.ptable = torch.where(b.ptable < n, b.ptable + npages - n, b.ptable)
    b.table = torch.where(b.table >= 0, b.table + npages - n, b.table)
    got = b.call()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("nseq", [3, 40])
def test_more_than_65536_tiles_a_cta(dev, nseq):
    """The longest prefix, 2^30 cells, of which all pages are one: every wait of 110,000 tiles a CTA has its turn.
    Keys of zeros weigh every cell 1, and values are -1, 0 or 1: a CTA's sums are integers below 110,400 x 128 < 2^24,
    so exact. Joining rounds to 2^-24 some 80 times (5e-6, a share of lse's 20.8 2e-6): far from half a step of
    bfloat16 beside the mean of 128 such values, which it holds exactly."""
    g = torch.Generator(device=dev).manual_seed(0)
    k = torch.zeros((1, 128, 2, 128), device=dev, dtype=BF16)
    v = torch.randint(-1, 2, k.shape, generator=g, device=dev).to(BF16)
    q = torch.randn((nseq, 8, 128), generator=g, device=dev, dtype=BF16)
    table = torch.zeros((1, 2 ** 23), dtype=torch.int32, device=dev)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    own, none = torch.zeros((nseq, 0), dtype=torch.int32, device=dev), torch.zeros(nseq, dtype=torch.int32, device=dev)
    out, lse = qsa.prefix_attn(q, k, v, table, ints(2 ** 30), ints(0, nseq), own, none)
    assert qsa.device_error(dev) == 0
    want = v[0].float().mean(0).to(BF16).repeat_interleave(4, 0)
    assert torch.equal(out, want.expand_as(out))
    assert float((lse - 30 * math.log(2)).abs().max()) <= 2e-5


@pytest.mark.parametrize("kv,qt", KINDS)
@pytest.mark.parametrize("members", [1, 3])
def test_long_sums(dev, members, kv, qt):
    """152 groups of 2^18 cells, so that a CTA holds all of one: 32 times the same 8,192, pages in an order of their own
    each time, whose values lie around 1. Tensor cores cut a sum off, by 2^-23 of it at every step of 16 cells: always
    towards zero, so that all results are off alike. The mean of their errors is bounded by 2^-23 of the sums of |p v| for
    each step of 256 tiles (fp32 queries: 32, with two steps), and 2^-23 for each part that is added."""
    groups, n, pages = 152, 2 ** 18, 64
    g = torch.Generator(device=dev).manual_seed(members)
    k, v = (torch.randn((pages, 128, 1, 128), generator=g, device=dev) for _ in range(2))
    v += 1
    ks = vs = None
    if kv == I8:
        ks, vs = ((x.abs().amax(-1) / 127).to(F16) for x in (k, v))
        k, v = ((x / sc.float()[..., None]).round().clamp(-127, 127) for x, sc in ((k, ks), (v, vs)))
    k, v = k.to(kv), v.to(kv)
    q = (4 * torch.randn((groups * members, 64, 128), generator=g, device=dev)).to(qt)
    table = torch.rand((groups, n // (128 * pages), pages), generator=g, device=dev).argsort(-1).to(torch.int32).reshape(groups, -1)
    own, none = torch.zeros((len(q), 0), dtype=torch.int32, device=dev), torch.zeros(len(q), dtype=torch.int32, device=dev)
    cu = torch.arange(0, len(q) + 1, members, dtype=torch.int32, device=dev)
    lens = torch.full((groups,), n, dtype=torch.int32, device=dev)
    out, lse = qsa.prefix_attn(q, k, v, table, lens, cu, own, none, k_scale_f16=ks, v_scale_f16=vs)
    assert qsa.device_error(dev) == 0
    (kd, seen), (vd, _) = (ref.paged_cells(x, sc, torch.arange(pages, device=dev), 128 * pages, 0, 128) for x, sc in ((k, ks), (v, vs)))
    chain = 32 if qt == F32 else 256
    steps, parts = chain * (16 if qt == F32 else 8), n // 128 // chain
    p_half = 2.0 ** -22 if qt == F32 else ref.half_step(BF16 if kv == BF16 else F16)
    off = total = 0.0
    for s in range(0, len(q), 76):
        o, l, _, size, S = ref.attend(q[s:s + 76].reshape(1, -1, 128), kd, vd, seen[None], 128 ** -0.5)
        tol, ltol = ref.bounds(o, l, size, S, 128 * chain + parts, qt, p_half)
        tol = tol + 2 * 128 * pages * 2.0 ** -32 * size.amax(-1, keepdim=True)
        got = out[s:s + 76].reshape(1, -1, 128)
        ref.check(got, o, tol, ("out", s))
        ref.check(lse[s:s + 76].reshape(1, -1), l + math.log(n // (128 * pages)), ltol + 2.0 ** -20, ("lse", s))
        off, total = off + float((got.double() - o).sum()), total + float(size.sum())
    assert abs(off) <= (steps + parts) * 2.0 ** -23 * total


def repeated(dev, qt, kv, lens, members, spread, seed):
    """Groups of `members` sequences of 64 heads, whose prefixes are the same 8,192 cells of one KV head, `lens` times, pages
    in an order of their own each time; values lie around 1. Returns the calls' results and the plain form's inputs."""
    pages = 64
    g = torch.Generator(device=dev).manual_seed(seed)
    k, v = (torch.randn((pages, 128, 1, 128), generator=g, device=dev) for _ in range(2))
    v += 1
    ks = vs = None
    if kv == I8:
        ks, vs = ((x.abs().amax(-1) / 127).to(F16) for x in (k, v))
        k, v = ((x / sc.float()[..., None]).round().clamp(-127, 127) for x, sc in ((k, ks), (v, vs)))
    k, v = k.to(kv), v.to(kv)
    q = (spread * torch.randn((sum(members), 64, 128), generator=g, device=dev)).to(qt)
    table = torch.rand((len(lens), max(lens), pages), generator=g, device=dev).argsort(-1).to(torch.int32).reshape(len(lens), -1)
    own, none = torch.zeros((len(q), 0), dtype=torch.int32, device=dev), torch.zeros(len(q), dtype=torch.int32, device=dev)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    cu = ints([sum(members[:i]) for i in range(len(members) + 1)])
    out, lse = qsa.prefix_attn(q, k, v, table, ints([128 * pages * n for n in lens]), cu, own, none, k_scale_f16=ks, v_scale_f16=vs)
    assert qsa.device_error(dev) == 0
    (kd, seen), (vd, _) = (ref.paged_cells(x, sc, torch.arange(pages, device=dev), 128 * pages, 0, 128) for x, sc in ((k, ks), (v, vs)))
    return q, out, lse, kd, vd, seen


@pytest.mark.parametrize("kv,qt", KINDS)
@pytest.mark.parametrize("lens,members", [([300, 700, 123, 511, 402], [3, 1, 4, 2, 1]), ([7, 5, 9, 3, 8, 6, 7], [1, 1, 2, 1, 5, 1, 1])])
def test_long_sums_of_several_blocks(dev, lens, members, kv, qt):
    """Ranges of some 860 tiles a CTA, and of 19 (of a row tile; fp32 queries' blocks are more): of two blocks, mostly, with
    sums that end in each of them and go on. Sums of at most 256 tiles (2 for fp32 queries), and as many parts as there are."""
    q, out, lse, kd, vd, seen = repeated(dev, qt, kv, lens, members, 4, 5)
    p_half = 2.0 ** -22 if qt == F32 else ref.half_step(BF16 if kv == BF16 else F16)
    s = 0
    for n, m in zip(lens, members):
        o, l, _, size, S = ref.attend(q[s:s + m].reshape(1, -1, 128), kd, vd, seen[None], 128 ** -0.5)
        chain = 2 if qt == F32 else 256
        tol, ltol = ref.bounds(o, l, size, S, 128 * chain + 64 * n // chain + 152, qt, p_half)
        tol = tol + 2 * 8192 * 2.0 ** -32 * size.amax(-1, keepdim=True)
        ref.check(out[s:s + m].reshape(1, -1, 128), o, tol, ("out", s))
        ref.check(lse[s:s + m].reshape(1, -1), l + math.log(n), ltol + 2.0 ** -20, ("lse", s))
        s += m


def test_sums_of_fp32_queries_end_early(dev):
    """A CTA has 64 tiles of one text here, 32 for either stream, and adds up weights that are nearly equal with values around
    1, so that sums grow evenly. Tensor cores cut them off at each of 16 steps a tile, by less than 2^-23 of the sum so far: over
    the 32 steps of 2 tiles less than 16.5 x 2^-23 of the sum at the end, 17 as growth is not quite even. Putting 16 such sums
    together, and the streams, rounds by 2^-24 some 16 times, to either side. (Sums of 16 tiles, 256 steps: 128.5 x 2^-23 at most,
    and 39 when they were so.)"""
    q, out, _, kd, vd, seen = repeated(dev, F32, I8, [1] * 152, [1] * 152, 0.25, 6)
    off = total = 0.0
    for s in range(0, 152, 19):
        o, _, _, size, _ = ref.attend(q[s:s + 19].reshape(1, -1, 128), kd, vd, seen[None], 128 ** -0.5)
        off, total = off + float((out[s:s + 19].reshape(1, -1, 128).double() - o).sum()), total + float(size.sum())
    assert abs(off) <= (17 + 8) * 2.0 ** -23 * total, off / total * 2 ** 23


def test_binding_refusals(dev):
    b = Shared(dev, [(2, 50), (2, 20)], [5, 5, 5, 5], 2, 4, 16, BF16, BF16)
    base = dict(q=b.q, k=b.k, v=b.v, pt=b.ptable, pl=b.plens, cu=b.cu, t=b.table, ln=b.lens, ks=None)
    for bad in (dict(q=b.q.half()), dict(q=b.q[:, :7]), dict(q=b.q[:3]), dict(q=b.q[..., :64]), dict(pt=b.ptable.long()),
                dict(pl=b.plens[:1]), dict(cu=b.cu[:2]), dict(cu=b.cu.long()), dict(t=b.table[:3]), dict(ln=b.lens[:3]),
                dict(ks=torch.ones(1, device=dev)), dict(v=b.v[:1]), dict(pt=b.ptable.cpu())):
        d = dict(base, **bad)
        with pytest.raises(ValueError):
            qsa.prefix_attn(d["q"], d["k"], d["v"], d["pt"], d["pl"], d["cu"], d["t"], d["ln"], k_scale_f16=d["ks"])
    with pytest.raises(ValueError):
        b.call(scratch=torch.empty(16, dtype=torch.uint8, device=dev))
    with pytest.raises(qsa.QSAError):
        b.call(scale=0.0)
