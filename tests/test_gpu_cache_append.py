"""cache_append on the GPU: every cell, query and key against the 64-bit rotation and the int8 form by IEEE steps."""
import math

import pytest
import torch

import sparse_attention_kv_qsa_gb300 as qsa
import token_ref

pytestmark = pytest.mark.gpu
BF16, F16, F32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8
KINDS = [(BF16, BF16), (F32, BF16), (F16, F16), (F32, F16), (F32, I8), (BF16, I8), (F16, I8)]   # rows, pages


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


class Batch:
    """New tokens of ragged sequences and the pool that takes them, filled with a mark."""

    def __init__(self, dev, new, context, nkv, group, page, rows, kv, layout="nhd", pairs=64, axes=1, seed=0, spare=2):
        g = torch.Generator(device=dev).manual_seed(seed)
        self.new, self.page, self.nkv, self.kv, self.dev = list(new), page, nkv, kv, dev
        self.length = [a + b for a, b in zip(new, context)]
        nseq, ntok, heads = len(new), sum(new), nkv * group
        self.cols = max(-(-n // page) for n in self.length + [1])
        npages = nseq * self.cols + spare
        shape = {"nhd": (npages, page, nkv, 128), "hnd": (npages, nkv, page, 128), "joint": (npages, 2, page, nkv, 128)}[layout]
        mark = lambda s: torch.full(s, 5, device=dev).to(kv)  # noqa: E731
        if layout == "joint":
            self.k, self.v = mark(shape).unbind(1)
        else:
            self.k, self.v = mark(shape), mark(shape)
            if layout == "hnd":
                self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        self.ks = self.vs = None
        if kv == I8:
            self.ks, self.vs = (torch.full((npages, nkv, page), 3.0, device=dev, dtype=F16).transpose(1, 2) for _ in range(2))
        self.table = torch.randperm(npages, generator=g, device=dev).to(torch.int32)[:nseq * self.cols].view(nseq, self.cols)
        self.lens = torch.tensor(self.length, dtype=torch.int32, device=dev)
        self.cu = torch.tensor([sum(self.new[:i]) for i in range(nseq + 1)], dtype=torch.int32, device=dev)
        fused = torch.randn((ntok, heads + 2 * nkv, 128), generator=g, device=dev).to(rows)
        self.q, self.kx, self.vx = fused[:, :heads], fused[:, heads:heads + nkv], fused[:, heads + nkv:]
        self.freqs = torch.pow(torch.tensor(10000.0, dtype=torch.float64), -torch.arange(pairs) / pairs).float().to(dev)
        self.positions = torch.randint(0, 9000, (axes, ntok), generator=g, device=dev, dtype=torch.int32)
        self.axis = (torch.arange(pairs, device=dev) % axes).to(torch.int32) if axes > 1 else None

    def cells(self):
        """Sequence and cell of every token."""
        seq = [s for s, n in enumerate(self.new) for _ in range(n)]
        cell = [self.length[s] - n + i for s, n in enumerate(self.new) for i in range(n)]
        return torch.tensor(seq, device=self.dev, dtype=torch.long), torch.tensor(cell, device=self.dev, dtype=torch.long)

    def call(self, **kw):
        d = dict(cu=self.cu, k_scale_f16=self.ks, v_scale_f16=self.vs, q=self.q, positions=self.positions, freqs=self.freqs,
                 axis=self.axis)
        d.update(kw)
        return qsa.cache_append(self.kx, self.vx, self.k, self.v, self.table, self.lens, **d)

    def check(self, q_out, k_out, positions="given", interleaved=False, wrote=None):
        """`wrote`: which tokens' cells were written (default all). Everything else of the pool keeps its mark."""
        seq, cell = self.cells()
        ntok = seq.numel()
        wrote = torch.ones(ntok, dtype=torch.bool, device=self.dev) if wrote is None else wrote
        pos = self.positions if positions == "given" else cell.to(torch.int32)
        axis = self.axis if positions == "given" else None
        pairs = self.freqs.numel()

        def near(got, x, dtype):
            want = token_ref.rotate(x, pos, self.freqs, axis, interleaved)
            tol = token_ref.rotate_tol(x, want, dtype, pairs, interleaved)
            err = (got.cpu().double() - want).abs()
            assert bool((err <= tol).all()), float((err - tol).max())
            return want, tol

        if q_out is not None:
            near(q_out, self.q, self.q.dtype)
        if k_out is not None:
            near(k_out, self.kx, self.kx.dtype)
        page, slot = self.table[seq, cell.clamp(0, self.cols * self.page - 1) // self.page].long()[wrote], (cell % self.page)[wrote]
        if self.kv == I8:
            codes, scale = token_ref.codes(self.vx[wrote])
            assert torch.equal(self.v[page, slot].cpu(), codes) and torch.equal(self.vs[page, slot].cpu(), scale)
            want = token_ref.rotate(self.kx, pos, self.freqs, axis, interleaved)
            tol = token_ref.rotate_tol(self.kx, want, F32, pairs, interleaved)[wrote.cpu()]
            want = want[wrote.cpu()]
            if k_out is not None and self.kx.dtype == F32:    # the very numbers that were made codes
                codes, scale = token_ref.codes(k_out[wrote])
                assert torch.equal(self.k[page, slot].cpu(), codes) and torch.equal(self.ks[page, slot].cpu(), scale)
            f = self.ks[page, slot].cpu().double()
            # the scale is max / 127 to half a step of binary16 (2^-11), or 2^-25 below its normal numbers
            amax = want.abs().amax(-1)
            assert bool(((f - amax / 127).abs() <= amax / 127 * (2.0 ** -11 + 2.0 ** -22) + tol.amax(-1) / 127 + 2.0 ** -25).all())
            got = self.k[page, slot].cpu().double() * f[..., None]
            # a code is off by half a step, and by up to 127 x 2^-11 of one where it was cut at 127
            assert bool(((got - want).abs() <= f[..., None] * (0.5 + 127 * 2.0 ** -11 + 2.0 ** -16) + tol).all())
        else:
            near_k = token_ref.rotate(self.kx, pos, self.freqs, axis, interleaved)
            tol = token_ref.rotate_tol(self.kx, near_k, self.kv, pairs, interleaved)
            assert bool(((self.k[page, slot].cpu().double() - near_k[wrote.cpu()]).abs() <= tol[wrote.cpu()]).all())
            assert torch.equal(self.v[page, slot], self.vx[wrote].to(self.kv))
        untouched = torch.ones(self.k.shape[:2], dtype=torch.bool, device=self.dev)
        untouched[page, slot] = False
        for t, mark in ((self.k, 5), (self.v, 5)) + (((self.ks, 3), (self.vs, 3)) if self.kv == I8 else ()):
            assert bool((t[untouched] == mark).all())


@pytest.mark.parametrize("layout", ["nhd", "hnd", "joint"])
@pytest.mark.parametrize("rows,kv", KINDS)
@pytest.mark.parametrize("new,context,nkv,group,page,pairs,axes",
                         [([1], [0], 1, 1, 16, 64, 1), ([1] * 7, [0, 5, 15, 16, 17, 100, 31], 8, 4, 16, 64, 1),
                          ([3, 0, 1, 40, 0, 0, 129, 2], [9, 4, 0, 7, 0, 77, 1, 30], 2, 3, 24, 48, 3),
                          ([700], [13], 1, 7, 7, 8, 2), ([1] * 300, [i % 50 for i in range(300)], 2, 1, 8, 32, 1),
                          ([5] * 130, [i % 3 for i in range(130)], 3, 5, 1, 64, 4)])
def test_ragged_batches(dev, new, context, nkv, group, page, pairs, axes, rows, kv, layout):
    b = Batch(dev, new, context, nkv, group, page, rows, kv, layout, pairs, axes)
    for interleaved in (False, True):
        k_out = torch.empty((sum(new), nkv, 128), device=dev, dtype=rows)
        b.check(*b.call(k_out=k_out, interleaved=interleaved), interleaved=interleaved)


@pytest.mark.parametrize("rows,kv", KINDS)
def test_positions_are_the_cells(dev, rows, kv):
    b = Batch(dev, [4, 1, 19], [30, 8000, 0], 2, 4, 16, rows, kv)
    b.check(*b.call(positions=None), positions="cells")


@pytest.mark.parametrize("rows,kv", KINDS)
def test_one_token_each_without_cu_and_without_queries(dev, rows, kv):
    b = Batch(dev, [1] * 5, [3, 0, 70, 16, 15], 4, 2, 16, rows, kv)
    q_out, k_out = b.call(cu=None, q=None)
    assert q_out is None and k_out is None
    b.check(None, None)


@pytest.mark.parametrize("rows,kv", KINDS)
def test_without_rotation(dev, rows, kv):
    """Keys as they are, odd values among them: copied bit for bit where the type is the same."""
    b = Batch(dev, [6, 2], [5, 0], 2, 1, 16, rows, kv)
    b.kx[0, 0, :3] = torch.tensor([math.inf, -math.inf, math.nan], device=dev).to(rows)
    b.kx[1, 1] = 0
    b.vx[2, 0] = 1e-6 * b.vx[2, 0]
    b.vx[3, 1, 7] = math.nan
    if rows == F32:
        b.vx[4, 0] = 1e30 * b.vx[4, 0]
        b.vx[5, 1] = 1e-42 * b.vx[5, 1]
        b.vx[7, 1] = 1e7 * b.vx[7, 1]       # a scale of binary16's largest numbers
    assert qsa.cache_append(b.kx, b.vx, b.k, b.v, b.table, b.lens, cu=b.cu, k_scale_f16=b.ks, v_scale_f16=b.vs) == (None, None)
    seq, cell = b.cells()
    page, slot = b.table[seq, cell // b.page].long(), cell % b.page
    for pool, scales, x in ((b.k, b.ks, b.kx), (b.v, b.vs, b.vx)):
        if kv == I8:
            codes, scale = token_ref.codes(x)
            assert torch.equal(pool[page, slot].cpu(), codes)
            assert torch.equal(scales[page, slot].cpu().nan_to_num(-1.0), scale.nan_to_num(-1.0))
        else:
            assert torch.equal(pool[page, slot].nan_to_num(-9.0, 8.0, -8.0), x.to(kv).nan_to_num(-9.0, 8.0, -8.0))


def test_tokens_of_no_sequence_and_cells_of_no_page(dev):
    b = Batch(dev, [2, 3, 4, 5], [10, 0, 20, 2], 2, 2, 16, BF16, BF16)
    whole, lengths = b.cu.clone(), list(b.length)
    seq, cell = b.cells()
    # sequence 2's second page is none, sequence 3 claims fewer cells than it has new tokens
    b.table[2, 1] = b.k.shape[0]
    b.lens[3] = 3
    b.length[3] = 3
    b.cu[-1] = 13                       # the last token is of no sequence; sequence 3 has 4 new tokens
    b.new[3] = 4
    q_out = torch.full((14, 4, 128), -3.0, device=dev, dtype=BF16)
    k_out = torch.full((14, 2, 128), -3.0, device=dev, dtype=BF16)
    b.call(q_out=q_out, k_out=k_out)
    assert bool((q_out[13] == -3).all()) and bool((k_out[13] == -3).all())
    b.q, b.kx, b.vx, b.positions = b.q[:13], b.kx[:13], b.vx[:13], b.positions[:, :13]
    wrote = torch.ones(13, dtype=torch.bool, device=dev)
    wrote[5:9] = False                  # cells 20 to 23 lie in that page
    wrote[9] = False                    # cell -1
    b.check(q_out[:13], k_out[:13], wrote=wrote)
    assert whole.tolist() == [0, 2, 5, 9, 14] and lengths == [12, 3, 24, 7]


@pytest.mark.parametrize("cu,lens", [([5, 9, 9], [2000, 3]), ([-3, 4, 100], [4, 6]), ([9, 3, 0], [5, 5]), ([0, 0, 0], [1, 1]),
                                     ([0, 5, 9], [-2 ** 31, 2 ** 31 - 1])])
def test_whatever_cu_and_lens_hold(dev, cu, lens):
    """Garbage in device memory: nothing but the batch's own cells is written."""
    b = Batch(dev, [5, 4], [40, 30], 2, 2, 16, BF16, BF16)
    b.cu.copy_(torch.tensor(cu, dtype=torch.int32))
    b.lens.copy_(torch.tensor(lens, dtype=torch.int32))
    b.call()
    torch.cuda.synchronize()
    untouched = torch.ones(b.k.shape[0], dtype=torch.bool, device=dev)
    untouched[b.table.long().flatten()] = False
    assert bool((b.k[untouched] == 5).all()) and bool((b.v[untouched] == 5).all())


def test_page_numbers_out_of_range(dev):
    for bad in (-1, -2 ** 31, 2 ** 31 - 1):
        b = Batch(dev, [3, 2], [0, 14], 2, 2, 16, F32, I8)
        b.table.fill_(bad)
        b.check(*b.call(), wrote=torch.zeros(5, dtype=torch.bool, device=dev))


def test_a_table_without_columns(dev):
    b = Batch(dev, [1, 1], [0, 3], 1, 2, 16, BF16, BF16)
    want, _ = b.call(cu=None)
    b2 = Batch(dev, [1, 1], [0, 3], 1, 2, 16, BF16, BF16)
    b2.table = torch.zeros((2, 0), dtype=torch.int32, device=dev)
    got, _ = b2.call(cu=None)
    assert torch.equal(got, want) and bool((b2.k == 5).all()) and bool((b2.v == 5).all())


def test_in_place(dev):
    b = Batch(dev, [9, 300], [0, 12], 2, 4, 16, BF16, BF16, axes=3)
    want_q, _ = b.call()
    want_k = b.k.clone()
    k_out = torch.empty_like(b.kx)
    b.call(k_out=k_out)
    b.call(q_out=b.q, k_out=b.kx)
    assert torch.equal(b.q, want_q) and torch.equal(b.kx, k_out) and torch.equal(b.k, want_k)


def test_no_tokens(dev):
    b = Batch(dev, [0, 0], [3, 3], 2, 4, 16, BF16, BF16)
    q_out, _ = b.call(positions=None)
    assert q_out.shape == (0, 8, 128) and bool((b.k == 5).all())
    none = torch.zeros((0, 2, 128), device=dev, dtype=BF16)
    assert qsa.cache_append(none, none, b.k, b.v, b.table[:0], b.lens[:0]) == (None, None)


def test_past_32_bit_offsets(dev):
    """Pages whose elements lie past 2^31."""
    npages = 2 ** 31 // (16 * 2 * 128) + 3
    k, v = (torch.zeros((npages, 16, 2, 128), device=dev, dtype=BF16) for _ in range(2))
    x = torch.randn((2, 2, 128), device=dev).to(BF16)
    table = torch.tensor([[npages - 1], [0]], dtype=torch.int32, device=dev)
    lens = torch.tensor([5, 16], dtype=torch.int32, device=dev)
    qsa.cache_append(x, -x, k, v, table, lens)
    assert torch.equal(k[npages - 1, 4], x[0]) and torch.equal(v[npages - 1, 4], -x[0]) and torch.equal(k[0, 15], x[1])
    assert int(torch.count_nonzero(k.view(npages, -1).any(1))) == 2


def test_captured_and_on_another_stream(dev):
    """A captured call follows lengths, tables and positions in place."""
    b = Batch(dev, [1] * 6, [3, 9, 0, 15, 31, 40], 2, 4, 16, BF16, I8)
    q_out = torch.empty_like(b.q, memory_format=torch.contiguous_format)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        got, _ = b.call(cu=None)
    torch.cuda.current_stream(dev).wait_stream(side)
    b.check(got, None)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.lens.add_(1)
        b.call(cu=None, q_out=q_out, positions=None)
    for t in (b.k, b.v):
        t.fill_(5)
    for t in (b.ks, b.vs):
        t.fill_(3)
    b.length = [n + 1 for n in b.length]
    g.replay()
    torch.cuda.synchronize()
    b.check(q_out, None, positions="cells")


def test_binding_refusals(dev):
    b = Batch(dev, [2, 3], [1, 1], 2, 2, 16, BF16, BF16)
    base = dict(kx=b.kx, vx=b.vx, k=b.k, v=b.v, table=b.table, lens=b.lens, cu=b.cu, q=b.q, positions=b.positions, freqs=b.freqs,
                axis=None, ks=None, vs=None, q_out=None, k_out=None)
    for bad in (dict(kx=b.kx.half()), dict(vx=b.vx.float()), dict(kx=b.kx[:, :1]), dict(vx=b.vx[:4]), dict(q=b.q.float()),
                dict(q=b.q[:4]), dict(freqs=None), dict(freqs=None, q=None, positions=None, k_out=torch.empty_like(b.kx)),
                dict(freqs=None, q=None), dict(cu=b.cu[:2]), dict(cu=None), dict(cu=b.cu.long()), dict(lens=b.lens[:1]),
                dict(table=b.table.long()), dict(ks=b.freqs), dict(positions=None, axis=torch.zeros(64, dtype=torch.int32, device=dev)),
                dict(q=None, q_out=torch.empty_like(b.q)), dict(q_out=torch.empty_like(b.q).float()), dict(k=b.k.cpu()),
                dict(lens=b.lens.cpu())):
        d = dict(base, **bad)
        with pytest.raises(ValueError):
            qsa.cache_append(d["kx"], d["vx"], d["k"], d["v"], d["table"], d["lens"], cu=d["cu"], k_scale_f16=d["ks"],
                             v_scale_f16=d["vs"], q=d["q"], positions=d["positions"], freqs=d["freqs"], axis=d["axis"],
                             q_out=d["q_out"], k_out=d["k_out"])
    one = b.k[:1].expand(b.k.shape)
    with pytest.raises(qsa.QSAError):                       # pages that are all one page
        qsa.cache_append(b.kx, b.vx, one, one, b.table, b.lens, cu=b.cu)
    assert bool((b.k == 5).all()) and bool((b.v == 5).all())


@pytest.mark.parametrize("rows,kv", KINDS)
def test_one_pool_for_keys_and_values(dev, rows, kv):
    """Without a rotation the same rows may go to the same pages as keys and as values."""
    b, one = (Batch(dev, [3, 1, 40], [5, 0, 9], 2, 1, 16, rows, kv) for _ in range(2))
    qsa.cache_append(b.kx, b.kx, b.k, b.v, b.table, b.lens, cu=b.cu, k_scale_f16=b.ks, v_scale_f16=b.vs)
    qsa.cache_append(b.kx, b.kx, one.k, one.k, b.table, b.lens, cu=b.cu, k_scale_f16=one.ks, v_scale_f16=one.ks)
    assert torch.equal(b.k, b.v) and torch.equal(one.k, b.k)
    if kv == I8:
        assert torch.equal(one.ks, b.ks) and torch.equal(b.ks, b.vs)
    with pytest.raises(qsa.QSAError):
        qsa.cache_append(b.kx, b.vx, one.k, one.k, b.table, b.lens, cu=b.cu, k_scale_f16=one.ks, v_scale_f16=one.ks)
    with pytest.raises(qsa.QSAError):
        qsa.cache_append(b.kx, b.kx, one.k, one.k, b.table, b.lens, cu=b.cu, k_scale_f16=one.ks, v_scale_f16=one.ks, freqs=b.freqs)
