"""The bounded-cache operators refuse bad arguments before anything is
launched (CPU only: fake device addresses, no call here reaches a kernel),
and the 64-bit forms that the GPU tests compare with are right on cases that
can be written down by hand."""
import ctypes
import math

import pytest
import torch

import cache_ref
from sparse_attention_kv_qsa_gb300 import build as qsa_build
from sparse_attention_kv_qsa_gb300 import qsa

OK, INVALID, UNSUPPORTED = qsa.QSA_OK, qsa.QSA_ERR_INVALID, qsa.QSA_ERR_UNSUPPORTED
A, B, MIS = 0x10000, 0x20000, 0x20002     # fake addresses, the last aligned to 2 bytes only


@pytest.fixture(scope="module")
def lib():
    qsa_build.build()
    return qsa.lib()


def pages(**kw):
    d = dict(k=A, v=B, k_scale_f16=None, v_scale_f16=None, dtype=qsa.BF16, npages=100, page_size=16, nkv=2,
             page_stride=16 * 2 * 128, cell_stride=2 * 128, head_stride=128, scale_page_stride=0, scale_cell_stride=0,
             scale_head_stride=0)
    d.update(kw)
    return ctypes.byref(qsa.KVPages(**d))


BIG = 1 << 40


def paged(lib, kv=None, **kw):
    d = dict(q=A, q_dtype=qsa.BF16, qs=1024, qh=128, nseq=2, nheads=8, table=A, cols=4, tstride=4, lens=A, window=-1,
             sinks=0, scale=0.1, out=A, lse=A, mass=None, mass_out=None, mstride=0, scratch=A, bytes=BIG)
    d.update(kw)
    return lib.qsa_paged_attn(d["q"], d["q_dtype"], d["qs"], d["qh"], d["nseq"], d["nheads"], kv or pages(), d["table"],
                              d["cols"], d["tstride"], d["lens"], d["window"], d["sinks"], d["scale"], d["out"],
                              d["lse"], d["mass"], d["mass_out"], d["mstride"], d["scratch"], d["bytes"], None)


BAD_PAGES = [dict(dtype=qsa.F32), dict(dtype=7), dict(npages=-1), dict(page_size=0), dict(nkv=0), dict(k=None),
             dict(v=MIS), dict(page_stride=-4096), dict(cell_stride=129), dict(head_stride=4),
             dict(k_scale_f16=A, v_scale_f16=A),                       # scales beside 16-bit cells
             dict(dtype=qsa.I8), dict(dtype=qsa.I8, k_scale_f16=A, v_scale_f16=A + 1),
             dict(dtype=qsa.I8, k_scale_f16=A, v_scale_f16=A, head_stride=8),
             dict(dtype=qsa.I8, k_scale_f16=A, v_scale_f16=A, scale_cell_stride=-1)]


@pytest.mark.parametrize("bad", BAD_PAGES)
def test_bad_pages(lib, bad):
    assert paged(lib, pages(**bad)) == INVALID
    assert evict(lib, pages(**bad)) == INVALID


@pytest.mark.parametrize("bad", [dict(nseq=-1), dict(nheads=0), dict(nheads=7), dict(sinks=-1), dict(scale=0.0),
                                 dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(q_dtype=qsa.F32),
                                 dict(q_dtype=qsa.F16), dict(cols=-1), dict(tstride=3), dict(qs=-128), dict(qh=4),
                                 dict(q=None), dict(q=MIS), dict(out=None), dict(out=MIS), dict(lens=None),
                                 dict(table=None), dict(lse=MIS), dict(mass=A), dict(mass_out=A),
                                 dict(mass=A, mass_out=A, mstride=63), dict(mass=MIS, mass_out=A, mstride=64),
                                 dict(scratch=None), dict(scratch=A + 4), dict(bytes=0)])
def test_paged_attn_argument_errors(lib, bad):
    assert paged(lib, **bad) == INVALID


def test_paged_attn_limits(lib):
    assert paged(lib, nseq=0, q=None, out=None, lens=None, table=None, scratch=None, bytes=0) == OK
    assert paged(lib, nseq=65536) == UNSUPPORTED
    assert paged(lib, nheads=65536) == UNSUPPORTED
    assert paged(lib, nseq=65535, nheads=32768) == UNSUPPORTED
    assert paged(lib, cols=1 << 27, tstride=1 << 27) == UNSUPPORTED
    assert paged(lib, nseq=65535, nheads=16000, cols=1 << 20, tstride=1 << 20) == UNSUPPORTED
    assert paged(lib, pages(dtype=qsa.I8, k_scale_f16=A, v_scale_f16=A), q_dtype=qsa.I8) == INVALID
    n = qsa.paged_attn_scratch_bytes
    assert n(0, 8, 2, 4, 16) == 0 and n(2, 7, 2, 4, 16) == 0
    assert n(4, 32, 8, 64, 16, True) >= n(4, 32, 8, 64, 16) > 0


def window(lib, **kw):
    d = dict(q=A, k=A, v=A, dtype=qsa.BF16, strides=(1024, 128, 256, 128, 256, 128), cu_q=A, cu_k=A, nseq=2, total_q=50,
             total_k=60, max_q=40, nheads=8, nkv=2, window=-1, sinks=0, scale=0.1, out=A, lse=A, scratch=A, bytes=BIG)
    d.update(kw)
    st = None if d["strides"] is None else (ctypes.c_int64 * 6)(*d["strides"])
    return lib.qsa_window_attn(d["q"], d["k"], d["v"], d["dtype"], st, d["cu_q"], d["cu_k"], d["nseq"], d["total_q"],
                               d["total_k"], d["max_q"], d["nheads"], d["nkv"], d["window"], d["sinks"], d["scale"],
                               d["out"], d["lse"], d["scratch"], d["bytes"], None)


@pytest.mark.parametrize("bad", [dict(dtype=qsa.F32), dict(dtype=qsa.I8), dict(nseq=-1), dict(total_q=-1),
                                 dict(total_k=-1), dict(max_q=-1), dict(nheads=9), dict(nheads=0), dict(nkv=0),
                                 dict(sinks=-1), dict(scale=0.0), dict(scale=math.nan), dict(strides=None),
                                 dict(strides=(1024, 4, 256, 128, 256, 128)), dict(strides=(1024, 128, -256, 128, 256, 128)),
                                 dict(strides=(1024, 128, 256, 128, 256, 129)), dict(q=None), dict(k=MIS), dict(v=None),
                                 dict(cu_q=None), dict(cu_k=MIS), dict(out=MIS), dict(lse=MIS)])
def test_window_attn_argument_errors(lib, bad):
    assert window(lib, **bad) == INVALID


def test_window_attn_scratch_stays_bounded(lib):
    """Partial results are kept for few items only, however many empty sequences are named."""
    n = qsa.window_attn_scratch_bytes
    for nseq, total_q, nheads, nkv in ((1, 1, 8, 8), (65535, 10, 32, 8), (76, 1, 8, 8), (300, 300, 1, 1), (1, 100000, 8, 1),
                                       (4, 2000, 32, 8), (1, 2 ** 30, 1, 1)):
        assert n(nseq, total_q, total_q, nheads, nkv) <= 256 << 20


def test_window_attn_limits(lib):
    assert window(lib, nseq=0, q=None, out=None) == OK
    assert window(lib, total_q=0, max_q=0, q=None, out=None, cu_q=None) == OK
    assert window(lib, nseq=65536) == UNSUPPORTED
    assert window(lib, nheads=258, nkv=2) == UNSUPPORTED
    assert window(lib, total_q=2 ** 30, nheads=2) == UNSUPPORTED


def evict(lib, kv=None, **kw):
    d = dict(nseq=2, table=A, cols=8, tstride=8, lens=A, mass=A, mstride=128, new=A, new_cols=4, nstride=4, budget=64,
             sinks=4, recent=16, kept=B, new_lens=B, new_mass=B, nmstride=64, nmcols=64)
    d.update(kw)
    return lib.qsa_cache_evict(kv or pages(), d["nseq"], d["table"], d["cols"], d["tstride"], d["lens"], d["mass"],
                               d["mstride"], d["new"], d["new_cols"], d["nstride"], d["budget"], d["sinks"], d["recent"],
                               d["kept"], d["new_lens"], d["new_mass"], d["nmstride"], d["nmcols"], None)


@pytest.mark.parametrize("bad", [dict(nseq=-1), dict(budget=0), dict(sinks=-1), dict(recent=-1),
                                 dict(sinks=40, recent=25), dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1),
                                 dict(budget=65), dict(nmcols=63), dict(nmstride=63), dict(mstride=127),
                                 dict(tstride=7), dict(nstride=3), dict(lens=None), dict(table=None), dict(mass=MIS),
                                 dict(new=None), dict(kept=MIS), dict(new_lens=None), dict(new_mass=MIS),
                                 dict(new_lens=A), dict(new_mass=A)])
def test_cache_evict_argument_errors(lib, bad):
    assert evict(lib, **bad) == INVALID


def test_cache_evict_limits(lib):
    assert evict(lib, nseq=0, table=None, mass=None, new=None, lens=None, kept=None, new_lens=None, new_mass=None) == OK
    assert evict(lib, nseq=65536) == UNSUPPORTED
    assert evict(lib, cols=1 << 27, tstride=1 << 27, mstride=1 << 31) == UNSUPPORTED


def test_binding_refuses_what_is_not_on_the_gpu():
    t = torch.zeros((1, 16, 1, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qsa.paged_attn(torch.zeros((1, 1, 128), dtype=torch.bfloat16), t, t, torch.zeros((1, 1), dtype=torch.int32),
                       torch.ones(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        qsa.window_attn(t[0], t[0], t[0], torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 1)
    with pytest.raises(ValueError):
        qsa.cache_evict(t, t, torch.zeros((1, 1), dtype=torch.int32), torch.ones(1, dtype=torch.int32),
                        torch.zeros((1, 16)), torch.zeros((1, 1), dtype=torch.int32), 4)


def test_reference_attention_by_hand():
    q = torch.zeros((1, 2, 128)); q[0, 0, 0] = 1.0                 # the second query sees nothing
    k = torch.zeros((3, 128)); k[1, 0] = math.log(3.0); k[2] = math.nan
    v = torch.stack([torch.full((128,), 1.0), torch.full((128,), 5.0), torch.full((128,), math.nan)])
    seen = torch.tensor([[True, True, False], [False, False, False]])
    out, lse, p, _, _ = cache_ref.attend(q, k, v, seen, 1.0)
    assert torch.allclose(out[0, 0], torch.full((128,), 4.0, dtype=torch.float64))     # (1 * 1 + 3 * 5) / 4
    assert abs(float(lse[0, 0]) - math.log(4.0)) < 1e-7 and float(lse[0, 1]) == -math.inf
    assert torch.count_nonzero(out[0, 1]) == 0 and torch.count_nonzero(p[0, 1]) == 0


def test_reference_eviction_by_hand():
    mass = [9.0, 1.0, 5.0, 5.0, math.nan, 5.0, 0.0, 0.0]
    assert cache_ref.evict(mass, 8, 8, 0, 0) == list(range(8))
    assert cache_ref.evict(mass, 8, 4, 1, 1) == [0, 2, 3, 7]        # of three fives, the two lowest
    assert cache_ref.evict(mass, 8, 2, 1, 1) == [0, 7]
    assert cache_ref.evict(mass, 8, 7, 0, 0) == [0, 1, 2, 3, 5, 6, 7]   # NaN goes first
    assert cache_ref.evict(mass, 3, 4, 1, 1) == [0, 1, 2]
