"""The new-token calls refuse bad arguments before anything is launched (CPU only: fake device addresses, no call here
reaches a kernel), and the 64-bit forms that the GPU tests compare with are right where they can be written down by hand."""
import ctypes
import math
import os
import sys

import pytest
import torch

import token_ref
from sparse_attention_kv_qsa_gb300 import build as qsa_build
from sparse_attention_kv_qsa_gb300 import qsa
from test_cache_abi import A, B, BAD_PAGES, MIS, pages

OK, INVALID, UNSUPPORTED = qsa.QSA_OK, qsa.QSA_ERR_INVALID, qsa.QSA_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    qsa_build.build()
    return qsa.lib()


def rotation(**kw):
    d = dict(freqs=A, axis=None, positions=A, position_stride=100, npairs=64, naxes=1, interleaved=0, inverse=0)
    d.update(kw)
    return ctypes.byref(qsa.Rotation(**d))


BAD_ROTATIONS = [dict(freqs=None), dict(freqs=MIS), dict(axis=MIS), dict(positions=MIS), dict(position_stride=-1), dict(npairs=0),
                 dict(npairs=12), dict(npairs=72), dict(npairs=-8), dict(naxes=0), dict(naxes=-1)]


def rotate(lib, rot=None, **kw):
    d = dict(x=A, dtype=qsa.BF16, strides=(1024, 128, 1024, 128), ntok=5, nheads=8, out=B)
    d.update(kw)
    st = None if d["strides"] is None else (ctypes.c_int64 * 4)(*d["strides"])
    return lib.qsa_rotate(d["x"], d["dtype"], st, d["ntok"], d["nheads"], None if rot == "none" else rot or rotation(), d["out"], None)


@pytest.mark.parametrize("bad", BAD_ROTATIONS + [dict(positions=None)])
def test_rotate_bad_rotations(lib, bad):
    assert rotate(lib, rotation(**bad)) == INVALID


@pytest.mark.parametrize("bad", [dict(x=None), dict(x=MIS), dict(out=None), dict(out=MIS), dict(dtype=qsa.I8), dict(dtype=9),
                                 dict(strides=None), dict(ntok=-1), dict(nheads=0), dict(strides=(1024, 4, 1024, 128)),
                                 dict(strides=(-1024, 128, 1024, 128)), dict(strides=(0, 0, 0, 128)),
                                 dict(strides=(0, 0, 1024, 0)), dict(strides=(0, 0, 64, 128)), dict(rot="none")])
def test_rotate_argument_errors(lib, bad):
    assert rotate(lib, **bad) == INVALID


def test_rotate_limits(lib):
    assert rotate(lib, ntok=0, x=None, out=None) == OK
    assert rotate(lib, nheads=65536) == UNSUPPORTED
    assert rotate(lib, rotation(naxes=65536)) == UNSUPPORTED


def append(lib, kv=None, rot=None, **kw):
    d = dict(k=A, v=A, q=A, dtype=qsa.BF16, strides=(256, 128, 256, 128, 1024, 128, 1024, 128, 256, 128), ntok=5, nheads=8, table=A,
             cols=4, tstride=4, lens=A, cu=A, nseq=2, q_out=B, k_out=B)
    d.update(kw)
    st = None if d["strides"] is None else (ctypes.c_int64 * 10)(*d["strides"])
    return lib.qsa_cache_append(d["k"], d["v"], d["q"], d["dtype"], st, d["ntok"], d["nheads"], kv or pages(), d["table"], d["cols"],
                                d["tstride"], d["lens"], d["cu"], d["nseq"], None if rot == "none" else rot or rotation(), d["q_out"],
                                d["k_out"], None)


INT8 = dict(dtype=qsa.I8, k_scale_f16=A, v_scale_f16=A, scale_page_stride=32, scale_cell_stride=2, scale_head_stride=1)


@pytest.mark.parametrize("bad", BAD_PAGES + [dict(page_stride=0), dict(cell_stride=0), dict(head_stride=64),
                                             dict(INT8, scale_page_stride=0), dict(INT8, scale_cell_stride=0),
                                             dict(INT8, scale_head_stride=0)])
def test_append_bad_pages(lib, bad):
    assert append(lib, pages(**bad)) == INVALID


@pytest.mark.parametrize("bad", BAD_ROTATIONS + [dict(inverse=1), dict(positions=None, naxes=2)])
def test_append_bad_rotations(lib, bad):
    assert append(lib, rot=rotation(**bad)) == INVALID


def strides(i, n):
    s = [256, 128, 256, 128, 1024, 128, 1024, 128, 256, 128]
    s[i] = n
    return tuple(s)


@pytest.mark.parametrize("bad", [dict(k=None), dict(k=MIS), dict(v=None), dict(q=None), dict(q_out=None), dict(q_out=MIS), dict(k_out=MIS),
                                 dict(dtype=qsa.F16), dict(dtype=qsa.I8), dict(strides=None), dict(ntok=-1), dict(nheads=-1),
                                 dict(nseq=-1), dict(cu=None), dict(cu=MIS), dict(lens=None), dict(table=None), dict(cols=-1),
                                 dict(tstride=3), dict(rot="none"), dict(rot="none", nheads=0, q=None, q_out=None)]
                         + [dict(strides=strides(i, -128)) for i in range(10)] + [dict(strides=strides(i, 4)) for i in range(10)]
                         + [dict(strides=strides(i, 0)) for i in range(6, 10)])
def test_append_argument_errors(lib, bad):
    assert append(lib, **bad) == INVALID


def test_in_place_with_other_strides(lib):
    """Rows would be read after others have been written there."""
    for st in ((0, 128, 1024, 128), (1024, 128, 2048, 128), (128, 640, 1024, 128)):
        assert rotate(lib, strides=st, out=A) == INVALID
        q, k = (256, 128, 256, 128) + st + (256, 128), (0, 128, 256, 128, 1024, 128, 1024, 128, 256, 128)
        assert append(lib, strides=q, q_out=A) == INVALID and append(lib, strides=k, k_out=A) == INVALID
    # a dimension of one element has no stride: these get as far as the device, which is not there
    if not torch.cuda.is_available():
        assert rotate(lib, ntok=1, strides=(0, 128, 1024, 128), out=A) not in (OK, INVALID)
        assert rotate(lib, nheads=1, strides=(1024, 0, 1024, 128), out=A) not in (OK, INVALID)


def far(**kw):
    """Pages whose values lie far from their keys."""
    d = dict(v=A + (1 << 30), v_scale_f16=A + (1 << 31) if "k_scale_f16" in kw else None)
    d.update({k: v for k, v in kw.items() if k != "v_scale_f16"})
    return pages(**d)


OVER_ONE_ANOTHER = [(128, 128), (640, 128), (128, 512), (896, 128), (136, 128), (1024, 8)]      # of 5 tokens of 8 heads


@pytest.mark.parametrize("st", OVER_ONE_ANOTHER)
def test_rows_written_over_one_another(lib, st):
    """Row [t][h] is also row [t + 1][h - i], or begins inside of it."""
    assert rotate(lib, strides=(1024, 128) + st) == INVALID
    assert append(lib, far(), strides=(256, 128, 256, 128, 1024, 128) + st + (256, 128)) == INVALID
    if st[1] == 128 and st[0] < 256 or st[1] < 128:                                             # 2 KV heads
        assert append(lib, far(), strides=(256, 128, 256, 128, 1024, 128, 1024, 128) + st) == INVALID


@pytest.mark.parametrize("bad", [dict(page_stride=128), dict(page_stride=256), dict(page_stride=4096 - 8), dict(cell_stride=128),
                                 dict(head_stride=256), dict(head_stride=2048, cell_stride=256),
                                 dict(INT8, scale_page_stride=31), dict(INT8, scale_cell_stride=1), dict(INT8, scale_head_stride=2),
                                 dict(INT8, scale_page_stride=1, scale_cell_stride=1, scale_head_stride=1)])
def test_cells_written_over_one_another(lib, bad):
    assert append(lib, far(**bad)) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="gets as far as the device, which must not be there")
@pytest.mark.parametrize("st", [(1024, 128), (128, 640), (1152, 144), (6144, 128), (1032, 128), (136, 1024), (1 << 40, 1 << 50), (1 << 55, 128)])
def test_rows_apart_in_any_order(lib, st):
    """Tokens outside heads, heads outside tokens, slices of something wider."""
    assert rotate(lib, strides=(1024, 128) + st) not in (OK, INVALID)
    assert append(lib, far(), strides=(256, 128, 256, 128, 1024, 128) + st + (256, 128)) not in (OK, INVALID)


@pytest.mark.skipif(torch.cuda.is_available(), reason="gets as far as the device, which must not be there")
@pytest.mark.parametrize("good", [dict(head_stride=16 * 128, cell_stride=128), dict(page_stride=8192), dict(cell_stride=512, page_stride=16 * 512),
                                  dict(head_stride=256, cell_stride=512, page_stride=16 * 512), dict(npages=1, page_stride=0),
                                  dict(page_size=1, cell_stride=0), dict(nkv=1, head_stride=0),
                                  dict(INT8, scale_cell_stride=1, scale_head_stride=16), dict(page_stride=256, cell_stride=100 * 256)])
def test_cells_apart_in_any_order(lib, good):
    assert append(lib, far(**good)) not in (OK, INVALID)


@pytest.mark.parametrize("ntok", [2 ** 31 - 63, 2 ** 31 - 1])
def test_more_tokens_than_numbers(lib, ntok):
    """Their numbers, and those behind them in the last CTA, would pass 32 bits. Rows of stride 0 need no memory for that."""
    assert rotate(lib, ntok=ntok, nheads=1, strides=(0, 0, 128, 128)) == UNSUPPORTED
    assert append(lib, far(), ntok=ntok, nheads=2, strides=(0, 0, 0, 0, 0, 0, 256, 128, 256, 128)) == UNSUPPORTED


def rows_of(at, strides, ntok, nheads, size=128):
    """The bytes that rows of bfloat16 elements lie at, as a set of 16-byte pieces."""
    return {(at + 2 * (t * strides[0] + h * strides[1])) // 16 + i for t in range(ntok) for h in range(nheads) for i in range(size // 8)}


def test_rows_over_the_rows_that_are_read(lib):
    """Whatever 16 bytes the output begins behind or before the input: refused where any row of it lies on one that is read,
    but for the very same rows; what gets past is what a plain list of all pieces finds apart."""
    at = 1 << 20
    for st, ntok, nheads in (((1024, 128), 5, 8), ((128, 640), 5, 8), ((1152, 144), 3, 8), ((2048, 256), 4, 3), ((512, 128), 1, 3), ((264, 64), 4, 1)):
        read = rows_of(at, st, ntok, nheads)
        for off in [i for i in range(-700, 700)] + [5 * 1024 // 8, -5 * 1024 // 8, 1 << 20]:
            out = at + 16 * off
            meets = off != 0 and not read.isdisjoint(rows_of(out, st, ntok, nheads))
            if meets or not torch.cuda.is_available():   # others get as far as the device, which must not be there
                assert (rotate(lib, x=at, out=out, strides=st + st, ntok=ntok, nheads=nheads) == INVALID) == meets, (st, off)
    st = (1024, 128)
    for off in (2048, -2048, 256, 4096, 16):             # tokens, heads, and part of a row
        assert append(lib, far(), q=at, q_out=at + off) == INVALID
        if abs(off) < 4096:                              # k's tokens are 256 elements apart
            assert append(lib, far(), k=at, k_out=at + off) == INVALID


@pytest.mark.parametrize("bad", [dict(v=A), dict(v=A + 256), dict(k=A + 4096, v=A), dict(v=A + 16), dict(v=A + 2 * 4096 * 99),
                                 dict(INT8, v=A + (1 << 30), v_scale_f16=A), dict(INT8, v=A + (1 << 30), v_scale_f16=A + 64 * 99),
                                 dict(INT8, v=A + (1 << 30), k_scale_f16=A + 2, v_scale_f16=A)])
def test_keys_cells_over_values_cells(lib, bad):
    assert append(lib, pages(**bad)) == INVALID


def test_one_pool_for_keys_and_values(lib):
    """The same rows to the same cells: refused where they would differ."""
    plain = dict(rot="none", nheads=0, q=None, q_out=None, k_out=None)
    int8 = dict(INT8, v=A, k_scale_f16=B, v_scale_f16=B)
    for kv in (dict(v=A), int8):
        assert append(lib, pages(**kv), **dict(plain, v=B)) == INVALID
        assert append(lib, pages(**kv), **dict(plain, strides=strides(2, 512))) == INVALID
        assert append(lib, pages(**kv)) == INVALID                                              # keys are turned
        if not torch.cuda.is_available():
            assert append(lib, pages(**kv), **plain) not in (OK, INVALID)
    assert append(lib, pages(**dict(int8, v_scale_f16=B + 2)), **plain) == INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="gets as far as the device, which must not be there")
@pytest.mark.parametrize("good", [dict(v=A + 2 * 4096, page_stride=8192), dict(k=A + 2 * 4096, v=A, page_stride=8192),
                                  dict(v=A + 256, head_stride=256, cell_stride=512, page_stride=8192), dict(v=A + 2 * 4096 * 100),
                                  dict(INT8, v=A + (1 << 30), v_scale_f16=A + 64, scale_page_stride=64), dict(v=A + 512, npages=1, page_stride=0, page_size=1)])
def test_keys_cells_beside_values_cells(lib, good):
    assert append(lib, pages(**good)) not in (OK, INVALID)


def test_append_limits(lib):
    assert append(lib, ntok=0, k=None, v=None, q=None, q_out=None, lens=None) == OK
    assert append(lib, nseq=0) == OK
    assert append(lib, nseq=65536) == UNSUPPORTED
    assert append(lib, nheads=65536) == UNSUPPORTED
    assert append(lib, rot=rotation(naxes=65536)) == UNSUPPORTED
    assert append(lib, cols=1 << 27, tstride=1 << 27) == UNSUPPORTED


def test_binding_refuses_what_is_not_on_the_gpu():
    x, p = torch.zeros((1, 1, 128)), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        qsa.rotate(x, p, torch.ones(64))
    t = torch.zeros((1, 16, 1, 128))
    with pytest.raises(ValueError):
        qsa.cache_append(x, x, t, t, torch.zeros((1, 1), dtype=torch.int32), p)


def test_reference_rotation_by_hand():
    x = torch.zeros((2, 1, 128)); x[..., 0], x[..., 8], x[..., 1] = 3.0, 4.0, 5.0
    f = torch.zeros(8); f[0] = 0.5
    p = torch.tensor([0, 7], dtype=torch.int32)
    y = token_ref.rotate(x, p, f)
    assert torch.equal(y[0], x[0].double())
    # below, 7 times some 4 roundings of 2^-53 (the reduced angle's, cosine's, product's and sum's): 3.2e-15
    c, s = math.cos(3.5), math.sin(3.5)
    assert abs(y[1, 0, 0] - (3 * c - 4 * s)) < 4e-15 and abs(y[1, 0, 8] - (4 * c + 3 * s)) < 4e-15 and y[1, 0, 1] == 5
    y = token_ref.rotate(x, p, f, interleaved=True, inverse=True)
    assert abs(y[1, 0, 0] - (3 * c + 5 * s)) < 4e-15 and abs(y[1, 0, 1] - (5 * c - 3 * s)) < 4e-15 and y[1, 0, 8] == 4
    y = token_ref.rotate(x, torch.stack((p, p + 1)), f, torch.tensor([1] + [0] * 7))
    assert abs(y[0, 0, 0] - (3 * math.cos(0.5) - 4 * math.sin(0.5))) < 4e-15
    # a whole number of turns of a far position: 2^31 - 1 times 1 radian
    far = token_ref.rotate(torch.eye(128)[:1, None], torch.tensor([2 ** 31 - 1], dtype=torch.int32), torch.ones(8))
    assert abs(float(far[0, 0, 0]) - math.cos(2 ** 31 - 1)) < 1e-9


def test_reference_far_angles_by_hand():
    assert token_ref.inv_two_pi(48) == int(2 ** 48 / (2 * math.pi))
    p, f = torch.tensor([7, -3, 2 ** 31 - 1], dtype=torch.int32), torch.tensor([0.5, 2.0, 1e4])
    far = token_ref.far_angles(p, f)
    # the product is below 2^45 and so exact in 64 bits; cos and sin of it are the C library's
    for i, a in enumerate(p.tolist()):
        for j, b in enumerate(f.tolist()):
            assert abs(math.cos(far[i, j]) - math.cos(a * b)) < 1e-14 and abs(math.sin(far[i, j]) - math.sin(a * b)) < 1e-14
    # 2^100 radians: its fraction of a turn from 1 / (2 pi) to 500 places
    turns = (token_ref.inv_two_pi(500) << 100) % (1 << 500) / (1 << 500)
    want = token_ref.far_angles(torch.tensor([1]), torch.tensor([2.0 ** 100]))
    assert abs(float(want) - 2 * math.pi * (turns - round(turns))) < 1e-14


def test_reference_codes_by_hand():
    x = torch.zeros((4, 128)); x[0, 0], x[0, 1], x[0, 2] = 127.0, -63.5, 0.5
    x[2, 3], x[3, 0] = 1e-9, math.inf
    q, s = token_ref.codes(x)
    assert s[0] == 1.0 and q[0, :3].tolist() == [127, -64, 0]           # halves to even
    assert s[1] == 0.0 and not q[1].any() and s[2] == 0.0 and not q[2].any()
    assert math.isnan(s[3]) and not q[3].any()


def prefix(lib, kv=None, **kw):
    d = dict(q=A, q_dtype=qsa.BF16, qs=1024, qh=128, nseq=4, nheads=8, pt=A, pcols=4, pstride=4, pl=A, cu=A, ngroups=2, table=A, cols=4,
             tstride=4, lens=A, scale=0.1, out=A, lse=A, scratch=A, bytes=1 << 40)
    d.update(kw)
    return lib.qsa_prefix_attn(d["q"], d["q_dtype"], d["qs"], d["qh"], d["nseq"], d["nheads"], kv or pages(), d["pt"], d["pcols"],
                               d["pstride"], d["pl"], d["cu"], d["ngroups"], d["table"], d["cols"], d["tstride"], d["lens"], d["scale"],
                               d["out"], d["lse"], d["scratch"], d["bytes"], None)


@pytest.mark.parametrize("bad", BAD_PAGES)
def test_prefix_bad_pages(lib, bad):
    assert prefix(lib, pages(**bad)) == INVALID


@pytest.mark.parametrize("bad", [dict(nseq=-1), dict(ngroups=-1), dict(nheads=0), dict(nheads=7), dict(scale=0.0), dict(scale=-1.0),
                                 dict(scale=math.inf), dict(scale=3e38), dict(q_dtype=qsa.F16), dict(q_dtype=qsa.F32), dict(pcols=-1),
                                 dict(cols=-1), dict(pstride=3), dict(tstride=3), dict(qs=-128), dict(qh=4), dict(q=None), dict(q=MIS),
                                 dict(out=None), dict(out=MIS), dict(lse=MIS), dict(pt=None), dict(pl=None), dict(cu=None), dict(cu=MIS),
                                 dict(table=None), dict(lens=None), dict(scratch=None), dict(scratch=A + 4), dict(bytes=0)])
def test_prefix_argument_errors(lib, bad):
    assert prefix(lib, **bad) == INVALID


def test_prefix_limits(lib):
    assert prefix(lib, nseq=0, q=None, out=None, lens=None, cu=None, scratch=None, bytes=0) == OK
    assert prefix(lib, nseq=65536) == UNSUPPORTED
    assert prefix(lib, ngroups=65536) == UNSUPPORTED
    assert prefix(lib, nheads=65536) == UNSUPPORTED
    assert prefix(lib, nheads=258) == UNSUPPORTED
    assert prefix(lib, pages(**INT8), q_dtype=qsa.F32, nheads=258) == UNSUPPORTED
    assert prefix(lib, pcols=1 << 27, pstride=1 << 27) == UNSUPPORTED
    assert prefix(lib, cols=1 << 27, tstride=1 << 27) == UNSUPPORTED
    n = qsa.prefix_attn_scratch_bytes
    assert n(0, 1, 8, 2, 4, 4, 16) == 0 and n(4, 1, 7, 2, 4, 4, 16) == 0 and n(4, -1, 8, 2, 4, 4, 16) == 0
    assert n(64, 3, 32, 8, 4096, 64, 16) >= n(4, 1, 32, 8, 4096, 64, 16) > 0 and n(4, 0, 8, 2, 0, 0, 16) > 0
    # partial results do not grow with the lengths: bounded by the GPU, the sequences and the groups
    assert n(64, 1, 32, 8, 1 << 25, 1 << 25, 16) == n(64, 1, 32, 8, 1 << 20, 1 << 20, 16) <= 128 << 20


# nseq, groups, heads, KV heads, prefix columns, columns, page size: each just past a limit, and just within
@pytest.mark.parametrize("within,past", [((65535, 1, 16384, 16384, 1, 1, 16), (65535, 1, 16385, 16385, 1, 1, 16)),
                                         ((2048, 2048, 64, 1, 1 << 20, 1, 128), (2048, 2049, 64, 1, 1 << 20, 1, 128)),
                                         ((128, 1, 64, 1, 1, 1 << 26, 16), (512, 1, 64, 1, 1, 1 << 26, 16)),
                                         ((4, 1, 128, 1, 1, 1, 16), (4, 1, 129, 1, 1, 1, 16)), ((4, 65535, 8, 8, 1, 1, 16), (4, 65536, 8, 8, 1, 1, 16))])
def test_no_scratch_for_what_is_refused(lib, within, past):
    assert qsa.prefix_attn_scratch_bytes(*within) > 0
    assert qsa.prefix_attn_scratch_bytes(*past) == 0
    nseq, ngroups, heads, nkv, pcols, cols, page = past
    kv = pages(nkv=nkv, page_size=page, head_stride=128, cell_stride=128 * nkv, page_stride=128 * nkv * page)
    assert prefix(lib, kv, nseq=nseq, ngroups=ngroups, nheads=heads, pcols=pcols, pstride=pcols, cols=cols, tstride=cols) == UNSUPPORTED


@pytest.mark.parametrize("bad", [dict(text=0), dict(text=-5), dict(texts=0), dict(readers=0), dict(question=0), dict(steps=0)])
def test_example_refuses_what_it_cannot_run(bad):
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import shared_prefix as ex
    with pytest.raises(ValueError, match="at least"):
        ex.generate(**bad)


def test_scratch_of_many_groups(lib):
    """What the GPU's CTAs leave (66 MB at most), 1.1 KB a sequence and head, and 4.2 KB a group and KV head."""
    n = qsa.prefix_attn_scratch_bytes
    for heads, nkv in ((8, 1), (8, 8), (32, 8), (128, 1), (64, 4)):
        for nseq, ngroups in ((1, 1), (512, 1), (512, 64), (512, 512), (4096, 4096)):
            assert n(nseq, ngroups, heads, nkv, 1 << 20, 1 << 20, 16) <= 66e6 + 1100 * nseq * heads + 4200 * ngroups * nkv
