"""Rotation by position on the GPU against its formula in 64 bits."""
import math

import numpy as np
import pytest
import torch

import sparse_attention_kv_qsa_gb300 as qsa
import token_ref

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def inputs(dev, ntok, heads, dtype, pairs=64, axes=1, far=5000, seed=0, extra=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn((ntok, heads + extra, 128), generator=g, device=dev).to(dtype)[:, :heads]
    freqs = torch.pow(torch.tensor(10000.0, dtype=torch.float64), -torch.arange(pairs) / pairs).to(torch.float32).to(dev)
    positions = torch.randint(0, far, (axes, ntok), generator=g, device=dev, dtype=torch.int32)
    axis = (torch.arange(pairs, device=dev) % axes).to(torch.int32) if axes > 1 else None
    return x, positions, freqs, axis


def check(x, got, positions, freqs, axis=None, interleaved=False, inverse=False):
    want = token_ref.rotate(x, positions, freqs, axis, interleaved, inverse)
    tol = token_ref.rotate_tol(x, want, x.dtype, freqs.numel(), interleaved)
    assert got.dtype == x.dtype and got.shape == x.shape
    err = (got.cpu().to(torch.float64) - want).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    assert torch.equal(got[..., 2 * freqs.numel():], x[..., 2 * freqs.numel():])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("ntok,heads,pairs,axes,extra", [(1, 1, 64, 1, 0), (1, 32, 64, 1, 16), (3, 40, 64, 3, 0), (17, 5, 48, 2, 3),
                                                        (1000, 1, 8, 1, 0), (700, 3, 32, 3, 1), (3000, 17, 40, 4, 0),
                                                        (2, 300, 16, 1, 0), (20011, 1, 56, 2, 0), (0, 4, 64, 1, 0)])
def test_against_the_formula(dev, ntok, heads, pairs, axes, extra, dtype, interleaved):
    x, positions, freqs, axis = inputs(dev, ntok, heads, dtype, pairs, axes, extra=extra)
    if ntok == 0:
        assert qsa.rotate(x, positions, freqs).shape == (0, heads, 128)
        return
    for inverse in (False, True):
        check(x, qsa.rotate(x, positions, freqs, axis=axis, interleaved=interleaved, inverse=inverse), positions, freqs,
              axis, interleaved, inverse)


@pytest.mark.parametrize("freq", [1.0, -1.0, 0.7320508, 1e-5, 3.0e-38, 1e-42, 0.0, 123.456, 3.0e7, 1.5e20])
def test_every_position(dev, freq):
    """Positions of the whole range of int32, and frequencies far outside the usual: the angle is reduced exactly."""
    freqs = torch.full((64,), freq, device=dev)
    freqs[1::2] *= 0.999
    p = torch.tensor([0, 1, -1, 2, 1000, 999999, -999999, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32,
                     device=dev)
    # 1.5e20 x 2^31 has more bits than the reference's longest type reduces: small positions only
    if freq > 1e8:
        p = torch.tensor([0, 1, -1], dtype=torch.int32, device=dev)
    if freq > 1e6:
        # the factor is held to freq x 2^-64 turns: some 2^-39 at 3e7 (times 1,000 still 2^-29); at 1.5e20 angles mean nothing
        if freq > 1e8:
            y = qsa.rotate(torch.ones((3, 1, 128), device=dev), p, freqs)
            assert torch.isfinite(y).all() and float((y.abs().max())) <= math.sqrt(2) * (1 + 2.0 ** -20)
            return
        p = p[:5]
    g = torch.Generator(device=dev).manual_seed(3)
    x = torch.randn((p.numel(), 2, 128), generator=g, device=dev)
    check(x, qsa.rotate(x, p, freqs), p, freqs)


@pytest.mark.parametrize("freq", [1.0, 1e4, 16777216.0, 3.0e7, -1.2345e9, 9.2e18, 2.5e19, 1.5e20, -7.7e30, 3.4028234663852886e38])
def test_every_frequency(dev, freq):
    """Angles of the largest frequencies at positions of all of int32, to the same tolerance as others'."""
    freqs = torch.full((64,), freq, device=dev)
    freqs[1::2] *= 0.999
    freqs[2::3] *= 0.7654321
    p = torch.tensor([0, 1, -1, 3, 1000, -999999, 2 ** 24 + 1, 2 ** 30 + 12345, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(4)
    x = torch.randn((p.numel(), 2, 128), generator=g, device=dev)
    angle = token_ref.far_angles(p, freqs)[:, None]
    a, b = x.cpu().double().chunk(2, -1)
    want = torch.cat((a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()), -1)
    err = (qsa.rotate(x, p, freqs).cpu().double() - want).abs()
    assert bool((err <= token_ref.rotate_tol(x, want, F32, 64)).all()), float(err.max())


def test_odd_frequencies_and_axes(dev):
    x, positions, freqs, _ = inputs(dev, 9, 2, F32, axes=2)
    axis = torch.zeros(64, dtype=torch.int32, device=dev)
    axis[5], axis[6], axis[7] = 2, -1, 1        # the first two name no axis: not turned
    y = qsa.rotate(x, positions, freqs, axis=axis)
    check(x, y, positions, freqs, axis)
    assert torch.equal(y[..., 5:7], x[..., 5:7])
    freqs[3], freqs[4] = math.inf, math.nan
    z = qsa.rotate(x, positions, freqs, axis=axis)
    assert torch.isnan(z[..., [3, 4, 67, 68]]).all()
    keep = [i for i in range(128) if i not in (3, 4, 67, 68)]
    assert torch.equal(z[..., keep], y[..., keep])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_and_into_a_slice(dev, dtype, interleaved):
    x, positions, freqs, _ = inputs(dev, 130, 6, dtype, extra=4)
    whole = x._base.clone() if x._base is not None else x.clone()
    want = qsa.rotate(x, positions, freqs, interleaved=interleaved)
    into = torch.full((130, 9, 128), -7.0, device=dev, dtype=dtype)
    assert qsa.rotate(x, positions, freqs, interleaved=interleaved, out=into[:, 2:8]).data_ptr() == into[:, 2:8].data_ptr()
    assert torch.equal(into[:, 2:8], want) and bool((into[:, :2] == -7).all()) and bool((into[:, 8:] == -7).all())
    qsa.rotate(x, positions, freqs, interleaved=interleaved, out=x)
    assert torch.equal(x, want)
    assert torch.equal(x._base[:, 6:], whole[:, 6:])


def test_broadcast_rows_and_strided_positions(dev):
    """x of stride 0 (one row for all tokens), positions as part of a wider table."""
    _, wide, freqs, axis = inputs(dev, 64, 1, F32, axes=3)
    x = torch.randn((1, 4, 128), device=dev).expand(33, 4, 128)
    p = wide[:, 10:43]
    check(x, qsa.rotate(x, p, freqs, axis=axis), p, freqs, axis)


def test_back_and_gradient(dev):
    """inverse undoes the rotation, and is its gradient: <w, R x> = <R' w, x>, also by differences."""
    x, positions, freqs, axis = inputs(dev, 50, 3, F32, axes=3, far=100000)
    there = qsa.rotate(x, positions, freqs, axis=axis)
    back = qsa.rotate(there, positions, freqs, axis=axis, inverse=True)
    # twice 4 x 2^-24 of |a| + |b|, which the turn keeps below sqrt(2) of itself
    assert float((back - x).abs().max()) <= 3 * 4 * 2.0 ** -24 * 2 * float(x.abs().max())
    w = torch.randn_like(x)
    grad = qsa.rotate(w, positions, freqs, axis=axis, inverse=True).double()
    d = torch.randn_like(x)
    up = (w.double() * (qsa.rotate(x + d, positions, freqs, axis=axis).double() - there.double())).sum()
    down = (grad * ((x + d).double() - x.double())).sum()
    n = x.numel()
    # linear: only roundings differ, 4 x 2^-24 x (|a| + |b|) of some 6 each, added with random signs
    assert abs(float(up - down)) <= 6 * math.sqrt(n) * 3 * 4 * 2.0 ** -24 * 8 * 4


def test_streams_and_graphs(dev):
    x, positions, freqs, _ = inputs(dev, 300, 8, BF16)
    want = qsa.rotate(x, positions, freqs)
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        y = qsa.rotate(x, positions, freqs)
    torch.cuda.current_stream(dev).wait_stream(side)
    assert torch.equal(y, want)
    out = torch.zeros_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qsa.rotate(x, positions, freqs, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    positions += 17
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, qsa.rotate(x, positions, freqs)) and not torch.equal(out, want)


def test_past_32_bit_offsets(dev):
    """Rows 2^31 elements apart."""
    base = torch.zeros((2 ** 31 + 4096,), device=dev, dtype=BF16)
    x = base.as_strided((2, 1, 128), (2 ** 31, 128, 1))
    x.copy_(torch.randn((2, 1, 128), device=dev))
    p = torch.tensor([3, 5], dtype=torch.int32, device=dev)
    _, _, freqs, _ = inputs(dev, 1, 1, BF16)
    check(x, qsa.rotate(x, p, freqs), p, freqs)


def test_binding_refusals(dev):
    x, positions, freqs, axis = inputs(dev, 4, 2, BF16, axes=2)
    bad = [dict(x=x.int()), dict(x=x[..., :64]), dict(x=x[0]), dict(x=x.transpose(1, 2)), dict(positions=positions.long()),
           dict(positions=positions[:, :3]), dict(positions=positions.cpu()), dict(positions=positions[:0]), dict(freqs=freqs[:12]),
           dict(freqs=freqs[:0]), dict(freqs=freqs.double()), dict(freqs=torch.cat((freqs, freqs))), dict(axis=axis[:8]),
           dict(axis=axis.long()), dict(out=x.float()), dict(out=x[:, :1]), dict(x=x.cpu()), dict(positions=None)]
    for b in bad:
        kw = dict(x=x, positions=positions, freqs=freqs, axis=axis, out=None)
        kw.update(b)
        with pytest.raises(ValueError):
            qsa.rotate(kw["x"], kw["positions"], kw["freqs"], axis=kw["axis"], out=kw["out"])
    one = torch.zeros((1, 2, 128), device=dev, dtype=BF16).expand(4, 2, 128)
    with pytest.raises(qsa.QSAError):                      # rows written over one another
        qsa.rotate(x, positions, freqs, out=one)
    odd = torch.zeros((4 * 2 * 132,), device=dev, dtype=BF16).as_strided((4, 2, 128), (264, 132, 1))
    with pytest.raises(qsa.QSAError):                      # rows 264 bytes apart
        qsa.rotate(odd, positions, freqs)


def test_what_is_neither_true_nor_false(dev):
    """Its own error, and nothing has been launched."""
    x, positions, freqs, _ = inputs(dev, 4, 2, BF16)
    out = torch.full_like(x, 5)
    for odd in (np.zeros(2), torch.zeros(2)):
        for name in ("interleaved", "inverse"):
            with pytest.raises((ValueError, RuntimeError), match="ambiguous"):
                qsa.rotate(x, positions, freqs, out=out, **{name: odd})
        k_pages, v_pages = (torch.full((1, 16, 2, 128), 5, device=dev, dtype=BF16) for _ in range(2))
        with pytest.raises((ValueError, RuntimeError), match="ambiguous"):
            qsa.cache_append(x, x, k_pages, v_pages, torch.zeros((4, 1), dtype=torch.int32, device=dev),
                             torch.arange(1, 5, dtype=torch.int32, device=dev), freqs=freqs, interleaved=odd)
        assert bool((k_pages == 5).all()) and bool((v_pages == 5).all())
    assert bool((out == 5).all())
