"""The bounded-cache calls at the limits of their arguments, on the GPU."""
import math

import pytest
import torch

import sparse_attention_kv_qsa_gb300 as qsa
from test_gpu_paged_attn import Cache, queries

pytestmark = pytest.mark.gpu
BF16, F16, F32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("kv,qt", [(BF16, BF16), (F16, F16), (I8, F32)])
@pytest.mark.parametrize("nseq,heads,nkv", [(1, 1, 1), (3, 8, 2), (700, 16, 1)])
def test_a_table_without_columns(dev, nseq, heads, nkv, kv, qt, mass):
    """No sequence can have a cell, whatever lens says: 0 and -infinity, and no mass."""
    k = torch.ones((2, 16, nkv, 128), device=dev).to(kv)
    scale = torch.ones((2, 16, nkv), device=dev, dtype=F16) if kv == I8 else None
    table = torch.zeros((nseq, 0), dtype=torch.int32, device=dev)
    lens = torch.full((nseq,), 5, dtype=torch.int32, device=dev)
    out = torch.full((nseq, heads, 128), math.nan, device=dev, dtype=qt)
    lse = torch.full((nseq, heads), math.nan, device=dev)
    kw = {}
    if mass:
        kw = dict(mass=torch.full((nseq, 9), 2.0, device=dev), mass_out=torch.full((nseq, 9), -5.0, device=dev))
    qsa.paged_attn(torch.ones((nseq, heads, 128), device=dev, dtype=qt), k, k.clone(), table, lens, k_scale_f16=scale,
                   v_scale_f16=scale, out=out, lse=lse, **kw)
    assert torch.count_nonzero(out) == 0 and bool((lse == -math.inf).all())
    if mass:
        assert bool((kw["mass"] == 2.0).all()) and bool((kw["mass_out"] == -5.0).all())


def prompt(dev, n, nkv, group, dtype, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda h: torch.randn((n, h, 128), generator=g, device=dev, dtype=dtype)  # noqa: E731
    return r(nkv * group), r(nkv), r(nkv), torch.tensor([0, n], dtype=torch.int32, device=dev)


def test_rows_summed_again_take_longer_than_a_wait_may(dev):
    """NaN in the values of the last token, which all rows of its key tile but its own read as hidden: thousands of
    keys are summed again for each while the pipeline's waits, cut to 1 ms, stand. Nothing gives up, all rows come."""
    n = 6000
    q, k, v, cu = prompt(dev, n, 8, 4, BF16)
    want, want_lse = qsa.window_attn(q, k, v, cu, cu, n)
    v[n - 1] = math.nan
    out, lse = torch.full_like(q, math.nan), torch.full(q.shape[:2], math.nan, device=dev)
    torch.cuda.synchronize()
    assert qsa.device_error(dev) == 0
    qsa.debug_inject(0, 1_000_000)
    try:
        qsa.window_attn(q, k, v, cu, cu, n, out=out, lse=lse)
        torch.cuda.synchronize()
    finally:
        qsa.debug_inject(0)
    assert qsa.device_error(dev) == 0
    assert torch.isnan(out[n - 1]).all() and torch.equal(lse, want_lse)
    # both forms are within half a step of bfloat16 (2^-8 of the weights, 2^-8 of the result) of the formula
    err = (out[:-1].float() - want[:-1].float()).abs().max()
    assert float(err) <= 2 * (2.0 ** -8 + 2.0 ** -8) * float(v[:-1].abs().max())


@pytest.mark.parametrize("n", [130, 600, 5000])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_visible_infinities_and_nan_reach_their_columns_alone(dev, n, dtype):
    """Columns 0 to 3: an infinity, a negative one, both, NaN in values that the later rows see. The weights'
    sum does not depend on them, nor does any other column of a row."""
    q, k, v, cu = prompt(dev, n, 2, 4, dtype)
    want, want_lse = qsa.window_attn(q, k, v, cu, cu, n)
    at = 70
    v[at, 0, 0] = math.inf
    v[at, 0, 1] = -math.inf
    v[at, 0, 2], v[at + 1, 0, 2] = math.inf, -math.inf
    v[at, 0, 3] = math.nan
    out, lse = qsa.window_attn(q, k, v, cu, cu, n)
    assert torch.equal(lse, want_lse)
    sees = out[at + 1:, :4]
    assert bool((sees[..., 0] == math.inf).all()) and bool((sees[..., 1] == -math.inf).all())
    assert torch.isnan(sees[..., 2:4]).all()
    assert torch.equal(out[at:, :4, 4:], want[at:, :4, 4:]) and torch.equal(out[:, 4:], want[:, 4:])
    tol = 2 * (2 * torch.finfo(dtype).eps) * float(v[:at].abs().max())   # two forms, each half a step for weights and result
    assert float((out[:at].float() - want[:at].float()).abs().max()) <= tol


def test_a_visible_nan_costs_little(dev):
    """Every row sees a NaN in token 0's values: no row is summed again (each is found NaN at its first key)."""
    n = 4096
    q, k, v, cu = prompt(dev, n, 8, 4, BF16)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=dev)

    def least():
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        times = []
        for _ in range(5):
            a.record()
            qsa.window_attn(q, k, v, cu, cu, n, out=out, lse=lse)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    fine = least()
    v[0] = math.nan
    slow = least()
    assert torch.isnan(out).all() and torch.isfinite(lse).all()
    assert slow < 20 * fine, (slow, fine)    # a thousand times when every row's keys were gone through again


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("qt", [F32, BF16])
@pytest.mark.parametrize("at", [0, 77, 299])
def test_value_scales_do_not_reach_the_weights(dev, qt, at, bad):
    """An infinite or NaN scale of an int8 cell's values spoils the results of its KV head, not lse and mass."""
    c = Cache(dev, [300, 20000], 2, 16, I8)
    q = queries(dev, 2, 8, qt)
    mass = torch.zeros((2, c.cols * 16), device=dev)
    want, _ = c.call(q, mass=torch.zeros_like(mass))
    places = [(c.table[s, at // 16].long(), at % 16, 1) for s in (0, 1)]
    kept = [c.vs[p].clone() for p in places]
    for p in places:
        c.vs[p] = bad
    out, lse = c.call(q, mass=mass)
    assert not torch.isfinite(out[:, 4:]).any() and torch.equal(out[:, :4], want[:, :4])
    for p, x in zip(places, kept):
        c.vs[p] = x
    c.check(q, want, lse, mass=torch.zeros_like(mass), mass_out=mass)


@pytest.mark.parametrize("qmul,scale", [(1e36, 1e-37), (3e37, 3e-38), (1e-36, 1e35), (1e-37, 1e36)])
def test_queries_of_the_whole_range_over_int8_cells(dev, qmul, scale):
    """fp32 queries near both ends of their range whose logits are ordinary numbers."""
    c = Cache(dev, [300, 5000], 2, 16, I8)
    q = (queries(dev, 2, 8, F32).clamp(-4, 4) * qmul)
    assert torch.isfinite(q).all()
    out, lse = c.call(q, scale=scale)
    c.check(q, out, lse, scale=scale)


@pytest.mark.parametrize("expanded", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_infinities_whose_weights_vanish(dev, dtype, expanded):
    """Each key outweighs the one before it, so that an infinity among the first values has a weight below fp32's
    range in later rows: by the formula it is positive still. Both by tensor copies and row by row (a token stride of 0)."""
    n = 300
    _, _, v, cu = prompt(dev, n, 1, 4, dtype)
    q = torch.zeros((1, 4, 128), device=dev, dtype=dtype)
    q[..., 0] = 1.0
    q = q.expand(n, 4, 128) if expanded else q.repeat(n, 1, 1)
    k = torch.zeros((n, 1, 128), device=dev, dtype=dtype)
    k[:, 0, 0] = 4.0 * torch.arange(n, device=dev)
    k[40:, 0, 0] += 400.0                                   # there all weights so far vanish at once
    v[2, 0, 5], v[3, 0, 6], v[4, 0, 7] = math.inf, -math.inf, math.nan
    out, lse = qsa.window_attn(q, k, v, cu, cu, n, scale=1.0)
    assert bool((out[2:, :, 5] == math.inf).all()) and bool((out[3:, :, 6] == -math.inf).all())
    assert torch.isnan(out[4:, :, 7]).all() and torch.isfinite(lse).all()
    rest = [c for c in range(128) if c not in (5, 6, 7)]
    assert torch.isfinite(out[..., rest]).all() and torch.isfinite(out[:2]).all()


def test_items_that_take_longer_than_a_wait_may(dev):
    """Whole items of 800 to 860 key tiles, some milliseconds each, under a limit of 1 ms for every wait."""
    nq, nk = 10000, 110000
    g = torch.Generator(device=dev).manual_seed(4)
    q = torch.randn((nq, 8, 128), generator=g, device=dev, dtype=BF16)
    k, v = (torch.randn((nk, 8, 128), generator=g, device=dev, dtype=BF16) for _ in range(2))
    cu_q, cu_k = (torch.tensor([0, n], dtype=torch.int32, device=dev) for n in (nq, nk))
    want, want_lse = qsa.window_attn(q, k, v, cu_q, cu_k, nq)
    out, lse = torch.full_like(q, math.nan), torch.full_like(want_lse, math.nan)
    torch.cuda.synchronize()
    assert qsa.device_error(dev) == 0
    qsa.debug_inject(0, 1_000_000)
    try:
        qsa.window_attn(q, k, v, cu_q, cu_k, nq, out=out, lse=lse)
        torch.cuda.synchronize()
    finally:
        qsa.debug_inject(0)
    assert qsa.device_error(dev) == 0
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
