"""qsa_window_attn (prompt attention, causal, sliding window and sinks)
against the plain 64-bit form. Tolerances: cache_ref.bounds; the weights
enter the product with the values rounded once to the inputs' type."""
import math

import pytest
import torch

import cache_ref as ref
import sparse_attention_kv_qsa_gb300 as qsa

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def dev():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return torch.device("cuda:0")


def starts(n, dev):
    return torch.tensor([sum(n[:i]) for i in range(len(n) + 1)], dtype=torch.int32, device=dev)


def inputs(dev, nq, nk, nkv, group, dtype, seed=0):
    g = torch.Generator(device=dev).manual_seed(seed)
    r = lambda n, h: torch.randn((n, h, 128), generator=g, device=dev, dtype=dtype)  # noqa: E731
    return r(sum(nq), nkv * group), r(sum(nk), nkv), r(sum(nk), nkv)


def check(q, k, v, nq, nk, out, lse, window=-1, sinks=0, scale=128 ** -0.5):
    dev, nkv = q.device, k.shape[1]
    g = q.shape[1] // nkv
    a = x = 0
    for n, m in zip(nq, nk):
        pos = (torch.arange(n, device=dev) + m - n)[:, None]
        j = torch.arange(m, device=dev)
        seen = j <= pos
        if window >= 0:
            seen = seen & ((j > pos - window) | (j < sinks))
        for h in range(nkv):
            hs = slice(h * g, (h + 1) * g)
            o, l, _, size, S = ref.attend(q[a:a + n, hs].transpose(0, 1), k[x:x + m, h], v[x:x + m, h], seen, scale)
            tol, ltol = ref.bounds(o, l, size, S, m, q.dtype, ref.half_step(q.dtype))
            ref.check(out[a:a + n, hs].transpose(0, 1), o, tol, ("out", n, m, h))
            ref.check(lse[a:a + n, hs].T, l, ltol, ("lse", n, m, h))
        a, x = a + n, x + m


def both(dev, nq, nk, nkv=2, group=4, dtype=BF16, **kw):
    q, k, v = inputs(dev, nq, nk, nkv, group, dtype)
    out, lse = qsa.window_attn(q, k, v, starts(nq, dev), starts(nk, dev), max(nq), **kw)
    check(q, k, v, nq, nk, out, lse, **kw)
    return q, k, v, out, lse


LENS = [1, 0, 2, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255, 257, 300]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("nkv,group", [(1, 1), (2, 4), (3, 3), (1, 8), (2, 5), (1, 7), (1, 16), (1, 128), (1, 100)])
def test_every_length(dev, dtype, nkv, group):
    q, k, v, out, lse = both(dev, LENS, LENS, nkv, group, dtype)
    cu = starts(LENS, dev)
    again, lse2 = qsa.window_attn(q, k, v, cu, cu, max(LENS))
    assert torch.equal(out, again) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window,sinks", [(0, 0), (0, 3), (1, 0), (1, 1), (7, 2), (64, 4), (128, 16), (129, 17),
                                          (200, 0), (250, 130), (4096, 4), (16, 5000), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("group", [1, 4, 6])
def test_windows_and_sinks(dev, window, sinks, group):
    n = [700, 1, 300, 129, 0, 513]
    q, k, v, out, lse = both(dev, n, n, 2, group, window=window, sinks=sinks)
    if window == 0 and sinks == 0:
        assert torch.count_nonzero(out) == 0 and bool((lse == -math.inf).all())


@pytest.mark.parametrize("window,sinks", [(-1, 0), (100, 4), (1000, 40)])
def test_chunks_of_prompts(dev, window, sinks):
    """Queries that are the last of their keys; more queries than keys leaves the first rows empty."""
    nq, nk = [1, 5, 64, 130, 40, 7, 300, 9], [1, 1000, 64, 2000, 33, 0, 299, 4000]
    _, _, _, out, lse = both(dev, nq, nk, window=window, sinks=sinks)
    first = sum(nq[:4])
    assert torch.count_nonzero(out[first:first + 7]) == 0 and bool((lse[first:first + 7] == -math.inf).all())


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("nq,nk,kw", [([1500], [1500], {}), ([2500], [2500], dict(window=333, sinks=5)),
                                      ([40], [20000], {}), ([1, 1], [30000, 100], {}),
                                      ([64, 3], [5000, 9000], dict(window=4000, sinks=64))])
def test_long(dev, dtype, nq, nk, kw):
    both(dev, nq, nk, 2, 4, dtype, **kw)


@pytest.mark.parametrize("nq,nk,kw", [([320], [1537], {}), ([320], [8200], dict(window=5000, sinks=20)),
                                      ([300, 150], [2600, 1200], {}), ([640], [2050], dict(window=1500, sinks=3)),
                                      ([100, 1, 540], [700, 3000, 5000], {}), ([1216], [4100], {}),
                                      ([2000, 301], [7000, 1000], dict(window=6000, sinks=1))])
def test_parts_of_every_size(dev, nq, nk, kw):
    """A quarter to two items per SM: keys split into 2 to 8 parts that fall in size, some rows' all masked."""
    both(dev, nq, nk, 8, 4, **kw)


def test_many_sequences(dev):
    n = [(7 * i) % 23 for i in range(600)]
    both(dev, n, n, 1, 2, window=9, sinks=2)


def test_empty_sequences(dev):
    """No keys at all, and a few tokens among thousands of empty sequences."""
    both(dev, [5, 70], [0, 0])
    n = [0] * 3000
    n[17], n[2999] = 3, 200
    both(dev, n, n, 2, 4)


@pytest.mark.parametrize("nseq,total_q,nheads,nkv", [(1, 1, 8, 8), (65535, 10, 32, 8), (76, 1, 8, 8), (300, 300, 1, 1),
                                                     (1, 100000, 8, 1), (4, 2000, 32, 8)])
def test_scratch_stays_bounded(dev, nseq, total_q, nheads, nkv):
    """However many empty sequences are named; on the device's own SM count."""
    assert qsa.window_attn_scratch_bytes(nseq, total_q, total_q, nheads, nkv) <= 256 << 20


def test_strided_arguments(dev):
    """Slices of a fused projection, and tensors with heads outside tokens."""
    n, cu = [150, 70], starts([150, 70], dev)
    fused = torch.randn((220, 8 + 2 + 2, 128), device=dev, dtype=BF16)
    q, k, v = fused[:, :8], fused[:, 8:10], fused[:, 10:]
    out, lse = qsa.window_attn(q, k, v, cu, cu, 150, window=60, sinks=2)
    check(q, k, v, n, n, out, lse, 60, 2)
    q, k, v = (torch.randn((h, 220, 128), device=dev, dtype=BF16).transpose(0, 1) for h in (8, 2, 2))
    buf = torch.empty((220, 8, 128), device=dev, dtype=BF16)
    out, lse = qsa.window_attn(q, k, v, cu, cu, 1000, out=buf)
    assert out is buf
    check(q, k, v, n, n, out, lse)
    k1 = k[:, :1].expand(220, 2, 128)                                # a head stride of zero
    out, lse = qsa.window_attn(q, k1, v, cu, cu, 150)
    check(q, k1, v, n, n, out, lse)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_hidden_values_never_reach_a_result(dev, bad):
    """Infinities and NaN in keys and values that a row does not see (a later
    token, one before its window, another sequence's) leave the row alone."""
    n, cu = [130, 90, 200], starts([130, 90, 200], dev)
    q, k, v = inputs(dev, n, n, 2, 4, BF16)
    at = 130 + 90 + 120                                              # token 120 of the last sequence
    for t in (k, v):
        t[130:220] = bad                                             # the whole second sequence
        t[at] = bad
    out, lse = qsa.window_attn(q, k, v, cu, cu, 200, window=40, sinks=3)
    clean_k, clean_v = k.clone(), v.clone()
    for t in (clean_k, clean_v):
        t[130:220] = 0
        t[at] = 0
    want_out, want_lse = qsa.window_attn(q, clean_k, clean_v, cu, cu, 200, window=40, sinks=3)
    fine = torch.ones(420, dtype=torch.bool, device=dev)
    fine[130:220] = False
    fine[at:at + 40] = False                                         # the rows that see token 120
    check(q, clean_k, clean_v, n, n, want_out, want_lse, 40, 3)
    assert torch.isfinite(out[fine]).all()
    err = (out[fine].float() - want_out[fine].float()).abs().max()
    assert float(err) <= 2.0 ** -6 * float(want_out[fine].abs().max())
    assert float((lse[fine] - want_lse[fine]).abs().max()) < 1e-4
    assert not torch.isfinite(out[at]).all()                         # and a row that sees it shows it


@pytest.mark.parametrize("qmul,scale", [(60.0, 128 ** -0.5), (1e-6, 128 ** -0.5), (1.0, 3.0), (1.0, 1e-30)])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_input_ranges(dev, qmul, scale, dtype):
    n, cu = [300, 40], starts([300, 40], dev)
    q, k, v = inputs(dev, n, n, 2, 4, dtype)
    q = (q.float() * qmul).to(dtype)
    out, lse = qsa.window_attn(q, k, v, cu, cu, 300, scale=scale)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    check(q, k, v, n, n, out, lse, scale=scale)


def test_growing_logits(dev):
    """Each later block of keys beats all before it by far: the running maximum moves at every step."""
    n, cu = [900], starts([900], dev)
    q, k, v = inputs(dev, n, n, 1, 4, BF16)
    q = q.abs()
    k = (k.abs() * torch.linspace(0.1, 8.0, 900, device=dev)[:, None, None]).to(BF16)
    out, lse = qsa.window_attn(q, k, v, cu, cu, 900)
    check(q, k, v, n, n, out, lse)


def test_agrees_with_the_decode_form(dev):
    """The last token's row equals paged attention over the same cells."""
    n = 700
    q, k, v = inputs(dev, [n], [n], 2, 4, BF16)
    cu = starts([n], dev)
    out, lse = qsa.window_attn(q, k, v, cu, cu, n, window=300, sinks=4)
    pad = lambda t: torch.nn.functional.pad(t, (0, 0, 0, 0, 0, 4)).view(44, 16, 2, 128)  # noqa: E731
    one, l1 = qsa.paged_attn(q[-1:], pad(k), pad(v), torch.arange(44, dtype=torch.int32, device=dev)[None],
                             torch.tensor([n], dtype=torch.int32, device=dev), window=300, sinks=4)
    assert float((one[0].float() - out[-1].float()).abs().max()) <= 2.0 ** -6
    assert float((l1[0] - lse[-1]).abs().max()) < 1e-4


def test_starts_out_of_range_are_clamped(dev):
    q, k, v = inputs(dev, [50], [50], 1, 4, BF16)
    cu = torch.tensor([-9, 20, 10 ** 9], dtype=torch.int32, device=dev)
    out, lse = qsa.window_attn(q, k, v, cu, cu, 50)
    check(q, k, v, [20, 30], [20, 30], out, lse)


def test_other_stream_and_graph(dev):
    q, k, v = inputs(dev, [260], [260], 2, 4, BF16)
    cu = starts([100, 160], dev)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=dev)
    need = qsa.window_attn_scratch_bytes(2, 260, 260, 8, 2)
    scratch = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    call = lambda: qsa.window_attn(q, k, v, cu, cu, 260, window=90, sinks=3, out=out, lse=lse, scratch=scratch)  # noqa: E731
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):
        call()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            call()
    for step in range(12):
        cu[1] = 20 * step
        q.copy_(torch.randn_like(q))
        out.fill_(math.nan)
        scratch.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        check(q, k, v, [20 * step, 260 - 20 * step], [20 * step, 260 - 20 * step], out, lse, 90, 3)
    assert qsa.device_error(dev) == 0


def test_refusals_of_the_binding(dev):
    q, k, v = inputs(dev, [30], [30], 2, 4, BF16)
    cu = starts([30], dev)
    for args in ((q.float(), k, v, cu, cu, 30), (q, k.half(), v, cu, cu, 30), (q[..., :64], k, v, cu, cu, 30),
                 (q[:, :7], k, v, cu, cu, 30), (q, k, v[:29], cu, cu, 30), (q, k, v, cu.long(), cu, 30),
                 (q, k, v, cu, cu[:1], 30), (q, k, v, cu, cu, -1), (q.cpu(), k, v, cu, cu, 30)):
        with pytest.raises(ValueError):
            qsa.window_attn(*args)
    with pytest.raises(qsa.QSAError):
        qsa.window_attn(q, k, v, cu, cu, 30, scale=-1.0)
    with pytest.raises(qsa.QSAError):
        qsa.window_attn(q, k, v, cu, cu, 30, sinks=-1)
    none = qsa.window_attn(q[:0], k[:0], v[:0], cu[:1], cu[:1], 0)
    assert none[0].shape == (0, 8, 128)
