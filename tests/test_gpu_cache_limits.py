"""The bounded-cache calls at the limits of their arguments, on the GPU."""
import math

import pytest
import torch

import sparse_attention_kv_qsa_gb300 as qsa

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
