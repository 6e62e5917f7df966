"""The bounded waits' failure path of prompt attention, made to run on the GPU
without a fault: a diagnostic call shortens every wait's limit and CTA 0 never
copies its first key tile. The call must end soon, report the time-out, and
leave the device usable. Where the keys of an item are split into parts, the
kernel that adds them must not depend on what the given-up CTA left unwritten
in scratch, whatever lies there."""
import time

import pytest
import torch

import sparse_attention_kv_qsa_gb300 as qsa
from sparse_attention_kv_qsa_gb300 import qsa as Q
from test_gpu_window_attn import BF16, check, dev, inputs, starts  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu
LIMIT_NS = 1_000_000   # 1 ms


@pytest.mark.parametrize("left", [0x00, 0x01, 0x7F, 0xFF])
@pytest.mark.parametrize("nq,nk", [([300], [2600]),               # few items, each in equal parts
                                   ([640], [2050]), ([100, 1, 540], [700, 3000, 5000]),   # parts that fall in size
                                   ([3000], [3000])])             # whole items, several a CTA
def test_a_wait_runs_out(dev, nq, nk, left):  # noqa: F811
    q, k, v = inputs(dev, nq, nk, 8, 4, BF16)
    cu_q, cu_k = starts(nq, dev), starts(nk, dev)
    need = qsa.window_attn_scratch_bytes(len(nq), sum(nq), max(nq), 32, 8)
    scratch = torch.full((max(need, 16),), left, dtype=torch.uint8, device=dev)
    out = torch.empty_like(q)
    assert qsa.device_error(dev) == 0
    torch.cuda.synchronize()
    Q.debug_inject(Q.INJECT_WINDOW_STALL, LIMIT_NS)
    try:
        t0 = time.perf_counter()
        qsa.window_attn(q, k, v, cu_q, cu_k, max(nq), out=out, scratch=scratch)
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        Q.debug_inject(0)
    code = qsa.device_error(dev)
    assert code == 0x10000, hex(code)
    assert dt < 0.5, f"the call took {dt:.3f} s"
    again, lse = qsa.window_attn(q, k, v, cu_q, cu_k, max(nq), scratch=scratch)
    check(q, k, v, nq, nk, again, lse)
    assert qsa.device_error(dev) == 0
