"""The bounded waits' failure path of the shared prefix's attention, made to run on the GPU without a fault: a diagnostic
call shortens every wait's limit and CTA 0 never hands over its first key tile. The call must end soon, report the
time-out, and leave the device usable, whatever lies in scratch."""
import time

import pytest
import torch

import sparse_attention_kv_qsa_gb300 as qsa
from sparse_attention_kv_qsa_gb300 import qsa as Q
from test_gpu_prefix_attn import KINDS, Shared, dev, lens_of  # noqa: F401 (dev is a fixture)

pytestmark = pytest.mark.gpu
LIMIT_NS = 1_000_000   # 1 ms


@pytest.mark.parametrize("left", [0x00, 0x01, 0x7F, 0xFF])
@pytest.mark.parametrize("kv,qt", KINDS)
@pytest.mark.parametrize("groups", [[(6, 3000)], [(150, 400)], [(2, 10), (1, 500), (40, 130)]])
def test_a_wait_runs_out(dev, groups, kv, qt, left):  # noqa: F811
    b = Shared(dev, groups, lens_of(sum(m for m, _ in groups)), 2, 4, 16, kv, qt)
    n = len(b.lens_list)
    need = qsa.prefix_attn_scratch_bytes(n, len(groups), 8, 2, b.ptable.shape[1], b.table.shape[1], 16)
    scratch = torch.full((need,), left, dtype=torch.uint8, device=dev)
    assert qsa.device_error(dev) == 0
    torch.cuda.synchronize()
    Q.debug_inject(Q.INJECT_PREFIX_STALL, LIMIT_NS)
    try:
        t0 = time.perf_counter()
        b.call(scratch=scratch)
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        Q.debug_inject(0)
    code = qsa.device_error(dev)
    assert code == 0x20000, hex(code)
    assert dt < 0.5, f"the call took {dt:.3f} s"
    out, lse = b.call(scratch=scratch)
    b.check(out, lse, only=list(range(0, n, 9)))
    assert qsa.device_error(dev) == 0
