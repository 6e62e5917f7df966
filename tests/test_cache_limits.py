"""The bounded-cache calls at the limits of their arguments, as far as that is
decided on the host (CPU only: fake device addresses, a call that passes the
checks finds no device)."""
import pytest

from sparse_attention_kv_qsa_gb300 import qsa
from test_cache_abi import A, lib, paged, window  # noqa: F401 (lib is a fixture)

INVALID = qsa.QSA_ERR_INVALID


@pytest.mark.parametrize("mass", [False, True])
@pytest.mark.parametrize("nseq,nheads,nkv", [(1, 1, 1), (2, 8, 2), (300, 40, 1)])
def test_a_table_without_columns_needs_scratch(lib, nseq, nheads, nkv, mass):  # noqa: F811
    """The kernels note in scratch what is to be joined, and the empty rows' sums, whatever the table's width."""
    need = qsa.paged_attn_scratch_bytes(nseq, nheads, nkv, 0, 16, mass)
    assert need >= 16 + (4 * nseq * nheads if mass else 0)
    assert qsa.paged_attn_scratch_bytes(nseq, nheads, nkv, 1, 16, mass) >= need


@pytest.mark.parametrize("kw", [dict(), dict(mass=A, mass_out=A, mstride=0)])
def test_a_table_without_columns_is_refused_without_scratch(lib, kw):  # noqa: F811
    need = qsa.paged_attn_scratch_bytes(2, 8, 2, 0, 16, "mass" in kw)
    for bad in (dict(scratch=None, bytes=0), dict(scratch=None), dict(bytes=need - 1), dict(scratch=A + 4)):
        assert paged(lib, cols=0, tstride=0, table=None, **bad, **kw) == INVALID


def test_prompt_attention_has_a_fault_bit(lib):  # noqa: F811
    assert lib.qsa_debug_inject(qsa.INJECT_WINDOW_STALL, 10 ** 6) == qsa.QSA_OK      # nothing is launched
    assert lib.qsa_debug_inject(16, 10 ** 6) == INVALID
    assert lib.qsa_debug_inject(0, qsa.WAIT_LIMIT_DEFAULT_NS) == qsa.QSA_OK


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_a_scale_that_overflows_in_base_2_is_refused(lib, scale):  # noqa: F811
    assert paged(lib, scale=scale) == INVALID and window(lib, scale=scale) == INVALID
