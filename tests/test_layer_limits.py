"""Sizes past what a call can do are refused on the host (no GPU needed: every call below comes
back before anything is launched)."""
import pytest

from bit_floating_point_amd import _lib as L
from bit_floating_point_amd import layer as Y

FAKE = 0x10000  # never dereferenced


def grid():
    g = L.fp4_grid()
    g.kind, g.e, g.m = 0, 4, 3
    return g


@pytest.mark.parametrize("slots", [(1 << 31) - (1 << 18), (1 << 31) - 1])
def test_experts_slots(slots):
    """All tiles of rows have to fit one launch."""
    d = Y.fp4_gemm_experts_desc(slots=slots, N=64, K=256, experts=1024, slots_per_row=(1 << 31) - 1, a=FAKE, lda=256, a_scales=FAKE,
                                lda_s=2, a_grid=grid(), w=FAKE, ldw=256, stride_w=64 * 256, w_scales=FAKE, w_grid=grid(),
                                offsets=FAKE, slot_list=FAKE, y=FAKE, ldy=64, y_dtype=L.FP4_BF16)
    assert Y._call("fp4_gemm_experts")(d, None) == L.FP4_ERR_UNSUPPORTED


@pytest.mark.parametrize("terms,status", [(1, L.FP4_ERR_ALIGNMENT), (2, L.FP4_ERR_UNSUPPORTED), (64, L.FP4_ERR_UNSUPPORTED)])
def test_norm_span_of_all_terms(terms, status):
    """x has rows * terms rows: their byte offsets have to fit 64 bits.  (What passes stops at
    gamma's alignment.)"""
    d = Y.fp4_rmsnorm_desc(rows=1 << 24, cols=256, x=FAKE, ldx=(1 << 36) - 64, x_dtype=L.FP4_F32, terms=terms, gamma=FAKE + 4,
                           gamma_dtype=L.FP4_F32, residual_dtype=L.FP4_BF16, eps=1e-6, y_dtype=L.FP4_BF16, y=FAKE, ldy=256)
    assert Y._call("fp4_rmsnorm_quant")(d, None) == status
