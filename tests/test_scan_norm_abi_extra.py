"""Refusals of the norms' entry points that go by the width (no GPU needed: device pointers
are made up and never followed)."""
import ctypes

import pytest

import ssm_decode_02_b200 as rsq

P = 1 << 20
INVAL = rsq.RSQ_E_INVAL


def config(rows, width, dtype, stride=0):
    return rsq.rsq_norm_config(rows, width, 0, 0, dtype, dtype, dtype, 1e-5, stride, stride)


@pytest.mark.parametrize("width,stride", [(63, 0), (64, 65)])
def test_vectors_of_an_odd_row_need_the_alignment_of_an_element(width, stride):
    """Rows that are worked on element by element may start anywhere."""
    cfg = config(0, width, rsq.RSQ_BF16, stride)       # no rows: checked, and nothing launched
    assert rsq.lib.rsq_gated_norm(ctypes.byref(cfg), None, None, P + 4, None, 0) == rsq.RSQ_OK
    assert rsq.lib.rsq_residual_norm(ctypes.byref(cfg), None, None, P + 4, P + 8, None, None, 0) == rsq.RSQ_OK
    assert rsq.lib.rsq_gated_norm(ctypes.byref(cfg), None, None, P + 2, None, 0) == INVAL
    assert rsq.lib.rsq_residual_norm(ctypes.byref(cfg), None, None, P + 2, P, None, None, 0) == INVAL


@pytest.mark.parametrize("width,dtype,off", [(63, rsq.RSQ_BF16, 1), (63, rsq.RSQ_F32, 2), (64, rsq.RSQ_BF16, 8), (64, rsq.RSQ_F32, 4)])
def test_misaligned_arrays_are_refused(width, dtype, off):
    cfg = ctypes.byref(config(4, width, dtype))
    lib = rsq.lib

    def each(call, n, skip=()):
        for k in range(n):
            if k not in skip:
                a = [P] * n
                a[k] = P + off
                assert call(a) == INVAL, (k, rsq.lib.rsq_last_error())

    each(lambda a: lib.rsq_gated_norm(cfg, *a, 0), 4, skip=())
    each(lambda a: lib.rsq_gated_norm_backward(cfg, *a, None, 0, 0), 7, skip=())      # and a dw needs a workspace
    each(lambda a: lib.rsq_residual_norm(cfg, *a, 0), 6, skip=())
    each(lambda a: lib.rsq_residual_norm_backward(cfg, *a, None, 0, 0), 10)
