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


def bytes_without_segments(slots, H, N, P, backward):
    """The workspace of a scan whose sequences are not cut into segments."""
    cells, state = slots * H, N * 64 * -(-P // 64)
    sizes = [4, slots * 8, cells * 128 * 8, cells * 128 * 4]
    sizes += [cells * state * 4, cells * state * 4, 2 * cells * 4] if backward else [cells * state * 2]
    return sum(-(-k // 256) * 256 for k in sizes)


@pytest.mark.parametrize("tokens,H,N,P,segments", [(128 * 40 + 17, 2, 16, 16, True), (128 * 33 + 5, 1, 16, 16, True),
                                                   (128 * 18 + 70, 2, 64, 64, True), (128 * 15, 2, 64, 64, False), (128 * 40, 80, 128, 64, False)])
def test_which_sequences_are_cut_into_segments(tokens, H, N, P, segments):
    """The long sequences of the GPU tests are, forward and backward: a change of the rule shows here."""
    s = rsq.Scan(1, tokens, H, N, P)
    for got, backward in ((s.workspace_bytes, False), (s.backward_workspace_bytes, True)):
        whole = bytes_without_segments(-(-tokens // 128), H, N, P, backward)
        assert (got > whole) if segments else (got == whole), backward
