"""Calls without tokens: arrays of no elements have no address (no GPU needed: nothing is
read or written, with or without a device)."""
import ctypes

import pytest

import ssm_decode_02_b200 as rsq


@pytest.mark.parametrize("ragged", [0, 1])
def test_no_tokens_need_no_arrays(ragged):
    """Empty dt, x, B and C are null pointers, as torch gives them out."""
    s = rsq.Scan(2, 0, 2, 64, 64, ragged=bool(ragged))
    none = rsq.rsq_scan_inputs(None, None, None, None, None, None, None, 0, 0, 0)
    if not ragged:      # a ragged call would read its bounds
        assert rsq.lib.rsq_scan(ctypes.byref(s.cfg), ctypes.byref(none), None, None, None, None, None, 0, 0) in (rsq.RSQ_OK, rsq.RSQ_E_CUDA)
    grads = rsq.rsq_scan_grads()
    # refused for the workspace alone, the last thing that is checked
    assert rsq.lib.rsq_scan_backward(ctypes.byref(s.cfg), ctypes.byref(none), 16 if ragged else None, None, None, None,
                                     ctypes.byref(grads), None, 0, 0) == rsq.RSQ_E_INVAL
    assert b"workspace" in rsq.lib.rsq_last_error()
