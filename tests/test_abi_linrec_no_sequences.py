"""Calls of rows without a sequence (no GPU needed): a step, like
gdr_recurrent_fwd, has nothing to do; the scans refuse them, like gdr_chunk_fwd."""
from tests.test_abi_linrec_norm import INVALID, _bwd, _fwd, _step, lib  # noqa: F401


def test_a_step_of_no_sequence_is_ok(lib):  # noqa: F811
    assert _step(lib, N=0, T=8) == 0
    assert lib.gdr_last_error() == b""
    assert _step(lib, N=0, T=8, dtype=7) != 0              # sizes and types are checked all the same


def test_a_scan_of_no_sequence_is_refused(lib):  # noqa: F811
    assert _fwd(lib, N=0, T=8) == INVALID
    assert _bwd(lib, N=0, T=8) == INVALID
