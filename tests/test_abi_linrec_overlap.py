"""Host-side refusal of states that overlap in part (no GPU needed)."""
import pytest

from tests.test_abi_linrec_norm import INVALID, P, _bwd, _fwd, lib  # noqa: F401

N, D = 3, 64
SIZE = 4 * N * D
AT = 1 << 20
NEAR = [0, 16, -16, 4 * D, -4 * D, SIZE - 16, -(SIZE - 16)]


def refused(lib, code):  # noqa: F811
    return code == INVALID and "overlap" in lib.gdr_last_error().decode()


@pytest.mark.parametrize("off", NEAR)
@pytest.mark.parametrize("T", [0, 8])
def test_overlapping_states_are_refused(lib, off, T):  # noqa: F811
    assert refused(lib, _fwd(lib, N=N, T=T, h0=P(AT), hT=P(AT + off)))
    assert refused(lib, _bwd(lib, N=N, T=T, h0=P(AT), d0=P(AT + off)))
    assert refused(lib, _bwd(lib, N=N, T=T, df=P(AT), d0=P(AT + off)))


@pytest.mark.parametrize("off", [SIZE, -SIZE, SIZE + 16, -SIZE - 16])
def test_states_beside_one_another_are_not(lib, off):  # noqa: F811
    """The next refusal is another: without a workspace nothing is launched."""
    big = dict(T=1 << 20, D=D, wn=16)
    assert not refused(lib, _fwd(lib, N=N, h0=P(AT), hT=P(AT + off), **big))
    assert not refused(lib, _bwd(lib, N=N, h0=P(AT), d0=P(AT + off), **big))
    assert not refused(lib, _bwd(lib, N=N, df=P(AT), d0=P(AT + off), **big))
