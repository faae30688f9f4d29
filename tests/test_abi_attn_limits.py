"""The longest prefix that a step takes: that of the table's positions (no GPU needed)."""
import ctypes

import pytest

import gated_delta_rule_37_gb300 as gdr
from tests.test_abi_attn import BF16, F32, UNSUPPORTED, _step, lib  # noqa: F401

LONGEST = 2 ** 31 - 257


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefix_len", [LONGEST + 1, 2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 63, 2 ** 31 - 1])
def test_longer_prefixes_are_refused(lib, prefix_len, dtype):
    out = ctypes.c_size_t(0)
    assert lib.gdr_attn_step_workspace_size(2, 4, 8, 2, 64, prefix_len, dtype, ctypes.byref(out)) == UNSUPPORTED
    assert "prefix_len" in lib.gdr_last_error().decode()
    ld = dict(ldq=512, ldo=512)
    assert _step(lib, pl=prefix_len, dtype=dtype, wn=1 << 62, **ld) == UNSUPPORTED
    assert "prefix_len" in lib.gdr_last_error().decode()
    with pytest.raises(gdr.GdrError, match="prefix_len"):
        gdr.attn_step_workspace_size(2, 4, 8, 2, 64, prefix_len=prefix_len, dtype=dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_the_longest_prefix_has_a_workspace(lib, dtype):
    """One that grows with the rows, not with the keys: as many partial results of a row as one a hundredth as long."""
    size = [gdr.attn_step_workspace_size(2, 4, 8, 2, 64, prefix_len=n, dtype=dtype) for n in (LONGEST // 100, LONGEST)]
    assert 0 < size[1] < 2 * size[0] < 1 << 24


@pytest.mark.parametrize("prefix_len", [2 ** 31, 2 ** 32, 2 ** 32 + 100])
def test_the_binding_passes_no_other_prefix(lib, prefix_len):
    """Lengths that 32 bits would wrap to a shorter one."""
    with pytest.raises(gdr.GdrError, match="prefix_len"):
        gdr.attn_step_workspace_size(2, 4, 8, 2, 64, prefix_len=prefix_len, dtype=BF16)
